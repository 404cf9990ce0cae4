"""pq_distill and pq_distill_bwd on the GPU against binary64."""
import pytest
import torch

import layer_ref as R
from gpu_util import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
# (rows, vocab, k): one word to more than any block holds, ends inside a chunk, lists as long as they get
SHAPES = [(1, 1, 1), (3, 5, 2), (7, 64, 64), (2, 1000, 1), (5, 8191, 33), (4, 8192, 100), (3, 8193, 7), (3, 32000, 64), (2, 32768, 1024),
          (2, 32769, 16), (3, 50257, 256), (2, 65536, 8), (2, 65537, 9), (2, 128256, 64), (1, 131072, 1000), (2, 131073, 3), (1, 200001, 20),
          (700, 300, 12)]


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_amd import pq as _pq
    assert torch.cuda.is_available()
    return _pq


def make(rows, v, k, dtype, seed=0, top_dtype=torch.float32):
    g = torch.Generator().manual_seed(seed + rows + v + k)
    z = (torch.randn(rows, v, generator=g) * 3).to(dtype).to(DEV)
    index = torch.stack([torch.randperm(v, generator=g)[:k] for _ in range(rows)]).to(torch.int32)
    index = torch.cat([index, index.new_full((rows, k - index.shape[1]), -1)], 1).to(DEV)
    top = (torch.randn(rows, k, generator=g) * 2 + 4).to(top_dtype).to(DEV)
    return z, index, top


def check(z, index, top, temp, weight, loss, dz, scale, what=""):
    want, dwant, p, q = R.distill(z, index, top, temp, weight)
    w = torch.ones(len(z), device=DEV, dtype=torch.float64) if weight is None else weight.double().abs()
    if loss is not None:
        # p and q to 2^-18 (exponents of up to 64 in fp32, products and sums), weighed by the terms' sizes
        lp = torch.log(p.clamp_min(1e-300))
        size = (p * (lp.abs() + torch.log(q.clamp_min(1e-300)).abs())).sum(-1) + 1
        lim = temp ** 2 * w * size * 2.0 ** -18 + 2.0 ** -24 * want.abs()
        bad = ~((loss.double() - want).abs() <= lim)
        assert not bool(bad.any()), f"{what} loss {loss[bad][0].item()} for {want[bad][0].item()}"
    if dz is not None:
        dwant = dwant * scale
        u = R.U[dz.dtype] if dz.dtype != torch.float32 else 0
        lim = u * dwant.abs() + temp * abs(scale) * w[:, None] * (p + q) * 2.0 ** -17 * (1 + u) + R.TINY[dz.dtype]
        bad = ~((dz.double() - dwant).abs() <= lim)
        assert not bool(bad.any()), f"{what} dz: {int(bad.sum())} off, first at {bad.nonzero()[0].tolist()}: " \
                                    f"{dz[bad][0].item()} for {dwant[bad][0].item()}"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_distill(pq, shape, dtype):
    print(f"[distill {shape} {dtype}]", flush=True)
    rows, v, k = shape
    temp = [1.0, 2.0, 0.7][(v + k) % 3]
    z, index, top = make(*shape, dtype)
    weight = (torch.rand(rows, generator=torch.Generator().manual_seed(1)) + 0.1).to(DEV)
    loss, stats, dz = Guarded((rows,), torch.float32), Guarded((rows, 2), torch.float32), Guarded((rows, v), dtype)
    pq.pq_distill(z, index, top, loss.t, stats.t, dz.t, temperature=temp, row_weight=weight, grad_scale=0.25)
    check(z, index, top, temp, weight, loss.t, dz.t, 0.25, "fused")
    for g in (loss, stats, dz):
        g.check("fused")
    only, again = torch.empty(rows, device=DEV), torch.empty(rows, 2, device=DEV)
    pq.pq_distill(z, index, top, only, again, temperature=temp, row_weight=weight)
    assert torch.equal(only, loss.t) and torch.equal(again, stats.t)
    dloss = torch.full((rows,), -0.5, device=DEV)
    dz2 = Guarded((rows, v), dtype)
    pq.pq_distill_bwd(z, index, top, stats.t, dloss, dz2.t, temperature=temp, row_weight=weight)
    check(z, index, top, temp, weight, None, dz2.t, -0.5, "bwd")
    dz2.check("bwd")
    keep = z.clone()                                                  # over the logits themselves
    pq.pq_distill_bwd(z, index, top, stats.t, dloss, z, temperature=temp, row_weight=weight)
    assert torch.equal(z, dz2.t)
    pq.pq_distill(keep, index, top, dlogits=keep, temperature=temp, row_weight=weight, grad_scale=0.25)
    assert torch.equal(keep, dz.t)


@pytest.mark.parametrize("top_dtype", DTYPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_lists_with_holes(pq, dtype, top_dtype):
    """Words named twice and more, entries outside the vocabulary, logits of -inf, rows of nothing, rows of weight 0."""
    rows, v, k = 9, 3001, 40
    z, index, top = make(rows, v, k, dtype, 5, top_dtype)
    index[0, 1] = index[0, 0]
    index[1] = index[1, 0]                      # one word only: p = 1 there
    index[2, 7:] = -1
    index[3, ::2], index[3, 1::4] = v, -2 ** 31
    index[4] = -5                               # nothing counts
    index[5, 1:20] = index[5, 0] ^ 1            # two words of one chunk
    top[6, 1:] = float("-inf")
    weight = torch.ones(rows, device=DEV)
    weight[7], weight[8] = 0.0, -1.5
    z[7] = float("nan")                         # a row of padding may hold anything
    z[4, 3] = float("inf")
    loss, dz, stats = torch.full((rows,), 9.0, device=DEV), torch.full((rows, v), 9.0, dtype=dtype, device=DEV), \
        torch.empty(rows, 2, device=DEV)
    pq.pq_distill(z, index, top, loss, stats, dz, temperature=1.5, row_weight=weight)
    keep = [r for r in range(rows) if r not in (4, 7)]
    check(z[keep], index[keep], top[keep], 1.5, weight[keep], loss[keep], dz[keep], 1.0)
    assert float(loss[4]) == 0 and float(loss[7]) == 0 and torch.count_nonzero(dz[[4, 7]]) == 0
    dz2 = torch.full_like(dz, 9.0)
    pq.pq_distill_bwd(z, index, top, stats, torch.ones(rows, device=DEV), dz2, temperature=1.5, row_weight=weight)
    check(z[keep], index[keep], top[keep], 1.5, weight[keep], None, dz2[keep], 1.0)
    assert torch.count_nonzero(dz2[[4, 7]]) == 0
    assert abs(float(loss[1])) < 1e3 and int(torch.isfinite(dz.float()).sum()) == dz.numel()


def test_logits_of_no_number(pq):
    """-inf logits are words of probability 0; NaN, +inf and nothing but -inf make a row NaN, and that row alone."""
    rows, v = 6, 70
    z, index, top = make(rows, v, 4, torch.float32, 6)
    z[0, :30] = float("-inf")
    index[0] = torch.tensor([40, 50, 60, 69])
    z[1, 5], z[2, 6], z[3] = float("nan"), float("inf"), float("-inf")
    z[4, int(index[4, 0])] = float("-inf")                  # a word that the teacher wants
    loss, dz = torch.empty(rows, device=DEV), torch.empty(rows, v, device=DEV)
    pq.pq_distill(z, index, top, loss, dlogits=dz)
    check(z[[0, 5]], index[[0, 5]], top[[0, 5]], 1.0, None, loss[[0, 5]], dz[[0, 5]], 1.0)
    assert torch.count_nonzero(dz[0, :30]) == 0
    assert bool(loss[1:4].isnan().all()) and bool(dz[1:4].isnan().any(-1).all())
    assert float(loss[4]) == float("inf") and bool(dz[4].isfinite().all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides(pq, dtype):
    rows, v, k = 5, 777, 9
    z, index, top = make(rows, v, k, dtype, 7)
    wide = torch.full((rows, 900), 50.0, dtype=dtype, device=DEV)
    wide[:, 3:3 + v] = z
    out = torch.full((rows, 801), 7.0, dtype=dtype, device=DEV)
    loss, stats = torch.empty(rows, device=DEV), torch.empty(rows, 2, device=DEV)
    pq.pq_distill(wide[:, 3:3 + v], index, top, loss, stats, out[:, 5:5 + v])
    check(z, index, top, 1.0, None, loss, out[:, 5:5 + v], 1.0)
    assert bool((out[:, :5] == 7).all()) and bool((out[:, 5 + v:] == 7).all())
    want = z.float().amax(-1)
    assert torch.equal(stats[:, 0], want)
    total = torch.exp(z.double() - want.double()[:, None]).sum(-1)
    assert bool(((stats[:, 1].double() - total).abs() <= 2.0 ** -18 * total).all())


def test_empty_and_extreme_temperatures(pq):
    e = torch.empty(0, 10, device=DEV)
    pq.pq_distill(e, torch.empty(0, 2, dtype=torch.int32, device=DEV), torch.empty(0, 2, device=DEV), torch.empty(0, device=DEV))
    z, index, top = make(4, 500, 6, torch.float32, 8)
    for temp in (0.25, 100.0):
        loss, dz = torch.empty(4, device=DEV), torch.empty_like(z)
        pq.pq_distill(z, index, top, loss, dlogits=dz, temperature=temp)
        check(z, index, top, temp, None, loss, dz, 1.0, str(temp))


def test_gradient_against_differences(pq):
    rows, v, k = 16, 400, 10
    z, index, top = make(rows, v, k, torch.float32, 9)
    d = torch.randn(rows, v, generator=torch.Generator().manual_seed(10)).to(DEV)
    loss, dz = torch.empty(rows, device=DEV), torch.empty_like(z)
    pq.pq_distill(z, index, top, loss, dlogits=dz, temperature=2.0)
    e = 2.0 ** -6

    def f(z):
        pq.pq_distill(z, index, top, loss, temperature=2.0)
        return loss.double().clone()
    slope = (f(z + e * d) - f(z - e * d)) / (2 * e)
    # third derivative of T^2 log-sum-exp(z / T) along d: at most max|d|^3 / T; a loss of up to 100 is rounded to 2^-18
    assert float((slope - (dz.double() * d.double()).sum(-1)).abs().max()) < e * e * 4.5 ** 3 / 2 / 6 * 4 + 2.0 ** -17 / e


def test_more_rows_than_a_launch(pq):
    """Rows past 2^21, which go in a second launch."""
    rows, v, k = (1 << 21) + 3, 17, 2
    z = torch.randn(rows, v, device=DEV).to(torch.bfloat16)
    index = (torch.arange(rows, device=DEV, dtype=torch.int32)[:, None] * 3 + torch.tensor([0, 5], dtype=torch.int32, device=DEV)) % v
    top, weight = torch.randn(rows, k, device=DEV), (torch.rand(rows, device=DEV) < 0.9).float()
    loss, stats, dz = torch.empty(rows, device=DEV), torch.empty(rows, 2, device=DEV), torch.empty_like(z)
    pq.pq_distill(z, index, top, loss, stats, dz, row_weight=weight)
    check(z, index, top, 1.0, weight, loss, dz, 1.0)
    dz2 = torch.empty_like(z)
    pq.pq_distill_bwd(z, index, top, stats, torch.ones(rows, device=DEV), dz2, row_weight=weight)
    check(z, index, top, 1.0, weight, None, dz2, 1.0)


@pytest.mark.parametrize("fill", [float("-inf"), 0.0])
def test_lists_filled_up_with_one_word(pq, fill):
    """A list of 1024 entries that is one word for the most part, with and without weight: the sum over it is exact."""
    rows, v = 3, 5000
    z, index, top = make(rows, v, 1024, torch.float32, 11)
    index[:, 20:], top[:, 20:] = 7, fill
    loss, dz = torch.empty(rows, device=DEV), torch.empty_like(z)
    pq.pq_distill(z, index, top, loss, dlogits=dz)
    check(z, index, top, 1.0, None, loss, dz, 1.0)
    again = torch.empty_like(dz)
    pq.pq_distill(z, index, top, dlogits=again)
    assert torch.equal(again, dz)
