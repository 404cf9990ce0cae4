"""Attention over values at the edges of what a cache can hold: rows that were
never written, scales of either sign, infinities in attended places."""
import math

import pytest
import torch

import serving_ref as R
from test_gpu_attn import Case
from test_gpu_kv import FMT

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_amd import pq as _pq
    assert torch.cuda.is_available()
    return _pq


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("heads,group,dim", [(2, 4, 64), (1, 12, 80), (1, 2, 256)])
def test_a_new_cache_reads_as_zeros(pq, fmt, heads, group, dim):
    """A cache as allocate() makes it: every row 0, so out = 0 and lse = ln len; unsplit, then split rows."""
    page, pages = 16, 100
    cache = pq.KVCache.allocate(FMT[fmt][0], pages, page, heads, dim)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    q = torch.randn(1, heads * group, dim, generator=torch.Generator().manual_seed(dim)).to(torch.bfloat16).to(DEV)
    for n in (1, 16, 31, 32, 33, 64, 300, 1600):
        out, lse = torch.empty_like(q), torch.empty(1, heads * group, device=DEV)
        pq.pq_attn_decode(cache, q, table, torch.tensor([n], dtype=torch.int32, device=DEV), out, lse)
        assert torch.count_nonzero(out) == 0, (fmt, n)
        # the scores are 0 exactly; the logarithm is off by 2^-20 of its size at most
        assert float((lse.double() - math.log(n)).abs().max()) <= 2.0 ** -20 * max(1.0, math.log(n)), (fmt, n)


def zero_rows(c, page, unwritten):
    """Rows (sequence, token) become what a new cache holds."""
    for b, t in unwritten:
        at = int(c.table[b, t // page])
        for x in c.cache.tensors:
            if x is not None:
                x[at, :, t % page] = 0
        for held in (c.k, c.v, *c.mag):
            held[b][t] = 0


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("heads,group,dim", [(2, 4, 64), (1, 12, 80), (1, 2, 256)])
def test_written_rows_among_new_ones(pq, fmt, heads, group, dim):
    """Tokens whose append was skipped: a whole beginning, all but the last, every third, all but one in the middle."""
    page = 16
    c = Case(pq, fmt, [500, 260, 200, 1500, 90], heads, group, dim, page, torch.bfloat16, seed=dim)
    zero_rows(c, page, [(0, t) for t in range(400)] + [(1, t) for t in range(259)] + [(2, t) for t in range(200) if t % 3] +
              [(3, t) for t in range(1500) if t != 700])
    c.check(*c.run(pq))
    c.check(*c.run(pq, window=150), window=150)


@pytest.mark.parametrize("fmt", ["kv8", "kv4"])
def test_scales_of_either_sign(pq, fmt):
    """Pairs (s, z) that another program wrote: x^ = z + s n holds for a negative s and for s = 0 too."""
    page, d, n = 16, 64, 300
    c = Case(pq, fmt, [n], 1, 4, d, page, torch.bfloat16)
    at, off = c.table[0, torch.arange(n) // page].long(), torch.arange(n) % page
    for i, (held, par) in enumerate(((c.k, c.cache.tensors[2]), (c.v, c.cache.tensors[3]))):
        codes, pairs = c.cache.tensors[i].cpu(), par.cpu()
        pairs[at, 0, off, 0] *= torch.tensor([1.0, -1.0, 0.0, -1.0, 1.0])[torch.arange(n) % 5].to(torch.bfloat16)
        par.copy_(pairs)
        rows, p = codes[at, 0, off], pairs[at, 0, off].double()
        nn = R.unpack(rows, c.bits).double()
        held[0] = (p[:, 1:] + p[:, :1] * nn)[:, None]
        c.mag[i][0] = (p[:, 1:].abs() + p[:, :1].abs() * nn)[:, None]
    c.check(*c.run(pq))


@pytest.mark.parametrize("fmt", ["kv8", "kv4"])
@pytest.mark.parametrize("size", [1e16, 2.0 ** 100])
def test_large_constant_values(pq, fmt, size):
    """Value rows of one large number each: the smallest scale beside a zero of any size."""
    n, d, page = 200, 64, 16
    c = Case(pq, fmt, [n], 1, 2, d, page, torch.bfloat16)
    v = (torch.ones(n, 1, d) * size * (1 + torch.arange(n)[:, None, None] % 3)).to(torch.bfloat16)
    k = c.k[0].to(torch.float32).to(torch.bfloat16)
    t = torch.arange(n)
    slots = c.table[0, t // page].long() * page + t % page
    pq.pq_kv_append(c.cache, k.to(DEV), v.to(DEV), slots.to(DEV))
    for i, (x, held) in enumerate(((k, c.k), (v, c.v))):
        m, p = R.quantise(x.float(), c.bits)
        held[0] = R.values(R.pack(m, c.bits), p, c.bits)
        c.mag[i][0] = p.double()[..., 1:].abs() + p.double()[..., :1] * m.double()
    c.check(*c.run(pq))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 128, 192, 208, 256])
def test_keys_with_an_infinity(pq, dim, dtype):
    """A score of minus infinity is a weight of 0, whatever channel of the key it comes from."""
    page, n = 16, 70
    for channel in sorted({0, dim // 2 - 1, dim - 8, dim - 1}):
        c = Case(pq, "kv16", [n, 9], 2, 3, dim, page, dtype, seed=channel)
        c.q[..., channel] = -1.0
        for t in (0, 37, 69):
            at = int(c.table[0, t // page])
            c.cache.tensors[0][at, :, t % page, channel] = float("inf")
        c.check(*c.run(pq), hidden={(0, t) for t in (0, 37, 69)})


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 80, 192])
@pytest.mark.parametrize("n", [33, 700, 3000])
def test_values_with_an_infinity(pq, n, dim, dtype):
    """An attended infinity is the sum's: with its sign, in its channel and nowhere else; two of opposite signs are NaN."""
    page, inf = 16, float("inf")
    c = Case(pq, "kv16", [n], 2, 3, dim, page, dtype, seed=n)
    put = {1: [(n // 2, inf)], 9: [(0, -inf)], dim - 2: [(3, inf), (n - 1, -inf)], dim - 1: [(t, -inf) for t in range(5, n, 7)]}
    for channel, places in put.items():
        for t, x in places:
            c.cache.tensors[1][int(c.table[0, t // page]), :, t % page, channel] = x
    out, lse = c.run(pq)
    assert bool((out[0, :, 1] == inf).all()) and bool((out[0, :, 9] == -inf).all())
    assert bool(out[0, :, dim - 2].isnan().all()) and bool((out[0, :, dim - 1] == -inf).all())
    for channel in put:                             # the others are what they are without
        c.v[0][:, :, channel] = c.mag[1][0][:, :, channel] = 0
        out[0, :, channel] = 0
    c.check(out, lse)


def test_values_with_an_infinity_and_little_weight(pq):
    """bf16 keeps the infinity of a token whose weight is too small for binary32."""
    page, n, d, inf = 16, 400, 128, float("inf")
    c = Case(pq, "kv16", [n], 2, 4, d, page, torch.bfloat16, gain=30.0)
    for t in range(n):
        c.cache.tensors[1][int(c.table[0, t // page]), :, t % page, t % d] = inf
    out, _ = c.run(pq, scale=0.5)
    assert bool((out == inf).all())


@pytest.mark.parametrize("fmt", list(FMT))
def test_the_longest_window(pq, fmt):
    """A window of 2^63 - 1 tokens is no window: the row is split over the blocks as without one."""
    c = Case(pq, fmt, [5000], 1, 4, 64, 16, torch.bfloat16)
    table, lens = c.table.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    size = pq.pq_attn_decode_workspace_bytes(c.cache, 1, 4)
    got = []
    for window in (0, 2 ** 63 - 1, 2 ** 31):
        out, ws = torch.empty(1, 4, 64, dtype=torch.bfloat16, device=DEV), torch.full((size,), 0xA5, dtype=torch.uint8, device=DEV)
        pq.pq_attn_decode(c.cache, c.q.to(DEV), table, lens, out, window=window, workspace=ws)
        got.append((out, ws))
    for out, ws in got[1:]:
        assert torch.equal(out, got[0][0])
        assert bool((ws != 0xA5).any()), "not split"


@pytest.mark.parametrize("fmt", ["kv8", "kv4"])
@pytest.mark.parametrize("bad", ["inf", "-inf", "range"])
def test_rows_without_a_finite_scale(pq, fmt, bad):
    """A row that holds an infinity, or whose range passes binary32, reads as NaN; attention over it is NaN too."""
    page, n, d = 16, 40, 64
    f, bits = FMT[fmt]
    for which in (0, 1):
        cache = pq.KVCache.allocate(f, 3, page, 2, d)
        g = torch.Generator().manual_seed(which)
        rows = [torch.randn(n, 2, d, generator=g) for _ in range(2)]
        x = rows[which]
        if bad == "range":
            x[7, 0, 3], x[7, 0, 50] = 3e38, -3e38
        else:
            x[7, 0, 3] = float(bad)
        pq.pq_kv_append(cache, rows[0].to(DEV), rows[1].to(DEV), torch.arange(n, device=DEV))
        table, cu = torch.arange(3, dtype=torch.int32, device=DEV)[None], torch.tensor([0, n], dtype=torch.int32, device=DEV)
        back = [torch.empty(n, 2, d, device=DEV) for _ in range(2)]
        pq.pq_kv_load(cache, table, None, cu, *back)
        assert bool(back[which][7, 0].isnan().all()) and int(back[which].isnan().sum()) == d
        q = torch.randn(1, 32, d, generator=g).to(torch.bfloat16).to(DEV)
        out = torch.empty_like(q)
        pq.pq_attn_decode(cache, q, table, cu[1:], out)
        assert bool(out[0, :16].isnan().all()) and bool(out[0, 16:].isfinite().all())
