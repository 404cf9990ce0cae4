"""pq_rope_table and pq_rope on the GPU against binary64."""
import numpy as np
import pytest
import torch

import serving_ref as R
from gpu_util import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_amd import pq as _pq
    assert torch.cuda.is_available()
    return _pq


@pytest.mark.parametrize("kind,factor,trained", [("plain", 1.0, 0), ("linear", 4.0, 0), ("ntk", 8.0, 0),
                                                 ("yarn", 16.0, 4096), ("bands", 8.0, 8192)])
@pytest.mark.parametrize("rot,base,rows", [(64, 10000.0, 4097), (128, 500000.0, 300), (6, 10000.0, 33)])
def test_table(pq, kind, factor, trained, rot, base, rows):
    k = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}[kind]
    s = pq.rope_scaling(k, factor, trained) if k else None
    got = pq.pq_rope_table(rows, rot, base, scaling=s).cpu().double().numpy()
    f, m = R.rope_freqs(rot, base, kind, factor, trained, 4.0 if kind == "bands" else 32.0, 1.0)
    ang = np.arange(rows)[:, None] * f
    want = m * np.stack([np.cos(ang), np.sin(ang)], -1)
    # one rounding to binary32; the angles' own binary64 error is 4097 * 2^-50
    assert np.all(np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 1e-10)


def table_of(rot, rows, seed=0):
    """Angles without structure, so that a wrong row or pair shows."""
    g = torch.Generator().manual_seed(seed)
    a = torch.rand(rows, rot // 2, dtype=torch.float64, generator=g) * 6.28
    return torch.stack([a.cos(), a.sin()], -1).float()


def check(got, x, want, dtype):
    """|got - want| <= the type's rounding of the result and three binary32 roundings of terms of |x1| + |x2|."""
    scale = x.double().abs().amax(-1, keepdim=True) * 2
    lim = (R.U[dtype] if dtype != torch.float32 else 0) * want.abs() + 3 * 2.0 ** -24 * scale + R.TINY[dtype]
    bad = ~((got.double() - want).abs() <= lim)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


SHAPES = [(1, 12, 64, 64), (5, 3, 128, 128), (33, 40, 128, 128), (3, 25, 80, 40), (7, 5, 80, 80), (2, 1, 96, 48), (4, 2, 256, 256),
          (3, 2, 20, 6), (5, 3, 17, 10), (2, 2, 1024, 1024), (2, 3, 300, 300), (3, 1, 32, 0), (300, 2, 16, 16), (2, 70, 40, 24)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_rope(pq, shape, half, dtype):
    n, h, d, rot = shape
    print(f"[rope {shape} half={half} {dtype}]", flush=True)
    g = torch.Generator().manual_seed(n + d)
    x = torch.randn(n, h, d, generator=g).to(dtype)
    table = table_of(rot, 50)
    pos = torch.randint(0, 50, (n,), generator=g, dtype=torch.int32)
    layout = pq.PQ_ROPE_HALF if half else pq.PQ_ROPE_INTERLEAVED
    xd, td, pd = x.to(DEV), table.to(DEV), pos.to(DEV)
    for inverse in (False, True):
        y = Guarded((n, h, d), dtype)
        pq.pq_rope(xd, pd, td, y.t, layout=layout, inverse=inverse)
        torch.cuda.synchronize()
        y.check("y")
        check(y.t.cpu(), x, R.rope(x.double(), table, pos, half, inverse), dtype)
        z = Guarded((n, h, d), dtype)
        z.t.copy_(xd)
        pq.pq_rope(z.t, pd, td, layout=layout, inverse=inverse)        # in place
        torch.cuda.synchronize()
        z.check("in place")
        assert torch.equal(z.t, y.t)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("offset,pad", [(0, 8), (0, 4), (1, 3), (4, 12)])
def test_rope_strided_and_unaligned(pq, half, offset, pad):
    """Heads of a fused buffer, at element offsets that allow vectors of 8, of 4 and none."""
    n, h, d = 6, 3, 64
    g = torch.Generator().manual_seed(9)
    buf = torch.randn(n * (h * (d + pad)) + offset + 64, generator=g).to(torch.bfloat16).to(DEV)
    view = buf[offset:offset + n * h * (d + pad)].view(n, h, d + pad)[..., :d]
    before, table = buf.clone(), table_of(d, 20)
    pos = torch.tensor([0, 19, 7, 3, 3, 11], dtype=torch.int32)
    want = R.rope(view.cpu().double(), table, pos, half)
    x = view.cpu().clone()
    layout = pq.PQ_ROPE_HALF if half else pq.PQ_ROPE_INTERLEAVED
    y = torch.zeros(h, n, d, dtype=torch.bfloat16, device=DEV).transpose(0, 1)     # heads outermost
    pq.pq_rope(view, pos.to(DEV), table.to(DEV), y, layout=layout)
    check(y.cpu(), x, want, torch.bfloat16)
    pq.pq_rope(view, pos.to(DEV), table.to(DEV), layout=layout)
    check(view.cpu(), x, want, torch.bfloat16)
    view.copy_(x)
    assert torch.equal(buf, before)                 # nothing between the heads was written


def test_rope_positions_outside_the_table(pq):
    x = torch.randn(4, 2, 64).to(torch.bfloat16)
    table = table_of(32, 5)
    pos = torch.tensor([-1, 4, 5, -2 ** 31], dtype=torch.int32)
    y = torch.empty_like(x, device=DEV)
    pq.pq_rope(x.to(DEV), pos.to(DEV), table.to(DEV), y)
    y = y.cpu()
    assert torch.equal(y[0], x[0]) and torch.equal(y[3], x[3])
    assert bool(y[2, :, :32].isnan().all()) and torch.equal(y[2, :, 32:], x[2, :, 32:])
    assert not bool(y[1].isnan().any())


def test_rope_special_values_are_copied_bit_for_bit(pq):
    """Channels past `rot` and rows of padding keep their bits, NaN and infinities included."""
    x = torch.randn(2, 1, 64)
    x[0, 0, 40:44] = torch.tensor([float("nan"), float("inf"), -0.0, 1e-42])
    x[1] = x[0].flip(-1)
    y = torch.empty_like(x, device=DEV)
    pq.pq_rope(x.to(DEV), torch.tensor([1, -1], dtype=torch.int32, device=DEV), table_of(32, 4).to(DEV), y)
    got = y.cpu().view(torch.int32)
    assert torch.equal(got[0, :, 32:], x.view(torch.int32)[0, :, 32:]) and torch.equal(got[1], x.view(torch.int32)[1])


@pytest.mark.parametrize("half", [True, False])
def test_gradient(pq, half):
    """The inverse call is the gradient: <dy, R x> = <R^T dy, x>, by the formula and by differences of sum(w * R x)."""
    n, h, d, rot = 4, 2, 48, 32
    g = torch.Generator().manual_seed(4)
    x, w, e = (torch.randn(n, h, d, generator=g).to(DEV) for _ in range(3))
    table = (table_of(rot, 9) * 1.25).to(DEV)       # with a magnitude: the transpose is not the inverse
    pos = torch.tensor([0, 8, 3, 5], dtype=torch.int32, device=DEV)
    layout = pq.PQ_ROPE_HALF if half else pq.PQ_ROPE_INTERLEAVED

    def fwd(v):
        y = torch.empty_like(v)
        pq.pq_rope(v, pos, table, y, layout=layout)
        return y.double()
    grad = torch.empty_like(w)
    pq.pq_rope(w, pos, table, grad, layout=layout, inverse=True)
    xa = x.cpu().double().requires_grad_(True)
    R_x = [R.rope(xa[i:i + 1], table.cpu(), pos.cpu()[i:i + 1], half) for i in range(n)]
    (torch.cat(R_x) * w.cpu().double()).sum().backward()
    assert torch.allclose(grad.cpu().double(), xa.grad, rtol=0, atol=3 * 2.0 ** -24 * 2.5 * float(w.abs().max()))
    diff = ((fwd(x + e) - fwd(x - e)) / 2 * w.double()).sum()
    # the map is linear: the difference quotient is exact but for the roundings of x +- e and R
    bound = 2.0 ** -22 * float((w.abs() * 2.5 * (x.abs() + e.abs()).amax()).double().sum())
    assert abs(float(diff - (grad.double() * e.double()).sum())) <= bound


def test_rope_long_positions_and_offsets_past_32_bits(pq):
    """Rows 2^31 elements apart, and a table row far down."""
    n, h, d = 2, 1, 16
    big = torch.empty((1 << 31) + 64, dtype=torch.bfloat16, device=DEV)
    x = torch.as_strided(big, (n, h, d), ((1 << 31) + 16, 16, 1))
    src = torch.randn(n, h, d).to(torch.bfloat16)
    x.copy_(src)
    table = torch.empty(1 << 20, 8, 2, device=DEV)
    t = table_of(16, 3)
    table[-1], table[0] = t[0], t[1]
    pos = torch.tensor([(1 << 20) - 1, 0], dtype=torch.int32, device=DEV)
    pq.pq_rope(x, pos, table)
    check(x.cpu(), src, R.rope(src.double(), t, torch.tensor([0, 1]), True), torch.bfloat16)


def test_rope_other_stream(pq):
    x = torch.randn(64, 8, 128, dtype=torch.bfloat16, device=DEV)
    table, pos = table_of(128, 64).to(DEV), torch.arange(64, dtype=torch.int32, device=DEV)
    want = torch.empty_like(x)
    pq.pq_rope(x, pos, table, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(x)
    side.wait_stream(torch.cuda.current_stream())
    pq.pq_rope(x, pos, table, y, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
