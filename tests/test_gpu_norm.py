"""pq_rmsnorm, pq_rmsnorm_bwd and pq_quantize_rows on the GPU against binary64."""
import pytest
import torch

import layer_ref as R
from gpu_util import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
# (rows, cols): every team and chunk count, ends inside a chunk, one element, rows past a grid of teams
SHAPES = [(1, 1), (1, 576), (3, 7), (5, 64), (2, 513), (7, 1000), (4, 1024), (3, 1025), (6, 2048), (2, 2049), (5, 4096), (3, 4100),
          (2, 6144), (3, 6145), (2, 8192), (2, 8193), (1, 16384), (2, 16385), (1, 32768), (2, 20001), (1031, 72), (4500, 64), (1500, 1200)]


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_amd import pq as _pq
    assert torch.cuda.is_available()
    return _pq


def make(shape, dtype, seed, spread=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g)
    if spread:
        x = x * torch.logspace(-2, 2, shape[0])[:, None]
    return x.to(dtype).to(DEV)


def within(got, want, lim, what):
    bad = ~((got.double() - want).abs() <= lim)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


# fp32 work: a sum of squares over a thread's (at most 64) values one after the other and ten joining steps, halved by the
# root, and some ten roundings beside it
FP32 = 2.0 ** -24 * (64 / 2 + 10 + 12)


def check_norm(y, h, w, eps, dtype):
    want, _ = R.norm(h, w, eps)
    within(y, want, (R.U[dtype] if dtype != torch.float32 else 0) * want.abs() + FP32 * want.abs() + R.TINY[dtype], "y")


def check_rows(q, scale, y, slack):
    """Codes and scales of rows y (f64), known to a relative error of slack each."""
    want = R.row_scale(y)
    within(scale, want, (slack + 2.0 ** -22) * want, "scale")
    # half a step, and what the error of quotients of up to 127 moves a border by
    within(q.double() * scale.double()[:, None], y, scale.double()[:, None] * (0.5 + 127 * 2 * (slack + 2.0 ** -22)) * torch.ones_like(y),
           "values")
    full = want > R.MIN_SCALE
    assert bool((q.abs().amax(-1)[full] == 127).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_norm(pq, shape, dtype):
    print(f"[norm {shape} {dtype}]", flush=True)
    rows, cols = shape
    x, r = make(shape, dtype, 1), make(shape, dtype, 2, False)
    w = (torch.rand(cols, generator=torch.Generator().manual_seed(3)) + 0.5).to(DEV)
    y, s, q = Guarded(shape, dtype), Guarded(shape, dtype), Guarded(shape, torch.int8)
    rstd, scale = Guarded((rows,), torch.float32), Guarded((rows,), torch.float32)
    pq.pq_rmsnorm(x, w, y=y.t, rstd=rstd.t, eps=1e-5)
    check_norm(y.t, x, w, 1e-5, dtype)
    want = R.norm(x, w, 1e-5)[1]
    within(rstd.t, want, FP32 * want, "rstd")
    wd = w.to(torch.bfloat16) if dtype == torch.float32 else w.to(dtype)
    pq.pq_rmsnorm(x, wd, residual=r, sum=s.t, q=q.t, scale=scale.t, eps=1e-5)
    h = (x.float() + r.float()).to(dtype)
    assert torch.equal(s.t, h)
    check_rows(q.t, scale.t, R.norm(h, wd, 1e-5)[0], FP32)
    for g, what in ((y, "y"), (s, "sum"), (q, "q"), (rstd, "rstd"), (scale, "scale")):
        g.check(what)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES + [(2, 40000), (1, 65536), (3, 65535)])
def test_rows(pq, shape, dtype):
    print(f"[rows {shape} {dtype}]", flush=True)
    x = make(shape, dtype, 4)
    q, scale = Guarded(shape, torch.int8), Guarded((shape[0],), torch.float32)
    pq.pq_quantize_rows(x, q.t, scale.t)
    check_rows(q.t, scale.t, x.double(), 0.0)
    q.check("q")
    scale.check("scale")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_norm_bwd(pq, shape, dtype):
    print(f"[norm_bwd {shape} {dtype}]", flush=True)
    rows, cols = shape
    h, dy, ds = make(shape, dtype, 5), make(shape, dtype, 6, False), make(shape, dtype, 7, False)
    w = (torch.rand(cols, generator=torch.Generator().manual_seed(8)) + 0.5).to(DEV)
    rstd = R.norm(h, w, 1e-5)[1].float()
    dx, dw = Guarded(shape, dtype), Guarded((cols,), torch.float32)
    for more in (None, ds):
        pq.pq_rmsnorm_bwd(h, w, rstd, dy, dx.t, dsum=more, dweight=dw.t)
        want, dwant, size, dsize = R.norm_grad(h, w, rstd, dy, more)
        # the row's sum: 64 values one after the other, ten joining steps, a dozen roundings around it
        within(dx.t, want, (R.U[dtype] if dtype != torch.float32 else 0) * want.abs() + 2.0 ** -24 * 86 * size + R.TINY[dtype], "dx")
        # at most 9 rows a team here, 4096 / 16 teams one after the other, 16 joined
        within(dw.t, dwant, 2.0 ** -24 * (9 + 256 + 16 + 4) * dsize, "dweight")
    dx.check("dx")
    dw.check("dweight")


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_and_places(pq, dtype):
    """Rows of a wider array at an odd offset, sum over the residual, y over x, dx over dy and dsum."""
    rows, cols, w = 37, 203, (torch.rand(203, generator=torch.Generator().manual_seed(9)) + 0.5).to(DEV)
    wide = make((rows, 411), dtype, 10)
    before = wide.clone()
    x, r = wide[:, 5:208], make((rows, 300), dtype, 11)[:, 1:204]
    h = (x.float() + r.float()).to(dtype)
    q = torch.zeros(rows, 301, dtype=torch.int8, device=DEV)
    scale = torch.empty(rows, device=DEV)
    pq.pq_rmsnorm(x, w, residual=r, sum=r, q=q[:, 3:206], scale=scale)
    assert torch.equal(r, h) and torch.equal(wide, before)
    check_rows(q[:, 3:206], scale, R.norm(h, w, 1e-6)[0], FP32)
    assert torch.count_nonzero(q[:, :3]) == 0 and torch.count_nonzero(q[:, 206:]) == 0
    want = R.norm(x, w, 1e-6)[0]
    old = x.clone()
    pq.pq_rmsnorm(x, w, y=x)
    check_norm(x, old, w, 1e-6, dtype)
    assert torch.equal(wide[:, :5], before[:, :5]) and torch.equal(wide[:, 208:], before[:, 208:]) and want.shape == x.shape
    rstd = R.norm(h, w, 1e-6)[1].float()
    dy, ds = make((rows, 411), dtype, 12)[:, 7:210], make((rows, cols), dtype, 13)
    fresh = torch.empty(rows, cols, dtype=dtype, device=DEV)
    pq.pq_rmsnorm_bwd(h, w, rstd, dy, fresh, dsum=ds)
    for place in ("dy", "dsum"):
        a, b = make((rows, 411), dtype, 12)[:, 7:210], ds.clone()
        pq.pq_rmsnorm_bwd(h, w, rstd, a, a if place == "dy" else b, dsum=b)
        assert torch.equal(a if place == "dy" else b, fresh), place


def test_edges_of_rows(pq):
    """Rows of zeros, of one value, of the type's ends, of what is no number."""
    x = torch.zeros(8, 96, device=DEV)
    x[1] = 3.0
    x[2, 5] = -7.0
    x[3] = 2.0 ** -100
    x[4, 0] = float("inf")
    x[5, 95] = float("nan")
    x[6] = torch.linspace(-3e38, 3e38, 96, dtype=torch.float64)      # in fp32 the range itself is infinite
    x[7, 1] = float("-inf")
    q, scale = torch.empty(8, 96, dtype=torch.int8, device=DEV), torch.empty(8, device=DEV)
    pq.pq_quantize_rows(x, q, scale)
    assert torch.count_nonzero(q[0]) == 0 and float(scale[0]) == R.MIN_SCALE
    assert bool((q[1] == 127).all()) and int(q[2, 5]) == -127 and int(q[2].abs().sum()) == 127
    assert torch.count_nonzero(q[3]) == 0 and float(scale[3]) == R.MIN_SCALE
    assert bool(scale[[4, 5, 7]].isnan().all()) and int(q[6, 0]) == -127 and int(q[6, 95]) == 127
    w, y, rstd = torch.ones(96, device=DEV), torch.empty(8, 96, device=DEV), torch.empty(8, device=DEV)
    pq.pq_rmsnorm(x, w, y=y, rstd=rstd, eps=1e-6)
    assert torch.count_nonzero(y[0]) == 0 and abs(float(rstd[0]) - 1000.0) < 1e-3
    assert bool(y[5].isnan().all()) and bool(y[4, 0].isnan()) and bool(y[7, 1].isnan())
    pq.pq_rmsnorm(x, w, q=q, scale=scale, eps=1e-6)
    assert torch.count_nonzero(q[0]) == 0 and bool(scale[[4, 5, 7]].isnan().all()) and bool(scale[:4].isfinite().all())


def test_empty_and_repeatable(pq):
    w = torch.ones(64, device=DEV)
    e = torch.empty(0, 64, device=DEV)
    pq.pq_rmsnorm(e, w, y=e)
    pq.pq_quantize_rows(e, e.to(torch.int8), torch.empty(0, device=DEV))
    dw = torch.full((64,), 3.0, device=DEV)
    pq.pq_rmsnorm_bwd(e, w, torch.empty(0, device=DEV), e, e, dweight=dw)
    assert torch.count_nonzero(dw) == 0                    # a sum over no rows
    h, dy = make((5000, 640), torch.bfloat16, 20), make((5000, 640), torch.bfloat16, 21)
    w, rstd = torch.ones(640, device=DEV), torch.rand(5000, device=DEV)
    got = []
    for _ in range(3):
        dx, dw = torch.empty_like(h), torch.empty(640, device=DEV)
        pq.pq_rmsnorm_bwd(h, w, rstd, dy, dx, dweight=dw)
        got.append((dx, dw))
    assert all(torch.equal(a, got[0][0]) and torch.equal(b, got[0][1]) for a, b in got)


def test_gradient_against_differences(pq):
    """dx and dweight along a direction, against differences of the forward call (both in fp32: the step balances them)."""
    rows, cols = 64, 320
    x, dy, d = (make((rows, cols), torch.float32, s, False) for s in (30, 31, 32))
    w, v = (torch.rand(cols, generator=torch.Generator().manual_seed(s)).to(DEV) + 0.5 for s in (33, 34))
    y, rstd, dx, dw = torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty_like(x), torch.empty(cols, device=DEV)
    pq.pq_rmsnorm(x, w, y=y, rstd=rstd)
    pq.pq_rmsnorm_bwd(x, w, rstd, dy, dx, dweight=dw)
    e = 2.0 ** -7

    def f(x, w):
        pq.pq_rmsnorm(x, w, y=y)
        return (y.double() * dy.double()).sum()
    slope = (f(x + e * d, w + e * v) - f(x - e * d, w - e * v)) / (2 * e)
    want = (dx.double() * d.double()).sum() + (dw.double() * v.double()).sum()
    # third derivative: e^2 / 6 of terms of size |dy| |d|^3; rounding: 2^-23 |y| |dy| / e, both over 20480 values in quadrature
    assert abs(float(slope - want)) < 20480 ** 0.5 * (e * e * 4 + 2.0 ** -22 * 3 / e)


def test_more_rows_than_a_launch(pq):
    """Rows past 2^21, which go in a second launch."""
    rows, cols = (1 << 21) + 5, 8
    x = torch.randn(rows, cols, device=DEV, dtype=torch.float32).to(torch.bfloat16)
    w, q, scale, rstd = torch.ones(cols, device=DEV), torch.empty(rows, cols, dtype=torch.int8, device=DEV), \
        torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    s = torch.empty_like(x)
    pq.pq_rmsnorm(x, w, residual=x, sum=s, q=q, scale=scale, rstd=rstd)
    assert torch.equal(s, x + x)
    check_rows(q, scale, R.norm(s, w, 1e-6)[0], FP32)
    want = R.norm(s, w, 1e-6)[1]
    within(rstd, want, FP32 * want, "rstd")
    pq.pq_quantize_rows(x, q, scale)
    check_rows(q, scale, x.double(), 0.0)
    dx, dw = torch.empty_like(x), torch.empty(cols, device=DEV)
    pq.pq_rmsnorm_bwd(x, w, rstd, s, dx, dweight=dw)
    dxw, dww, size, dsize = R.norm_grad(x, w, rstd, s)
    within(dx, dxw, R.U[x.dtype] * dxw.abs() + 2.0 ** -24 * 86 * size + R.TINY[x.dtype], "dx")
    # 512 rows one after the other in each of 4096 waves, then 16 and 64 sums
    within(dw, dww, 2.0 ** -24 * (512 + 96) * dsize, "dweight")
