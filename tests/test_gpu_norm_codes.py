"""The 8-bit output of pq_rmsnorm is that of its y, bit for bit, also where h weight overflows; weights of every type in its gradient."""
import pytest
import torch

import layer_ref as R
from gpu_util import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
# every team and number of chunks, ends inside a chunk
SHAPES = [(1, 1), (5, 64), (300, 576), (7, 1000), (40, 2048), (33, 4100), (9, 6144), (6, 8192), (5, 16384), (3, 20001), (2, 32768)]


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_amd import pq as _pq
    assert torch.cuda.is_available()
    return _pq


def rows8(y):
    """Codes and scales of fp32 rows by the header's formulas, in fp32 on the CPU."""
    y = y.cpu()
    scale = (y.abs().amax(-1) * torch.tensor(1 / 127, dtype=torch.float32)).clamp_min(R.MIN_SCALE)
    return torch.round(y * (1.0 / scale)[:, None]).to(torch.int8), scale


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_codes_are_those_of_y(pq, shape, dtype):
    print(f"[norm codes {shape} {dtype}]", flush=True)
    rows, cols = shape
    g = torch.Generator().manual_seed(rows + cols)
    x, r = ((torch.randn(rows, cols, generator=g) * torch.logspace(-2, 2, rows)[:, None]).to(dtype).to(DEV) for _ in range(2))
    w = (torch.rand(cols, generator=g) + 0.5).to(dtype).to(DEV)
    h, q, scale, rstd = torch.empty_like(x), Guarded(shape, torch.int8), Guarded((rows,), torch.float32), torch.empty(rows, device=DEV)
    pq.pq_rmsnorm(x, w, residual=r, sum=h, q=q.t, scale=scale.t, rstd=rstd, eps=1e-5)
    y, same = torch.empty(rows, cols, device=DEV), torch.empty(rows, device=DEV)
    pq.pq_rmsnorm(h.float(), w, y=y, rstd=same, eps=1e-5)              # y before its rounding to the type
    assert torch.equal(rstd, same)
    want, swant = rows8(y)
    assert torch.equal(scale.t.cpu(), swant) and torch.equal(q.t.cpu(), want)
    q.check("q")
    scale.check("scale")


@pytest.mark.parametrize("cols", [64, 576, 4096, 16384])
def test_products_past_the_range(pq, cols):
    """h weight is infinite where y is not: rows of a norm without end (y is 0) and rows whose y is finite."""
    x, w = torch.zeros(4, cols, device=DEV), torch.full((cols,), 1.5, device=DEV)
    x[0] = 3e38                     # squares past the range: rstd and y are 0
    x[1, ::2], x[1, 1::2] = -3e38, 2e38
    x[2, 5], w[5] = 1e19, 1e20      # one square of 1e38: y = sqrt(cols) 1e20
    x[3] = 2.0
    q, scale, y = torch.empty(4, cols, dtype=torch.int8, device=DEV), torch.empty(4, device=DEV), torch.empty(4, cols, device=DEV)
    pq.pq_rmsnorm(x, w, q=q, scale=scale)
    pq.pq_rmsnorm(x, w, y=y)
    assert torch.count_nonzero(y[:2]) == 0 and torch.count_nonzero(q[:2]) == 0 and bool((scale[:2] == R.MIN_SCALE).all())
    want = cols ** 0.5 * 1e20 / 127
    assert abs(float(scale[2]) - want) < 1e-5 * want and int(q[2, 5]) == 127 and torch.count_nonzero(q[2]) == 1
    codes, s = rows8(y)
    assert torch.equal(q.cpu(), codes) and torch.equal(scale.cpu(), s)
    w[7] = float("inf")             # a y that is infinite or no number has no scale
    pq.pq_rmsnorm(x, w, q=q, scale=scale)
    assert bool(scale.isnan().all())


@pytest.mark.parametrize("w_dtype", DTYPES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(3, 7), (70, 576), (9, 1025), (40, 4096), (5, 8192), (7, 16384), (3, 20001), (3, 32768)])
def test_gradient_with_every_weight(pq, shape, dtype, w_dtype):
    print(f"[norm bwd weights {shape} {dtype} {w_dtype}]", flush=True)
    rows, cols = shape
    g = torch.Generator().manual_seed(rows + cols)
    h, dy, ds = (torch.randn(rows, cols, generator=g).to(dtype).to(DEV) for _ in range(3))
    w = (torch.rand(cols, generator=g) + 0.5).to(w_dtype).to(DEV)
    rstd = R.norm(h, w, 1e-5)[1].float()
    dx, dw = Guarded(shape, dtype), Guarded((cols,), torch.float32)
    pq.pq_rmsnorm_bwd(h, w, rstd, dy, dx.t, dsum=ds, dweight=dw.t)
    want, dwant, size, dsize = R.norm_grad(h, w, rstd, dy, ds)
    # the row's sum: at most 32 values a thread one after the other and 22 joining steps, a dozen roundings around it
    u = R.U[dtype] if dtype != torch.float32 else 0.0
    assert bool(((dx.t.double() - want).abs() <= u * want.abs() + 2.0 ** -24 * 86 * size + R.TINY[dtype]).all())
    # a row a team, joined by fours, then by at most 16 and 64 partial sums, with a dozen roundings beside
    assert bool(((dw.t.double() - dwant).abs() <= 2.0 ** -24 * 96 * dsize).all())
    dx.check("dx")
    dw.check("dweight")
