"""Strides of 0 (an input that is the same row for all) and below 0 (rows from the last to the first) around the packed product."""
import ctypes

import pytest
import torch

from test_gpu_a8 import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_amd import pq as _pq
    assert torch.cuda.is_available()
    return _pq


def last(t):
    """Address of the last row and the stride that walks back from it."""
    return t[-1].data_ptr(), -t.stride(0)


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("rows,cols", [(5, 70), (9, 1500), (3, 9000)])
def test_norm(pq, rows, cols):
    g = torch.Generator().manual_seed(cols)
    x, r, dy = (torch.randn(rows, cols, generator=g).to(torch.bfloat16).to(DEV) for _ in range(3))
    w = (torch.rand(cols, generator=g) + 0.5).to(DEV)
    new = torch.empty_like
    # the same row for all
    same, s, q, scale = x[:1].expand(rows, cols), new(x), torch.empty(rows, cols, dtype=torch.int8, device=DEV), torch.empty(rows, device=DEV)
    s2, q2, scale2 = new(s), new(q), new(scale)
    pq.pq_rmsnorm(same, w, residual=r, sum=s, q=q, scale=scale)
    pq.pq_rmsnorm(same.contiguous(), w, residual=r, sum=s2, q=q2, scale=scale2)
    assert torch.equal(s, s2) and torch.equal(q, q2) and torch.equal(scale, scale2)
    # all rows backwards, inputs and outputs
    bf = pq.PQ_BF16
    assert pq.lib.pq_rmsnorm(bf, rows, cols, *last(x), *last(r), *last(s2), w.data_ptr(), pq.PQ_F32, 1e-6, None, 0, *last(q2),
                             scale2.data_ptr(), None, stream()) == 0
    pq.pq_rmsnorm(x, w, residual=r, sum=s, q=q, scale=scale)
    assert torch.equal(s, s2) and torch.equal(q, q2) and torch.equal(scale.flip(0), scale2)
    assert pq.lib.pq_quantize_rows(bf, rows, cols, *last(x), *last(q2), scale2.data_ptr(), stream()) == 0
    pq.pq_quantize_rows(x, q, scale)
    assert torch.equal(q, q2) and torch.equal(scale.flip(0), scale2)
    rstd, dx, dx2, dw = torch.rand(rows, device=DEV), new(x), new(x), torch.empty(cols, device=DEV)
    back = rstd.flip(0).contiguous()
    pq.pq_rmsnorm_bwd(x, w, rstd, dy, dx, dsum=same, dweight=dw)
    assert pq.lib.pq_rmsnorm_bwd(bf, rows, cols, *last(x), w.data_ptr(), pq.PQ_F32, back.data_ptr(), *last(dy), same.data_ptr(), 0,
                                 *last(dx2), None, None, 0, stream()) == 0
    assert torch.equal(dx, dx2)


@pytest.mark.parametrize("m,n,k", [(5, 70, 320), (30, 70, 320), (40, 31, 8256), (300, 600, 576), (2100, 2500, 192)])
def test_product(pq, m, n, k):
    c = Case(2, m, n, k, seed=9)
    row = c.random(1, n, dtype=torch.bfloat16)
    y, y2 = torch.empty(m, n, dtype=torch.bfloat16, device=DEV), torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    pq.pq_gemm_a8(2, c.x, c.x_scale, c.packed, c.alpha, y, other=row.expand(m, n), combine=pq.PQ_COMBINE_MUL)
    c.check(y, other=row.expand(m, n), mul=True)
    other = c.random(m, n, dtype=torch.bfloat16)
    pq.pq_gemm_a8(2, c.x, c.x_scale, c.packed, c.alpha, y, other=other)
    e = pq.pq_epilogue()
    kept = other.flip(0).contiguous()
    e.other, e.other_stride = last(kept)
    need = pq.pq_gemm_a8_workspace_bytes(2, m, n, k)
    ws = torch.empty(need + 16, dtype=torch.uint8, device=DEV)
    assert pq.lib.pq_gemm_a8(2, m, n, k, c.x.data_ptr(), k, c.x_scale.data_ptr(), c.packed.data_ptr(), c.alpha.data_ptr(), pq.PQ_BF16,
                             ctypes.addressof(e), pq.PQ_BF16, *last(y2), ws.data_ptr(), need, stream()) == 0
    assert torch.equal(y2.flip(0), y)


@pytest.mark.parametrize("v", [300, 9001, 70000])
def test_distill(pq, v):
    rows, k = 4, 6
    g = torch.Generator().manual_seed(v)
    z = torch.randn(rows, v, generator=g).to(torch.bfloat16).to(DEV)
    index = torch.randint(0, v, (rows, k), generator=g).to(torch.int32).to(DEV)
    top = torch.randn(rows, k, generator=g).to(DEV)
    loss, loss2, stats, dz, dz2 = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV), torch.empty(rows, 2, device=DEV), \
        torch.empty_like(z), torch.empty_like(z)
    same = z[:1].expand(rows, v)
    pq.pq_distill(same, index, top, loss, stats, dz)
    pq.pq_distill(same.contiguous(), index, top, loss2, stats, dz2)
    assert torch.equal(loss, loss2) and torch.equal(dz, dz2)
    one = torch.ones(rows, device=DEV)
    pq.pq_distill_bwd(same, index, top, stats, one, dz)
    pq.pq_distill_bwd(same.contiguous(), index, top, stats, one, dz2)
    assert torch.equal(dz, dz2)
    pq.pq_distill(z, index, top, loss, stats, dz)
    i2, t2, bf = index.flip(0).contiguous(), top.flip(0).contiguous(), pq.PQ_BF16
    assert pq.lib.pq_distill(bf, rows, v, *last(z), k, i2.data_ptr(), t2.data_ptr(), pq.PQ_F32, 1.0, None, loss2.data_ptr(), None, 1.0,
                             *last(dz2), stream()) == 0
    assert torch.equal(loss2.flip(0), loss) and torch.equal(dz2, dz)
    back = stats.flip(0).contiguous()
    pq.pq_distill_bwd(z, index, top, stats, one, dz)
    assert pq.lib.pq_distill_bwd(bf, rows, v, *last(z), k, i2.data_ptr(), t2.data_ptr(), pq.PQ_F32, 1.0, None, back.data_ptr(),
                                 one.data_ptr(), *last(dz2), stream()) == 0
    assert torch.equal(dz2, dz)
