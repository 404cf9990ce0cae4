"""Words that a teacher's list of pq_distill names more than once: the gradient's sum over them at every size, the loss by entries."""
import math

import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_amd import pq as _pq
    assert torch.cuda.is_available()
    return _pq


@pytest.mark.parametrize("temp", [1.0, 0.25])
@pytest.mark.parametrize("times", [2, 3, 300])
def test_small_sums(pq, times, temp):
    """A word named again and again with next to no weight: its gradient is as near to the formula as any other."""
    depths = [0, 5, 10, 15, 20, 25, 30, 35, 40]                 # p = e^-depth an entry
    rows, v, k = len(depths), 4000, times + 1
    g = torch.Generator().manual_seed(times)
    z = torch.randn(rows, v, generator=g)
    index = torch.full((rows, k), 1234, dtype=torch.int32)
    index[:, 0] = 77
    z[:, 1234] = -60.0 * temp                                   # q is e^-60 there: the gradient is the teacher's alone
    top = torch.zeros(rows, k)
    top[:, 1:] = -torch.tensor(depths, dtype=torch.float32)[:, None] * temp
    top[:, 2::3] -= 0.5 * temp                                  # entries of two sizes
    z, index, top = z.to(DEV), index.to(DEV), top.to(DEV)
    loss, stats, dz, dz2 = torch.empty(rows, device=DEV), torch.empty(rows, 2, device=DEV), torch.empty_like(z), torch.empty_like(z)
    pq.pq_distill(z, index, top, loss, stats, dz, temperature=temp)
    pq.pq_distill_bwd(z, index, top, stats, torch.ones(rows, device=DEV), dz2, temperature=temp)
    _, want, p, q = R.distill(z, index, top, temp)
    # exponents of up to 58 (86 where q is, e^-20 of p): two roundings each, times ln 2: 2^-17.7; a few more for sums and products
    for got in (dz, dz2):
        bad = ~((got.double() - want).abs() <= temp * (p + q) * 2.0 ** -17)
        assert not bool(bad.any()), (bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item())
    again = torch.empty_like(z)
    pq.pq_distill(z, index, top, dlogits=again, temperature=temp)
    assert torch.equal(again, dz)


@pytest.mark.parametrize("k", [1, 2, 40])
def test_loss_counts_entries(pq, k):
    """One word k times: every entry has p = 1 / k, so the loss is T^2 (-ln k - ln q); the gradient's p is 1."""
    z = torch.randn(3, 500, generator=torch.Generator().manual_seed(k)).to(DEV)
    index, top = torch.full((3, k), 9, dtype=torch.int32, device=DEV), torch.full((3, k), 2.5, device=DEV)
    loss, dz = torch.empty(3, device=DEV), torch.empty_like(z)
    pq.pq_distill(z, index, top, loss, dlogits=dz, temperature=2.0)
    log_q = torch.log_softmax(z.double() / 2, -1)
    want = 4 * (-math.log(k) - log_q[:, 9])
    assert bool(((loss.double() - want).abs() <= 4 * 2.0 ** -18 * (1 + math.log(k) + log_q[:, 9].abs())).all())
    p = torch.zeros_like(log_q)
    p[:, 9] = 1
    assert bool(((dz.double() - 2 * (log_q.exp() - p)).abs() <= 2 * (p + log_q.exp()) * 2.0 ** -17).all())
