"""A gradient of pq_distill that is large enough to be written past the caches is that of its rows by themselves, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_amd import pq as _pq
    assert torch.cuda.is_available()
    return _pq


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,v", [(2200, 32000), (2200, 32005), (530, 140008)])
def test_past_the_caches(pq, rows, v, dtype):
    print(f"[distill past the caches {rows} {v} {dtype}]", flush=True)
    assert rows * v * 2 > 1 << 27
    g = torch.Generator(device=DEV).manual_seed(v)
    z = (torch.randn(rows, v, generator=g, device=DEV) * 3).to(dtype)
    index = torch.randint(0, v, (rows, 20), generator=g, device=DEV, dtype=torch.int32)
    top = torch.randn(rows, 20, generator=g, device=DEV)
    loss, stats, dz, dz2 = torch.empty(rows, device=DEV), torch.empty(rows, 2, device=DEV), torch.empty_like(z), torch.empty_like(z)
    one = torch.ones(rows, device=DEV)
    pq.pq_distill(z, index, top, loss, stats, dz, temperature=1.5)
    pq.pq_distill_bwd(z, index, top, stats, one, dz2, temperature=1.5)
    for a in range(0, rows, 300):
        b = slice(a, min(a + 300, rows))
        n = b.stop - a
        part, part2, only, st = torch.empty(n, v, dtype=dtype, device=DEV), torch.empty(n, v, dtype=dtype, device=DEV), \
            torch.empty(n, device=DEV), torch.empty(n, 2, device=DEV)
        pq.pq_distill(z[b], index[b], top[b], only, st, part, temperature=1.5)
        pq.pq_distill_bwd(z[b], index[b], top[b], st, one[b], part2, temperature=1.5)
        assert torch.equal(only, loss[b]) and torch.equal(st, stats[b])
        assert torch.equal(part, dz[b]) and torch.equal(part2, dz2[b])
