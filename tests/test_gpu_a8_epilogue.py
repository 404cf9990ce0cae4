"""pq_gemm_a8's epilogue in every kernel that ends with it (split K, 17 to 32 rows through the stream, small tiles)."""
import pytest
import torch

import layer_ref as R
from test_gpu_a8 import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_amd import pq as _pq
    assert torch.cuda.is_available()
    return _pq


# (mode, m, n, k, whether K is split)
SPLIT = [(0, 18, 90, 8192, True), (2, 40, 31, 8256, True), (2, 48, 96, 8192, True), (3, 33, 257, 16384, True), (4, 100, 64, 16448, True)]
STREAM = [(2, 20, 90, 320, False), (2, 32, 6300, 192, False), (4, 17, 6201, 320, False), (3, 31, 12400, 192, False), (0, 16, 70, 576, False)]
TILES = [(0, 20, 90, 320, False), (4, 40, 130, 448, False)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", range(5))
@pytest.mark.parametrize("mode,m,n,k,split", SPLIT + STREAM + TILES)
def test_epilogue(pq, mode, m, n, k, split, kind, dtype):
    """Bias, activation, both combinations, rows of wider arrays, in place."""
    print(f"[a8 epilogue {mode} {m} {n} {k} act={kind} {dtype}]", flush=True)
    need = pq.pq_gemm_a8_workspace_bytes(mode, m, n, k)
    assert (need > 0) == split                          # else this is a test of another kernel
    c = Case(mode, m, n, k, seed=8)
    bias = c.random(n, dtype=DTYPES[(kind + 1) % 3])
    wide = c.random(m, n + 9, dtype=dtype)
    other, before = wide[:, 4:4 + n], wide.clone()
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    for mul in (False, True):
        combine = pq.PQ_COMBINE_MUL if mul else pq.PQ_COMBINE_ADD
        y = torch.full((m, n + 5), 3.0, dtype=dtype, device=DEV)
        pq.pq_gemm_a8(mode, c.x, c.x_scale, c.packed, c.alpha, y[:, 3:3 + n], bias=bias, activation=kind, other=other, combine=combine,
                      workspace=ws)
        c.check(y[:, 3:3 + n], kind, bias, other, mul)
        assert bool((y[:, :3] == 3).all()) and bool((y[:, 3 + n:] == 3).all()) and bool((ws[need:] == 0x5A).all())
        assert torch.equal(wide, before)
        place = wide.clone()
        inner = place[:, 4:4 + n]
        pq.pq_gemm_a8(mode, c.x, c.x_scale, c.packed, c.alpha, inner, bias=bias, activation=kind, other=inner, combine=combine)
        assert torch.equal(inner, y[:, 3:3 + n])
        assert torch.equal(place[:, :4], before[:, :4]) and torch.equal(place[:, 4 + n:], before[:, 4 + n:])
    alone = torch.empty(m, n, dtype=dtype, device=DEV)
    pq.pq_gemm_a8(mode, c.x, c.x_scale, c.packed, c.alpha.float(), alone, activation=kind, workspace=ws)
    c.check(alone, kind)
