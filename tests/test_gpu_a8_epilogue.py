"""pq_gemm_a8's epilogue in every kernel that ends with it (split K, 17 to 32 rows through the stream, small tiles), and its
activations where they are small."""
import math

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


@pytest.mark.parametrize("kind", [2, 3, 4])
@pytest.mark.parametrize("m", [1, 200])
def test_activations_keep_their_small_values(pq, kind, m):
    """Far on the negative side an activation is tiny; it is so to a few units of its own last place there too.

    One column of weights of +1 and one activation a row that is not 0, so that v = x_scale is exact."""
    n, k = 16, 64
    v = -torch.logspace(-6, 1.1, 997, dtype=torch.float64) if kind == 3 else -torch.logspace(-6, 1.9, 997, dtype=torch.float64)
    if kind == 4:
        v = v[v > -9]
    v = torch.cat([v, -v]).float()
    codes = torch.ones(n, k, dtype=torch.uint8)
    packed = R.pack(codes, 1).to(DEV)                   # binary: code 1 is +1
    x = torch.zeros(m, k, dtype=torch.int8)
    x[:, 0] = 1
    x, alpha = x.to(DEV), torch.ones(n, device=DEV)
    for a in range(0, len(v), m):
        s = v[a:a + m]
        if len(s) < m:
            break
        y = torch.empty(m, n, device=DEV)
        pq.pq_gemm_a8(0, x, s.to(DEV), packed, alpha, y, activation=kind)
        t = s.double().to(DEV)[:, None]
        want = R.act(t, kind).expand(m, n)
        # e^u: u (|v|, v^2 / 2 or 2 sqrt(2 / pi) (|v| + 0.044715 |v|^3), of at most six roundings), log2 e and the product of both
        # are rounded; a dozen units for the rest
        u = t.abs() if kind == 2 else t * t / 2 if kind == 3 else 1.6 * (t.abs() + 0.044715 * t.abs() ** 3)
        lim = 2.0 ** -24 * (12 + 9 * u) * want.abs() + 2.0 ** -126
        bad = ~((y.double() - want).abs() <= lim)
        assert not bool(bad.any()), (float(t[bad.nonzero()[0][0]]), y[bad][0].item(), want[bad][0].item())


def test_activations_of_infinity(pq):
    """+inf stays, under every activation."""
    codes, x = torch.ones(16, 64, dtype=torch.uint8), torch.ones(3, 64, dtype=torch.int8, device=DEV)
    packed, y = R.pack(codes, 1).to(DEV), torch.empty(3, 16, device=DEV)
    bias = torch.full((16,), math.inf, device=DEV)
    for kind in range(5):
        pq.pq_gemm_a8(0, x, torch.ones(3, device=DEV), packed, torch.ones(16, device=DEV), y, bias=bias, activation=kind)
        assert bool((y == math.inf).all()), kind
        big = torch.full((16,), 2e38, device=DEV)       # squares past the range
        pq.pq_gemm_a8(0, x, torch.ones(3, device=DEV), packed, torch.ones(16, device=DEV), y, bias=big, activation=kind)
        assert bool((y == 2e38).all()), kind
        pq.pq_gemm_a8(0, x, torch.ones(3, device=DEV), packed, torch.ones(16, device=DEV), y, bias=-big, activation=kind)
        assert bool((y == (-2e38 if kind == 0 else 0.0)).all()), kind
