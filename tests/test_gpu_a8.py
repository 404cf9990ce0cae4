"""pq_gemm_a8 on the GPU against binary64: the sums are exact, so only scales, epilogue and the last rounding differ."""
import pytest
import torch

import layer_ref as R
from gpu_util import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_amd import pq as _pq
    assert torch.cuda.is_available()
    return _pq


def pack(codes, bits):
    """layer_ref.pack with tensor operations (equal to it: the first test)."""
    n, k = codes.shape
    if bits == 2:
        c = codes.view(n, -1, 16).to(torch.int32)
        rows = torch.stack([c[..., 2 * j] | c[..., 8 + 2 * j] << 2 | c[..., 2 * j + 1] << 4 | c[..., 9 + 2 * j] << 6 for j in range(4)], -1)
    else:
        c = codes.view(n, -1, 8 // bits).to(torch.int32)
        rows = sum(c[..., i] << (bits * i) for i in range(8 // bits))
    rows = rows.reshape(n, -1).to(torch.uint8)
    g, np_ = -(-rows.shape[1] // 64), -(-n // 16) * 16
    full = torch.zeros(np_, g * 64, dtype=torch.uint8, device=codes.device)
    full[:n, :rows.shape[1]] = rows
    return full.view(np_ // 16, 16, g, 64).permute(2, 0, 1, 3).contiguous().view(-1)


class Case:
    def __init__(self, mode, m, n, k, seed=0):
        bits, count, *_ = R.LEVELS[mode]
        g = torch.Generator().manual_seed(seed + 7 * m + n + k)
        self.mode = mode
        self.x = torch.randint(-127, 128, (m, k), generator=g).to(torch.int8).to(DEV)
        self.codes = torch.randint(0, count, (n, k), generator=g, dtype=torch.uint8).to(DEV)
        self.packed = pack(self.codes, bits)
        self.x_scale = (torch.rand(m, generator=g) * 0.05 + 0.001).to(DEV)
        self.alpha = (torch.rand(n, generator=g) * k ** -0.5 + 0.001).to(torch.bfloat16).to(DEV)
        self.g = g

    def random(self, *shape, dtype=torch.float32):
        return torch.randn(*shape, generator=self.g).to(dtype).to(DEV)

    def check(self, y, kind=0, bias=None, other=None, mul=False, alpha=None):
        want, err = R.product(self.x, self.x_scale, R.levels(self.codes, self.mode), self.alpha if alpha is None else alpha, bias, kind,
                              other, mul)
        u = R.U[y.dtype] if y.dtype != torch.float32 else 0
        bad = ~((y.double() - want).abs() <= u * (want.abs() + err) + err + R.TINY[y.dtype])
        assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: " \
                                    f"{y[bad][0].item()} for {want[bad][0].item()}"


@pytest.mark.parametrize("mode", sorted(R.LEVELS))
def test_packing(mode):
    bits, count, *_ = R.LEVELS[mode]
    c = torch.randint(0, count, (21, 320), generator=torch.Generator().manual_seed(mode), dtype=torch.uint8)
    assert torch.equal(pack(c, bits), R.pack(c, bits))


# one row to many, ragged columns, K that ends inside a 64-byte group of each width, sizes on both sides of the tiles
SHAPES = [(1, 1, 64), (1, 16, 128), (2, 17, 192), (7, 40, 576), (15, 33, 320), (16, 64, 1024), (17, 48, 256), (31, 100, 704), (33, 64, 64),
          (63, 129, 448), (64, 256, 1536), (65, 300, 512), (100, 576, 960), (128, 128, 2048), (129, 257, 384), (200, 513, 640),
          (257, 255, 1088), (300, 1000, 128), (513, 520, 832), (1, 1030, 4352), (9, 2000, 8192), (40, 31, 8256), (1025, 272, 576),
          # few rows over one, two and four column tiles a block; 17 to 32 rows on both sides of the stream kernel's limits
          (1, 13000, 64), (5, 6300, 640), (16, 12500, 192), (20, 6200, 320), (32, 12400, 576), (18, 90, 8192), (18, 90, 8256)]


@pytest.mark.parametrize("mode", [0, 2, 3, 4])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(pq, shape, mode):
    print(f"[a8 mode={mode} {shape}]", flush=True)
    c = Case(mode, *shape)
    y = Guarded(shape[:2], torch.bfloat16)
    pq.pq_gemm_a8(mode, c.x, c.x_scale, c.packed, c.alpha, y.t)
    c.check(y.t)
    y.check("y")


# many tiles: 64 x 128 ones in two groups of waves and in one, 128 x 256 ones; a last stage that is whole, half, the only one
LARGE = [(1500, 1100, 320), (1411, 1153, 64), (2100, 2100, 192), (2049, 2200, 1088), (2200, 4100, 448), (4000, 2177, 128), (2051, 4097, 1600)]


@pytest.mark.parametrize("mode", [0, 2, 3, 4])
@pytest.mark.parametrize("shape", LARGE)
def test_large(pq, shape, mode):
    print(f"[a8 large mode={mode} {shape}]", flush=True)
    c = Case(mode, *shape)
    y = Guarded(shape[:2], torch.bfloat16)
    pq.pq_gemm_a8(mode, c.x, c.x_scale, c.packed, c.alpha, y.t)
    c.check(y.t)
    y.check("y")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1500, 1100, 320), (2100, 2100, 192), (2200, 4100, 448), (2304, 3840, 256)])
def test_large_epilogue(pq, shape, dtype):
    """Every type, both combinations, rows of wider arrays; whole tiles and ragged ones."""
    print(f"[a8 large epilogue {shape} {dtype}]", flush=True)
    m, n, _ = shape
    c = Case(2, *shape, seed=6)
    bias, other = c.random(n, dtype=dtype), c.random(m, n + 3, dtype=dtype)[:, 1:1 + n]
    y = torch.full((m, n + 5), 3.0, dtype=dtype, device=DEV)
    for kind, mul in ((2, True), (4, False)):
        pq.pq_gemm_a8(2, c.x, c.x_scale, c.packed, c.alpha, y[:, 2:2 + n], bias=bias, activation=kind, other=other,
                      combine=pq.PQ_COMBINE_MUL if mul else pq.PQ_COMBINE_ADD)
        c.check(y[:, 2:2 + n], kind, bias, other, mul)
    assert bool((y[:, :2] == 3).all()) and bool((y[:, 2 + n:] == 3).all())
    pq.pq_gemm_a8(2, c.x, c.x_scale, c.packed, c.alpha, other, bias=bias, activation=4, other=other)         # in place
    assert torch.equal(other, y[:, 2:2 + n])


def test_output_past_the_caches(pq):
    """An output so large that it is written with streaming stores."""
    c = Case(2, 8192, 8200, 64, seed=7)
    y = torch.empty(8192, 8200, dtype=torch.bfloat16, device=DEV)
    pq.pq_gemm_a8(2, c.x, c.x_scale, c.packed, c.alpha, y)
    c.check(y)


@pytest.mark.parametrize("mode", sorted(R.LEVELS))
@pytest.mark.parametrize("shape", [(5, 50, 640), (150, 300, 1216), (600, 600, 1024)])
def test_modes(pq, shape, mode):
    print(f"[a8 mode={mode} {shape}]", flush=True)
    c = Case(mode, *shape, seed=1)
    y, alpha = torch.empty(shape[:2], device=DEV), c.alpha.float() * 1.001
    pq.pq_gemm_a8(mode, c.x, c.x_scale, c.packed, alpha, y)
    c.check(y, alpha=alpha)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", range(5))
@pytest.mark.parametrize("shape", [(3, 70, 256), (70, 200, 448), (515, 530, 256)])
def test_epilogue(pq, shape, kind, dtype):
    print(f"[a8 epilogue {shape} act={kind} {dtype}]", flush=True)
    m, n, _ = shape
    c = Case(2, *shape, seed=2)
    for mul in (False, True):
        bias, other = c.random(n, dtype=dtype), c.random(m, n, dtype=dtype)
        y = torch.empty(m, n, dtype=dtype, device=DEV)
        pq.pq_gemm_a8(2, c.x, c.x_scale, c.packed, c.alpha, y, bias=bias, activation=kind, other=other,
                      combine=pq.PQ_COMBINE_MUL if mul else pq.PQ_COMBINE_ADD)
        c.check(y, kind, bias, other, mul)
        pq.pq_gemm_a8(2, c.x, c.x_scale, c.packed, c.alpha, other, bias=bias, activation=kind, other=other,
                      combine=pq.PQ_COMBINE_MUL if mul else pq.PQ_COMBINE_ADD)                     # in place
        assert torch.equal(y, other)


@pytest.mark.parametrize("m,n,k", [(4, 90, 320), (77, 90, 320), (530, 270, 320)])
def test_strides(pq, m, n, k):
    """Rows of wider arrays: x 16 bytes apart at least, y and other at odd offsets; what lies between rows stays."""
    c = Case(2, m, n, k, seed=3)
    wide = torch.full((m, k + 48), 99, dtype=torch.int8, device=DEV)
    wide[:, 16:16 + k] = c.x
    y = torch.full((m, n + 13), 5.0, dtype=torch.bfloat16, device=DEV)
    other = c.random(m, n + 7, dtype=torch.bfloat16)[:, 3:3 + n]
    pq.pq_gemm_a8(2, wide[:, 16:16 + k], c.x_scale, c.packed, c.alpha, y[:, 1:1 + n], other=other)
    c.check(y[:, 1:1 + n], other=other)
    assert bool((y[:, :1] == 5).all()) and bool((y[:, 1 + n:] == 5).all())


@pytest.mark.parametrize("m", [1, 40, 300])
@pytest.mark.parametrize("mode,code", [(4, 0), (3, 0), (2, 0), (2, 3), (0, 0)])
def test_largest_sums(pq, mode, code, m):
    """K at its limit, every value at its end: the sums come near 2^31."""
    k, n = (1 << 17) - 64, 20
    bits, count, step, shift, unit = R.LEVELS[mode]
    codes = torch.full((n, k), code, dtype=torch.uint8, device=DEV)
    codes[1] = count - 1
    for value in (127, -127, -128):
        x = torch.full((m, k), value, dtype=torch.int8, device=DEV)
        y = torch.empty(m, n, device=DEV)
        pq.pq_gemm_a8(mode, x, torch.ones(m, device=DEV), pack(codes, bits), torch.ones(n, device=DEV), y)
        want = torch.full((m, n), value * k * (code * step - shift) * unit, dtype=torch.float64, device=DEV)
        want[:, 1] = value * k * ((count - 1) * step - shift) * unit
        assert bool(((y.double() - want).abs() <= 3 * 2.0 ** -24 * want.abs()).all()), (value, mode)


def test_what_is_no_number(pq):
    """A row whose scale is NaN is NaN, the others are not; other rows of 0 under a product keep their sign of nothing."""
    c = Case(2, 40, 64, 256, seed=4)
    c.x_scale[3] = float("nan")
    y = torch.empty(40, 64, device=DEV)
    pq.pq_gemm_a8(2, c.x, c.x_scale, c.packed, c.alpha, y, activation=pq.PQ_ACT_RELU)
    assert bool(y[3].isnan().all()) and bool(y[:3].isfinite().all()) and bool(y[4:].isfinite().all())
    c.x[:] = 0
    pq.pq_gemm_a8(2, c.x, torch.ones(40, device=DEV), c.packed, c.alpha, y, activation=pq.PQ_ACT_GELU)
    assert torch.count_nonzero(y) == 0


def test_empty(pq):
    c = Case(2, 1, 16, 64)
    e = torch.empty(0, 64, dtype=torch.int8, device=DEV)
    pq.pq_gemm_a8(2, e, torch.empty(0, device=DEV), c.packed, c.alpha, torch.empty(0, 16, device=DEV))
    pq.pq_gemm_a8(2, c.x, c.x_scale, torch.empty(0, dtype=torch.uint8, device=DEV), torch.empty(0, device=DEV), torch.empty(1, 0, device=DEV))


@pytest.mark.parametrize("m,n,k", [(1, 500, 2048), (48, 96, 8192), (333, 1600, 4352), (700, 900, 512), (1600, 1100, 576), (2100, 4000, 320)])
def test_workspace_and_repeats(pq, m, n, k):
    """A workspace of any contents, larger than needed, shared by calls one after the other: the same bits every time."""
    c = Case(2, m, n, k, seed=5)
    need = pq.pq_gemm_a8_workspace_bytes(2, m, n, k)
    y0 = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    pq.pq_gemm_a8(2, c.x, c.x_scale, c.packed, c.alpha, y0)
    c.check(y0)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        y = torch.empty_like(y0)
        pq.pq_gemm_a8(2, c.x, c.x_scale, c.packed, c.alpha, y, workspace=ws)
        assert torch.equal(y, y0)
    assert bool((ws[need:] == 0xA5).all())
