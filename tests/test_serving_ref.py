"""The serving references against independent statements of the same things (CPU)."""
import math

import pytest
import torch

import serving_ref as R


@pytest.mark.parametrize("half", [True, False])
def test_rope_is_a_complex_product(half):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(5, 2, 16, dtype=torch.float64, generator=g)
    f, m = R.rope_freqs(12, 10000.0)
    ang = torch.arange(9, dtype=torch.float64)[:, None] * torch.from_numpy(f)
    table = torch.stack([ang.cos(), ang.sin()], -1)
    pos = torch.tensor([0, 3, 8, -1, 2])
    y = R.rope(x, table, pos, half)
    a, b = R.pair_index(12, half)
    w = torch.polar(torch.ones(5, 6, dtype=torch.float64), ang[pos.clamp_min(0)] * (pos >= 0)[:, None])[:, None]
    z = torch.complex(x[..., a], x[..., b]) * w
    assert torch.allclose(y[..., a], z.real) and torch.allclose(y[..., b], z.imag)
    assert torch.equal(y[..., 12:], x[..., 12:]) and m == 1.0
    assert torch.allclose(R.rope(y, table, pos, half, inverse=True), x)


def test_rope_scalings_meet_at_factor_one():
    plain, _ = R.rope_freqs(64, 10000.0)
    for kind in ("linear", "ntk", "yarn", "bands"):
        f, m = R.rope_freqs(64, 10000.0, kind, 1.0, 4096.0, 32.0 if kind == "yarn" else 4.0, 1.0)
        assert abs(f - plain).max() < 1e-15 and m == 1.0, kind


@pytest.mark.parametrize("bits", [8, 4])
def test_quantiser_error(bits):
    g = torch.Generator().manual_seed(2)
    x = torch.randn(50, 32, generator=g) * torch.logspace(-3, 3, 50)[:, None] + 0.5
    n, p = R.quantise(x, bits)
    assert int(n.max()) == R.TOP[bits]
    got = R.values(R.pack(n, bits), p, bits)
    mn, mx = x.amin(-1, keepdim=True).double(), x.amax(-1, keepdim=True).double()
    # half a step, and what the rounded (s, z) cut off at the ends
    lim = p[:, :1].double() * 0.5001 + 2.0 ** -8 * (mn.abs() + (mx - mn)) * 1.01
    assert bool(((got - x.double()).abs() <= lim).all())
    assert torch.equal(R.unpack(R.pack(n, bits), bits), n)


def test_quantiser_constant_row():
    n, p = R.quantise(torch.full((1, 16), 0.3), 4)
    # bf16(0.3) = 0.30078 lies above 0.3: every channel is code 0
    assert int(n.max()) == 0 and abs(float(p[0, 1]) - 0.3) < 2e-3 and float(p[0, 0]) == R.MIN_SCALE


def test_attention_is_softmax():
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(n, 8, dtype=torch.float64, generator=g) for n in (3, 11, 11))
    out, lse, _ = R.attention(q, k, v, 0.25)
    x = 0.25 * q @ k.T
    assert torch.allclose(out, torch.softmax(x, -1) @ v) and torch.allclose(lse, torch.logsumexp(x, -1))
    out, lse, _ = R.attention(q, k[:0], v[:0], 1.0)
    assert torch.count_nonzero(out) == 0 and lse[0] == -math.inf
