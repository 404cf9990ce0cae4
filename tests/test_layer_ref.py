"""The references of tests/layer_ref.py against independent statements of the same things (CPU)."""
import math

import pytest
import torch

import layer_ref as R
import oracle as O


def test_norm_gradient_is_autograd_and_differences():
    g = torch.Generator().manual_seed(0)
    h, dy = (torch.randn(5, 13, dtype=torch.float64, generator=g) for _ in range(2))
    w = torch.rand(13, dtype=torch.float64, generator=g) + 0.5
    hh, ww = h.clone().requires_grad_(), w.clone().requires_grad_()
    y, rstd = R.norm(hh, ww, 1e-3)
    dx, dw, _, _ = R.norm_grad(h, w, rstd.detach(), dy)
    y.backward(dy)
    assert torch.allclose(dx, hh.grad, rtol=1e-12) and torch.allclose(dw, ww.grad, rtol=1e-12)
    d = torch.randn(5, 13, dtype=torch.float64, generator=g)
    e = 1e-5
    slope = ((R.norm(h + e * d, w, 1e-3)[0] - R.norm(h - e * d, w, 1e-3)[0]) * dy).sum() / (2 * e)
    assert abs(slope - (dx * d).sum()) < 1e-8


@pytest.mark.parametrize("mode", sorted(R.LEVELS))
def test_packing_and_levels_are_the_oracle_s(mode):
    bits, count, *_ = R.LEVELS[mode]
    codes = torch.randint(0, count, (19, 192), generator=torch.Generator().manual_seed(mode), dtype=torch.uint8)
    per = 8 // bits
    rows = sum(codes[:, i::per].to(torch.int32) << (bits * i) for i in range(per)).to(torch.uint8).numpy()
    want = O.tile_codes(rows, bits)
    assert R.pack(codes, bits).numpy().tobytes() == want.tobytes()
    lev = {0: [-1, 1], 1: [-2 / 3, 0, 2 / 3], 2: [-.75, -.25, .25, .75], 3: range(-4, 4), 4: range(-8, 8), 5: range(-2, 2),
           6: [-1, 0, 1]}[mode]
    got = R.levels(torch.arange(count, dtype=torch.uint8), mode)
    assert torch.allclose(got, torch.tensor(list(lev), dtype=torch.float64), atol=3e-8)


def test_activations():
    v = torch.linspace(-8, 8, 1001, dtype=torch.float64)
    assert torch.allclose(R.act(v, 2), torch.nn.functional.silu(v))
    assert torch.allclose(R.act(v, 3), torch.nn.functional.gelu(v), atol=1e-14)
    assert torch.allclose(R.act(v, 4), torch.nn.functional.gelu(v, approximate="tanh"), atol=1e-14)


@pytest.mark.parametrize("temp", [1.0, 2.5])
def test_distillation_gradient_is_autograd(temp):
    g = torch.Generator().manual_seed(3)
    z = torch.randn(6, 20, dtype=torch.float64, generator=g, requires_grad=True)
    index = torch.stack([torch.randperm(20, generator=g)[:4] for _ in range(6)]).to(torch.int32)
    index[1, 2:] = -1
    index[2] = -1
    index[3, 1] = index[3, 0]                   # the same word twice
    top = torch.randn(6, 4, dtype=torch.float64, generator=g)
    w = torch.tensor([1.0, 2.0, 1.0, 0.5, 0.0, 1.0], dtype=torch.float64)
    loss, dz, target, q = R.distill(z, index, top, temp, w)
    loss.sum().backward()
    assert torch.allclose(z.grad, dz, atol=1e-14)
    assert loss[2] == 0 and loss[4] == 0 and torch.count_nonzero(dz[2]) == 0
    assert torch.allclose(q.sum(-1), torch.ones(6, dtype=torch.float64))
    # the whole vocabulary as the teacher's list: the divergence of the two distributions, 0 where they agree
    every = torch.arange(20, dtype=torch.int32).expand(6, 20)
    same, _, _, _ = R.distill(z.detach(), every, z.detach() + 3.0, temp)
    assert same.abs().max() < 1e-12 and math.isclose(float(target[0].sum()), 1.0)
