"""The decode example on the GPU: its attention against the cache's values, and the graph against plain calls."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_decode_steps(example, bits):
    steps = 37                          # ends inside a page
    layer = example.Layer(3, steps, hidden=512, heads=8, kv_heads=2, kv_bits=bits)
    x = example.run(layer, steps)
    assert layer.lens.tolist() == [steps] * 3 and torch.isfinite(x.float()).all()
    want = layer.plain_attention()
    # outputs are bf16: half a unit of 8 bits, doubled for the kernel's own sums
    assert ((layer.attn.double() - want).abs() <= 2 ** -8 * want.abs() + 2 ** -8 * want.abs().amax()).all()


def test_recorded_steps_are_the_same(example):
    layers = [example.Layer(3, 20, hidden=512, heads=8, kv_heads=2) for _ in range(2)]
    plain, replayed = (example.run(layer, 20, graph=g) for layer, g in zip(layers, (False, True)))
    torch.cuda.synchronize()
    assert torch.equal(plain, replayed) and torch.equal(layers[0].attn, layers[1].attn)
