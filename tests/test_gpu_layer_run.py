"""The operators around the packed product together, as a model's feed-forward
part and a training step use them: one by one, recorded, on other streams."""
import pytest
import torch

import layer_ref as R
from test_gpu_a8 import pack

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_amd import pq as _pq
    assert torch.cuda.is_available()
    return _pq


class Linear:
    """Weights quantised and exported by the library, and their values."""

    def __init__(self, pq, mode, n, k, seed):
        w = (torch.randn(n, k, generator=torch.Generator().manual_seed(seed)) * k ** -0.5).to(DEV)
        alpha, codes = torch.zeros(n, device=DEV), torch.empty(n, pq.pq_code_row_bytes(mode, k), dtype=torch.uint8, device=DEV)
        pq.pq_quantize_fwd(mode, n, k, w, alpha, pq.PQ_INIT_ALPHA, None, None, codes)
        self.packed = torch.empty(pq.pq_packed_bytes(mode, n, k), dtype=torch.uint8, device=DEV)
        self.alpha = torch.empty(n, dtype=torch.bfloat16, device=DEV)
        pq.pq_pack(mode, n, k, w, alpha, self.packed, self.alpha)
        bits = R.LEVELS[mode][0]
        c = torch.stack([(codes >> (bits * i)) & (2 ** bits - 1) for i in range(8 // bits)], -1).view(n, k)
        assert torch.equal(pack(c, bits), self.packed)
        self.mode, self.n, self.k, self.levels = mode, n, k, R.levels(c, mode)


class FeedForward:
    """Norm to 8 bits, up and gated products, rows to 8 bits, down product onto the residual stream."""

    def __init__(self, pq, tokens, hidden, inner, modes, seed=0):
        self.pq, self.tokens = pq, tokens
        self.up, self.gate, self.down = (Linear(pq, m, n, k, seed + i) for i, (m, n, k) in
                                         enumerate(zip(modes, (inner, inner, hidden), (hidden, hidden, inner))))
        self.weight = (torch.rand(hidden, generator=torch.Generator().manual_seed(seed)) + 0.5).to(DEV)
        e = lambda *s, d=torch.bfloat16: torch.empty(*s, dtype=d, device=DEV)  # noqa: E731
        self.sum, self.x8, self.xs = e(tokens, hidden), e(tokens, hidden, d=torch.int8), e(tokens, d=torch.float32)
        self.u, self.h = e(tokens, inner), e(tokens, inner)
        self.h8, self.hs = e(tokens, inner, d=torch.int8), e(tokens, d=torch.float32)
        self.spaces = [pq.a8_workspace(p.mode, tokens, p.n, p.k) for p in (self.up, self.gate, self.down)]

    def __call__(self, x, residual, stream=None):
        pq, s = self.pq, {"stream": stream}
        pq.pq_rmsnorm(x, self.weight, residual=residual, sum=self.sum, q=self.x8, scale=self.xs, **s)
        pq.pq_gemm_a8(self.up.mode, self.x8, self.xs, self.up.packed, self.up.alpha, self.u, workspace=self.spaces[0], **s)
        pq.pq_gemm_a8(self.gate.mode, self.x8, self.xs, self.gate.packed, self.gate.alpha, self.h, activation=pq.PQ_ACT_SILU,
                      other=self.u, combine=pq.PQ_COMBINE_MUL, workspace=self.spaces[1], **s)
        pq.pq_quantize_rows(self.h, self.h8, self.hs, **s)
        pq.pq_gemm_a8(self.down.mode, self.h8, self.hs, self.down.packed, self.down.alpha, self.sum, other=self.sum,
                      workspace=self.spaces[2], **s)
        return self.sum

    def steps(self):
        """Every tensor that a call wrote (the sum holds the last product's result)."""
        return [t.clone() for t in (self.x8, self.xs, self.u, self.h, self.h8, self.hs, self.sum)]


def near(got, want, err, dtype):
    assert bool(((got.double() - want).abs() <= R.U[dtype] * (want.abs() + err) + err + R.TINY[dtype]).all())


@pytest.mark.parametrize("tokens,hidden,inner,modes", [(1, 576, 1536, (2, 2, 2)), (16, 320, 832, (0, 3, 4)), (77, 576, 1536, (2, 2, 4)),
                                                       (600, 640, 1088, (1, 2, 2))])
def test_feed_forward(pq, tokens, hidden, inner, modes):
    f = FeedForward(pq, tokens, hidden, inner, modes)
    g = torch.Generator().manual_seed(1)
    x, r = (torch.randn(tokens, hidden, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    out = f(x, r).clone()
    h = (x.float() + r.float()).to(torch.bfloat16)
    y, _ = R.norm(h, f.weight, 1e-6)
    # each step from what the step before it left
    assert bool(((f.x8.double() * f.xs.double()[:, None] - y).abs() <= f.xs.double()[:, None] * 0.501).all())
    near(f.u, *R.product(f.x8, f.xs, f.up.levels, f.up.alpha), torch.bfloat16)
    near(f.h, *R.product(f.x8, f.xs, f.gate.levels, f.gate.alpha, None, 2, f.u, True), torch.bfloat16)
    assert bool(((f.h8.double() * f.hs.double()[:, None] - f.h.double()).abs() <= f.hs.double()[:, None] * 0.501).all())
    near(out, *R.product(f.h8, f.hs, f.down.levels, f.down.alpha, None, 0, h, False), torch.bfloat16)


def test_recorded_and_on_a_stream(pq):
    """Recorded without a call before it, replayed between eager work on the same tensors' copies; then on a side stream."""
    f, plain = (FeedForward(pq, 48, 576, 1536, (2, 2, 4)) for _ in range(2))
    g = torch.Generator().manual_seed(2)
    x, r = (torch.randn(48, 576, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        f(x, r)
    for i in range(4):
        x.copy_(torch.randn(48, 576, generator=g).to(torch.bfloat16))
        plain(x, r)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(f.steps(), plain.steps())), i
        torch.randn(1 << 20, device=DEV).mul_(2.0)
    torch.cuda.synchronize()
    f(x, r, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(f.steps(), plain.steps()))


def test_two_streams_at_once(pq):
    """Two calls in flight with tensors and workspaces of their own do not disturb each other."""
    fs = [FeedForward(pq, m, 576, 1536, (2, 2, 2), seed=m) for m in (100, 101)]
    g = torch.Generator().manual_seed(3)
    xs = [torch.randn(m, 576, generator=g).to(torch.bfloat16).to(DEV) for m in (100, 101)]
    want = []
    for f, x in zip(fs, xs):
        f(x, x)
        torch.cuda.synchronize()
        want.append(f.steps())
    streams = [torch.cuda.Stream() for _ in fs]
    for _ in range(5):
        for f, x, s in zip(fs, xs, streams):
            s.wait_stream(torch.cuda.current_stream())
            f(x, x, stream=s)
    torch.cuda.synchronize()
    for f, w in zip(fs, want):
        assert all(torch.equal(a, b) for a, b in zip(f.steps(), w))


class Step:
    """A training step's gradients: norm, fake-quantised head, distillation, and back."""

    def __init__(self, pq, rows, hidden, vocab, k, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.pq = pq
        self.x = torch.randn(rows, hidden, generator=g).to(DEV)
        self.weight = (torch.rand(hidden, generator=g) + 0.5).to(DEV)
        self.W = (torch.randn(vocab, hidden, generator=g) * 0.3).to(DEV)
        self.alpha, self.Wq = torch.zeros(vocab, device=DEV), torch.empty(vocab, hidden, device=DEV)
        pq.pq_quantize_fwd(pq.PQ_W2_SEQ, vocab, hidden, self.W, self.alpha, pq.PQ_INIT_ALPHA, None, self.Wq, None)
        self.index = torch.stack([torch.randperm(vocab, generator=g)[:k] for _ in range(rows)]).to(torch.int32).to(DEV)
        self.top = (torch.randn(rows, k, generator=g) * 2).to(DEV)
        self.keep = (torch.rand(rows, generator=g) < 0.8).float().to(DEV)
        e = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
        self.y, self.rstd, self.loss, self.dz = e(rows, hidden), e(rows), e(rows), e(rows, vocab)
        self.dW, self.dalpha, self.dx, self.dweight = e(vocab, hidden), e(vocab), e(rows, hidden), e(hidden)
        self.space = pq.rmsnorm_bwd_workspace(rows, hidden)

    def __call__(self):
        pq = self.pq
        pq.pq_rmsnorm(self.x, self.weight, y=self.y, rstd=self.rstd)
        self.z = self.y @ self.Wq.t()
        pq.pq_distill(self.z, self.index, self.top, self.loss, dlogits=self.dz, temperature=2.0, row_weight=self.keep,
                      grad_scale=1.0 / len(self.x))
        self.dWq = self.dz.t() @ self.y
        pq.pq_quantize_bwd(pq.PQ_W2_SEQ, *self.W.shape, self.W, self.alpha, self.dWq, pq.PQ_G_F32, 0.01, self.dW, self.dalpha)
        pq.pq_rmsnorm_bwd(self.x, self.weight, self.rstd, self.dz @ self.Wq, self.dx, dweight=self.dweight, workspace=self.space)
        return [t.clone() for t in (self.loss, self.dz, self.dW, self.dalpha, self.dx, self.dweight)]


def test_training_step(pq):
    """Gradients against autograd of the same step in binary64."""
    s = Step(pq, 40, 192, 504, 12)
    loss, dz, dW, dalpha, dx, dweight = s()
    x, w, Wq = (t.double().clone().requires_grad_() for t in (s.x, s.weight, s.Wq))
    y = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
    log_q = torch.log_softmax((y @ Wq.t()) / 2.0, -1)
    p = torch.softmax(s.top.double() / 2.0, -1)
    want = (4.0 * (p * (p.log() - log_q.gather(1, s.index.long()))).sum(-1) * s.keep.double())
    (want.sum() / 40).backward()
    assert float((loss.double() - want.detach()).abs().max()) < 1e-4
    # products of 504 and 192 terms in fp32: 2^-24 sqrt(504) of the terms' sizes is far below 1e-5 of the largest gradient
    for got, ref in ((dx, x.grad), (dweight, w.grad), (s.dWq, Wq.grad)):
        assert float((got.double() - ref).abs().max()) <= 1e-5 * float(ref.abs().max())
    assert torch.count_nonzero(dz[s.keep == 0]) == 0 and bool((dW[dW != 0] == s.dWq[dW != 0]).all())


def test_training_step_recorded(pq):
    s = Step(pq, 24, 256, 1000, 8, seed=4)
    want = s()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s()
    for i in range(3):
        for t in (s.loss, s.dz, s.dW, s.dalpha, s.dx, s.dweight):
            t.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = (s.loss, s.dz, s.dW, s.dalpha, s.dx, s.dweight)
        for a, b in zip(got, want):
            assert float((a - b).abs().max()) <= 1e-5 * float(b.abs().max()), i
        torch.randn(1 << 20, device=DEV).mul_(2.0)
