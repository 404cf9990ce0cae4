"""Answering with a packed-weight attention layer, one token per sequence and
step, on one GPU:

    python examples/decode_step.py [--batch 8] [--steps 512] [--kv 16|8|4] [--graph]

A step is four calls: the packed projection to q, k and v (pq_gemm), the
append that rotates q and k and writes k and v into the paged cache
(pq_kv_append), the attention over the cache (pq_attn_decode) and the packed
output projection (pq_gemm).  Positions, lengths and slots live on the GPU and
are advanced there, so that the step can be recorded once into a graph and
replayed.  At the end the cache is read back (pq_kv_load) and the last step's
attention is computed from it once more in binary64.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_quantization_aware_amd import pq  # noqa: E402

FORMATS = {16: pq.PQ_KV_16, 8: pq.PQ_KV_8, 4: pq.PQ_KV_4}


class Linear:
    """Packed 2-bit weights (rows x cols) and the call that multiplies by them."""

    def __init__(self, rows, cols, generator, device):
        w = (torch.randn(rows, cols, generator=generator) * cols ** -0.5).to(device)
        alpha = torch.zeros(rows, dtype=torch.float32, device=device)
        codes = torch.empty(rows, pq.pq_code_row_bytes(pq.PQ_W2_SEQ, cols), dtype=torch.uint8, device=device)
        pq.pq_quantize_fwd(pq.PQ_W2_SEQ, rows, cols, w, alpha, pq.PQ_INIT_ALPHA, None, None, codes)
        self.packed = torch.empty(pq.pq_packed_bytes(pq.PQ_W2_SEQ, rows, cols), dtype=torch.uint8, device=device)
        self.alpha = torch.empty(rows, dtype=torch.bfloat16, device=device)
        pq.pq_pack(pq.PQ_W2_SEQ, rows, cols, w, alpha, self.packed, self.alpha)
        self.rows, self.cols = rows, cols

    def prepare(self, tokens, device):
        self.out = torch.empty(tokens, self.rows, dtype=torch.bfloat16, device=device)
        self.workspace = pq.gemm_workspace(pq.PQ_W2_SEQ, tokens, self.rows, self.cols, device)
        return self

    def __call__(self, x):
        pq.pq_gemm(pq.PQ_W2_SEQ, x.shape[0], self.rows, self.cols, x, self.packed, self.alpha, self.out,
                   workspace=self.workspace)
        return self.out


class Layer:
    """Attention with its cache for a fixed batch of sequences of up to max_len tokens."""

    def __init__(self, batch, max_len, hidden=1024, heads=16, kv_heads=4, kv_bits=8, page=16, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.batch, self.heads, self.kv_heads, self.dim, self.page = batch, heads, kv_heads, hidden // heads, page
        self.qkv = Linear((heads + 2 * kv_heads) * self.dim, hidden, g, device).prepare(batch, device)
        self.o = Linear(hidden, hidden, g, device).prepare(batch, device)
        per_seq = -(-max_len // page)
        self.cache = pq.KVCache.allocate(FORMATS[kv_bits], batch * per_seq, page, kv_heads, self.dim, device=device)
        # pages in any order, as an allocator would have left them
        self.pages = torch.randperm(batch * per_seq, generator=g).to(torch.int32).view(batch, per_seq).to(device)
        self.angles = pq.pq_rope_table(max_len, self.dim, device=device)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.positions = torch.zeros_like(self.lens)
        self.slots = torch.zeros(batch, dtype=torch.int64, device=device)
        self.q = torch.empty(batch, heads, self.dim, dtype=torch.bfloat16, device=device)
        self.attn = torch.empty_like(self.q)
        self.lse = torch.empty(batch, heads, dtype=torch.float32, device=device)
        self.workspace = pq.attn_workspace(self.cache, batch, heads, device)

    def step(self, x):
        """x [batch, hidden]: the new tokens' inputs; returns the layer's outputs."""
        self.positions.copy_(self.lens)
        at = self.pages.gather(1, (self.positions // self.page).long().unsqueeze(1)).squeeze(1)
        self.slots.copy_(at.long() * self.page + self.positions % self.page)
        self.lens.add_(1)
        q, k, v = self.qkv(x).view(self.batch, -1, self.dim).split([self.heads, self.kv_heads, self.kv_heads], dim=1)
        pq.pq_kv_append(self.cache, k, v, self.slots, positions=self.positions, table=self.angles, q=q, q_out=self.q)
        pq.pq_attn_decode(self.cache, self.q, self.pages, self.lens, self.attn, self.lse, workspace=self.workspace)
        return self.o(self.attn.view(self.batch, -1))

    def stored(self):
        """Every sequence's keys and values, as the cache holds them: [tokens, kv_heads, dim] each, in f32."""
        lens = self.lens.cpu()
        cu = torch.cat([torch.zeros(1, dtype=torch.int32), lens.cumsum(0).to(torch.int32)])
        k, v = (torch.empty(int(cu[-1]), self.kv_heads, self.dim, dtype=torch.float32, device=self.q.device)
                for _ in range(2))
        pq.pq_kv_load(self.cache, self.pages, None, cu.to(self.q.device), k, v)
        return k.split(lens.tolist()), v.split(lens.tolist())

    def plain_attention(self):
        """The last step's attention, from the cache's values in binary64."""
        out = []
        for q, k, v in zip(self.q, *self.stored()):
            q = q.double().view(self.kv_heads, -1, self.dim)
            p = (q @ k.double().permute(1, 2, 0).contiguous() * self.dim ** -0.5).softmax(-1)
            out.append((p @ v.double().transpose(0, 1).contiguous()).reshape(self.heads, self.dim))
        return torch.stack(out)


def run(layer, steps, graph=False, seed=1):
    """`steps` tokens for every sequence, each one's output (scaled to unit size) the next one's input."""
    device = layer.q.device
    x = torch.randn(layer.batch, layer.heads * layer.dim, generator=torch.Generator().manual_seed(seed))
    x = x.to(torch.bfloat16).to(device)

    def advance():
        y = layer.step(x).float()
        x.copy_(y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6))
    if not graph:
        for _ in range(steps):
            advance()
        return x
    if steps > 0:
        advance()                       # the first step of a process loads the kernels
    recorded = torch.cuda.CUDAGraph()
    with torch.cuda.graph(recorded):
        advance()
    for _ in range(steps - 1):
        recorded.replay()
    return x


def main():
    ap = argparse.ArgumentParser(description="decode steps of a packed-weight attention layer")
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--steps", type=int, default=512)
    ap.add_argument("--kv", type=int, default=8, choices=sorted(FORMATS))
    ap.add_argument("--graph", action="store_true")
    args = ap.parse_args()
    run(Layer(args.batch, args.steps, kv_bits=args.kv), min(args.steps, 4), args.graph)
    layer = Layer(args.batch, args.steps, kv_bits=args.kv)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    run(layer, args.steps, args.graph)
    torch.cuda.synchronize()
    t1 = time.perf_counter()
    want = layer.plain_attention()
    off = (layer.attn.double() - want).norm() / want.norm()
    print(f"{args.batch} sequences, {args.steps} steps, {args.kv}-bit cache: {(t1 - t0) * 1e6 / args.steps:.1f} us a step, "
          f"last attention off by {off:.2g} of its size")


if __name__ == "__main__":
    main()
