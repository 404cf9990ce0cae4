"""pq_attn_decode on the GPU against binary64 attention over the values that
the cache holds, and a decode step through append and attention."""
import math

import pytest
import torch

import serving_ref as R
from gpu_util import Guarded
from test_gpu_kv import FMT, make_cache

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_amd import pq as _pq
    assert torch.cuda.is_available()
    return _pq


class Case:
    """A filled cache with its page table; k, v: the values it holds, binary64 [tokens, heads, dim] per sequence."""

    def __init__(self, pq, fmt, lens, heads, group, dim, page, dtype, seed=0, token_major=False, gain=1.0, stale=None):
        f, bits = FMT[fmt]
        g = torch.Generator().manual_seed(seed)
        need = [max(1, -(-n // page)) for n in lens]
        pages = sum(need) + 2
        perm = torch.randperm(pages, generator=g).tolist()
        self.cache = make_cache(pq, fmt, pages, page, heads, dim, dtype, token_major, fill=0xFF)      # NaN patterns
        self.table = torch.full((len(lens), max(need) + 2), 1 << 30, dtype=torch.int32)               # never followed
        self.lens, self.dtype, self.heads, self.group, self.dim, self.bits = lens, dtype, heads, group, dim, bits
        b = 0
        for i, n in enumerate(need):
            self.table[i, :n] = torch.tensor(perm[b:b + n])
            b += n
        total = sum(lens)
        self.k, self.v, self.mag = [], [], []
        if total:
            k = torch.randn(total, heads, dim, generator=g) * gain
            k[..., ::16] *= 4.0
            v = torch.randn(total, heads, dim, generator=g) + 0.5
            k, v = k.to(dtype), v.to(dtype)
            seq = torch.cat([torch.full((n,), i) for i, n in enumerate(lens)])
            at = torch.cat([torch.arange(n) for n in lens])
            slots = self.table[seq, at // page].long() * page + at % page
            pq.pq_kv_append(self.cache, k.to(DEV), v.to(DEV), slots.to(DEV))
            for x, keep in ((k, self.k), (v, self.v)):
                if bits == 16:
                    val, mag = x.double(), x.double().abs()
                else:
                    n, p = R.quantise(x.float(), bits)
                    val = R.values(R.pack(n, bits), p, bits)
                    mag = p.double()[..., 1:].abs() + p.double()[..., :1] * n.double()
                keep += list(val.split(lens))
                self.mag.append(list(mag.split(lens)))
        else:
            z = torch.zeros(0, heads, dim, dtype=torch.float64)
            self.k, self.v, self.mag = [z] * len(lens), [z] * len(lens), [[z] * len(lens)] * 2
        self.q = torch.randn(len(lens), heads * group, dim, generator=g).to(dtype)

    def run(self, pq, window=0, max_len=0, scale=None, q=None, stream=None, workspace=None):
        b, hq = len(self.lens), self.heads * self.group
        q = self.q.to(DEV) if q is None else q
        out, lse = Guarded((b, hq, self.dim), self.dtype), Guarded((b, hq), torch.float32)
        n = pq.pq_attn_decode_workspace_bytes(self.cache, b, hq)
        ws = Guarded((n,), torch.uint8)
        pq.pq_attn_decode(self.cache, q, self.table.to(DEV), torch.tensor(self.lens, dtype=torch.int32, device=DEV),
                          out.t, lse.t, scale, window, max_len, ws.t)
        torch.cuda.synchronize()
        for x, what in ((out, "out"), (lse, "lse"), (ws, "workspace")):
            x.check(what)
        return out.t.cpu(), lse.t.cpu()

    def check(self, out, lse, window=0, scale=None, hidden=()):
        """Bounds, all derived from the arithmetic: x_t sums dim products of
        f16 or bf16 values in binary32, off by dx = 2^-24 (dim + 8) scale sum
        |q| (|z| + s n); the weights are two 16-bit pieces (2^-14 covers both
        types) and the sums of weights and values binary32; out is rounded
        once."""
        scale = self.dim ** -0.5 if scale is None else scale
        for b, n in enumerate(self.lens):
            first = max(0, n - window) if window else 0
            keep = torch.tensor([t for t in range(first, n) if (b, t) not in hidden], dtype=torch.long)
            for h in range(self.heads):
                rows = slice(h * self.group, (h + 1) * self.group)
                q = self.q[b, rows].double()
                o, s, p = R.attention(q, self.k[b][keep, h], self.v[b][keep, h], scale)
                got, gs = out[b, rows].double(), lse[b, rows].double()
                if not len(keep):
                    assert torch.count_nonzero(got) == 0 and bool((gs == -math.inf).all())
                    continue
                dx = 2.0 ** -24 * (self.dim + 8) * abs(scale) * float((q.abs() @ self.mag[0][b][keep, h].T).max())
                spread = p @ self.mag[1][b][keep, h]
                lim = R.U[self.dtype] * 1.01 * o.abs() + (2.0 ** -14 + 4 * dx) * spread + R.TINY[self.dtype]
                bad = ~((got - o).abs() <= lim)
                assert not bool(bad.any()), f"b={b} len={n} head={h}: {int(bad.sum())} of {bad.numel()} off, " \
                    f"worst {float(((got - o).abs() / lim).max()):.2f} x the bound"
                assert bool(((gs - s).abs() <= 2 * dx + 2.0 ** -20 * s.abs().clamp_min(1)).all()), (b, n, h)


SHAPES = [  # heads, group, dim, page
    (1, 1, 16, 16), (3, 3, 64, 16), (2, 4, 128, 64), (5, 4, 80, 32), (1, 8, 256, 16), (2, 2, 192, 128), (1, 16, 96, 16),
    (2, 20, 64, 32), (1, 71, 32, 16), (4, 5, 48, 16), (1, 7, 208, 64), (8, 1, 128, 16)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("shape", SHAPES)
def test_attention(pq, shape, fmt, dtype):
    heads, group, dim, page = shape
    print(f"[attn {shape} {fmt} {dtype}]", flush=True)
    lens = [0, 1, 15, 16, 17, 31, 33, 127, 128, 129, 300]
    c = Case(pq, fmt, lens, heads, group, dim, page, dtype, seed=dim + group)
    c.check(*c.run(pq))
    for window in (1, 16, 100):
        c.check(*c.run(pq, window=window), window=window)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("lens", [[1], [5000], [4096, 1, 0, 2500], [3, 9001], [700] * 9, [0, 0], [0]])
def test_split_rows(pq, fmt, lens):
    """Rows over many blocks, rows inside one, both in one call, none."""
    print(f"[attn split {fmt} {lens}]", flush=True)
    c = Case(pq, fmt, lens, 2, 4, 64, 16, torch.bfloat16, seed=len(lens))
    out, lse = c.run(pq)
    c.check(out, lse)
    again = c.run(pq)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])         # the same in every run
    for hint in (max(1, max(lens)), 1 << 20):
        c.check(*c.run(pq, max_len=hint))
    for most in (1, 130, 700):                                              # longer sequences count as max_len
        got = c.run(pq, max_len=most)
        full, c.lens = c.lens, [min(n, most) for n in c.lens]
        c.check(*got)
        c.lens = full


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("shape", [(1, 4, 80, 32), (2, 1, 128, 16), (1, 12, 128, 64), (1, 5, 256, 16), (2, 3, 48, 16), (1, 20, 80, 16)])
def test_split_rows_of_every_shape(pq, shape, fmt):
    """More tokens than one block takes, row ends inside a share and inside a tile; windows that start in the middle."""
    heads, group, dim, page = shape
    print(f"[attn split {shape} {fmt}]", flush=True)
    c = Case(pq, fmt, [2300, 0, 1041, 2, 4111], heads, group, dim, page, torch.bfloat16, seed=dim)
    c.check(*c.run(pq))
    c.check(*c.run(pq, window=1900), window=1900)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("seqs", [127, 128])
def test_unsplit_rows_where_there_are_many(pq, fmt, seqs):
    """Rows of up to 1200 tokens, just too few and just enough of them for one block each."""
    lens = [3 * i for i in range(seqs - 2)] + [1200, 0]
    print(f"[attn many {fmt} {seqs}]", flush=True)
    c = Case(pq, fmt, lens, 2, 2, 32, 16, torch.float16, seed=seqs)
    c.check(*c.run(pq, max_len=1200))


@pytest.mark.parametrize("fmt", list(FMT))
def test_token_major_pages_and_strided_q(pq, fmt):
    c = Case(pq, fmt, [77, 200], 3, 2, 64, 32, torch.bfloat16, token_major=True)
    fused = torch.randn(2, 12, 64).to(torch.bfloat16)
    fused[:, :6] = c.q
    c.check(*c.run(pq, q=fused.to(DEV)[:, :6]))


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("gain", [30.0, 1e-6])
def test_peaked_and_flat_scores(pq, fmt, gain):
    """Scores over several hundred (one token takes all) and all but equal ones."""
    c = Case(pq, fmt, [400, 130], 2, 4, 128, 16, torch.bfloat16, gain=gain)
    c.check(*c.run(pq))
    c.check(*c.run(pq, scale=0.5), scale=0.5)
    c.check(*c.run(pq, scale=0.0), scale=0.0)
    c.check(*c.run(pq, scale=-0.02), scale=-0.02)


@pytest.mark.parametrize("fmt", list(FMT))
def test_rising_scores(pq, fmt):
    """Every tile brings a new maximum: the running reference moves each time."""
    n, d = 900, 64
    c = Case(pq, fmt, [n], 1, 4, d, 16, torch.bfloat16)
    k = torch.randn(n, 1, d) * 0.1
    k[:, 0, 0] = torch.arange(n) * 0.5
    v = torch.randn(n, 1, d)
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    at = torch.arange(n)
    slots = c.table[0, at // 16].long() * 16 + at % 16
    pq.pq_kv_append(c.cache, k.to(DEV), v.to(DEV), slots.to(DEV))
    c.k, c.v, c.mag = [], [], []
    for x, keep in ((k, c.k), (v, c.v)):
        if c.bits == 16:
            keep.append(x.double())
            c.mag.append([x.double().abs()])
        else:
            m, p = R.quantise(x.float(), c.bits)
            keep.append(R.values(R.pack(m, c.bits), p, c.bits))
            c.mag.append([p.double()[..., 1:].abs() + p.double()[..., :1] * m.double()])
    c.q[..., 0] = 1.0
    c.check(*c.run(pq, scale=1.0), scale=1.0)
    c.q[..., 0] = -1.0
    c.check(*c.run(pq, scale=1.0), scale=1.0)


@pytest.mark.parametrize("fmt", ["kv8", "kv4"])
def test_scales_of_every_size(pq, fmt):
    """Value rows from 1e-12 to 1e12 in one sequence, constant rows (the smallest scale) among them."""
    n, d = 200, 64
    c = Case(pq, fmt, [n], 1, 2, d, 16, torch.bfloat16)
    k = (torch.randn(n, 1, d) * 0.5).to(torch.bfloat16)
    v = (torch.randn(n, 1, d) * torch.logspace(-12, 12, n)[:, None, None]).to(torch.bfloat16)
    v[::7] = 0.25
    at = torch.arange(n)
    slots = c.table[0, at // 16].long() * 16 + at % 16

    def refill():
        pq.pq_kv_append(c.cache, k.to(DEV), v.to(DEV), slots.to(DEV))
        c.k, c.v, c.mag = [], [], []
        for x, keep in ((k, c.k), (v, c.v)):
            m, p = R.quantise(x.float(), c.bits)
            keep.append(R.values(R.pack(m, c.bits), p, c.bits))
            c.mag.append([p.double()[..., 1:].abs() + p.double()[..., :1] * m.double()])
    refill()
    c.check(*c.run(pq))
    v[:] = 0.25                                     # nothing but constant rows
    refill()
    c.check(*c.run(pq))


def test_q_of_every_size(pq):
    c = Case(pq, "kv8", [50], 1, 4, 64, 16, torch.bfloat16)
    c.q = (c.q.float() * torch.tensor([1e-20, 1e-4, 1.0, 0.0])[None, :, None]).to(torch.bfloat16)
    c.check(*c.run(pq))


@pytest.mark.parametrize("fmt", list(FMT))
def test_hidden_pages(pq, fmt):
    """Page ids outside the cache hide their tokens, also all of them."""
    c = Case(pq, fmt, [150, 60, 20], 2, 3, 64, 16, torch.bfloat16)
    c.table[0, 2], c.table[0, 9], c.table[1, 0] = -1, 1 << 29, c.cache.num_pages
    c.table[2, :2] = -5
    hidden = {(0, t) for t in range(32, 48)} | {(0, t) for t in range(144, 160)} | {(1, t) for t in range(16)} | \
        {(2, t) for t in range(20)}
    c.check(*c.run(pq), hidden=hidden)


@pytest.mark.parametrize("fmt", list(FMT))
def test_what_is_not_attended_is_not_used(pq, fmt):
    """The cache's NaN patterns past len are in every test; here also infinities and the type's lowest values
    before the window, and lengths past the page table."""
    c = Case(pq, fmt, [120], 2, 2, 64, 16, torch.bfloat16)
    want = c.run(pq, window=40)
    for bad in (float("nan"), float("inf"), torch.finfo(torch.bfloat16).min):
        x = torch.full((80, 2, 64), bad, dtype=torch.bfloat16, device=DEV)
        at = torch.arange(80)
        slots = c.table[0, at // 16].long() * 16 + at % 16
        pq.pq_kv_append(c.cache, x, x, slots.to(DEV))
        got = c.run(pq, window=40)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c = Case(pq, fmt, [128], 1, 1, 32, 16, torch.bfloat16)
    c.table = c.table[:, :8].contiguous()           # 128 tokens
    want = c.run(pq)
    c.lens = [2 ** 31 - 1]
    got = c.run(pq)
    assert torch.equal(got[0], want[0])
    c.lens = [-3]
    out, lse = c.run(pq)
    assert torch.count_nonzero(out) == 0 and bool((lse == -math.inf).all())


def test_values_that_are_attended_spread(pq):
    """An infinite or NaN value of an attended token reaches its channel of the output and no other sequence."""
    c = Case(pq, "kv16", [40, 40], 1, 2, 64, 16, torch.bfloat16)
    x = c.v[0][7].to(torch.bfloat16).clone()
    k = c.k[0][7].to(torch.bfloat16)
    x[0, 3], x[0, 9] = float("inf"), float("nan")
    slot = c.table[0, 0].long() * 16 + 7
    pq.pq_kv_append(c.cache, k[None].to(DEV), x[None].to(DEV), slot[None].to(DEV))
    out, lse = c.run(pq)
    assert bool(out[0, :, 9].isnan().all()) and not bool(out[0, :, 3].isfinite().any())
    ok = [i for i in range(64) if i not in (3, 9)]
    assert bool(out[0][:, ok].isfinite().all()) and bool(out[1].isfinite().all()) and bool(lse.isfinite().all())


def test_many_sequences(pq):
    """More sequences than one launch takes."""
    g = torch.Generator().manual_seed(5)
    lens = [int(x) for x in torch.randint(0, 20, (1100,), generator=g)]
    c = Case(pq, "kv8", lens, 1, 2, 16, 16, torch.bfloat16)
    c.check(*c.run(pq))


@pytest.mark.parametrize("fmt", list(FMT))
def test_offsets_past_32_bits(pq, fmt):
    """Pages 3 GiB apart."""
    f, bits = FMT[fmt]
    page, d, n = 16, 64, 45
    row, stride = d * bits // 8, 3 << 30
    kind = torch.bfloat16 if bits == 16 else torch.uint8
    size = kind.itemsize
    raw = [torch.empty(2 * stride + 16 * row + 64, dtype=torch.uint8, device=DEV) for _ in range(2)]
    views = [torch.as_strided(r.view(kind), (3, 1, page, row // size), (stride // size, page * row // size, row // size, 1))
             for r in raw]
    par = [] if bits == 16 else [torch.zeros(3, 1, page, 2, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    c = Case(pq, fmt, [n], 1, 2, d, page, torch.bfloat16)
    c.table = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    old = c.cache
    c.cache = pq.KVCache(f, page, *views, *par)
    for t in range(3):                              # the same rows, in the pages far apart
        src = Case(pq, fmt, [n], 1, 2, d, page, torch.bfloat16).table[0, t]
        for a, b in zip(c.cache.tensors, old.tensors):
            if a is not None:
                a[int(c.table[0, t])] = b[int(src)]
    c.check(*c.run(pq))


@pytest.mark.parametrize("fmt", list(FMT))
def test_decode_step_in_a_graph(pq, fmt):
    """Append (rotating q and k) and attention of one step, captured and replayed with other work in between."""
    f, bits = FMT[fmt]
    b, h, g, d, page = 3, 2, 4, 64, 16
    c = Case(pq, fmt, [40, 17, 1], h, g, d, page, torch.bfloat16)
    q = torch.randn(b, h * g, d, dtype=torch.bfloat16, device=DEV)
    k, v = (torch.randn(b, h, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    lens = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    pos, table = (lens - 1).to(torch.int32), c.table.to(DEV)
    slots = table[torch.arange(b, device=DEV), (pos // page).long()].long() * page + pos % page
    angles = pq.pq_rope_table(64, d)
    q_out, ws = torch.empty_like(q), pq.attn_workspace(c.cache, b, h * g)

    def step(out, stream=None):
        pq.pq_kv_append(c.cache, k, v, slots, positions=pos, table=angles, q=q, q_out=q_out, stream=stream)
        pq.pq_attn_decode(c.cache, q_out, table, lens, out, workspace=ws, stream=stream)
    want, got = torch.empty_like(q), torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(got, stream=side)
    step(want)
    torch.cuda.synchronize()
    for _ in range(3):
        got.fill_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        torch.randn(1 << 20, device=DEV).mul_(3.0)
        torch.cuda.synchronize()
    del graph


def test_without_workspace_on_another_stream(pq):
    c = Case(pq, "kv8", [3000], 2, 4, 64, 16, torch.bfloat16)
    want, _ = c.run(pq)
    side = torch.cuda.Stream()
    out, q = torch.empty(1, 8, 64, dtype=torch.bfloat16, device=DEV), c.q.to(DEV)
    table, lens = c.table.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    pq.pq_attn_decode(c.cache, q, table, lens, out, stream=side)
    side.synchronize()
    assert torch.equal(out.cpu(), want)


def test_one_workspace_for_calls_of_other_sizes(pq):
    """Calls in a row on one stream with one workspace: long and split, short, long again."""
    cases = [Case(pq, f, lens, 2, 4, 64, 16, torch.bfloat16, seed=i)
             for i, (f, lens) in enumerate([("kv8", [6000, 40]), ("kv4", [3]), ("kv16", [4000]), ("kv8", [0, 900, 2])])]
    ws = pq.attn_workspace(cases[0].cache, 3, 8)
    outs = []
    for c in cases * 2:
        b = len(c.lens)
        out, lse = torch.empty(b, 8, 64, dtype=torch.bfloat16, device=DEV), torch.empty(b, 8, device=DEV)
        pq.pq_attn_decode(c.cache, c.q.to(DEV), c.table.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV), out, lse,
                          workspace=ws)
        outs.append((c, out, lse))
    torch.cuda.synchronize()
    for c, out, lse in outs:
        c.check(out.cpu(), lse.cpu())


@pytest.mark.parametrize("fmt,dim", [("kv16", 64), ("kv16", 128), ("kv16", 256), ("kv8", 128), ("kv8", 256)])
@pytest.mark.parametrize("group", [4, 12])
def test_large_caches_are_streamed(pq, fmt, dim, group):
    """A page table that allows over 256 MB of cache takes the reads past the caches."""
    c = Case(pq, fmt, [0, 700, 33, 129], 2, group, dim, 64, torch.bfloat16, seed=dim)
    want = c.run(pq)
    wide = torch.full((4, 1 << 13), -1, dtype=torch.int32)
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    out, lse = c.run(pq)
    c.check(out, lse)
    c.check(*want)


def test_more_rows_than_one_launch_takes(pq):
    """300 sequences of 65520 heads: 19.7 million rows, of which a launch takes 16.8."""
    b, h, d, page = 300, 65520, 16, 16
    cache = pq.KVCache.allocate(pq.PQ_KV_8, 1, page, h, d)
    g = torch.Generator(device=DEV).manual_seed(3)
    k, v = (torch.randn(3, h, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    pq.pq_kv_append(cache, k, v, torch.arange(3, device=DEV))
    q = torch.randn(b, h, d, generator=g, device=DEV).to(torch.bfloat16)
    table, lens = torch.zeros(b, 1, dtype=torch.int32, device=DEV), torch.arange(b, device=DEV).to(torch.int32) % 4
    out = torch.full_like(q, 7.0)
    ws = pq.attn_workspace(cache, b, h)
    pq.pq_attn_decode(cache, q, table, lens, out, workspace=ws)
    part = torch.full_like(q[:100], 7.0)
    for b0 in (0, 100, 200):
        at = slice(b0, b0 + 100)
        pq.pq_attn_decode(cache, q[at], table[at], lens[at], part, workspace=ws)
        assert torch.equal(out[at], part)
    assert torch.count_nonzero(out[::4]) == 0 and bool((out[1::4] != 0).any())
