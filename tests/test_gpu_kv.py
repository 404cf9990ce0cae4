"""pq_kv_append and pq_kv_load on the GPU: codes and pairs bit for bit against
the header's binary32 steps, read-back against binary64."""
import pytest
import torch

import serving_ref as R
from gpu_util import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMT = {"kv16": (0, 16), "kv8": (1, 8), "kv4": (2, 4)}


@pytest.fixture(scope="module")
def pq():
    from bit_quantization_aware_amd import pq as _pq
    assert torch.cuda.is_available()
    return _pq


def make_cache(pq, fmt, pages, page, heads, dim, dtype=torch.bfloat16, token_major=False, fill=0xA5):
    f, bits = FMT[fmt]
    row = dim if bits != 4 else dim // 2
    kind = dtype if bits == 16 else torch.uint8
    shape = (pages, page, heads, row) if token_major else (pages, heads, page, row)
    k, v = (torch.full((*shape, kind.itemsize), fill, dtype=torch.uint8, device=DEV).view(kind).squeeze(-1) for _ in range(2))
    if token_major:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    if bits == 16:
        return pq.KVCache(f, page, k, v)
    par = [torch.full((pages, heads, page, 4), fill, dtype=torch.uint8, device=DEV).view(torch.bfloat16) for _ in range(2)]
    return pq.KVCache(f, page, k, v, *par)


def rows_at(t, slots, page):
    """t [pages, heads, page, x] -> [tokens, heads, x] on the CPU."""
    return t.cpu()[slots // page, :, slots % page]


def rot32(x, table, pos, half):
    return R.rope(x.float(), table, pos, half)      # one rounding an operation, as the kernel


def check_cache(cache, fmt, bits, dtype, slots, page, k, v):
    """k, v [tokens, heads, dim] f32: the values that were stored."""
    ck, cv, kp, vp = cache.tensors
    for c, p, x in ((ck, kp, k), (cv, vp, v)):
        got = rows_at(c, slots, page)
        if bits == 16:
            assert torch.equal(got.view(torch.int16), x.to(dtype).view(torch.int16))
        else:
            n, par = R.quantise(x, bits)
            assert torch.equal(rows_at(p, slots, page).view(torch.int16), par.view(torch.int16))
            assert torch.equal(got, R.pack(n, bits))


CASES = [("kv8", 1, 2, 64, 16), ("kv8", 5, 8, 128, 64), ("kv4", 7, 5, 80, 32), ("kv4", 3, 3, 16, 16), ("kv16", 4, 5, 80, 32),
         ("kv8", 2, 1, 256, 16), ("kv4", 2, 2, 256, 128), ("kv4", 33, 1, 48, 16), ("kv8", 300, 3, 32, 64), ("kv16", 2, 1, 16, 16),
         ("kv4", 6, 2, 208, 16), ("kv8", 2, 70, 64, 16)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rope", ["none", "half", "interleaved", "part"])
@pytest.mark.parametrize("case", CASES)
def test_append(pq, case, rope, dtype):
    fmt, n, h, d, page = case
    print(f"[append {case} {rope} {dtype}]", flush=True)
    f, bits = FMT[fmt]
    ct = torch.float16 if dtype == torch.float16 else torch.bfloat16
    g = torch.Generator().manual_seed(n + d)
    k, v = (torch.randn(n, h, d, generator=g).to(dtype) for _ in range(2))
    pages = (n + page - 1) // page + 2
    slots = torch.randperm(pages * page, generator=g)[:n]
    cache = make_cache(pq, fmt, pages, page, h, d, ct)
    before = [None if t is None else t.cpu().clone() for t in cache.tensors]
    kw, kk = {}, k.float()
    if rope != "none":
        rot = d if rope in ("half", "interleaved") else max(2, d // 2 - 4)     # part: no whole runs of 8 channels
        half = rope != "interleaved"
        a = torch.rand(40, rot // 2, generator=g) * 6.28
        table = torch.stack([a.cos(), a.sin()], -1)
        pos = torch.randint(0, 40, (n,), generator=g, dtype=torch.int32)
        q = torch.randn(n, 2 * h, d, generator=g).to(dtype)
        out = Guarded((n, 2 * h, d), dtype)
        kw = dict(positions=pos.to(DEV), table=table.to(DEV), layout=0 if half else 1, q=q.to(DEV), q_out=out.t)
        kk = rot32(k, table, pos, half)
    pq.pq_kv_append(cache, k.to(DEV), v.to(DEV), slots.to(DEV), **kw)
    torch.cuda.synchronize()
    check_cache(cache, fmt, bits, ct, slots, page, kk, v.float())
    other = torch.ones(pages * page, dtype=torch.bool)
    other[slots] = False
    rest = other.nonzero()[:, 0]
    for t, b in zip(cache.tensors, before):          # the other slots keep their bytes
        if t is not None:
            assert torch.equal(rows_at(t, rest, page).view(torch.uint8), rows_at(b, rest, page).view(torch.uint8))
    if rope != "none":
        out.check("q_out")
        assert torch.equal(out.t.cpu(), rot32(q, table, pos, half).to(dtype))
        qd = q.to(DEV)
        pq.pq_kv_append(cache, k.to(DEV), v.to(DEV), slots.to(DEV), **dict(kw, q=qd, q_out=None))      # in place
        assert torch.equal(qd, out.t)


@pytest.mark.parametrize("fmt", list(FMT))
def test_append_skips_bad_slots_and_takes_strides(pq, fmt):
    """Heads of a fused qkv buffer into token-major pages; slots of padding and past the cache."""
    f, bits = FMT[fmt]
    n, h, d, page, pages = 6, 3, 64, 16, 3
    buf = torch.randn(n, (2 * h + 4) * d).to(torch.bfloat16)
    k, v = buf[:, 4 * d:(4 + h) * d].view(n, h, d), buf[:, (4 + h) * d:].view(n, h, d)
    bd = buf.to(DEV)
    kd, vd = bd[:, 4 * d:(4 + h) * d].view(n, h, d), bd[:, (4 + h) * d:].view(n, h, d)
    slots = torch.tensor([-1, 5, pages * page, 47, -2 ** 62, 20])
    cache = make_cache(pq, fmt, pages, page, h, d, token_major=True)
    before = cache.tensors[0].cpu().clone()
    pq.pq_kv_append(cache, kd, vd, slots.to(DEV))
    ok = torch.tensor([1, 3, 5])
    check_cache(cache, fmt, bits, torch.bfloat16, slots[ok], page, k[ok].float(), v[ok].float())
    rest = torch.tensor([i for i in range(pages * page) if i not in (5, 47, 20)])
    assert torch.equal(rows_at(cache.tensors[0], rest, page).view(torch.uint8), rows_at(before, rest, page).view(torch.uint8))


@pytest.mark.parametrize("fmt", ["kv8", "kv4"])
def test_append_hard_rows(pq, fmt):
    """Constant, tiny, huge and one-outlier rows bit for bit; a NaN or an infinity makes the row read as NaN."""
    f, bits = FMT[fmt]
    d = 64
    k = torch.randn(10, 1, d)
    k[0], k[1], k[2] = 0.0, 0.3, -7.25
    k[3] *= 1e-30
    k[4] *= 1e30
    k[5, 0, 7] = 1e4
    k[6] = k[6].abs() + 100
    k[7] = torch.arange(d) * 0.5                    # many ties
    k[8, 0, 63] = float("nan")
    k[9, 0, 0] = float("inf")
    cache = make_cache(pq, fmt, 1, 16, 1, d)
    slots = torch.arange(10)
    pq.pq_kv_append(cache, k.to(DEV), k.to(DEV), slots.to(DEV))
    check_cache(cache, fmt, bits, None, slots[:8], 16, k[:8], k[:8])
    out = [torch.empty(10, 1, d, device=DEV) for _ in range(2)]
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    pq.pq_kv_load(cache, table, None, torch.tensor([0, 10], dtype=torch.int32, device=DEV), *out)
    assert bool(out[0][8:].isnan().all()) and not bool(out[0][:8].isnan().any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("case", [("kv8", 64, 3, 16, [1, 0, 40, 17]), ("kv4", 80, 5, 32, [33, 64, 7]), ("kv16", 128, 2, 16, [100]),
                                  ("kv4", 16, 1, 64, [0, 0, 3]), ("kv8", 256, 2, 16, [31, 32, 33]), ("kv4", 128, 8, 64, [300, 1]),
                                  ("kv16", 48, 3, 16, [5, 16]), ("kv8", 128, 40, 16, [18])])
def test_load(pq, case, dtype):
    """Ragged sequences from offsets inside them, against binary64."""
    fmt, d, h, page, counts = case
    print(f"[load {case} {dtype}]", flush=True)
    f, bits = FMT[fmt]
    ct = torch.float16 if dtype == torch.float16 else torch.bfloat16
    g = torch.Generator().manual_seed(d)
    starts = [3 * i for i in range(len(counts))]
    need = [(s + c + page - 1) // page + 1 for s, c in zip(starts, counts)]
    pages = sum(need)
    cache = make_cache(pq, fmt, pages, page, h, d, ct, fill=0xFF)            # NaN where nothing was written
    perm = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(counts), max(need) + 1), -7, dtype=torch.int32)   # never followed
    slots, b = [], 0
    for i, (s, c) in enumerate(zip(starts, counts)):
        mine = perm[b:b + need[i]]
        b += need[i]
        table[i, :len(mine)] = torch.tensor(mine)
        slots += [mine[t // page] * page + t % page for t in range(s, s + c)]
    n = len(slots)
    k, v = (torch.randn(n, h, d, generator=g).to(dtype) for _ in range(2))
    slots = torch.tensor(slots)
    pq.pq_kv_append(cache, k.to(DEV), v.to(DEV), slots.to(DEV))
    cu = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(DEV)
    out = [Guarded((n, h, d), dtype) for _ in range(2)]
    pq.pq_kv_load(cache, table.to(DEV), torch.tensor(starts, dtype=torch.int32, device=DEV), cu, out[0].t, out[1].t)
    torch.cuda.synchronize()
    for o, x in zip(out, (k, v)):
        o.check("k_out / v_out")
        if bits == 16:
            assert torch.equal(o.t.cpu(), x.to(ct).to(dtype))
            continue
        codes, par = R.quantise(x.float(), bits)
        want = R.values(R.pack(codes, bits), par, bits)
        # z + s n in binary32 (s n is exact), then the type's rounding
        lim = 2.0 ** -24 * want.abs() + (R.U[dtype] * want.abs() if dtype != torch.float32 else 0) * 1.01 + R.TINY[dtype]
        assert bool(((o.t.cpu().double() - want).abs() <= lim).all())


def test_load_without_a_source_reads_zero(pq):
    """Page ids outside the cache, tokens past the table's columns and rows past cu[batch]."""
    cache = make_cache(pq, "kv16", 2, 16, 1, 16, fill=0x3F)
    table = torch.tensor([[1, 5, -1]], dtype=torch.int32, device=DEV)
    k, v = (torch.full((70, 1, 16), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pq.pq_kv_load(cache, table, None, torch.tensor([0, 60], dtype=torch.int32, device=DEV), k, v)
    assert bool((k[:16] != 0).all()) and torch.count_nonzero(k[16:]) == 0 and torch.count_nonzero(v[16:]) == 0
    pq.pq_kv_load(cache, table[:, :0], None, torch.tensor([0, 60], dtype=torch.int32, device=DEV), k, v)
    assert torch.count_nonzero(k) == 0


def test_many_sequences(pq):
    """More sequences than tokens of a block, many of them empty."""
    g = torch.Generator().manual_seed(8)
    counts = [int(x) for x in torch.randint(0, 3, (700,), generator=g)]
    n = sum(counts)
    cache = make_cache(pq, "kv8", 700, 16, 1, 32)
    x = torch.randn(n, 1, 32, generator=g)
    seq = torch.cat([torch.full((c,), i, dtype=torch.int64) for i, c in enumerate(counts)])
    at = torch.cat([torch.arange(c) for c in counts])
    pq.pq_kv_append(cache, x.to(DEV), -x.to(DEV), (seq * 16 + at).to(DEV))
    out = [torch.empty(n, 1, 32, device=DEV) for _ in range(2)]
    cu = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(DEV)
    pq.pq_kv_load(cache, torch.arange(700, dtype=torch.int32, device=DEV)[:, None], None, cu, *out)
    codes, par = R.quantise(x, 8)
    assert torch.equal(out[0].cpu(), R.values(codes, par, 8).float())


@pytest.mark.parametrize("fmt", ["kv16", "kv8", "kv4"])
def test_offsets_past_32_bits(pq, fmt):
    """Pages 3 GiB apart."""
    f, bits = FMT[fmt]
    page, d = 16, 64
    row = R.unpack(torch.zeros(1, d, dtype=torch.uint8), 8).shape[1] * bits // 8
    stride = 3 << 30
    raw = [torch.empty(2 * stride + 16 * row + 64, dtype=torch.uint8, device=DEV) for _ in range(2)]
    kind = torch.bfloat16 if bits == 16 else torch.uint8
    size = kind.itemsize
    views = [torch.as_strided(r.view(kind), (3, 1, page, row // size), (stride // size, page * row // size, row // size, 1))
             for r in raw]
    par = [] if bits == 16 else [torch.zeros(3, 1, page, 2, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    cache = pq.KVCache(f, page, *views, *par)
    x = torch.randn(3, 1, d).to(torch.bfloat16)
    pq.pq_kv_append(cache, x.to(DEV), x.to(DEV), torch.tensor([5, 16 + 6, 32 + 15], device=DEV))
    out = [torch.empty(3, 1, d, device=DEV) for _ in range(2)]
    table = torch.tensor([[0], [1], [2]], dtype=torch.int32, device=DEV)
    pq.pq_kv_load(cache, table, torch.tensor([5, 6, 15], dtype=torch.int32, device=DEV),
                  torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV), *out)
    if bits == 16:
        want = x.float()
    else:
        n, p = R.quantise(x.float(), bits)
        want = R.values(R.pack(n, bits), p, bits).float()
    assert torch.equal(out[0].cpu(), want) and torch.equal(out[1].cpu(), want)


@pytest.mark.parametrize("dim", range(16, 257, 16))
@pytest.mark.parametrize("fmt", ["kv8", "kv4"])
def test_every_row_length(pq, fmt, dim):
    """Rows side by side over a wave's lanes, whatever their length; the smallest and the largest value on each lane in turn."""
    f, bits = FMT[fmt]
    n, h, page = dim // 8, 7, 16
    g = torch.Generator().manual_seed(dim)
    k, v = (torch.randn(n, h, dim, generator=g).to(torch.bfloat16) for _ in range(2))
    for i in range(n):
        k[i, :, 8 * i + 3], k[i, :, (8 * i + 11) % dim] = -9.0, 11.0
        v[i, :, (8 * i + 6) % dim], v[i, :, (8 * i - 4) % dim] = 12.0, -8.0
    slots = torch.randperm(2 * page, generator=g)[:n]
    cache = make_cache(pq, fmt, 2, page, h, dim)
    pq.pq_kv_append(cache, k.to(DEV), v.to(DEV), slots.to(DEV))
    check_cache(cache, fmt, bits, torch.bfloat16, slots, page, k.float(), v.float())
    out = [Guarded((n, h, dim), torch.float32) for _ in range(2)]       # the first n slots, in order
    pq.pq_kv_load(cache, torch.tensor([[0, 1]], dtype=torch.int32, device=DEV), None,
                  torch.tensor([0, n], dtype=torch.int32, device=DEV), out[0].t, out[1].t)
    at = {int(s): i for i, s in enumerate(slots)}
    for x, o in ((k, out[0]), (v, out[1])):
        codes, par = R.quantise(x.float(), bits)
        want = R.values(R.pack(codes, bits), par, bits)
        mag = par.double()[..., 1:].abs() + par.double()[..., :1] * codes.double()
        for t in range(n):
            if t in at:             # one binary32 product and sum
                err = (o.t[t].cpu().double() - want[at[t]]).abs()
                assert (err <= 2.0 ** -23 * mag[at[t]]).all()
        o.check("k_out / v_out")


@pytest.mark.parametrize("dim", range(16, 257, 16))
@pytest.mark.parametrize("fmt", list(FMT))
def test_every_row_length_reads_back(pq, fmt, dim):
    """Every token written is read and compared, wherever its slot is."""
    f, bits = FMT[fmt]
    n, h, page = 32, 5, 16
    g = torch.Generator().manual_seed(dim + 1)
    k, v = (torch.randn(n, h, dim, generator=g).to(torch.bfloat16) for _ in range(2))
    slots = torch.randperm(2 * page, generator=g)
    cache = make_cache(pq, fmt, 2, page, h, dim)
    pq.pq_kv_append(cache, k.to(DEV), v.to(DEV), slots.to(DEV))
    out = [Guarded((n, h, dim), torch.float32) for _ in range(2)]
    pq.pq_kv_load(cache, torch.tensor([[0, 1]], dtype=torch.int32, device=DEV), None,
                  torch.tensor([0, n], dtype=torch.int32, device=DEV), out[0].t, out[1].t)
    torch.cuda.synchronize()
    for x, o in ((k, out[0]), (v, out[1])):
        o.check("k_out / v_out")
        got = o.t.cpu()[slots].double()             # slot s is row s of the output
        assert got.shape[0] == n
        if bits == 16:
            assert torch.equal(got, x.double())
            continue
        codes, par = R.quantise(x.float(), bits)
        want = R.values(R.pack(codes, bits), par, bits)
        mag = par.double()[..., 1:].abs() + par.double()[..., :1] * codes.double()
        assert bool(((got - want).abs() <= 2.0 ** -23 * mag).all())       # one binary32 product and sum
