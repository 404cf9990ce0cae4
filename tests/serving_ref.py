"""Plain references of the serving operators on the CPU: rotation, the cache's
quantiser and attention, in binary64 (the quantiser also in binary32, step by
step as include/pq.h states it, for bit-exact comparisons)."""
import math

import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}      # unit roundoff
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}
TOP = {8: 255, 4: 15}
MIN_SCALE = 2.0 ** -60


def rope_freqs(rot, base, kind="plain", factor=1.0, trained=0.0, fast=32.0, slow=1.0):
    """(frequencies [rot / 2], magnitude) of a scaling, binary64."""
    if kind == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = np.array([base ** (-2.0 * c / rot) for c in range(rot // 2)])
    if kind in ("plain", "ntk"):
        return f, 1.0
    if kind == "linear":
        return f / factor, 1.0
    if kind == "yarn":
        def index(turns):
            return rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo = min(max(math.floor(index(fast)), 0), rot - 1)
        hi = min(max(math.ceil(index(slow)), 0), rot - 1)
        if hi <= lo:
            hi = lo + 0.001
        g = 1 - np.clip((np.arange(rot // 2) - lo) / (hi - lo), 0, 1)
        return f / factor * (1 - g) + f * g, 0.1 * math.log(factor) + 1.0
    assert kind == "bands"
    out = []
    for x in f:
        wave = 2 * math.pi / x
        if wave > trained / slow:
            out.append(x / factor)
        elif wave < trained / fast:
            out.append(x)
        else:
            g = (trained / wave - slow) / (fast - slow)
            out.append((1 - g) * x / factor + g * x)
    return np.array(out), 1.0


def pair_index(rot, half):
    """Channels (first, second) of each pair."""
    c = torch.arange(rot // 2)
    return (c, c + rot // 2) if half else (2 * c, 2 * c + 1)


def rope(x, table, positions, half, inverse=False):
    """x [tokens, heads, dim] of any float type, computed in x's type; table
    [max_pos, rot / 2, 2].  Positions below 0 leave the row, past the table give NaN."""
    y = x.clone()
    rot = 2 * table.shape[1]
    a, b = pair_index(rot, half)
    for t, p in enumerate(positions.tolist()):
        if p < 0:
            continue
        if p >= table.shape[0]:
            y[t, :, :rot] = float("nan")
            continue
        cos, sin = table[p, :, 0].to(x.dtype), table[p, :, 1].to(x.dtype)
        if inverse:
            sin = -sin
        y[t][:, a] = x[t][:, a] * cos - x[t][:, b] * sin
        y[t][:, b] = x[t][:, b] * cos + x[t][:, a] * sin
    return y


def quantise(x, bits):
    """Binary32 steps of the header: codes uint8 (unpacked) and bf16 pairs (s, z) of rows x [..., dim] f32."""
    top = np.float32(TOP[bits])
    x = x.float()
    mn, mx = x.amin(-1), x.amax(-1)
    s = ((mx - mn) * torch.tensor(np.float32(1) / top)).to(torch.bfloat16)
    s = torch.maximum(s.float(), torch.tensor(MIN_SCALE, dtype=torch.float32))
    z = mn.to(torch.bfloat16)
    r = torch.ones_like(s) / s
    n = torch.round((x - z.float()[..., None]) * r[..., None]).clamp(0, float(top))
    return n.to(torch.uint8), torch.stack([s.to(torch.bfloat16), z], -1)


def pack(n, bits):
    return n if bits == 8 else n[..., 0::2] | (n[..., 1::2] << 4)


def unpack(codes, bits):
    return codes if bits == 8 else torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def values(codes, param, bits):
    """What codes stand for, binary64."""
    p = param.double()
    return p[..., 1:] + p[..., :1] * unpack(codes, bits).double()


def attention(q, k, v, scale):
    """One sequence and cache head: q [group, dim], k, v [tokens, dim] in binary64 -> out, lse, weights."""
    g, d = q.shape
    if k.shape[0] == 0:
        return torch.zeros(g, d, dtype=torch.float64), torch.full((g,), -math.inf, dtype=torch.float64), \
            torch.zeros(g, 0, dtype=torch.float64)
    x = (q @ k.T) * scale
    m = x.max(-1, keepdim=True).values
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    return (p / total) @ v, (m + total.log())[:, 0], p / total
