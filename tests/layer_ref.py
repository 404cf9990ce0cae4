"""Binary64 references of the operators around the packed product, from the
formulas in include/pq.h: norm and its gradient, rows in 8 bits, the product of
8-bit activations with its epilogue, distillation and its gradient."""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}     # half a step, relative
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}   # half the smallest step
MIN_SCALE = 2.0 ** -60
# mode -> (code bits, number of codes, level = (step c - shift) unit)
LEVELS = {0: (1, 2, 2, 1, 1.0), 1: (2, 3, 1, 1, float(torch.tensor(2.0 / 3.0))), 2: (2, 4, 2, 3, 0.25), 3: (4, 8, 1, 4, 1.0),
          4: (4, 16, 1, 8, 1.0), 5: (2, 4, 1, 2, 1.0), 6: (2, 3, 1, 1, 1.0)}


def norm(h, weight, eps):
    """y and rstd of rows h, f64."""
    rstd = (h.double().square().mean(-1) + eps).rsqrt()
    return h.double() * rstd[:, None] * weight.double(), rstd


def norm_grad(h, weight, rstd, dy, dsum=None):
    """dx, dweight, and the sizes of what dx and dweight are sums of, f64."""
    n, dy = h.double() * rstd.double()[:, None], dy.double()
    g = dy * weight.double()
    dx = rstd.double()[:, None] * (g - n * (g * n).mean(-1, keepdim=True))
    size = rstd.double()[:, None] * (g.abs() + n.abs() * (g * n).abs().mean(-1, keepdim=True))
    if dsum is not None:
        dx, size = dx + dsum.double(), size + dsum.double().abs()
    return dx, (dy * n).sum(0), size, (dy * n).abs().sum(0)


def row_scale(y):
    return (y.double().abs().amax(-1) / 127).clamp_min(MIN_SCALE)


def pack(codes, bits):
    """Codes [n, k] uint8 in the export byte order, spelt out byte by byte from its definition."""
    n, k = codes.shape
    c = codes.to(torch.int64).tolist()
    rb = k * bits // 8
    groups, np_ = -(-rb // 64), -(-n // 16) * 16
    out = bytearray(groups * np_ * 64)
    for r in range(n):
        row = bytearray(rb)
        if bits == 2:
            for w in range(rb // 4):
                for j in range(4):
                    s = c[r][16 * w:16 * w + 16]
                    row[4 * w + j] = s[2 * j] | s[8 + 2 * j] << 2 | s[2 * j + 1] << 4 | s[9 + 2 * j] << 6
        else:
            per = 8 // bits
            for b in range(rb):
                row[b] = sum(c[r][per * b + i] << (bits * i) for i in range(per))
        for b in range(rb):
            out[(b // 64) * np_ * 64 + (r // 16) * 1024 + (r % 16) * 64 + b % 64] = row[b]
    return torch.frombuffer(out, dtype=torch.uint8).clone()


def levels(codes, mode):
    _, _, step, shift, unit = LEVELS[mode]
    return (codes.double() * step - shift) * unit


def act(v, kind):
    if kind == 1:
        return v.clamp_min(0.0)
    if kind == 2:
        return v * torch.sigmoid(v)
    if kind == 3:
        return 0.5 * v * torch.special.erfc(-v * math.sqrt(0.5))
    if kind == 4:
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def product(x, x_scale, lev, alpha, bias=None, kind=0, other=None, mul=False):
    """y and a bound of its binary32 error before the last rounding, f64."""
    s = (x.double() @ lev.T) * x_scale.double()[:, None] * alpha.double()
    b = torch.zeros_like(s) if bias is None else bias.double().expand_as(s)
    v = s + b
    # the scales' two products, the sum's conversion and the sum with the bias: a rounding each; no activation is steeper
    # than 1.13; evaluating one costs a few units of |v| in the last place
    err = 1.13 * 5 * 2.0 ** -24 * (s.abs() + b.abs()) + (2.0 ** -20 * v.abs() if kind else 0.0)
    y = act(v, kind)
    if other is not None:
        o = other.double()
        y, err = (y * o, err * o.abs() + 2.0 ** -24 * (y * o).abs()) if mul else (y + o, err + 2.0 ** -24 * (y + o).abs())
    return y, err


def distill(z, index, top, temp, weight=None):
    """Loss per row, its gradient to z, p spread over the words, q: f64."""
    rows, v = z.shape
    z, top = z.double() / temp, top.double() / temp
    valid = (index >= 0) & (index < v)
    at = index.long().clamp(0, v - 1)
    p = torch.softmax(top.masked_fill(~valid, -math.inf), -1)
    p = torch.where(valid, p, torch.zeros_like(p))
    log_q = torch.log_softmax(z, -1)
    terms = torch.where(p > 0, p * (torch.log(p) - log_q.gather(1, at)), torch.zeros_like(p))
    loss = temp ** 2 * terms.sum(-1)
    target = torch.zeros_like(z).scatter_add_(1, at, p)
    q = log_q.exp()
    dz = temp * (q - target)
    w = torch.ones(rows, dtype=torch.float64, device=z.device) if weight is None else weight.double()
    none = (~valid).all(-1) | (w == 0)
    loss = torch.where(none, torch.zeros_like(loss), loss * w)
    dz = torch.where(none[:, None], torch.zeros_like(dz), dz * w[:, None])
    return loss, dz, target, q
