"""Plain 64-bit definitions of the balance losses, the AdamW step and the FP8
weight quantizer, on CPU tensors, for their tests.  Written from the formulas;
shares no code with the package."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24     # half a step of f32, relative
BLOCK = 256


# --------------------------------------------------------------------------- balance losses

def softmax(x):
    """(p, lse, whether the token counts) of logits x [T, E], float64."""
    x = x.double()
    here = (x != -math.inf).any(1)
    odd = torch.isnan(x).any(1) | (x == math.inf).any(1)
    fine = torch.where((here & ~odd).unsqueeze(1), x, 0.0)
    top = fine.amax(1, keepdim=True)                       # taken off first: logits near f32's largest
    e = torch.exp(fine - top)
    total = e.sum(1, keepdim=True)
    lse = torch.where(odd, math.nan, torch.where(here, (top + torch.log(total)).squeeze(1), 0.0))
    p = e / total
    return torch.where(odd.unsqueeze(1), math.nan, torch.where(here.unsqueeze(1), p, 0.0)), lse, here


def balance(x, ids=None, counts=None):
    """(losses, counts, probs, n), float64 and integers."""
    T, E = x.shape
    p, lse, here = softmax(x)
    n = int(here.sum())
    if counts is None:
        flat = ids.reshape(-1).tolist()
        counts = torch.tensor([flat.count(e) for e in range(E)], dtype=torch.int64)
    c = counts.double().clamp(min=0)
    probs = p.sum(0) / max(n, 1)
    total = float(c.sum())
    first = E * float((c * probs).sum()) / total if n and total else 0.0
    second = float((lse * lse).sum()) / n if n else 0.0
    return torch.tensor([first, second], dtype=torch.float64), counts, probs, n


def balance_tolerances(x, T):
    """(relative error of probs and of the first loss, absolute error of the second).
    A probability: the rounded difference in the exponential (up to 104 before it vanishes) for itself and the
    sum, and 30 for exponentials, sums over 16 + 6 levels and the quotient.  Their sum over tokens is of
    positive terms: its levels are a lane's tokens, 2 + 16 in a block, the blocks' partials (256 of them in one
    chain at most) and 16 groups.  lse: the sum's relative error, 2 steps of the logarithm, the addition."""
    levels = -(-T // 4096) + 18 + 256 + 16
    relative = U32 * (2 * 104 + 30 + levels + 4)
    _, lse, here = softmax(x)
    lse = lse[here]
    n = max(1, lse.numel())
    one = U32 * (2 * 104 + 30 + 3 * lse.abs() + 3 * 7)
    z = float((2 * lse.abs() * one + one * one + U32 * (levels + 4) * lse * lse).sum()) / n
    return relative, z


def balance_bwd(dlosses, x, counts, n, add=None):
    """(dlogits, sum of the magnitudes of its terms) in float64."""
    E = x.shape[1]
    p, lse, here = softmax(x)
    c = counts.double().clamp(min=0)
    total = float(c.sum())
    a = float(dlosses[0]) * E / (n * total) if n and total else 0.0
    b = float(dlosses[1]) * 2 / n if n else 0.0
    c = c - total / E
    d = p * (a * (c - (p * c).sum(1, keepdim=True)) + b * lse.unsqueeze(1))
    mag = p * (abs(a) * (c.abs() + (p * c.abs()).sum(1, keepdim=True)) + abs(b) * lse.abs().unsqueeze(1))
    d = torch.where(here.unsqueeze(1), d, 0.0)
    return (d, mag) if add is None else (d + add.double(), mag + add.double().abs())


# --------------------------------------------------------------------------- AdamW

class Step:
    """An AdamW step's numbers, and one on tensors of float64."""

    def __init__(self, lr, step, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, scale=1.0):
        self.lr, self.t, (self.b1, self.b2), self.eps, self.wd, self.scale = lr, step, betas, eps, weight_decay, scale

    def __call__(self, p, g, m, v):
        """New p, m, v and their error bounds in f32 arithmetic.  A coefficient, a product and a sum round by U32
        each: m has 5 of them, v 7; the quotient's error comes from m's, half of v's, and 12 more (bias
        corrections, root, products, eps, division); p's own decay 4 and its sums 2."""
        g = g * self.scale
        m1, v1 = self.b1 * m + (1 - self.b1) * g, self.b2 * v + (1 - self.b2) * g * g
        em = 5 * U32 * (self.b1 * m.abs() + (1 - self.b1) * g.abs()) + 2.0 ** -148
        ev = 7 * U32 * v1 + 2.0 ** -148
        up = self.lr / (1 - self.b1 ** self.t)
        below = torch.sqrt(v1) / math.sqrt(1 - self.b2 ** self.t) + self.eps
        move = up * m1 / below
        p1 = p - (self.lr * self.wd * p + move)
        some = v1 > 0
        half = torch.where(some, ev / (2 * torch.where(some, v1, 1.0)), 0.0)
        ep = up * em / below + move.abs() * (half + 12 * U32) + 4 * U32 * self.lr * self.wd * p.abs() + \
            2 * U32 * (p.abs() + p1.abs() + move.abs()) + 2.0 ** -148
        return (p1, m1, v1), (ep, em, ev)


def _mix(x):
    m = 0xFFFFFFFF
    x = (x ^ (x >> 16)) * 0x6A09E667 & m
    x = (x ^ (x >> 15)) * 0xBB67AE85 & m
    return x ^ (x >> 16)


def noise(seed, step, tensor, size):
    """(u of m, u of r) in (0, 1) for a tensor's elements, float64 [size]."""
    m = 0xFFFFFFFF
    key = _mix((seed & m) + _mix((seed >> 32) + _mix(step & m) & m) & m)
    key = _mix(key + tensor & m)
    h = torch.empty(size, dtype=torch.int64)
    for b in range(-(-size // BLOCK)):
        kb = _mix(key + b & m)
        for j in range(min(BLOCK, size - b * BLOCK)):
            h[b * BLOCK + j] = _mix(kb + 0x9E3779B9 * j & m)
    return ((h & 0xFFFF).double() + 0.5) / 65536, ((h >> 16).double() + 0.5) / 65536


def e4m3(codes):
    """float64 values of e4m3fn codes, by the format."""
    c = codes.long()
    sign, e, f = 1 - 2 * (c >> 7), c >> 3 & 15, c & 7
    v = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2((e - 10).double()))
    return torch.where((c & 127) == 127, math.nan, sign * v)


def values(codes, scales):
    """float64 of a state's codes (any shape) and scales, flat."""
    c = e4m3(codes.reshape(-1))
    return c * scales.double().repeat_interleave(BLOCK)[:c.numel()]


def scales_of(x):
    """max |x| / 448 of each block."""
    n = x.numel()
    pad = torch.zeros(-(-n // BLOCK) * BLOCK, dtype=torch.float64)
    pad[:n] = x.abs()
    return pad.view(-1, BLOCK).amax(1) / 448


def held(x, scales, u, positive, error):
    """The lowest and the highest value (in units of its block's scale) that x may be held as, `error` off."""
    s = scales.repeat_interleave(BLOCK)[:x.numel()]
    q = torch.where(s > 0, x.abs() / torch.where(s > 0, s, 1.0), 0.0)
    off = torch.where(s > 0, error / torch.where(s > 0, s, 1.0), 0.0) + 8 * U32 * q + 2.0 ** -29
    out = []
    for v in ((q - off).clamp(min=0), q + off):
        d = torch.exp2(torch.floor(torch.log2(v.clamp(min=2.0 ** -6))) - 3)
        w = (torch.floor(v / d + u) * d).clamp(max=448)
        w = torch.where((x > 0) & (s > 0), w.clamp(min=2.0 ** -9), w) if positive else w
        out.append(torch.where(s > 0, w, 0.0))
    return out


# --------------------------------------------------------------------------- FP8 weights

def quantize_weights(w):
    """(values of the codes in float64, NaN for NaN codes; scales f32) of w [G, K, N]."""
    x = w.float()
    top = torch.where(torch.isnan(x), 0.0, x.abs()).amax(1).clamp(min=1e-12)
    scale = top / torch.tensor(448.0)                     # f32 divisions, correctly rounded on the CPU
    q = (x / scale.unsqueeze(1)).double()
    d = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))).clamp(max=8) - 3)
    return torch.where(torch.isnan(q), math.nan, (torch.round(q / d) * d).clamp(-448, 448)), scale
