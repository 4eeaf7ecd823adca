"""Plain 64-bit definitions of the routing, dispatch, combine and MXFP4 calls,
on CPU tensors, for their tests.  Written from the formulas; shares no code
with the package."""
from __future__ import annotations

import math

import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def route(logits, k, renorm):
    """(ids, weights in float64, group_sizes, row_of_slot, slot_of_row) of
    logits [T, E], one token at a time."""
    T, E = logits.shape
    x = logits.double()
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros((T, k), dtype=torch.float64)
    for t in range(T):
        row = x[t].tolist()
        key = lambda e: (0 if math.isnan(row[e]) else 1, 0.0 if math.isnan(row[e]) else -row[e], e)
        chosen = [e for e in sorted(range(E), key=key)[:k] if row[e] != -math.inf]
        if not chosen:
            continue
        top = row[chosen[0]]
        some = [row[e] for e in chosen] if renorm else row
        total = sum(math.exp(v - top) if v != -math.inf else 0.0 for v in some) if math.isfinite(top) else math.nan
        for j, e in enumerate(chosen):
            ids[t, j] = e
            w[t, j] = math.exp(row[e] - top) / total if math.isfinite(total) else math.nan
    flat = ids.reshape(-1).tolist()
    slots = sorted((s for s in range(T * k) if flat[s] >= 0), key=lambda s: (flat[s], s))
    rows = torch.full((T * k,), -1, dtype=torch.int32)
    slot_of_row = torch.full((T * k,), -1, dtype=torch.int32)
    for r, s in enumerate(slots):
        rows[s], slot_of_row[r] = r, s
    sizes = torch.tensor([flat.count(e) for e in range(E)], dtype=torch.int32)
    return ids, w, sizes, rows.view(T, k), slot_of_row


def route_bwd(dweights, logits, ids, weights, renorm):
    """(d logits, sum of the magnitudes of its terms) in float64."""
    x, w, dw = logits.double(), weights.double(), dweights.double()
    here = ids >= 0
    w, dw = torch.where(here, w, 0.0), torch.where(here, dw, 0.0)
    inner = (w * dw).sum(1, keepdim=True)
    inner_abs = (w * dw).abs().sum(1, keepdim=True)
    d, a = torch.zeros_like(x), torch.zeros_like(x)
    at = ids.clamp(min=0).long()
    d.scatter_add_(1, at, w * (dw - inner) if renorm else w * dw)
    a.scatter_add_(1, at, w * (dw.abs() + inner_abs) if renorm else (w * dw).abs())
    if not renorm:
        p = torch.nan_to_num(torch.softmax(x, 1))
        d, a = d - p * inner, a + p * inner_abs
    return d, a


def combine(y, rows, weights):
    """(sum, sum of magnitudes) in float64 of y's rows; rows outside y count as zero."""
    T, k = rows.shape
    out, mag = torch.zeros((T, y.shape[1]), dtype=torch.float64), torch.zeros((T, y.shape[1]), dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            r = int(rows[t, j])
            if 0 <= r < y.shape[0]:
                v = y[r].double() * (1.0 if weights is None else float(weights[t, j]))
                out[t] += v
                mag[t] += v.abs()
    return out, mag


def mxfp4(x):
    """(codes of one value a byte, E8M0 bytes) of x [.., K] in blocks of 32:
    the nearest of the sixteen values, the even code on a tie."""
    v = x.double().unflatten(-1, (-1, 32))
    amax = v.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    power = torch.where((amax > 0) & ~bad, torch.frexp(torch.where(bad, 1.0, amax))[1].double() - 3, -127.0)
    power = power.clamp(min=-127)
    u = torch.where(bad.unsqueeze(-1), 0.0, v) * torch.exp2(-power).unsqueeze(-1)
    table = torch.tensor(E2M1, dtype=torch.float64)
    dist = (u.abs().unsqueeze(-1) - table).abs()
    best = dist.amin(-1, keepdim=True)
    parity = torch.arange(8) % 2
    code = torch.where(dist == best, parity + 0 * dist, 9.0).argmin(-1)      # an even code wins a tie
    code = torch.where(torch.signbit(v), code + 8, code)
    byte = torch.where(bad, 255, power + 127)
    return code.to(torch.uint8).flatten(-2), byte.to(torch.uint8)


def mxfp4_values(code, byte):
    """float64 values of one code a byte [.., K] and E8M0 bytes [.., K/32]."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64)
    unit = torch.where(byte == 255, math.nan, torch.exp2(byte.double() - 127))
    return (table[code.long()].unflatten(-1, (-1, 32)) * unit.unsqueeze(-1)).flatten(-2)


def pack_weights(code, byte):
    """The library's layout of codes [G, N, K] and bytes [G, N, K/32]."""
    pair = code.unflatten(-1, (-1, 2))
    G, N, nb = byte.shape
    return (pair[..., 0] | (pair[..., 1] << 4)).contiguous(), byte.view(G, N, nb // 4, 4).transpose(1, 2).contiguous()
