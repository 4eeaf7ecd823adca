"""The cases on which the MoE layer's routing, dispatch, combine and MXFP4
operators are measured, with their plain forms in elementary torch operations.

A case is a dict of plain values; its ``kind`` names the operator.  ``run``
computes one pass in the plain form or, where ``own`` is set, through the
package's entry points.
"""
import math

import torch

own = False

BLOCK = 32  # values that share one scale of the microscaled format


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token choosing 8 of 256 experts: latency alone
        dict(name="route_token", kind="route", T=1, E=256, k=8, dtype="float32", renorm=True, masked=False),
        # a training batch of bf16 logits, whose ties are many
        dict(name="route_batch", kind="route", T=16384, E=256, k=8, dtype="bfloat16", renorm=True, masked=False),
        # the router's gradient with weights taken from the softmax over all experts, some of them masked
        dict(name="route_grad", kind="route_grad", T=16384, E=160, k=6, dtype="float32", renorm=False, masked=True),
        # the dropless width (7168) in training: each token's row to its experts' rows
        dict(name="permute_train", kind="permute", T=4096, H=7168, k=8, E=256),
        # the same on the way into the FP8 forward, an odd number of tokens
        dict(name="permute_fp8", kind="permute_fp8", T=2999, H=2048, k=6, E=64),
        # a few decoded tokens coming back from their experts
        dict(name="combine_few", kind="combine", T=16, H=7168, k=8, E=32, weighted=True),
        # a training batch coming back
        dict(name="combine_train", kind="combine", T=4096, H=7168, k=8, E=256, weighted=True),
        # its gradient, to the experts' rows and to the weights
        dict(name="combine_grad", kind="combine_grad", T=4096, H=7168, k=8, E=256),
        # a checkpoint's expert weights to 4 bits, seen through their values
        dict(name="mxfp4_weights", kind="mxfp4_weights", G=8, K=7168, N=2048),
        # one token's 8 experts of 32 in the first product: bound by the weights' bytes
        dict(name="mxfp4_token", kind="mxfp4", T=1, k=8, G=32, K=7168, N=4096, swiglu=True, skew=0.0),
        # the second product of a middling batch, short contraction, ragged groups
        dict(name="mxfp4_wo", kind="mxfp4", T=8190, k=1, G=8, K=768, N=2048, swiglu=False, skew=0.5),
        # the dropless first product of a large prefill over skewed groups
        dict(name="mxfp4_wi", kind="mxfp4", T=5000, k=4, G=32, K=7168, N=4096, swiglu=True, skew=1.1),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["route", "route_grad", "permute", "permute_fp8", "combine", "combine_grad", "mxfp4_weights",
                       "mxfp4", "mxfp4", "mxfp4"])
    if kind in ("route", "route_grad"):
        E = _log(rng, 8, 512)
        return dict(kind=kind, T=_log(rng, 1, 16384), E=E, k=rng.randint(1, min(E, 10)),
                    dtype=rng.choice(["float32", "bfloat16"]), renorm=rng.random() < 0.5, masked=rng.random() < 0.5)
    if kind in ("permute", "permute_fp8", "combine", "combine_grad"):
        c = dict(kind=kind, T=_log(rng, 1, 4096), H=128 * rng.randint(1, 56), k=rng.randint(1, 8),
                 E=_log(rng, 8, 256))
        if kind == "combine":
            c["weighted"] = rng.random() < 0.7
        return c
    if kind == "mxfp4_weights":
        return dict(kind=kind, G=rng.randint(1, 8), K=128 * rng.randint(1, 56), N=128 * rng.randint(1, 16))
    G = _log(rng, 2, 32)
    return dict(kind=kind, T=_log(rng, 1, 4096), k=rng.randint(1, min(G, 4)), G=G, K=128 * rng.randint(1, 56),
                N=256 * rng.randint(1, 16), swiglu=rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 1.1]))


def work(case):
    kind = case["kind"]
    if kind in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        b = 4 if case["dtype"] == "float32" else 2
        if kind == "route":
            return {"bytes": T * E * b + 16 * T * k + 4 * E, "flops": 0}
        return {"bytes": T * E * b * (1 if case["renorm"] else 2) + 12 * T * k, "flops": 0}
    if kind == "mxfp4_weights":
        n = case["G"] * case["K"] * case["N"]
        return {"bytes": 4 * n, "flops": 0}
    if kind == "mxfp4":
        M = case["T"] * case["k"]
        K, N = case["K"], case["N"]
        hit = min(case["G"], M)
        return {"bytes": hit * N * K * 17 / 32 + 2 * case["T"] * K + M * (4 + N * (1 if case["swiglu"] else 2)),
                "flops": 2 * M * K * N}
    T, H, k = case["T"], case["H"], case["k"]
    one, many = 2 * T * H, 2 * T * H * k
    if kind == "permute":
        return {"bytes": one + many + 4 * T * k, "flops": 0}
    if kind == "permute_fp8":
        return {"bytes": one + many // 2 + 8 * T * k, "flops": 0}
    if kind == "combine":
        return {"bytes": one + many + (8 if case["weighted"] else 4) * T * k, "flops": 2 * T * H * k}
    return {"bytes": one + 2 * many + 12 * T * k, "flops": 3 * T * H * k}


# --------------------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=g.device)


def _activations(g, rows, width):
    """N(0, 1) with one entry in a hundred 50 times as large."""
    x = _normal(g, rows, width)
    big = torch.rand((rows, width), generator=g, device=g.device) < 0.01
    return torch.where(big, 50 * x, x).to(torch.bfloat16)


def _logits(g, T, E, skew=0.5):
    """Router logits: some experts are liked more than others by every token."""
    return _normal(g, T, E) + skew * _normal(g, E)


def _routing(g, T, E, k, skew):
    """(ids, group_sizes, row_of_slot, slot_of_row) of random choices without
    repeats, as a program has them after its router."""
    ids = torch.topk(_logits(g, T, E, skew), k, dim=1).indices.to(torch.int32)
    return (ids,) + _sort(ids, E)


def _layout_mxfp4(values, exponents):
    """Codes [G, N, K/2] (the even k of a pair in the low half byte) and scales
    [G, K/128, N, 4] of quantized values [G, N, K] and their blocks' E8M0 bytes
    [G, N, K/32]."""
    G, N, K = values.shape
    m = values.abs()
    code = (2 * m).where(m < 2, (m + 2).where(m < 4, m / 2 + 4)).to(torch.uint8)
    code = torch.where(torch.signbit(values), code + 8, code).view(G, N, K // 2, 2)
    codes = code[..., 0] | (code[..., 1] << 4)
    scales = exponents.to(torch.uint8).view(G, N, K // 128, 4).transpose(1, 2).contiguous()
    return codes.contiguous(), scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = case["kind"]
    s = dict(case)
    if kind in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        x = _logits(g, T, E)
        if case["masked"]:  # a tenth of the experts masked, and one token in fifty without any
            x = x.masked_fill(torch.rand((T, E), generator=g, device="cuda") < 0.1, -math.inf)
            x = x.masked_fill(torch.rand((T, 1), generator=g, device="cuda") < 0.02, -math.inf)
        s["logits"] = x.to(getattr(torch, case["dtype"]))
        if kind == "route_grad":
            s["ids"], s["weights"] = _topk(s["logits"], k, case["renorm"])
            s["dweights"] = _normal(g, T, k)
        return s
    if kind == "mxfp4_weights":
        w = 0.02 * _normal(g, case["G"], case["K"], case["N"])
        s["w"] = w.to(torch.bfloat16)
        return s
    if kind == "mxfp4":
        T, k, G, K, N = (case[n] for n in ("T", "k", "G", "K", "N"))
        s["x"] = _activations(g, T, K)
        _, s["group_sizes"], _, slot_of_row = _routing(g, T, G, k, case["skew"])
        s["slot_of_row"] = slot_of_row
        s["most"] = int(s["group_sizes"].max())  # rows of the fullest expert, which a padded product needs
        codes, scales = [], []
        for _ in range(G):
            q, e = _mxfp4_values((0.02 * _normal(g, 1, N, K)).to(torch.bfloat16))
            c, v = _layout_mxfp4(q, e)
            codes.append(c)
            scales.append(v)
        s["codes"], s["scales"] = torch.cat(codes), torch.cat(scales)
        return s
    T, H, k, E = (case[n] for n in ("T", "H", "k", "E"))
    _, _, s["row_of_slot"], _ = _routing(g, T, E, k, 0.5)
    s["row_of_slot"] = s["row_of_slot"].view(T, k)
    if kind in ("permute", "permute_fp8"):
        s["x"] = _activations(g, T, H)
        return s
    s["y"] = _normal(g, T * k, H).to(torch.bfloat16)
    s["weights"] = torch.softmax(_normal(g, T, k), dim=1)
    if kind == "combine_grad":
        s["dout"] = (1e-3 * _normal(g, T, H)).to(torch.bfloat16)
    return s


# --------------------------------------------------------------------------- plain forms

def _topk(logits, k, renorm):
    x = logits.float()
    value, index = torch.sort(x, dim=1, descending=True, stable=True)
    value, index = value[:, :k], index[:, :k].to(torch.int32)
    none = value == -math.inf
    top = value[:, :1].masked_fill(none[:, :1], 0)
    e = torch.exp(value - top)
    total = (e if renorm else torch.exp(x - top)).sum(1, keepdim=True)
    return index.masked_fill(none, -1), torch.where(none, 0.0, e / total)


def _sort(ids, E):
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    sizes = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))
    slots = torch.sort(key, stable=True).indices
    place = torch.arange(n, device=ids.device)
    rows = torch.empty_like(place)
    rows[slots] = place
    kept = n - sizes[E]
    return (sizes[:E].to(torch.int32), torch.where(key < E, rows, -1).to(torch.int32),
            torch.where(place < kept, slots, -1).to(torch.int32))


def _mxfp4_values(x):
    """e2m1 values [.., K] (in units of their block's scale) and E8M0 bytes
    [.., K/32] of the last dimension's blocks of 32."""
    v = x.float().unflatten(-1, (-1, BLOCK))
    amax = v.abs().amax(-1, keepdim=True)
    power = (torch.frexp(amax).exponent - 3).clamp(min=-127).masked_fill(amax == 0, -127)
    q = torch.ldexp(v, -power)
    step = torch.where(q.abs() < 2, 0.5, torch.where(q.abs() < 4, 1.0, 2.0))
    q = (torch.round(q / step) * step).clamp(-6, 6)
    return q.flatten(-2), power.squeeze(-1) + 127


def _mxfp4_decode(codes, scales):
    """float32 [G, N, K] of codes [G, N, K/2] and scales [G, K/128, N, 4]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    q = torch.stack((codes & 15, codes >> 4), dim=-1).int()
    G, N, half = codes.shape
    e = scales.transpose(1, 2).reshape(G, N, half // 16, 1)
    return (table[q].view(G, N, half // 16, BLOCK) * torch.exp2(e.float() - 127)).view(G, N, 2 * half)


def _padded_product(s):
    """float32 [M, N] of the ragged product, its groups padded to the fullest."""
    q, e = _mxfp4_values(s["x"])
    a = (q.unflatten(-1, (-1, BLOCK)) * torch.exp2(e.float() - 127).unsqueeze(-1)).flatten(-2)
    w = _mxfp4_decode(s["codes"], s["scales"])
    token = s["slot_of_row"].long() // s["k"]
    M = token.numel()
    end = s["group_sizes"].long().cumsum(0)
    start = end - s["group_sizes"]
    row = (start.unsqueeze(1) + torch.arange(s["most"], device=end.device)).clamp(max=M - 1)
    y = torch.bmm(a[token[row]], w.transpose(1, 2)).flatten(0, 1)
    r = torch.arange(M, device=end.device)
    expert = torch.searchsorted(end, r, right=True)
    return y[expert * s["most"] + r - start[expert]]


def _plain(s):
    kind = s["kind"]
    if kind == "route":
        ids, weights = _topk(s["logits"], s["k"], s["renorm"])
        return (ids, weights) + _sort(ids, s["E"])
    if kind == "route_grad":
        x, ids, w, dw = s["logits"].float(), s["ids"].long(), s["weights"], s["dweights"]
        inner = (w * dw).sum(1, keepdim=True)
        here = torch.where(ids >= 0, w * (dw if not s["renorm"] else dw - inner), 0.0)
        d = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), here)
        if not s["renorm"]:
            top = x.amax(1, keepdim=True)
            e = torch.exp(x - top.masked_fill(top == -math.inf, 0))
            total = e.sum(1, keepdim=True)
            d = d - torch.where(total > 0, e / total, 0.0) * inner
        return d.to(s["logits"].dtype)
    if kind == "permute":
        rows = s["row_of_slot"].reshape(-1).long()
        out = torch.empty((rows.numel(), s["H"]), dtype=torch.bfloat16, device=rows.device)
        out[rows] = s["x"].repeat_interleave(s["k"], dim=0)
        return out
    if kind == "permute_fp8":
        # in 64 bits, so that the scale and the quotient are the correctly rounded 32-bit ones and no code crosses a border
        x = s["x"].double()
        scale = (x.abs().amax(1).clamp(min=1e-12) / 448).float()
        quotient = (x / scale.double().unsqueeze(1)).float()
        code = quotient.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        rows = s["row_of_slot"].reshape(-1).long()
        codes = torch.empty((rows.numel(), s["H"]), dtype=torch.uint8, device=rows.device)
        scales = torch.empty(rows.numel(), device=rows.device)
        codes[rows] = code.repeat_interleave(s["k"], dim=0)
        scales[rows] = scale.repeat_interleave(s["k"])
        return codes.view(torch.float8_e4m3fn), scales
    if kind == "combine":
        y = s["y"][s["row_of_slot"].long()].float()
        return (y * s["weights"].unsqueeze(2) if s["weighted"] else y).sum(1).to(torch.bfloat16)
    if kind == "combine_grad":
        rows = s["row_of_slot"].long()
        d = s["dout"].float().unsqueeze(1)
        dy = torch.empty_like(s["y"])
        dy[rows.reshape(-1)] = (d * s["weights"].unsqueeze(2)).to(torch.bfloat16).flatten(0, 1)
        return dy, (s["y"][rows].float() * d).sum(2)
    if kind == "mxfp4_weights":
        q, e = _mxfp4_values(s["w"].transpose(1, 2))
        return (q.unflatten(-1, (-1, BLOCK)) * torch.exp2(e.float() - 127).unsqueeze(-1)).flatten(-2).to(torch.bfloat16)
    y = _padded_product(s)
    if s["swiglu"]:
        gate, up = y.chunk(2, dim=1)
        y = gate / (1 + torch.exp(-gate)) * up
    return y.to(torch.bfloat16)


def run(state):
    if not own:
        return _plain(state)
    import fp8_moe_grouped_amd as lib
    s, kind = state, state["kind"]
    if kind == "route":
        r = lib.moe_route(s["logits"], s["k"], renormalize=s["renorm"])
        return r.ids, r.weights, r.group_sizes, r.row_of_slot.view(-1), r.slot_of_row
    if kind == "route_grad":
        return lib.moe_route_bwd(s["dweights"], s["logits"], s["ids"], s["weights"], renormalize=s["renorm"])
    if kind == "permute":
        return lib.moe_permute(s["x"], s["row_of_slot"])
    if kind == "permute_fp8":
        codes, scales = lib.moe_permute_fp8(s["x"], s["row_of_slot"])
        return codes.view(torch.float8_e4m3fn), scales
    if kind == "combine":
        return lib.moe_combine(s["y"], s["row_of_slot"], s["weights"] if s["weighted"] else None)
    if kind == "combine_grad":
        return lib.moe_combine_bwd(s["dout"], s["y"], s["row_of_slot"], s["weights"])
    if kind == "mxfp4_weights":
        return lib.dequantize_mxfp4(*lib.quantize_mxfp4_weights(s["w"]))
    product = lib.gmm_silu_mxfp4 if s["swiglu"] else lib.gmm_mxfp4_fwd
    return product(s["x"], s["codes"], s["scales"], s["group_sizes"], slot_of_row=s["slot_of_row"], topk=s["k"])


# --------------------------------------------------------------------------- definitions in 64 bits

def _choose_exactly(x, k):
    """(ids, chosen logits) by k times the largest, its lowest index first."""
    x, E = x.clone(), x.shape[1]
    place = torch.arange(E, device=x.device)
    ids, values = [], []
    for _ in range(k):
        m = x.amax(1, keepdim=True)
        i = torch.where(x == m, place, E).amin(1, keepdim=True)
        ids.append(torch.where(m == -math.inf, -1, i))
        values.append(m)
        x.scatter_(1, i, -math.inf)
    return torch.cat(ids, 1), torch.cat(values, 1)


def _quantize_exactly(x):
    """The values that x [.., K] is held as in the microscaled format."""
    v = x.double().unflatten(-1, (-1, BLOCK))
    amax = v.abs().amax(-1, keepdim=True)
    unit = torch.exp2((torch.floor(torch.log2(amax)) - 2).clamp(min=-127))
    v = v / unit
    size, held = v.abs(), torch.zeros_like(v)
    for border, up, to_even in ((0.25, 0.5, False), (0.75, 0.5, True), (1.25, 0.5, False), (1.75, 0.5, True),
                                (2.5, 1.0, False), (3.5, 1.0, True), (5.0, 2.0, False)):
        held += up * ((size >= border) if to_even else (size > border))
    return (torch.copysign(held, v) * unit).flatten(-2)


def _decode_exactly(codes, scales):
    """float64 [N, K] of one expert's codes [N, K/2] and scales [K/128, N, 4]."""
    n = torch.stack((codes % 16, codes // 16), dim=-1).flatten(1).long()
    sign, e, m = 1 - 2 * (n // 8), n // 2 % 4, n % 2
    v = sign * torch.where(e == 0, 0.5 * m, torch.exp2((e - 1).double()) * (1 + 0.5 * m))
    unit = torch.exp2(scales.permute(1, 0, 2).reshape(codes.shape[0], -1).double() - 127)
    return v * unit.repeat_interleave(BLOCK, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "route":
        x = s["logits"].double()
        ids, v = _choose_exactly(x, case["k"])
        lse = torch.logsumexp(v if case["renorm"] else x, 1, keepdim=True)
        return None, torch.where(ids < 0, 0.0, torch.exp(v - lse)), None, None, None
    if kind == "route_grad":
        # through the softmax's Jacobian, from the inputs' own weights
        x, w, dw = s["logits"].double(), s["weights"].double(), s["dweights"].double()
        hit = (s["ids"].unsqueeze(2) == torch.arange(case["E"], device=x.device)).double()
        if case["renorm"]:
            jac = torch.diag_embed(w) - w.unsqueeze(2) * w.unsqueeze(1)
            return torch.einsum("tj,tji,tie->te", dw, jac, hit)
        p = torch.nan_to_num(torch.softmax(x, 1))
        up = torch.einsum("tj,tje->te", dw, hit)
        # sum_j w_j dw_j holds the weights that came in, like the operator
        return p * up - p * (w * dw).sum(1, keepdim=True)
    if kind == "permute":
        out = torch.zeros((case["T"] * case["k"], case["H"]), dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            out[s["row_of_slot"][:, j].long()] = s["x"].double()
        return out
    if kind == "permute_fp8":
        x = s["x"].double()
        # the scale and the quotient are 32-bit numbers by definition
        scale = (x.abs().amax(1).clamp(min=1e-12) / 448).float().double()
        m = (x / scale.unsqueeze(1)).float().double().clamp(-448, 448)
        unit = torch.exp2(torch.floor(torch.log2(m.abs().clamp(min=2.0 ** -6))) - 3)
        held = torch.round(m / unit) * unit
        codes = torch.zeros((case["T"] * case["k"], case["H"]), dtype=torch.float64, device="cuda")
        scales = torch.zeros(case["T"] * case["k"], dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            rows = s["row_of_slot"][:, j].long()
            codes[rows], scales[rows] = held, scale
        return codes, scales
    if kind == "combine":
        out = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            y = s["y"][s["row_of_slot"][:, j].long()].double()
            out += y * s["weights"][:, j:j + 1].double() if case["weighted"] else y
        return out
    if kind == "combine_grad":
        dy = torch.zeros((case["T"] * case["k"], case["H"]), dtype=torch.float64, device="cuda")
        dw = torch.zeros((case["T"], case["k"]), dtype=torch.float64, device="cuda")
        d = s["dout"].double()
        for j in range(case["k"]):
            rows = s["row_of_slot"][:, j].long()
            dy[rows] = d * s["weights"][:, j:j + 1].double()
            dw[:, j] = (d * s["y"][rows].double()).sum(1)
        return dy, dw
    if kind == "mxfp4_weights":
        return _quantize_exactly(s["w"].transpose(1, 2))
    a = _quantize_exactly(s["x"])
    M = s["slot_of_row"].numel()
    out = torch.zeros((M, case["N"] // 2 if case["swiglu"] else case["N"]), dtype=torch.float64, device="cuda")
    at = 0
    for g, n in enumerate(s["group_sizes"].tolist()):
        if n == 0:
            continue
        token = torch.div(s["slot_of_row"][at:at + n].long(), case["k"], rounding_mode="floor")
        y = a[token] @ _decode_exactly(s["codes"][g], s["scales"][g]).t()
        if case["swiglu"]:
            half = case["N"] // 2
            y = y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]
        out[at:at + n] = y
        at += n
    return out
