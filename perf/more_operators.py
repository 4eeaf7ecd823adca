"""The cases on which the router's balance losses, the AdamW step and the FP8
weight quantizer are measured, with their plain forms in elementary torch
operations.

A case is a dict of plain values; its ``kind`` names the operator.  ``run``
computes one pass in the plain form or, where ``own`` is set, through the
package's entry points.  AdamW works in place in both.
"""
import math
import random

import torch

own = False

BLOCK = 256  # elements that share one scale of an 8-bit state
BETAS, EPS, DECAY = (0.9, 0.999), 1e-8, 0.01


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # a small debugging batch of a few experts: latency alone
        dict(name="balance_small", kind="balance", T=64, E=8, k=2, dtype="float32", masked=False),
        # a training batch of bf16 logits
        dict(name="balance_batch", kind="balance", T=16384, E=256, k=8, dtype="bfloat16", masked=False),
        # an odd batch with padding tokens and masked experts
        dict(name="balance_odd", kind="balance", T=10007, E=160, k=6, dtype="float32", masked=True),
        # the gradient joined to the router's own
        dict(name="balance_grad", kind="balance_grad", T=16384, E=256, k=8, dtype="float32", masked=False, add=True),
        # the gradient alone, of the same odd batch
        dict(name="balance_grad_odd", kind="balance_grad", T=10007, E=160, k=6, dtype="bfloat16", masked=True,
             add=False),
        # routers, norms and biases of a small model: many tensors, each a launch by itself
        dict(name="adamw_many", kind="adamw", shapes="", n=48, top=200000, pick=7, param="float32", grad="float32",
             scaled=True),
        # one layer's experts: f32 masters with the weight gradients that the backward leaves
        dict(name="adamw_experts", kind="adamw", shapes="8x2048x1536,8x768x2048", n=0, top=0, pick=0,
             param="float32", grad="float32", scaled=False),
        # the same step without masters, odd sizes
        dict(name="adamw_bf16", kind="adamw", shapes="4999x2048,2048x1537,77", n=0, top=0, pick=0, param="bfloat16",
             grad="bfloat16", scaled=True),
        # a small router and its neighbours with 8-bit states
        dict(name="adamw8_many", kind="adamw8", shapes="", n=10, top=300000, pick=3, param="float32", grad="bfloat16",
             scaled=True),
        # the dropless width's experts (7168) with 8-bit states, where the states' bytes count most
        dict(name="adamw8_experts", kind="adamw8", shapes="8x7168x4096,8x2048x7168", n=0, top=0, pick=0,
             param="float32", grad="float32", scaled=False),
        # a layer's second product's weights, bf16 masters, to codes
        dict(name="weights_wo", kind="weights", G=8, K=768, N=2048, dtype="bfloat16"),
        # the dropless first product's f32 masters to codes
        dict(name="weights_wi", kind="weights", G=8, K=7168, N=4096, dtype="float32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["balance", "balance_grad", "adamw", "adamw8", "weights"])
    if kind in ("balance", "balance_grad"):
        E = _log(rng, 8, 512)
        c = dict(kind=kind, T=_log(rng, 1, 16384), E=E, k=rng.randint(1, min(E, 10)),
                 dtype=rng.choice(["float32", "bfloat16"]), masked=rng.random() < 0.5)
        if kind == "balance_grad":
            c["add"] = rng.random() < 0.5
        return c
    if kind == "weights":
        return dict(kind=kind, G=rng.randint(1, 8), K=128 * rng.randint(1, 56), N=128 * rng.randint(1, 32),
                    dtype=rng.choice(["float32", "bfloat16"]))
    return dict(kind=kind, shapes="", n=_log(rng, 1, 48 if kind == "adamw" else 12), top=_log(rng, 100, 5000000),
                pick=rng.randint(1, 10 ** 6), param=rng.choice(["float32", "float32", "bfloat16"]),
                grad=rng.choice(["float32", "bfloat16"]), scaled=rng.random() < 0.5)


def _shapes(case):
    """The tensors' shapes: those named, or n of 1 to `top` elements, odd ones among them."""
    if case["shapes"]:
        return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]
    rng = random.Random(case["pick"])
    return [(_log(rng, 1, case["top"]),) for _ in range(case["n"])]


def _bytes(name):
    return 4 if name == "float32" else 2


def work(case):
    kind = case["kind"]
    if kind in ("balance", "balance_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        rows = T * E * _bytes(case["dtype"])
        if kind == "balance":
            return {"bytes": rows + 4 * T * k + 8 * E + 12, "flops": 4 * T * E}
        return {"bytes": rows * (3 if case["add"] else 2) + 4 * E + 12, "flops": 8 * T * E}
    if kind == "weights":
        n, columns = case["G"] * case["K"] * case["N"], case["G"] * case["N"]
        return {"bytes": n * (_bytes(case["dtype"]) + 1) + 4 * columns, "flops": 2 * n}
    n = sum(math.prod(s) for s in _shapes(case))
    one = 2 * _bytes(case["param"]) + _bytes(case["grad"])
    return {"bytes": n * (one + 16) if kind == "adamw" else n * (one + 4) + n / 16, "flops": 14 * n}


# --------------------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=g.device)


class _Many:
    """Tensors of the given shapes as views of one buffer, each at a multiple of
    256 elements, as a program has that keeps its parameters in one allocation."""

    def __init__(self, shapes):
        self.shapes, self.at, end = shapes, [], 0
        for s in shapes:
            self.at.append(end)
            end += -(-math.prod(s) // BLOCK) * BLOCK
        self.size = end

    def filled(self, g, dtype, draw):
        """(buffer, its views) with draw(number of elements) in the views, zeros between."""
        flat = torch.zeros(self.size, dtype=dtype, device="cuda")
        views = self.views(flat)
        for v in views:
            v.view(-1).copy_(draw(v.numel()))
        return flat, views

    def views(self, flat):
        return [flat[a:a + math.prod(s)].view(s) for a, s in zip(self.at, self.shapes)]

    def blocks(self, flat):
        """The views' scales, of a buffer with one for each 256 elements."""
        return [flat[a // BLOCK:a // BLOCK - (-math.prod(s) // BLOCK)] for a, s in zip(self.at, self.shapes)]


def _to_blocks(flat):
    """e4m3 codes and scales of a buffer whose blocks are its rows of 256."""
    x = flat.view(-1, BLOCK)
    scale = x.abs().amax(1) / 448
    q = torch.where(scale > 0, 1 / scale, 0.0).unsqueeze(1) * x
    return q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(-1), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = case["kind"]
    s = dict(case)
    if kind in ("balance", "balance_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        x = _normal(g, T, E) + 0.5 * _normal(g, E)   # some experts are liked more than others by every token
        if case["masked"]:  # a tenth of the experts masked, and one token in fifty is padding
            x = x.masked_fill(torch.rand((T, E), generator=g, device="cuda") < 0.1, -math.inf)
            x = x.masked_fill(torch.rand((T, 1), generator=g, device="cuda") < 0.02, -math.inf)
        s["logits"] = x.to(getattr(torch, case["dtype"]))
        value, ids = torch.topk(s["logits"].float(), k, dim=1)
        s["ids"] = ids.masked_fill(value == -math.inf, -1).to(torch.int32)
        if kind == "balance_grad":
            s["dlosses"] = torch.tensor([0.01, 0.001], device="cuda") * (1 + torch.rand(2, generator=g, device="cuda"))
            s["counts"], s["tokens"] = _counts(s["ids"], E), (value[:, 0] > -math.inf).sum().to(torch.int32).view(1)
            s["add_to"] = (1e-3 * _normal(g, T, E)).to(s["logits"].dtype) if case["add"] else None
        return s
    if kind == "weights":
        w = 0.02 * _normal(g, case["G"], case["K"], case["N"]) * (0.2 + torch.rand(case["N"], generator=g, device="cuda"))
        s["w"] = w.to(getattr(torch, case["dtype"]))
        return s
    many = _Many(_shapes(case))
    s["p_flat"], s["p"] = many.filled(g, getattr(torch, case["param"]), lambda n: 0.02 * _normal(g, n))
    s["g_flat"], s["g"] = many.filled(g, getattr(torch, case["grad"]), lambda n: 1e-3 * _normal(g, n))
    m_flat, m = many.filled(g, torch.float32, lambda n: 2e-4 * _normal(g, n))
    v_flat, v = many.filled(g, torch.float32, lambda n: (1e-3 * _normal(g, n)) ** 2 + 1e-8)
    s["lr"], s["step"] = 1e-3, 1000 + seed % 7
    s["scale"] = 0.5 + torch.rand(1, generator=g, device="cuda") if case["scaled"] else None
    if kind == "adamw":
        s.update(m_flat=m_flat, m=m, v_flat=v_flat, v=v)
        return s
    s["seed"] = seed
    blocks = torch.tensor([-(-math.prod(v) // BLOCK) for v in many.shapes], device="cuda")
    s["tensor"] = torch.arange(len(blocks), device="cuda").repeat_interleave(blocks)
    s["block"] = torch.arange(len(s["tensor"]), device="cuda") - (blocks.cumsum(0) - blocks)[s["tensor"]]
    for name, flat in (("m", m_flat), ("r", torch.sqrt(v_flat))):
        codes, scales = _to_blocks(flat)
        s[name + "_codes"], s[name + "_scales"] = codes, scales
        s[name] = list(zip(many.views(codes), many.blocks(scales)))
    return s


# --------------------------------------------------------------------------- plain forms

def _counts(ids, E):
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    return torch.zeros(E + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))[:E].to(
        torch.int32)


def _softmax(x):
    """(softmax, log of the sum of exponentials, whether the token counts) of rows x, zeros for a row of -inf."""
    top = x.amax(1, keepdim=True)
    here = top > -math.inf
    top = torch.where(here, top, 0.0)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    return (torch.where(here, e / total, 0.0), torch.where(here, top + torch.log(total), 0.0).squeeze(1),
            here.squeeze(1))


def _balance(s):
    E = s["E"]
    p, lse, here = _softmax(s["logits"].float())
    n = here.sum().to(torch.int32).view(1)
    counts = _counts(s["ids"], E)
    probs = p.sum(0) / n.clamp(min=1)
    share = counts / counts.sum().clamp(min=1)
    losses = torch.stack((E * (share * probs).sum(), (lse * lse).sum() / n[0].clamp(min=1)))
    return losses, counts, probs, n


def _balance_grad(s):
    c, n, E = s["counts"].float(), s["tokens"].clamp(min=1), s["E"]
    p, lse, _ = _softmax(s["logits"].float())
    c = c - c.mean()
    total = s["counts"].sum().clamp(min=1)
    a, b = s["dlosses"][0] * E / n / total, s["dlosses"][1] * 2 / n
    d = p * (a * (c - (p * c).sum(1, keepdim=True)) + b * lse.unsqueeze(1))
    return (d if s["add_to"] is None else d + s["add_to"]).to(s["logits"].dtype)


def _rates(s):
    """(lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t))."""
    return s["lr"] / (1 - BETAS[0] ** s["step"]), 1 / math.sqrt(1 - BETAS[1] ** s["step"])


def _adamw(s):
    """In place, over all tensors at once an elementary operation."""
    up, root = _rates(s)
    g = s["g"] if s["scale"] is None else torch._foreach_mul([t.float() for t in s["g"]], s["scale"].view(()))
    g = [t.float() for t in g]
    torch._foreach_mul_(s["m"], BETAS[0])
    torch._foreach_add_(s["m"], g, alpha=1 - BETAS[0])
    torch._foreach_mul_(s["v"], BETAS[1])
    torch._foreach_addcmul_(s["v"], g, g, value=1 - BETAS[1])
    below = torch._foreach_sqrt(s["v"])
    torch._foreach_mul_(below, root)
    torch._foreach_add_(below, EPS)
    p = [t.float() for t in s["p"]]
    d = torch._foreach_mul(p, s["lr"] * DECAY)
    torch._foreach_addcdiv_(d, s["m"], below, value=up)
    torch._foreach_copy_(s["p"], torch._foreach_sub(p, d))
    return s["p_flat"], s["m_flat"], s["v_flat"]


def _mix(x):
    x = ((x ^ (x >> 16)) * 0x6A09E667) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _noise(s):
    """32 random bits for each element of the whole buffer [blocks, 256]."""
    key = _mix((s["seed"] & 0xFFFFFFFF) + _mix((s["seed"] >> 32) + _mix(s["step"])) & 0xFFFFFFFF)
    key = _mix((_mix(s["tensor"] + key & 0xFFFFFFFF) + s["block"]) & 0xFFFFFFFF).unsqueeze(1)
    return _mix((key + torch.arange(BLOCK, device="cuda") * 0x9E3779B9) & 0xFFFFFFFF)


def _held(x, bits, least):
    """(codes, scales) of blocks x [blocks, 256], rounded up or down by chance; `least`: the smallest code of a value above zero."""
    scale = x.abs().amax(1) / 448
    q = torch.where(scale > 0, 1 / scale, 0.0).unsqueeze(1) * x.abs()
    step = torch.ldexp(torch.ones_like(q), torch.frexp(q).exponent.clamp(min=-5) - 4)
    q = (torch.floor(q / step + (bits + 0.5) / 65536) * step).clamp(max=448)
    q = torch.where(x != 0, q.clamp(min=least), q)
    return torch.copysign(q, x).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _adamw8(s):
    """In place, over the buffers that hold all tensors."""
    up, root = _rates(s)
    rows = lambda name: s[name].view(-1, BLOCK)
    old = lambda name: rows(name + "_codes").view(torch.float8_e4m3fn).float() * s[name + "_scales"].unsqueeze(1)
    g = rows("g_flat").float() if s["scale"] is None else rows("g_flat").float() * s["scale"]
    m, r = BETAS[0] * old("m") + (1 - BETAS[0]) * g, old("r")
    r = torch.sqrt(BETAS[1] * r * r + (1 - BETAS[1]) * g * g)
    p = rows("p_flat").float()
    rows("p_flat").copy_(p - (s["lr"] * DECAY * p + up * m / (r * root + EPS)))
    bits = _noise(s)
    codes, scales = _held(m, bits & 0xFFFF, 0.0)
    rows("m_codes").copy_(codes), s["m_scales"].copy_(scales)
    codes, scales = _held(r, bits >> 16, 2.0 ** -9)
    rows("r_codes").copy_(codes), s["r_scales"].copy_(scales)
    return _held_outputs(s)


def _held_outputs(s):
    e4m3 = torch.float8_e4m3fn
    return s["p_flat"], s["m_codes"].view(e4m3), s["m_scales"], s["r_codes"].view(e4m3), s["r_scales"]


def _weights(s):
    # in 64 bits, so that the scale and the quotient are the correctly rounded 32-bit ones and no code crosses a border
    scale = (s["w"].abs().amax(1).double().clamp(min=1e-12) / 448).float()
    q = (s["w"].double() / scale.double().unsqueeze(1)).float()
    return q.clamp(-448, 448).to(torch.float8_e4m3fn), scale


def run(state):
    s, kind = state, state["kind"]
    if not own:
        return {"balance": _balance, "balance_grad": _balance_grad, "adamw": _adamw, "adamw8": _adamw8,
                "weights": _weights}[kind](s)
    import fp8_moe_grouped_amd as lib
    if kind == "balance":
        return tuple(lib.moe_balance_loss(s["logits"], s["ids"]))
    if kind == "balance_grad":
        return lib.moe_balance_loss_bwd(s["dlosses"], s["logits"], s["counts"], s["tokens"], add=s["add_to"])
    if kind == "weights":
        codes, scales = lib.quantize_fp8_weights(s["w"])
        return codes.view(torch.float8_e4m3fn), scales
    how = dict(lr=s["lr"], step=s["step"], betas=BETAS, eps=EPS, weight_decay=DECAY, grad_scale=s["scale"])
    if kind == "adamw":
        lib.adamw_step(s["p"], s["g"], s["m"], s["v"], **how)
        return s["p_flat"], s["m_flat"], s["v_flat"]
    lib.adamw_step_8bit(s["p"], s["g"], s["m"], s["r"], seed=s["seed"], **how)
    return _held_outputs(s)


# --------------------------------------------------------------------------- definitions in 64 bits

def _exact_noise(seed, step, tensor, block, place):
    """The two random numbers in (0, 1) of elements `place` [..] of blocks `block` [..]."""
    def times(a, c):  # modulo 2^32, by halves
        return ((a * (c % 65536)) + ((a * (c // 65536)) % 65536) * 65536) % (1 << 32)

    def mixed(a):
        a = times(a ^ (a // 65536), 0x6A09E667)
        a = times(a ^ (a // 32768), 0xBB67AE85)
        return a ^ (a // 65536)

    word = lambda v: torch.tensor(v % (1 << 32), device="cuda")
    low = lambda a: a % (1 << 32)
    key = mixed(low(word(seed) + mixed(low(word(seed // (1 << 32)) + mixed(word(step))))))
    key = mixed(low(key + tensor))
    h = mixed(low(mixed(low(key + block)) + times(place, 0x9E3779B9)))
    return (h % 65536 + 0.5) / 65536, (h // 65536 + 0.5) / 65536


def _exact_update(s, p, g, m, r2):
    """One element's step: (p, m, v) new, all float64."""
    b1, b2 = BETAS
    g = g if s["scale"] is None else g * s["scale"].double()
    m = m * b1 + g * (1 - b1)
    v = r2 * b2 + g * g * (1 - b2)
    ahead = m / (1 - b1 ** s["step"])
    size = torch.sqrt(v / (1 - b2 ** s["step"]))
    return p * (1 - s["lr"] * DECAY) - s["lr"] * ahead / (size + EPS), m, v


def _exact_codes(x, u, positive):
    """(held values, scales) of blocks x [blocks, 256] by the grid of e4m3."""
    scale = x.abs().amax(1) / 448
    q = torch.nan_to_num(x.abs() / scale.unsqueeze(1))
    exponent = torch.floor(torch.log2(q.clamp(min=2.0 ** -6))).clamp(max=8)
    unit = torch.exp2(exponent - 3)
    down = torch.floor(q / unit)
    up = (q / unit - down) + u >= 1
    held = ((down + up.double()) * unit).clamp(max=448)
    if positive:
        held = torch.where((q > 0) & (held == 0), 2.0 ** -9, held)
    return torch.where(x < 0, -held, held), scale


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("balance", "balance_grad"):
        x, E = s["logits"].double(), case["E"]
        here = (x > -math.inf).any(1)
        x = x[here]
        n = max(1, x.shape[0])
        lse = torch.logsumexp(x, 1, keepdim=True)
        p = torch.exp(x - lse)
        if kind == "balance":
            c = torch.stack([(s["ids"] == e).sum() for e in range(E)]).double()
            probs = p.sum(0) / n
            balance = E * torch.dot(c, probs) / max(1.0, float(c.sum()))
            return torch.stack((balance, (lse ** 2).sum() / n)), None, probs, None
        c = s["counts"].double()
        a = s["dlosses"][0].double() * E / (n * max(1.0, float(c.sum())))
        out = torch.zeros((case["T"], E), dtype=torch.float64, device="cuda")
        out[here] = p * (a * (c - (p @ c).unsqueeze(1)) + s["dlosses"][1].double() * 2 / n * lse)
        return out if s["add_to"] is None else out + s["add_to"].double()
    if kind == "weights":
        scale = (s["w"].abs().amax(1).double().clamp(min=1e-12) / 448).float().double()
        # the scale and the quotient are 32-bit numbers by definition
        q = (s["w"].double() / scale.unsqueeze(1)).float().double().clamp(-448, 448)
        unit = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        return torch.round(q / unit) * unit, scale
    if kind == "adamw":
        p, m, v = (torch.zeros(s["p_flat"].numel(), dtype=torch.float64, device="cuda") for _ in range(3))
        place = _Many(_shapes(case))
        for i, (po, mo, vo) in enumerate(zip(place.views(p), place.views(m), place.views(v))):
            new = _exact_update(s, *(s[name][i].double() for name in ("p", "g", "m", "v")))
            for out, value in zip((po, mo, vo), new):
                out.copy_(value)
        return p, m, v
    place = _Many(_shapes(case))
    p, mv, rv = (torch.zeros(place.size, dtype=torch.float64, device="cuda") for _ in range(3))
    ms, rs = (torch.zeros(place.size // BLOCK, dtype=torch.float64, device="cuda") for _ in range(2))
    chunk = 1 << 16  # blocks at a time
    for i, shape in enumerate(place.shapes):
        n, at = math.prod(shape), place.at[i]
        for b in range(0, -(-n // BLOCK), chunk):
            lo, hi = b * BLOCK, min(n, (b + chunk) * BLOCK)
            blocks = -(-(hi - lo) // BLOCK)
            one = lambda t: torch.cat((t.view(-1)[lo:hi].double(), torch.zeros(
                blocks * BLOCK - (hi - lo), dtype=torch.float64, device="cuda"))).view(blocks, BLOCK)
            old = [one(c.view(torch.float8_e4m3fn).view(-1)) * v[b:b + blocks].double().unsqueeze(1)
                   for c, v in (s["m"][i], s["r"][i])]
            x, m, v = _exact_update(s, one(s["p"][i]), one(s["g"][i]), old[0], old[1] ** 2)
            number = torch.arange(b, b + blocks, device="cuda").unsqueeze(1)
            um, ur = _exact_noise(seed, s["step"], i, number, torch.arange(BLOCK, device="cuda"))
            mq, mscale = _exact_codes(m, um, False)
            rq, rscale = _exact_codes(torch.sqrt(v), ur, True)
            to = slice(at + lo, at + hi)
            for out, value in ((p, x), (mv, mq), (rv, rq)):
                out[to] = value.view(-1)[:hi - lo]
            to = slice(at // BLOCK + b, at // BLOCK + b + blocks)
            ms[to], rs[to] = mscale, rscale
    return p, mv, ms, rv, rs
