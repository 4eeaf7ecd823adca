"""One mixture-of-experts layer from its tokens to its tokens, through the
package's calls: a training step in FP8 and decoding on 4-bit weights.

    python examples/moe_layer.py [--tokens 4096] [--hidden 2048] [--inner 768] [--experts 64] [--topk 6]

Training (forward, then backward):

    logits = x @ router                                    (a library product, f32)
    route     ids, weights, group_sizes, row_of_slot       moe_route
    dispatch  xp[row_of_slot[t, j]] = x[t]                 moe_permute
    experts   y = FFN_e(xp)                                moe_ffn_fp8_fwd
    combine   out[t] = sum_j weights[t, j] y[row]          moe_combine

    dy, dweights = moe_combine_bwd(dout, ...);  dxp, dwi, dwo = moe_ffn_fp8_bwd(dy, ...)
    dlogits = moe_route_bwd(dweights, ...);     dx = moe_combine(dxp) + dlogits @ router^T

with the router's auxiliary losses, where they are asked for, between the two (their gradient joins the router's own):

    losses, counts, probs, tokens = moe_balance_loss(logits, counts=group_sizes)
    dlogits = moe_balance_loss_bwd(coefficients, logits, counts, tokens, add=dlogits)

and then the update of the f32 master weights, whose new codes the next step reads:

    adamw_step([router, wi, wo], gradients, ...)  or  adamw_step_8bit;   quantize_fp8_weights(wi), (wo)

(and quantize_mxfp4_weights, so that decoding follows the training; a program may leave that to the end)

Decoding has no dispatch of its own: the first product gathers its rows.

    h = gmm_silu_mxfp4(x, ..., slot_of_row, topk);  y = gmm_mxfp4_fwd(h, ...);  out = moe_combine(y, ...)
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_moe_grouped_amd as lib


class MoeLayer:
    """SwiGLU experts behind a top-k softmax router: router f32 [H, E], wi
    bf16 [E, H, 2I] ([gate | up]), wo bf16 [E, I, H].  Training keeps f32 masters
    of the experts' weights instead, whose e4m3 codes the products read."""

    def __init__(self, router, wi, wo, topk):
        self.router, self.topk = router, topk
        self.experts = [wi, wo]
        self.wi, self.wo = lib.quantize_fp8_weights(wi), lib.quantize_fp8_weights(wo)
        self.wi4, self.wo4 = lib.quantize_mxfp4_weights(wi), lib.quantize_mxfp4_weights(wo)

    def start_training(self, bits=32):
        """f32 masters of the weights, or those of the training so far, and AdamW's states, in 32 bits or 8."""
        self.experts = [w.float() for w in self.experts]
        self.masters = [self.router, *self.experts]
        self.bits, self.step = bits, 0
        self.states = (lib.adamw_8bit_states(self.masters) if bits == 8 else
                       [[torch.zeros_like(w) for w in self.masters] for _ in range(2)])

    def update(self, gradients, lr, **how):
        """One AdamW step on (drouter, dwi, dwo), and the experts' new codes, those for decoding too."""
        self.step += 1
        step = lib.adamw_step_8bit if self.bits == 8 else lib.adamw_step
        step(self.masters, list(gradients), *self.states, lr=lr, step=self.step, **how)
        for w, (codes, scales), (codes4, scales4) in zip(self.experts, (self.wi, self.wo), (self.wi4, self.wo4)):
            lib.quantize_fp8_weights(w, codes=codes, scales=scales)
            lib.quantize_mxfp4_weights(w.to(torch.bfloat16), codes=codes4, scales=scales4)

    def route(self, x):
        logits = x.float() @ self.router
        return logits, lib.moe_route(logits, self.topk)

    def forward(self, x):
        """out bf16 [T, H] and what backward needs."""
        logits, r = self.route(x)
        xp = lib.moe_permute(x, r.row_of_slot)
        y, h, preact = lib.moe_ffn_fp8_fwd(xp, *self.wi, *self.wo, r.group_sizes)
        out = lib.moe_combine(y, r.row_of_slot, r.weights)
        return out, (x, logits, r, xp, y, h, preact)

    def balance(self, saved):
        """The router's auxiliary losses of a forward pass."""
        _, logits, r, *_ = saved
        return lib.moe_balance_loss(logits, counts=r.group_sizes)

    def backward(self, dout, saved, balance=None, coefficients=None):
        """(dx bf16 [T, H], drouter f32 [H, E], dwi f32 [E, H, 2I], dwo f32 [E, I, H]), with balance's losses
        weighted by coefficients f32 [2]."""
        x, logits, r, xp, y, h, preact = saved
        dy, dweights = lib.moe_combine_bwd(dout, y, r.row_of_slot, r.weights)
        dxp, dwi, dwo, _ = lib.moe_ffn_fp8_bwd(xp, h, preact, dy, *self.wi, *self.wo, r.group_sizes)
        dlogits = lib.moe_route_bwd(dweights, logits, r.ids, r.weights)
        if balance is not None:
            lib.moe_balance_loss_bwd(coefficients, logits, balance.counts, balance.tokens, add=dlogits, out=dlogits)
        dx = (lib.moe_combine(dxp, r.row_of_slot).float() + dlogits @ self.router.t()).to(torch.bfloat16)
        return dx, x.float().t() @ dlogits, dwi, dwo

    def decode(self, x):
        """out bf16 [T, H] on 4-bit weights and activations."""
        _, r = self.route(x)
        h = lib.gmm_silu_mxfp4(x, *self.wi4, r.group_sizes, slot_of_row=r.slot_of_row, topk=self.topk)
        y = lib.gmm_mxfp4_fwd(h, *self.wo4, r.group_sizes)
        return lib.moe_combine(y, r.row_of_slot, r.weights)


def make_layer(hidden, inner, experts, topk, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    return MoeLayer(normal(hidden, experts) * hidden ** -0.5,
                    (normal(experts, hidden, 2 * inner) * hidden ** -0.5).to(torch.bfloat16),
                    (normal(experts, inner, hidden) * inner ** -0.5).to(torch.bfloat16), topk)


def _milliseconds(f, n=20):
    f()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(n):
        f()
    end.record()
    end.synchronize()
    return start.elapsed_time(end) / n


def main():
    p = argparse.ArgumentParser(description="Times a training step and decoding of one MoE layer.")
    for name, value in (("tokens", 4096), ("hidden", 2048), ("inner", 768), ("experts", 64), ("topk", 6)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    layer = make_layer(a.hidden, a.inner, a.experts, a.topk)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    dout = (1e-3 * torch.randn((a.tokens, a.hidden), device="cuda")).to(torch.bfloat16)

    coefficients = torch.tensor([1e-2, 1e-3], device="cuda")
    layer.start_training()

    def step():
        out, saved = layer.forward(x)
        return layer.backward(dout, saved, layer.balance(saved), coefficients)

    gradients = step()[1:]

    print(f"{a.tokens} tokens, {a.experts} experts of {a.hidden} x {a.inner}, top {a.topk}")
    print(f"  forward            {_milliseconds(lambda: layer.forward(x)):8.3f} ms")
    print(f"  forward + backward {_milliseconds(step):8.3f} ms")
    print(f"  update             {_milliseconds(lambda: layer.update(gradients, 1e-4)):8.3f} ms")
    for n in (1, 32, a.tokens):
        print(f"  decode {n:6d}      {_milliseconds(lambda: layer.decode(x[:n])):8.3f} ms")


if __name__ == "__main__":
    main()
