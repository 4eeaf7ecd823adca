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


def quantize_fp8_weights(w):
    """e4m3 codes [G, K, N] and f32 scales [G, N] of bf16 weights [G, K, N]."""
    scale = w.float().abs().amax(1).clamp(min=1e-12) / 448
    return (w.float() / scale.unsqueeze(1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale


class MoeLayer:
    """SwiGLU experts behind a top-k softmax router.  Master weights: router
    f32 [H, E], wi bf16 [E, H, 2I] ([gate | up]), wo bf16 [E, I, H]."""

    def __init__(self, router, wi, wo, topk):
        self.router, self.topk = router, topk
        self.wi, self.wo = quantize_fp8_weights(wi), quantize_fp8_weights(wo)
        self.wi4, self.wo4 = lib.quantize_mxfp4_weights(wi), lib.quantize_mxfp4_weights(wo)

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

    def backward(self, dout, saved):
        """(dx bf16 [T, H], drouter f32 [H, E], dwi f32 [E, H, 2I], dwo f32 [E, I, H])."""
        x, logits, r, xp, y, h, preact = saved
        dy, dweights = lib.moe_combine_bwd(dout, y, r.row_of_slot, r.weights)
        dxp, dwi, dwo, _ = lib.moe_ffn_fp8_bwd(xp, h, preact, dy, *self.wi, *self.wo, r.group_sizes)
        dlogits = lib.moe_route_bwd(dweights, logits, r.ids, r.weights)
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

    def step():
        out, saved = layer.forward(x)
        return layer.backward(dout, saved)

    print(f"{a.tokens} tokens, {a.experts} experts of {a.hidden} x {a.inner}, top {a.topk}")
    print(f"  forward            {_milliseconds(lambda: layer.forward(x)):8.3f} ms")
    print(f"  forward + backward {_milliseconds(step):8.3f} ms")
    for n in (1, 32, a.tokens):
        print(f"  decode {n:6d}      {_milliseconds(lambda: layer.decode(x[:n])):8.3f} ms")


if __name__ == "__main__":
    main()
