"""The example's layer on the GPU: its training step and its decoding against a
layer computed in 64 bits token by token, from the same quantized weights."""
import pytest
import torch

from tests import plain_moe as P

pytestmark = pytest.mark.gpu
H, I, E, K = 256, 128, 6, 3


def fp8_values(x):
    """float64 values of bf16 rows [.., K] after e4m3 quantization by row."""
    scale = x.float().abs().amax(-1, keepdim=True).clamp(min=1e-12) / 448
    return (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn).double() * scale.double()


def bf16(x):
    return x.to(torch.bfloat16).double()


def layer_and_input(T, seed):
    from examples.moe_layer import make_layer
    layer = make_layer(H, I, E, K, seed)
    x = torch.randn((T, H), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
    return layer, x


def experts(x, wi, wo, weights, ids, hold):
    """out [T, H]: hold quantizes a product's rows; h is rounded to bf16 before it, y after."""
    out = torch.zeros((x.shape[0], H), dtype=torch.float64)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            z = hold(x[t]) @ wi[e]
            h = bf16(z[:I] * torch.sigmoid(z[:I]) * z[I:])
            out[t] += weights[t, j] * bf16(hold(h) @ wo[e])
    return out


def rel(a, b):
    return float((a.double().cpu() - b).norm() / b.norm())


# What the chain adds to one call's error: an intermediate on a border of its bf16 or 8 or 4-bit rounding may
# fall on the other side.  A few entries in a thousand move by one bf16 step, of them one in 16 over a 4-bit
# border (half its value at most): sqrt(0.003 / 16) / 2 < 1 %; over an 8-bit border all, by 2^-4 at most:
# sqrt(0.003) / 16 < 0.4 %.  The outputs' own rounding is 2^-9.
@pytest.mark.parametrize("T", [1, 37])
def test_forward(T):
    layer, x = layer_and_input(T, T)
    out, saved = layer.forward(x)
    r = saved[2]
    value = lambda w: w[0].cpu().view(torch.float8_e4m3fn).double() * w[1].cpu().double().unsqueeze(1)
    want = experts(x.cpu(), value(layer.wi), value(layer.wo), r.weights.cpu().double(), r.ids.cpu(),
                   lambda v: fp8_values(v.to(torch.bfloat16)))
    assert rel(out, want) < 2.0 ** -7


@pytest.mark.parametrize("T", [1, 37])
def test_decode(T):
    layer, x = layer_and_input(T, 10 + T)
    out = layer.decode(x)
    _, r = layer.route(x)
    import fp8_moe_grouped_amd as G
    value = lambda w: G.dequantize_mxfp4(*w).cpu().double().transpose(1, 2)
    want = experts(x.cpu().double(), value(layer.wi4), value(layer.wo4), r.weights.cpu().double(), r.ids.cpu(),
                   lambda v: P.mxfp4_values(*P.mxfp4(v)))
    assert rel(out, want) < 2.0 ** -6


def test_backward():
    """Against autograd through the dequantized layer.  The weight gradients quantize both operands to 8
    bits (e4m3 3 %, e5m2 6 % of a value at most, less in the norm), the activations' gradients do not."""
    T = 60
    layer, x = layer_and_input(T, 5)
    dout = torch.randn((T, H), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    _, saved = layer.forward(x)
    dx, drouter, dwi, dwo = layer.backward(dout, saved)
    value = lambda w: (w[0].cpu().view(torch.float8_e4m3fn).float() * w[1].cpu().unsqueeze(1)).double()
    xs, router, wi, wo = (t.requires_grad_() for t in (x.cpu().double(), layer.router.cpu().double(),
                                                       value(layer.wi), value(layer.wo)))
    ids = saved[2].ids.cpu().long()
    weights = torch.softmax((xs @ router).gather(1, ids), dim=1)
    out = torch.zeros((T, H), dtype=torch.float64)
    for e in range(E):
        for j in range(K):
            t = (ids[:, j] == e).nonzero().flatten()
            z = xs[t] @ wi[e]
            y = (z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:]) @ wo[e]
            out = out.index_add(0, t, weights[t, j:j + 1] * y)
    out.backward(dout.cpu().double())
    # the forward's 8-bit activations enter every factor: 2^-4 of a value at most, their norm a third of it
    for got, want in ((dx, xs.grad), (drouter, router.grad), (dwi, wi.grad), (dwo, wo.grad)):
        assert rel(got, want) < 2.0 ** -4
        assert got.shape == want.shape


def test_example_runs(monkeypatch, capsys):
    import examples.moe_layer as M
    monkeypatch.setattr("sys.argv", ["moe_layer.py", "--tokens", "64", "--hidden", "256", "--inner", "128", "--experts",
                                     "8", "--topk", "2"])
    M.main()
    assert "decode" in capsys.readouterr().out
