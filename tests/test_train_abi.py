"""CPU tests of the balance losses, AdamW and the FP8 weight quantizer: what
the C ABI and the binding refuse (fake device pointers are never dereferenced),
and hand-computed pins of the plain definitions that the GPU tests compare with."""
import ctypes
import math
import os

import pytest
import torch

import fp8_moe_grouped_amd as G
from tests import plain_train as P

A = 0x10000          # fake, 16-byte aligned "device" address
BAD = 0x10008        # misaligned


def _lib():
    if not os.path.exists(G.LIB_PATH):
        pytest.skip("library not built")
    return G.lib()


def test_macros_match_binding():
    text = open(G.HEADER_PATH).read()
    assert "#define FP8GMM_OP_BALANCE 12 " in text and G.OP_BALANCE == 12
    assert "#define FP8GMM_ERR_OVERLAP (-8)" in text and G.ERR_OVERLAP == -8
    _lib()
    assert "overlap" in G.status_string(G.ERR_OVERLAP)


def test_balance_refusals():
    L = _lib()
    f = lambda **a: L.moe_balance_loss(a.get("x", A), a.get("dt", G.F32), a.get("ids", A), a.get("T", 4096),
                                       a.get("E", 64), a.get("k", 8), a.get("losses", A), a.get("counts", A),
                                       a.get("probs", A), a.get("tokens", A), a.get("ws", A), a.get("wsb", 1 << 30),
                                       None)
    for name in ("x", "losses", "counts", "probs", "tokens"):
        assert f(**{name: None}) == G.ERR_NULL, name
    assert f(T=-1) == G.ERR_SHAPE and f(E=0) == G.ERR_SHAPE and f(k=0) == G.ERR_SHAPE
    assert f(T=1 << 21, k=8) == G.ERR_SHAPE and f(T=(1 << 63) - 1) == G.ERR_SHAPE
    assert f(E=1025) == G.ERR_UNSUPPORTED and f(k=33) == G.ERR_UNSUPPORTED and f(dt=2) == G.ERR_UNSUPPORTED
    assert f(x=BAD) == G.ERR_ALIGN and f(ws=BAD) == G.ERR_ALIGN
    need = L.fp8gmm_workspace_bytes(G.OP_BALANCE, 4096, 64, 8, 1, 0)
    assert need > 0 and f(ws=None) == G.ERR_WORKSPACE and f(wsb=need - 1) == G.ERR_WORKSPACE
    assert f(ids=None, k=0, ws=None) == G.ERR_WORKSPACE         # k does not matter without ids
    assert L.fp8gmm_workspace_bytes(G.OP_BALANCE, 1, 64, 8, 1, 0) == 0
    assert L.fp8gmm_workspace_bytes(G.OP_BALANCE, 4096, 1025, 8, 1, 0) == 0
    b = lambda **a: L.moe_balance_loss_bwd(a.get("d", A), a.get("x", A), a.get("dt", G.F32), a.get("counts", A),
                                           a.get("tokens", A), a.get("T", 8), a.get("E", 64), a.get("add"),
                                           a.get("out", A), None)
    for name in ("d", "x", "counts", "tokens", "out"):
        assert b(**{name: None}) == G.ERR_NULL, name
    assert b(T=-1) == G.ERR_SHAPE and b(E=0) == G.ERR_SHAPE and b(T=1 << 24) == G.ERR_SHAPE
    assert b(E=1025) == G.ERR_UNSUPPORTED and b(dt=7) == G.ERR_UNSUPPORTED
    assert b(x=BAD) == G.ERR_ALIGN and b(add=BAD) == G.ERR_ALIGN and b(out=BAD) == G.ERR_ALIGN
    assert b(T=0, x=None, out=None) == G.OK


def _adamw(L, bits=32, n=1, size=1000, p=0x100000, g=0x200000, m=0x300000, v=0x400000, ms=0x500000, vs=0x600000,
           pd=G.F32, gd=G.F32, how=None, second=None, **rates):
    h = G._AdamW(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1)
    for k, x in rates.items():
        setattr(h, k, x)
    col = lambda a, key: None if a == "null" else (ctypes.c_void_p * 2)(a, (second or {}).get(key))
    sizes = (ctypes.c_int64 * 2)(size, (second or {}).get("size", 0))
    h = None if how == "null" else ctypes.byref(h)
    if bits == 32:
        return L.adamw_step(n, sizes, col(p, "p"), pd, col(g, "g"), gd, col(m, "m"), col(v, "v"), h, None)
    return L.adamw_step_8bit(n, sizes, col(p, "p"), pd, col(g, "g"), gd, col(m, "m"), col(ms, "ms"), col(v, "v"),
                             col(vs, "vs"), 5, h, None)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_refusals(bits):
    L = _lib()
    f = lambda **a: _adamw(L, bits, **a)
    names = ("p", "g", "m", "v") + (("ms", "vs") if bits == 8 else ())
    for name in names:
        assert f(**{name: None}) == G.ERR_NULL, name
        assert f(**{name: "null"}) == G.ERR_NULL, name
        if bits == 32 or name not in ("m", "v"):              # codes are bytes
            assert f(**{name: BAD + 2}) == G.ERR_ALIGN, name
    assert f(pd=G.BF16, p=0x100001) == G.ERR_ALIGN and f(gd=G.BF16, g=0x200001) == G.ERR_ALIGN
    assert f(how="null") == G.ERR_NULL
    assert f(n=-1) == G.ERR_SHAPE and f(size=-1) == G.ERR_SHAPE and f(size=(1 << 35) + 1) == G.ERR_SHAPE
    for bad in (dict(pd=2), dict(gd=-1), dict(lr=-1.0), dict(lr=math.nan), dict(lr=math.inf), dict(eps=-1e-9),
                dict(weight_decay=math.inf), dict(beta1=1.0), dict(beta2=-0.1), dict(beta1=math.nan), dict(step=0),
                dict(step=-5), dict(eps=1e-39), dict(eps=5e-324)):
        assert f(**bad) == G.ERR_UNSUPPORTED, bad
    for name, bad in (("lr_dev", 0x900002), ("step_dev", 0x900004), ("grad_scale", 0x900001)):
        assert f(**{name: bad}) == G.ERR_ALIGN, name
    # nothing to do: no launch
    assert f(n=0) == G.OK and f(size=0, p=None, g=None, m=None, v=None, ms=None, vs=None) == G.OK


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_overlaps(bits):
    """A written buffer overlaps another: refused on the host, whatever the order in which they are listed."""
    L = _lib()
    f = lambda **a: _adamw(L, bits, **a)
    assert f(p=0x200000 + 3984) == G.ERR_OVERLAP             # p's first bytes are g's last
    assert f(m=0x100000) == G.ERR_OVERLAP and f(v=0x300000) == G.ERR_OVERLAP and f(g=0x400000) == G.ERR_OVERLAP
    other = dict(size=500, p=0x700000, g=0x800000, m=0x900000, v=0xA00000, ms=0xB00000, vs=0xC00000)
    for twice, at in (("p", 0x100000), ("m", 0x300000), ("v", 0x400000), ("p", 0x200000 + 16), ("m", 0x100000 + 3200)):
        assert f(n=2, second={**other, twice: at}) == G.ERR_OVERLAP, (twice, at)
    if bits == 8:
        assert f(n=2, second={**other, "ms": 0x500000 + 8}) == G.ERR_OVERLAP
        assert f(vs=0x500000 + 12) == G.ERR_OVERLAP          # four scales a tensor of 1000
    # numbers on the device are read while the buffers are written
    for name in ("lr_dev", "step_dev", "grad_scale"):
        assert f(**{name: 0x100000 + 80}) == G.ERR_OVERLAP and f(**{name: 0x400000}) == G.ERR_OVERLAP, name


def test_quantize_refusals():
    L = _lib()
    f = lambda **a: L.quantize_fp8_weights(a.get("w", A), a.get("dt", G.F32), a.get("K", 256), a.get("N", 256),
                                           a.get("G", 2), a.get("codes", A), a.get("scales", A), a.get("ws", A),
                                           a.get("wsb", 1 << 30), None)
    for name in ("w", "codes", "scales"):
        assert f(**{name: None}) == G.ERR_NULL and f(**{name: BAD}) == G.ERR_ALIGN, name
    assert f(K=0) == G.ERR_SHAPE and f(N=-128) == G.ERR_SHAPE and f(G=0) == G.ERR_SHAPE
    assert f(K=96) == G.ERR_UNSUPPORTED and f(N=200) == G.ERR_UNSUPPORTED and f(G=1025) == G.ERR_UNSUPPORTED
    assert f(dt=2) == G.ERR_UNSUPPORTED and f(K=1 << 16, N=1 << 16) == G.ERR_UNSUPPORTED
    assert f(K=16384 + 128) == G.ERR_UNSUPPORTED and f(ws=BAD) == G.ERR_ALIGN
    for dt, small, large in ((G.F32, 384, 640), (G.BF16, 768, 1152)):
        assert L.fp8gmm_workspace_bytes(G.OP_QUANT_WEIGHTS, 0, small, 256, 2, dt) == 0
        need = L.fp8gmm_workspace_bytes(G.OP_QUANT_WEIGHTS, 0, large, 256, 2, dt)
        assert need == 2 * 256 * 2 * 4                        # a word for each column of each half
        assert f(dt=dt, K=large, ws=None) == G.ERR_WORKSPACE and f(dt=dt, K=large, wsb=need - 1) == G.ERR_WORKSPACE
    assert L.fp8gmm_workspace_bytes(G.OP_QUANT_WEIGHTS, 0, 7168, 256, 2, 2) == 0


def test_binding_refusals():
    _lib()
    x = torch.zeros(4, 8)
    ids = torch.zeros((4, 2), dtype=torch.int32)
    w = torch.zeros((1, 128, 128))
    p = [torch.zeros(10)]
    for call in (lambda: G.moe_balance_loss(x, ids), lambda: G.moe_balance_loss_bwd(x[0], x, ids[0], ids[0]),
                 lambda: G.quantize_fp8_weights(w), lambda: G.adamw_step(p, p, p, p, lr=1e-3, step=1),
                 lambda: G.adamw_step_8bit(p, p, *G.adamw_8bit_states(p), lr=1e-3, step=1)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        G.moe_balance_loss(x.half(), ids)
    with pytest.raises(TypeError):
        G.quantize_fp8_weights(w.half())
    with pytest.raises(ValueError, match="one length"):
        G.adamw_step(p, p + p, p, p, lr=1e-3, step=1)
    with pytest.raises(TypeError, match="pairs"):
        G.adamw_step_8bit(p, p, p, p, lr=1e-3, step=1)
    with pytest.raises(TypeError, match="float32 or all bfloat16"):
        G.adamw_step([torch.zeros(10, dtype=torch.float16)], p, p, p, lr=1e-3, step=1)
    with pytest.raises(TypeError, match="hold torch"):
        G.adamw_step([1.0], p, p, p, lr=1e-3, step=1)
    with pytest.raises(TypeError):
        G.adamw_step(None, p, p, p, lr=1e-3, step=1)


def test_8bit_states():
    m, r = G.adamw_8bit_states([torch.zeros(3, 100), torch.zeros(256), torch.zeros(0), torch.zeros(())])
    assert [tuple(c.shape) for c, _ in m] == [(3, 100), (256,), (0,), ()] and [s.numel() for _, s in r] == [2, 1, 0, 1]
    assert all(c.dtype == torch.uint8 and s.dtype == torch.float32 for c, s in m + r)


# --------------------------------------------------------------------------- the plain definitions

def test_plain_balance_by_hand():
    x = torch.tensor([[0.0, math.log(3.0)], [math.log(3.0), 0.0], [-math.inf, -math.inf], [0.0, -math.inf]])
    ids = torch.tensor([[1], [0], [-1], [0]])
    losses, counts, probs, n = P.balance(x, ids)
    assert counts.tolist() == [2, 1] and n == 3
    assert torch.allclose(probs, torch.tensor([2 / 3, 1 / 3], dtype=torch.float64), atol=1e-7)
    assert abs(float(losses[0]) - 2 * (2 / 3 * 2 / 3 + 1 / 3 * 1 / 3)) < 1e-7
    assert abs(float(losses[1]) - 2 * math.log(4.0) ** 2 / 3) < 1e-6
    even = P.balance(torch.zeros(6, 3), torch.tensor([[0], [1], [2], [0], [1], [2]]))[0]
    assert abs(float(even[0]) - 1) < 1e-12 and abs(float(even[1]) - math.log(3) ** 2) < 1e-12
    assert P.balance(x[2:3], ids[2:3])[0].tolist() == [0.0, 0.0]
    assert math.isnan(P.balance(torch.tensor([[0.0, math.nan]]), ids[:1])[0][0])


def test_plain_balance_gradient_by_differences():
    g = torch.Generator().manual_seed(2)
    x = torch.randn((5, 6), generator=g, dtype=torch.float64)
    x[1, 2] = x[3, :] = -math.inf
    counts, d = torch.tensor([3, 0, 4, 1, 1, 1]), (0.7, 0.2)
    grad, _ = P.balance_bwd(d, x, counts, 4)
    loss = lambda y: float((P.balance(y, counts=counts)[0] * torch.tensor(d, dtype=torch.float64)).sum())
    h = 1e-6
    for t in range(5):
        for e in range(6):
            if x[t, e] == -math.inf:
                assert grad[t, e] == 0
                continue
            up, down = x.clone(), x.clone()
            up[t, e] += h
            down[t, e] -= h
            assert abs((loss(up) - loss(down)) / (2 * h) - float(grad[t, e])) < 1e-8


def test_plain_adamw_against_torch():
    """Three steps of torch's optimizer in float64."""
    g = torch.Generator().manual_seed(3)
    p = torch.randn(50, generator=g, dtype=torch.float64).requires_grad_()
    opt = torch.optim.AdamW([p], lr=0.02, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    q, m, v = p.detach().clone(), torch.zeros(50, dtype=torch.float64), torch.zeros(50, dtype=torch.float64)
    for t in range(1, 4):
        p.grad = torch.randn(50, generator=g, dtype=torch.float64)
        (q, m, v), _ = P.Step(0.02, t, (0.8, 0.95), 1e-6, 0.1)(q, p.grad, m, v)
        opt.step()
        assert torch.allclose(p.detach(), q, rtol=1e-12, atol=1e-12)


def test_plain_codes_by_hand():
    assert P.e4m3(torch.tensor([0, 1, 7, 8, 0x38, 0x7E, 0xFE, 0x80])).tolist() == \
        [0, 2 ** -9, 7 * 2 ** -9, 2 ** -6, 1.0, 448.0, -448.0, 0.0]
    everyone = torch.arange(256, dtype=torch.uint8)
    assert torch.equal(torch.nan_to_num(P.e4m3(everyone), 500.0),
                       torch.nan_to_num(everyone.view(torch.float8_e4m3fn).double(), 500.0))
    # 448 sets the scale to 1; 1.0625 is half way between 1 and 1.125; 0.3 steps of 2^-9
    x = torch.tensor([448.0, 1.0625, -1.0625, 0.3 * 2 ** -9, 0.0], dtype=torch.float64)
    low = P.held(x, P.scales_of(x), torch.tensor([0.4, 0.49, 0.51, 0.69, 0.9], dtype=torch.float64), False, 0 * x)[0]
    assert low.tolist() == [448.0, 1.0, 1.125, 0.0, 0.0]
    assert P.held(x.abs(), P.scales_of(x), 0 * x + 0.5, True, 0 * x)[0].tolist()[3:] == [2 ** -9, 0.0]


def test_noise_is_even():
    """Of 40960 draws: mean within 5 deviations of 1/2, no correlation between m's and r's or neighbours."""
    a, b = P.noise((7 << 32) + 1, 12, 3, 40960)
    n = 40960
    for x in (a, b):
        assert abs(float(x.mean()) - 0.5) < 5 * (1 / 12 / n) ** 0.5
        assert abs(float(((x - 0.5) ** 2).mean()) - 1 / 12) < 5 * (1 / 180 / n) ** 0.5
        assert abs(float(((x[1:] - 0.5) * (x[:-1] - 0.5)).mean())) < 5 / 12 / n ** 0.5
        assert abs(float(((x[256:] - 0.5) * (x[:-256] - 0.5)).mean())) < 5 / 12 / n ** 0.5
    assert abs(float(((a - 0.5) * (b - 0.5)).mean())) < 5 / 12 / n ** 0.5


def test_plain_weights_by_hand():
    w = torch.tensor([[[448.0, math.nan, 0.0], [-1.0625, 2.05, 0.0], [1.1876, -4.48, 0.0]]])
    v, s = P.quantize_weights(w)
    assert s[0, 0] == 1.0 and abs(float(s[0, 1]) - 0.01) < 1e-9 and abs(float(s[0, 2]) * 448 - 1e-12) < 1e-18
    assert v[0, :, 0].tolist() == [448.0, -1.0, 1.25]        # 1.0625 ties to the even 1, 1.1876 is past 1.1875
    assert math.isnan(v[0, 0, 1]) and v[0, 1, 1] == 208.0 and v[0, 2, 1] == -448.0 and v[0, :, 2].tolist() == [0.0] * 3
    assert torch.equal(P.e4m3((w[:, :, :1] / s[:, None, :1]).to(torch.float8_e4m3fn).view(torch.uint8)), v[:, :, :1])
