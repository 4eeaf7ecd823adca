"""CPU tests of the routing, dispatch, combine and MXFP4 entry points: what the
C ABI and the binding refuse (fake device pointers are never dereferenced), and
hand-computed pins of the plain definitions that the GPU tests compare with."""
import math
import os

import pytest
import torch

import fp8_moe_grouped_amd as G
from tests import plain_moe as P

A = 0x10000          # fake, 16-byte aligned "device" address
BAD = 0x10008        # misaligned


def _lib():
    if not os.path.exists(G.LIB_PATH):
        pytest.skip("library not built")
    return G.lib()


def test_macros_match_binding():
    text = open(G.HEADER_PATH).read()
    for name, value in (("OP_ROUTE 10", G.OP_ROUTE), ("OP_MXFP4 11", G.OP_MXFP4), ("F32 0", G.F32), ("BF16 1", G.BF16)):
        assert f"#define FP8GMM_{name}" in text and int(name.split()[1]) == value


def test_route_refusals():
    L = _lib()
    f = lambda **a: L.moe_route(a.get("x", A), a.get("dt", G.F32), a.get("T", 4096), a.get("E", 64), a.get("k", 8), 1,
                                a.get("ids", A), A, a.get("gs", A), A, A, a.get("ws", A), a.get("wsb", 1 << 30), None)
    assert f(x=None) == G.ERR_NULL and f(ids=None) == G.ERR_NULL and f(gs=None) == G.ERR_NULL
    assert f(T=-1) == G.ERR_SHAPE and f(E=0) == G.ERR_SHAPE and f(k=0) == G.ERR_SHAPE
    assert f(k=65) == G.ERR_SHAPE and f(T=1 << 21, k=8) == G.ERR_SHAPE
    assert f(T=(1 << 63) - 1) == G.ERR_SHAPE
    assert f(E=1025) == G.ERR_UNSUPPORTED and f(k=33) == G.ERR_UNSUPPORTED and f(dt=2) == G.ERR_UNSUPPORTED
    assert f(x=BAD) == G.ERR_ALIGN
    need = L.fp8gmm_workspace_bytes(G.OP_ROUTE, 4096, 64, 8, 1, 0)
    assert need > 0 and f(ws=None) == G.ERR_WORKSPACE and f(wsb=need - 1) == G.ERR_WORKSPACE
    assert L.fp8gmm_workspace_bytes(G.OP_ROUTE, 1, 64, 8, 1, 0) == 0
    assert L.fp8gmm_workspace_bytes(G.OP_ROUTE, 4096, 64, 65, 1, 0) == 0
    b = lambda **a: L.moe_route_bwd(a.get("dw", A), a.get("x", A), a.get("dt", G.F32), A, A, a.get("T", 8),
                                    a.get("E", 64), a.get("k", 8), a.get("renorm", 0), a.get("out", A), None)
    assert b(dw=None) == G.ERR_NULL and b(x=None) == G.ERR_NULL and b(out=None) == G.ERR_NULL
    assert b(T=-1) == G.ERR_SHAPE and b(k=65) == G.ERR_SHAPE and b(E=1025) == G.ERR_UNSUPPORTED
    assert b(dt=7) == G.ERR_UNSUPPORTED and b(out=BAD) == G.ERR_ALIGN
    assert b(T=0, dw=None, x=None, out=None) == G.OK


def test_slot_refusals():
    L = _lib()
    calls = {
        "permute": lambda a: L.moe_permute(a["x"], a["map"], a["T"], a["k"], a["R"], a["H"], a["out"], None),
        "permute_fp8": lambda a: L.moe_permute_fp8(a["x"], a["map"], a["T"], a["k"], a["R"], a["H"], a["out"], A, None),
        "combine": lambda a: L.moe_combine(a["x"], a["map"], None, a["T"], a["k"], a["R"], a["H"], a["out"], None),
        "combine_bwd": lambda a: L.moe_combine_bwd(A, a["x"], a["map"], A, a["T"], a["k"], a["R"], a["H"], a["out"], A,
                                                   None),
    }
    base = dict(x=A, map=A, T=16, k=4, R=64, H=256, out=A)
    for name, f in calls.items():
        g = lambda **a: f({**base, **a})
        assert g(x=None) == G.ERR_NULL and g(map=None) == G.ERR_NULL and g(out=None) == G.ERR_NULL, name
        for bad in (dict(T=-1), dict(k=0), dict(R=-1), dict(R=1 << 24), dict(H=0), dict(T=1 << 23)):
            assert g(**bad) == G.ERR_SHAPE, (name, bad)
        for bad in (dict(k=33), dict(H=200), dict(H=16384 + 128)):
            assert g(**bad) == G.ERR_UNSUPPORTED, (name, bad)
        assert g(x=BAD) == G.ERR_ALIGN and g(out=BAD) == G.ERR_ALIGN, name
        assert g(T=0, x=None, map=None, out=None) in (G.OK,), name


def test_mxfp4_refusals():
    L = _lib()
    q = lambda **a: L.quantize_mxfp4_weights(a.get("w", A), a.get("K", 256), a.get("N", 256), a.get("G", 2),
                                             a.get("out", A), A, None)
    d = lambda **a: L.dequantize_mxfp4(a.get("w", A), A, a.get("K", 256), a.get("N", 256), a.get("G", 2),
                                       a.get("out", A), None)
    for f in (q, d):
        assert f(w=None) == G.ERR_NULL and f(out=None) == G.ERR_NULL
        assert f(K=0) == G.ERR_SHAPE and f(G=0) == G.ERR_SHAPE
        assert f(K=96) == G.ERR_UNSUPPORTED and f(N=200) == G.ERR_UNSUPPORTED and f(K=16384 + 128) == G.ERR_UNSUPPORTED
        assert f(G=1025) == G.ERR_UNSUPPORTED and f(w=BAD) == G.ERR_ALIGN and f(out=BAD) == G.ERR_ALIGN
    for name in ("gmm_mxfp4_fwd", "gmm_silu_mxfp4"):
        m = lambda **a: getattr(L, name)(a.get("x", A), a.get("w", A), A, a.get("gs", A), a.get("map", A),
                                         a.get("topk", 2), a.get("T", 32), a.get("M", 64), a.get("K", 256),
                                         a.get("N", 256), a.get("G", 4), a.get("out", A), a.get("ws", A),
                                         a.get("wsb", 1 << 30), None, None)
        assert m(x=None) == G.ERR_NULL and m(w=None) == G.ERR_NULL and m(gs=None) == G.ERR_NULL
        assert m(out=None) == G.ERR_NULL
        assert m(M=-1) == G.ERR_SHAPE and m(T=-1) == G.ERR_SHAPE and m(topk=0) == G.ERR_SHAPE
        assert m(T=1 << 24) == G.ERR_SHAPE and m(map=None) == G.ERR_SHAPE            # rows without a map: T != M
        assert m(K=192) == G.ERR_UNSUPPORTED and m(N=192) == G.ERR_UNSUPPORTED and m(G=1025) == G.ERR_UNSUPPORTED
        assert m(K=16384 + 128) == G.ERR_UNSUPPORTED and m(N=65536 + 256) == G.ERR_UNSUPPORTED
        assert m(x=BAD) == G.ERR_ALIGN and m(w=BAD) == G.ERR_ALIGN and m(out=BAD) == G.ERR_ALIGN
        need = L.fp8gmm_workspace_bytes(G.OP_MXFP4, 32, 256, 256, 4, 0)
        assert need >= 33 * (128 + 8)
        assert m(ws=None) == G.ERR_WORKSPACE and m(wsb=need - 1) == G.ERR_WORKSPACE
        assert m(M=0, x=None, out=None, ws=None, wsb=0) == G.OK
    assert L.gmm_silu_mxfp4(A, A, A, A, None, 1, 8, 8, 256, 384, 4, A, A, 1 << 30, None, None) == G.ERR_UNSUPPORTED


def test_binding_refusals():
    _lib()
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    rows = torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: G.moe_route(torch.zeros(4, 8), 2), lambda: G.moe_permute(x, rows),
                 lambda: G.moe_permute_fp8(x, rows), lambda: G.moe_combine(x, rows),
                 lambda: G.quantize_mxfp4_weights(torch.zeros((1, 128, 128), dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        G.moe_route(torch.zeros((4, 8), dtype=torch.float16), 2)
    with pytest.raises(TypeError):
        G.moe_route([[0.0]], 1)


@pytest.mark.parametrize("topk", [(1 << 32) + 1, 1 - (1 << 32), -(1 << 31) - 1, -(1 << 70)])
def test_binding_refuses_topk_past_32_bits(topk):
    """On either side: ctypes would keep the low 32 bits, 1 of 1 - 2^32."""
    _lib()
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    codes, scales = torch.zeros((2, 128, 64), dtype=torch.uint8), torch.zeros((2, 1, 128, 4), dtype=torch.uint8)
    with pytest.raises(ValueError, match="topk"):
        G.gmm_mxfp4_fwd(x, codes, scales, torch.zeros(2, dtype=torch.int32), topk=topk)


# --------------------------------------------------------------------------- the plain definitions

def test_plain_route_by_hand():
    inf = math.inf
    x = torch.tensor([[0.0, 1.0, 1.0, -inf], [-inf, -inf, 2.0, -inf], [-inf] * 4, [0.0, -0.0, 0.0, 5.0]])
    ids, w, sizes, rows, slots = P.route(x, 2, True)
    assert ids.tolist() == [[1, 2], [2, -1], [-1, -1], [3, 0]]
    assert w[0].tolist() == [0.5, 0.5] and w[1].tolist() == [1.0, 0.0] and w[2].tolist() == [0.0, 0.0]
    assert sizes.tolist() == [1, 1, 2, 1]
    # slots 0..7 hold experts 1 2 | 2 - | - - | 3 0
    assert rows.view(-1).tolist() == [1, 2, 3, -1, -1, -1, 4, 0]
    assert slots.tolist() == [7, 0, 1, 2, 6, -1, -1, -1]
    _, w, *_ = P.route(x, 2, False)
    assert abs(float(w[0, 0]) - math.e / (2 * math.e + 1)) < 1e-15
    nan = torch.tensor([[0.0, math.nan, inf]])
    ids, w, *_ = P.route(nan, 2, True)
    assert ids.tolist() == [[1, 2]] and all(math.isnan(v) for v in w[0].tolist())


@pytest.mark.parametrize("renorm", [True, False])
def test_plain_route_gradient_by_differences(renorm):
    g = torch.Generator().manual_seed(5)
    x = torch.randn((6, 7), generator=g, dtype=torch.float64)
    dw = torch.randn((6, 3), generator=g, dtype=torch.float64)
    ids, w, *_ = P.route(x, 3, renorm)
    d, _ = P.route_bwd(dw, x, ids, w, renorm)
    h = 1e-6
    for t in range(6):
        for e in range(7):
            up, down = x.clone(), x.clone()
            up[t, e] += h
            down[t, e] -= h
            iu, wu, *_ = P.route(up, 3, renorm)
            il, wl, *_ = P.route(down, 3, renorm)
            assert torch.equal(iu, ids) and torch.equal(il, ids)
            num = float(((wu - wl) * dw).sum()) / (2 * h)
            assert abs(num - float(d[t, e])) < 1e-8


def test_plain_mxfp4_by_hand():
    x = torch.zeros((1, 64))
    x[0, :12] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.26, -0.25, -0.3, -5.01])
    x[0, 32:34] = torch.tensor([7.9, 1.0])               # amax in [4, 8): saturates at 6
    code, byte = P.mxfp4(x)
    assert byte.tolist() == [[127, 127]]
    assert code[0, :12].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 1, 8, 9, 15]
    assert code[0, 32:34].tolist() == [7, 2]
    assert P.mxfp4_values(code, byte)[0, 32:34].tolist() == [6.0, 1.0]
    small = torch.full((1, 32), 2.0 ** -130)
    code, byte = P.mxfp4(small)
    assert byte.tolist() == [[0]] and code.unique().tolist() == [0]      # 2^-3 of the smallest unit
    assert P.mxfp4(torch.full((1, 32), 2.0 ** -128))[0].unique().tolist() == [1]
    bad = torch.ones((1, 64))
    bad[0, 3] = math.nan
    bad[0, 40] = -math.inf
    assert P.mxfp4(bad)[1].tolist() == [[255, 255]]
    packed, scales = P.pack_weights(torch.arange(128, dtype=torch.uint8).view(1, 1, 128) % 16,
                                    torch.arange(4, dtype=torch.uint8).view(1, 1, 4))
    assert packed[0, 0, :3].tolist() == [0x10, 0x32, 0x54] and scales.tolist() == [[[[0, 1, 2, 3]]]]
