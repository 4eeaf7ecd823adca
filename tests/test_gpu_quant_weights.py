"""GPU tests of the FP8 weight quantizer against its definition, bit for bit."""
import math

import pytest
import torch

from tests import plain_train as P

pytestmark = pytest.mark.gpu


def weights(G, K, N, dtype, seed):
    """Columns of very different sizes, one of zeros, one below the floor."""
    g = torch.Generator().manual_seed(seed)
    w = 0.02 * torch.randn((G, K, N), generator=g) * torch.exp2(torch.randint(-20, 20, (N,), generator=g).float())
    w[:, :, 3] = 0
    w[:, :, 5] *= 1e-20
    w[:, 1::3, ::7] = -0.0
    return w.to(dtype)


def check(codes, scales, w):
    value, scale = P.quantize_weights(w)
    assert codes.dtype == torch.uint8 and torch.equal(scales.cpu(), scale)
    got = P.e4m3(codes.cpu())
    assert torch.equal(torch.isnan(got), torch.isnan(value))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(value))
    signs = torch.signbit(got) == torch.signbit(w.double())
    assert bool(signs[~torch.isnan(value)].all())                # zeros keep theirs


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G_,K,N", [(1, 128, 128), (2, 256, 384), (3, 768, 256), (1, 7168, 128), (2, 1152, 640),
                                    (1, 16384, 128), (1, 1664, 256), (5, 128, 1920), (1, 3200, 384),
                                    (2, 2048, 1536), (3, 896, 6144), (40, 256, 640), (9, 1152, 2176)])
def test_quantize_fp8_weights(G_, K, N, dtype):
    import fp8_moe_grouped_amd as G
    w = weights(G_, K, N, dtype, K + N)
    check(*G.quantize_fp8_weights(w.cuda()), w)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_largest_anywhere(dtype):
    """Each row of a column in turn holds the largest magnitude: every lane's part of the maximum."""
    import fp8_moe_grouped_amd as G
    for K in (128, 640, 2304):
        w = torch.ones((1, K, 128 * (-(-K // 128))), dtype=dtype)
        k = torch.arange(K)
        w[0, k, k] = -(2.0 + k % 7).to(dtype)
        check(*G.quantize_fp8_weights(w.cuda()), w)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nan_and_inf(dtype):
    import fp8_moe_grouped_amd as G
    for K in (128, 8192):
        w = weights(1, K, 128, dtype, 1)
        w[0, K // 2, 7] = math.nan
        w[0, K - 1, 8] = -math.inf
        w[0, :, 9] = math.nan
        w[0, 0, 10], w[0, 1, 10] = math.inf, math.nan
        codes, scales = G.quantize_fp8_weights(w.cuda())
        check(codes, scales, w)
        assert torch.isfinite(scales[0, 7]) and torch.isinf(scales[0, 8]) and torch.isinf(scales[0, 10])


def test_every_quotient_border():
    """f32 weights next to the codes' borders, with scales of all mantissas: the quotient's own rounding decides."""
    import fp8_moe_grouped_amd as G
    g = torch.Generator().manual_seed(9)
    K, N = 512, 1024
    top = (1 + torch.rand(N, generator=g)) * torch.exp2(torch.randint(-12, 12, (N,), generator=g).float())
    scale = top / torch.tensor(448.0)
    every = P.e4m3(torch.arange(127, dtype=torch.uint8))
    border = (every[1:] + every[:-1]) / 2
    w = (border[torch.randint(0, 126, (K, N), generator=g)].float() * scale)
    near = torch.randint(-1, 2, (K, N), generator=g)             # one f32 step off, or none
    w = torch.where(near > 0, torch.nextafter(w, w * 2), torch.where(near < 0, torch.nextafter(w, 0 * w), w))
    w[0] = top
    w = torch.where(torch.rand((K, N), generator=g) < 0.5, w, -w).unsqueeze(0)
    check(*G.quantize_fp8_weights(w.cuda()), w)


def test_same_as_the_products_read():
    """The codes go into a product: its dequantized weights are the weights to half a step of e4m3."""
    import fp8_moe_grouped_amd as G
    w = weights(2, 256, 256, torch.float32, 4).cuda()
    codes, scales = G.quantize_fp8_weights(w)
    back = G.dequantize_fp8_codes(codes, scales).double()
    top = scales.double().unsqueeze(1)
    # half a step of e4m3 (2^-4, or of its smallest numbers 2^-10 scales), then of bf16; f32's on the way
    assert bool(((back - w).abs() <= w.abs().double() * (2.0 ** -4 + 2.0 ** -8) + top * 2.0 ** -10 + 1e-40).all())


def test_outputs_graph_and_stream():
    import fp8_moe_grouped_amd as G
    ws = [weights(2, 1024, 256, torch.float32, s).cuda() for s in range(3)]
    eager = [G.quantize_fp8_weights(w) for w in ws]
    codes = torch.full((2 * 1024 * 256 + 64,), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((2 * 256 + 16,), -7.0, device="cuda")
    c, s = codes[:-64].view(2, 1024, 256), scales[:-16].view(2, 256)
    a, b = G.quantize_fp8_weights(ws[1], codes=c, scales=s)
    assert a is c and b is s and torch.equal(c, eager[1][0]) and torch.equal(s, eager[1][1])
    assert bool((codes[-64:] == 0xAA).all()) and bool((scales[-16:] == -7).all())
    w = ws[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = G.quantize_fp8_weights(w)
    for i in (0, 1, 2, 0):
        w.copy_(ws[i])
        graph.replay()
        G.quantize_fp8_weights(ws[(i + 1) % 3])
        torch.cuda.synchronize()
        assert torch.equal(out[0], eager[i][0]) and torch.equal(out[1], eager[i][1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o = G.quantize_fp8_weights(ws[2])
    side.synchronize()
    assert torch.equal(o[0], eager[2][0])


def _launch(w, codes, scales, words, polls):
    """The library's launcher, which the C call hands its number of polls."""
    import ctypes

    import fp8_moe_grouped_amd as G
    f = G.lib()._ZN6fp8gmm24launch_quant_weights_fp8EPKvbiiiPhPfPviP12ihipStream_t
    p, i = ctypes.c_void_p, ctypes.c_int
    f.argtypes = [p, ctypes.c_bool, i, i, i, p, p, p, i, p]
    n, K, N = w.shape
    assert f(w.data_ptr(), w.dtype == torch.bfloat16, n, K, N, codes.data_ptr(), scales.data_ptr(), words.data_ptr(),
             polls, torch.cuda.current_stream().cuda_stream) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_block_that_waits_in_vain(dtype):
    """With no polls, or one, blocks compute the maxima of the strip's other blocks themselves: the same bits."""
    import fp8_moe_grouped_amd as G
    w = weights(3, 2432, 512, dtype, 5)
    w[1, 2000, 100] = math.nan
    w[1, 10, 101] = -math.inf
    dev = w.cuda()
    want = G.quantize_fp8_weights(dev)
    check(*want, w)
    for polls in (0, 1):
        codes, scales = torch.full_like(want[0], 0xAA), torch.full_like(want[1], -1.0)
        words = torch.full((3 * 512 * 7,), -1, dtype=torch.int32, device="cuda")
        _launch(dev, codes, scales, words, polls)
        assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G_,K,N", [(8, 4096, 2048), (2, 16384, 4224), (122, 1152, 1024), (1024, 128, 1152), (1, 6912, 640),
                                    (3, 2176, 2816)])
def test_large(G_, K, N, dtype):
    """Strips of 16 to 128 columns, one part to forty-three, against the definition on the GPU: 64-bit quotients of f32 numbers
    round to f32's own."""
    import fp8_moe_grouped_amd as G
    g = torch.Generator(device="cuda").manual_seed(K)
    w = torch.randn((G_, K, N), generator=g, device="cuda") * torch.exp2(torch.randint(-9, 9, (N,), generator=g,
                                                                                      device="cuda").float())
    w = w.to(dtype)
    w[0, K - 1, 5], w[G_ - 1, 0, N - 1], w[G_ // 2, K // 2, 77] = math.nan, math.inf, 1e4
    codes, scales = G.quantize_fp8_weights(w)
    for e in range(G_):
        x = w[e].float()
        top = torch.where(torch.isnan(x), 0.0, x.abs()).amax(0).clamp(min=1e-12)
        scale = (top.double() / 448).float()
        assert torch.equal(scales[e], scale)
        q = (x.double() / scale.double()).float().double()
        d = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))).clamp(max=8) - 3)
        want = torch.where(torch.isnan(q), 500.0, torch.round(q / d) * d)
        got = codes[e].view(torch.float8_e4m3fn).double()
        assert torch.equal(torch.where(torch.isnan(got), 500.0, got), want)


def test_given_workspace():
    import fp8_moe_grouped_amd as G
    w = weights(2, 2048, 256, torch.float32, 6).cuda()
    want = G.quantize_fp8_weights(w)
    need = G.workspace_bytes(G.OP_QUANT_WEIGHTS, 0, 2048, 256, 2, G.F32)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):                                           # whatever the last call left there
        got = G.quantize_fp8_weights(w, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((ws[need:] == 0xFF).all())
    with pytest.raises(ValueError, match="needed"):
        G.quantize_fp8_weights(w, workspace=ws[:need - 1])
    with pytest.raises(ValueError):
        G.quantize_fp8_weights(w, workspace=ws.cpu())


def test_two_at_once():
    """Two streams, many blocks of each waiting for others: every call ends with the same bits."""
    import fp8_moe_grouped_amd as G
    ws = [weights(2, 7168, 1024, torch.float32, s).cuda() for s in range(2)]
    want = [G.quantize_fp8_weights(w) for w in ws]
    streams = [torch.cuda.Stream() for _ in ws]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s, w in zip(streams, ws):
            with torch.cuda.stream(s):
                got.append(G.quantize_fp8_weights(w))
    torch.cuda.synchronize()
    for i, (c, s) in enumerate(got):
        assert torch.equal(c, want[i % 2][0]) and torch.equal(s, want[i % 2][1])


@pytest.mark.parametrize("n", [2, 4])
def test_several_at_once_of_the_longest_columns(n):
    """Strips in 22 parts from several streams, which together ask for more blocks than fit: what waits in vain reads for
    itself and for the others."""
    import fp8_moe_grouped_amd as G
    g = torch.Generator(device="cuda").manual_seed(n)
    ws = [torch.randn((2, 16384, 2048), generator=g, device="cuda") for _ in range(n)]
    want = [G.quantize_fp8_weights(w) for w in ws]
    streams = [torch.cuda.Stream() for _ in ws]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, w in zip(streams, ws):
            with torch.cuda.stream(s):
                got.append(G.quantize_fp8_weights(w))
        torch.cuda.synchronize()
        for (c, s), (wc, ws_) in zip(got, want):
            assert torch.equal(c, wc) and torch.equal(s, ws_)


def test_past_4_gib():
    """f32 weights of 9 GiB: the last expert's columns."""
    import fp8_moe_grouped_amd as G
    n, K, N = 9, 16384, 16384
    w = torch.zeros((n, K, N), device="cuda")
    w[n - 1] = weights(1, K, 128, torch.float32, 2).cuda().repeat(1, 1, N // 128)[0]
    codes, scales = G.quantize_fp8_weights(w)
    value = w[n - 1, :, -128:].cpu().unsqueeze(0)
    check(codes[n - 1, :, -128:].unsqueeze(0), scales[n - 1, -128:].unsqueeze(0), value)
    assert not bool(codes[:n - 1].any())


def test_refusals():
    import fp8_moe_grouped_amd as G
    w = torch.zeros((2, 128, 256), device="cuda")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    for call in (lambda: G.quantize_fp8_weights(w.transpose(1, 2)), lambda: G.quantize_fp8_weights(w[0]),
                 lambda: G.quantize_fp8_weights(w, codes=u8(2, 128, 128)),
                 lambda: G.quantize_fp8_weights(w, scales=torch.zeros((2, 128), device="cuda")),
                 lambda: G.quantize_fp8_weights(w, codes=u8(2, 128, 256).cpu())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        G.quantize_fp8_weights(w.half())
    for bad in (w[:, :100].contiguous(), w[:, :, :200].contiguous(), w[:0],
                torch.zeros((1, 16384 + 128, 128), device="cuda")):
        with pytest.raises(G.Fp8GmmError):
            G.quantize_fp8_weights(bad)
    torch.cuda.synchronize()
