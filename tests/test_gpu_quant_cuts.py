"""GPU tests of the FP8 weight quantizer's workspace, and of its widest f32
strips, whose rows are shared by many blocks.  A strip of 128 columns is taken from 2^19 elements a CU
(256 CUs: G K N >= 2^27) while K <= 9216; a block keeps 384 of its rows, and four
groups of threads look for the other blocks' maxima, each for every fourth one."""
import pytest
import torch

from tests.test_gpu_quant_weights import _launch

pytestmark = pytest.mark.gpu


def weights(G_, K, N):
    """Columns of very different sizes; a NaN, an Inf and a column's largest in each part of an expert's rows."""
    g = torch.Generator(device="cuda").manual_seed(K + N)
    w = torch.randn((G_, K, N), generator=g, device="cuda") * torch.exp2(
        torch.randint(-9, 9, (N,), generator=g, device="cuda").float())
    part = torch.arange(K, device="cuda") // 384
    w[1, torch.arange(K, device="cuda"), part] *= 8              # column i has its largest in part i, most probably
    w[0, K - 1, 5], w[G_ - 1, 0, N - 1], w[G_ // 2, K // 2, 77] = float("nan"), float("inf"), 1e4
    w[0, ::3, ::5] = -0.0
    return w


def check(codes, scales, w):
    """Against the definition on the GPU: 64-bit quotients of f32 numbers round to f32's own."""
    for e in range(w.shape[0]):
        x = w[e].float()
        top = torch.where(torch.isnan(x), 0.0, x.abs()).amax(0).clamp(min=1e-12)
        scale = (top.double() / 448).float()
        assert torch.equal(scales[e], scale)
        q = (x.double() / scale.double()).float().double()
        d = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))).clamp(max=8) - 3)
        want = torch.where(torch.isnan(q), 500.0, torch.round(q / d) * d)
        got = codes[e].view(torch.float8_e4m3fn).double()
        assert torch.equal(torch.where(torch.isnan(got), 500.0, got), want)
        assert torch.equal(torch.signbit(got)[want == 0], torch.signbit(x)[want == 0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G_,K,N", [(5, 9216, 2944), (5, 9344, 2944), (2, 16384, 4224), (1, 16384, 128), (1, 9216, 256),
                                    (8, 1664, 768)])
def test_a_workspace_of_the_stated_size(G_, K, N, dtype):
    """What the call says it needs is what it uses at most: nothing behind it changes."""
    import fp8_moe_grouped_amd as G
    w = weights(max(G_, 2), K, N)[:G_].to(dtype)
    need = G.workspace_bytes(G.OP_QUANT_WEIGHTS, 0, K, N, G_, G.BF16 if dtype == torch.bfloat16 else G.F32)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    codes, scales = G.quantize_fp8_weights(w, workspace=ws)
    assert bool((ws[need:] == 0xFF).all())
    check(codes, scales, w)


@pytest.mark.parametrize("G_,K,N", [(8, 7168, 2432), (5, 9216, 2944), (40, 1536, 2304), (12, 2944, 3968)])
def test_strips_of_128_columns(G_, K, N):
    """19 parts, 24 (the most of any cut), 4 and 8."""
    import fp8_moe_grouped_amd as G
    w = weights(G_, K, N)
    check(*G.quantize_fp8_weights(w), w)


@pytest.mark.parametrize("G_,K,N", [(8, 7168, 2432), (5, 9216, 2944)])
def test_wide_strips_that_wait_in_vain(G_, K, N):
    """With no polls, or one, a block reads the rows of the strip's other blocks itself, a group several of them."""
    import fp8_moe_grouped_amd as G
    w = weights(G_, K, N)
    codes, scales = G.quantize_fp8_weights(w)
    check(codes, scales, w)
    for polls in (0, 1):
        c, s = torch.full_like(codes, 0xAA), torch.full_like(scales, -1.0)
        words = torch.full((G_ * N * (K // 384 + 1),), -1, dtype=torch.int32, device="cuda")
        _launch(w, c, s, words, polls)
        assert torch.equal(c, codes) and torch.equal(s, scales)
