"""GPU tests of the FP8 weight quantizer's workspace."""
import pytest
import torch

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
