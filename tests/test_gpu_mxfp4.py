"""GPU tests of the MXFP4 calls: codes, scales and values bit for bit; products
within f32 accumulation and half a bf16 step of the plain 64-bit definition."""
import math

import pytest
import torch

from tests import plain_moe as P

pytestmark = pytest.mark.gpu


def special(w):
    """Blocks of zeros, signed zeros, ties, subnormals, the largest values."""
    flat = w.view(-1, w.shape[-1])                   # [.., N]: columns are channels
    flat[:32, 0] = 0
    flat[:32, 1] = -0.0
    flat[:16, 2] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -7.9])
    flat[16:32, 2] = 0
    flat[:32, 3] = 2.0 ** -133
    flat[:32, 4] = 3.38e38
    flat[:32, 5] = torch.linspace(-2.0 ** -124, 2.0 ** -125, 32)
    return w


@pytest.mark.parametrize("G_,K,N", [(1, 128, 128), (3, 384, 256), (2, 640, 384), (1, 7168, 128), (5, 256, 640)])
def test_weights(G_, K, N):
    import fp8_moe_grouped_amd as G
    w = torch.randn((G_, K, N), generator=torch.Generator().manual_seed(K)) * 0.02
    w = special(w).to(torch.bfloat16)
    code, byte = P.mxfp4(w.transpose(1, 2))
    want_c, want_s = P.pack_weights(code, byte)
    codes, scales = G.quantize_mxfp4_weights(w.cuda())
    assert torch.equal(codes.cpu(), want_c) and torch.equal(scales.cpu(), want_s)
    values = G.dequantize_mxfp4(codes, scales).cpu()
    want = P.mxfp4_values(code, byte).to(torch.bfloat16)
    assert torch.equal(values.view(torch.int16), want.view(torch.int16))


def test_weights_not_finite():
    import fp8_moe_grouped_amd as G
    w = torch.ones((1, 128, 128), dtype=torch.bfloat16)
    w[0, 3, 0], w[0, 40, 1], w[0, 127, 2] = math.nan, math.inf, -math.inf
    codes, scales = G.quantize_mxfp4_weights(w.cuda())
    s = scales.cpu()[0, 0]
    assert s[0].tolist() == [255, 125, 125, 125] and s[1].tolist() == [125, 255, 125, 125]
    assert s[2].tolist() == [125, 125, 125, 255]
    nan = torch.isnan(G.dequantize_mxfp4(codes, scales)).cpu()[0]
    assert nan[0, :32].all() and nan[1, 32:64].all() and nan[2, 96:].all() and int(nan.sum()) == 96


def activations(T, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, K), generator=g)
    return torch.where(torch.rand((T, K), generator=g) < 0.01, 50 * x, x).to(torch.bfloat16)


def weights(G_, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    code = torch.randint(0, 16, (G_, N, K), generator=g, dtype=torch.uint8)
    byte = torch.randint(118, 124, (G_, N, K // 32), generator=g, dtype=torch.uint8)
    return code, byte


def product(x, code, byte, sizes, tokens):
    """(sum, sum of magnitudes) in float64 of the valid rows."""
    a = P.mxfp4_values(*P.mxfp4(x))
    y, mag, at = [], [], 0
    for g, n in enumerate(sizes):
        w = P.mxfp4_values(code[g], byte[g])
        rows = torch.where((tokens[at:at + n] >= 0).unsqueeze(1), a[tokens[at:at + n].clamp(min=0)], 0.0)
        y.append(rows @ w.t())
        mag.append(rows.abs() @ w.abs().t())
        at += n
    return torch.cat(y), torch.cat(mag)


def check(out, y, mag, K, swiglu):
    # each instruction adds the sums of four blocks to f32: four roundings of at most the magnitudes'
    # sum, twice over for an adder that cuts off; a few more where partial sums are joined
    e = mag * 2.0 ** -23 * (4 * K / 128 + 16)
    if swiglu:
        I = y.shape[1] // 2
        g, u, eg, eu = y[:, :I], y[:, I:], e[:, :I], e[:, I:]
        sig = torch.sigmoid(g)
        silu, slope = g * sig, (sig * (1 + g * (1 - sig))).abs()
        # first order, the second order of the small errors, and the f32 evaluation (exp's argument, reciprocal)
        e = slope * u.abs() * eg + silu.abs() * eu + eg * eu * 1.1 + 0.5 * eg * eg * u.abs() \
            + 2.0 ** -20 * (4 + g.abs()) * (silu * u).abs()
        y = silu * u
    got = out.cpu().double()
    tol = e + y.abs() * 2.0 ** -8 + 2.0 ** -126
    bad = (got - y).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), float(((got - y).abs() / tol).max()))


def sizes_of(M, G_, seed, empty=True):
    g = torch.Generator().manual_seed(seed)
    p = torch.rand(G_, generator=g) ** 2
    if empty and G_ > 2:
        p[1] = 0
    n = (p / p.sum() * M).floor().int()
    n[-1] += M - int(n.sum())
    return n


GEMM = [(1, 1, 1, 128, 256), (1, 8, 8, 7168, 256), (3, 2, 5, 384, 512), (17, 1, 2, 256, 256), (33, 4, 4, 640, 768),
        (100, 3, 7, 1152, 512), (257, 1, 1, 512, 256), (300, 4, 6, 896, 1280), (64, 2, 32, 128, 256),
        (1500, 2, 3, 256, 512), (2100, 1, 2, 768, 1024)]


@pytest.mark.parametrize("T,k,G_,K,N", GEMM)
@pytest.mark.parametrize("swiglu", [False, True])
def test_product(T, k, G_, K, N, swiglu):
    """Gathered rows, ragged and empty groups, rows past the valid prefix, slots without a token."""
    import fp8_moe_grouped_amd as G
    M = T * k
    g = torch.Generator().manual_seed(T)
    tail = M // 10
    sizes = sizes_of(M - tail, G_, K)
    slots = torch.randperm(M, generator=g).int()
    if M > 4:
        slots[1], slots[3] = -1, M + 5               # no token: zeros
    x = activations(T, K, T)
    code, byte = weights(G_, N, K, N)
    codes, scales = P.pack_weights(code, byte)
    tokens = torch.where((slots >= 0) & (slots < M), slots // k, -1).long()
    n = M - tail
    slots[n:] = torch.iinfo(torch.int32).max
    out = torch.full((M, N // 2 if swiglu else N), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    f = G.gmm_silu_mxfp4 if swiglu else G.gmm_mxfp4_fwd
    f(x.cuda(), codes.cuda(), scales.cuda(), sizes.cuda(), slot_of_row=slots.cuda(), topk=k, out=out, dev_status=status)
    y, mag = product(x, code, byte, sizes.tolist(), tokens)
    assert int(status) == 0 and bool((out[n:] == 7.0).all())
    check(out[:n], y, mag, K, swiglu)


@pytest.mark.parametrize("M,N", [(9, 128), (70, 384), (900, 640)])
def test_product_plain_rows(M, N):
    """Without a map, and N a multiple of 128 only."""
    import fp8_moe_grouped_amd as G
    K = 512
    x = activations(M, K, 1)
    code, byte = weights(3, N, K, 2)
    codes, scales = P.pack_weights(code, byte)
    sizes = sizes_of(M, 3, 5)
    out = G.gmm_mxfp4_fwd(x.cuda(), codes.cuda(), scales.cuda(), sizes.cuda())
    check(out, *product(x, code, byte, sizes.tolist(), torch.arange(M)), K, False)


def test_product_not_finite():
    """An Inf or NaN activation makes its own rows NaN, a NaN scale its own column."""
    import fp8_moe_grouped_amd as G
    x = activations(40, 256, 1)
    x[3, 7], x[20, 200] = math.inf, math.nan
    code, byte = weights(2, 256, 256, 2)
    code = code & 7 | 1                              # no zero codes
    byte[1, 5, 2] = 255
    codes, scales = P.pack_weights(code, byte)
    sizes = torch.tensor([15, 25], dtype=torch.int32)
    out = G.gmm_mxfp4_fwd(x.cuda(), codes.cuda(), scales.cuda(), sizes.cuda()).cpu()
    nan = torch.isnan(out)
    want = torch.zeros_like(nan)
    want[3] = want[20] = True
    want[15:, 5] = True
    assert torch.equal(nan, want) and bool(torch.isfinite(out[~want]).all())


def test_product_repairs_sizes():
    import fp8_moe_grouped_amd as G
    x = activations(20, 256, 1)
    code, byte = weights(3, 256, 256, 2)
    codes, scales = P.pack_weights(code, byte)
    for sizes, fixed, flags in (([-4, 8, 30], [0, 8, 12], G.DEV_NEGATIVE_SIZE | G.DEV_SUM_CLAMPED), ([0, 0, 0], [0, 0, 0], 0),
                                ([3, 2, 1], [3, 2, 1], 0)):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((20, 256), 7.0, dtype=torch.bfloat16, device="cuda")
        G.gmm_mxfp4_fwd(x.cuda(), codes.cuda(), scales.cuda(), torch.tensor(sizes, dtype=torch.int32).cuda(), out=out,
                        dev_status=st)
        n = sum(fixed)
        assert int(st) == flags and bool((out[n:] == 7.0).all())
        if n:
            check(out[:n], *product(x, code, byte, fixed, torch.arange(20)), 256, False)


def test_product_agrees_with_values():
    """gmm_bf16_fwd on the dequantized weights and activations gives the same product."""
    import fp8_moe_grouped_amd as G
    M, K, N, G_ = 500, 1024, 512, 4
    x = activations(M, K, 1)
    w = (0.02 * torch.randn((G_, K, N), generator=torch.Generator().manual_seed(2))).to(torch.bfloat16)
    sizes = sizes_of(M, G_, 3).cuda()
    codes, scales = G.quantize_mxfp4_weights(w.cuda())
    got = G.gmm_mxfp4_fwd(x.cuda(), codes, scales, sizes).float()
    xv = P.mxfp4_values(*P.mxfp4(x)).to(torch.bfloat16).cuda()
    wv = G.dequantize_mxfp4(codes, scales).transpose(1, 2).contiguous()
    ref = G.gmm_bf16_fwd(xv, wv, sizes).float()
    assert float((got - ref).norm() / ref.norm()) < 2.0 ** -8


def test_product_graph_and_stream():
    import fp8_moe_grouped_amd as G
    M, K, N, G_ = 96, 768, 512, 5
    code, byte = weights(G_, N, K, 2)
    codes, scales = (t.cuda() for t in P.pack_weights(code, byte))
    xs = [activations(M, K, s).cuda() for s in range(3)]
    sz = [sizes_of(M, G_, s).cuda() for s in range(3)]
    eager = [G.gmm_silu_mxfp4(x, codes, scales, s) for x, s in zip(xs, sz)]
    x, s = xs[0].clone(), sz[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = G.gmm_silu_mxfp4(x, codes, scales, s)
    for i in (0, 1, 2, 1):
        x.copy_(xs[i])
        s.copy_(sz[i])
        graph.replay()
        G.gmm_silu_mxfp4(xs[(i + 1) % 3], codes, scales, sz[0])
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = G.gmm_silu_mxfp4(xs[2], codes, scales, sz[2])
    side.synchronize()
    assert torch.equal(out, eager[2])


def test_refusals():
    import fp8_moe_grouped_amd as G
    w = torch.zeros((2, 256, 256), dtype=torch.bfloat16, device="cuda")
    codes, scales = G.quantize_mxfp4_weights(w)
    x = torch.zeros((8, 256), dtype=torch.bfloat16, device="cuda")
    sizes = torch.tensor([4, 4], dtype=torch.int32, device="cuda")
    for call in (lambda: G.quantize_mxfp4_weights(w[:, :, :128]), lambda: G.dequantize_mxfp4(codes, scales[:1]),
                 lambda: G.gmm_mxfp4_fwd(x[:, :128].contiguous(), codes, scales, sizes),
                 lambda: G.gmm_mxfp4_fwd(x, codes, scales, sizes[:1]),
                 lambda: G.gmm_mxfp4_fwd(x, codes, scales, sizes, out=x[:4]),
                 lambda: G.gmm_mxfp4_fwd(x, codes, scales, sizes, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        G.quantize_mxfp4_weights(w.float())
    with pytest.raises(TypeError):
        G.gmm_mxfp4_fwd(x, codes, scales, sizes, slot_of_row=sizes.long())
    with pytest.raises(G.Fp8GmmError) as e:
        G.quantize_mxfp4_weights(torch.zeros((1, 96, 128), dtype=torch.bfloat16, device="cuda"))
    assert e.value.status == G.ERR_UNSUPPORTED
    with pytest.raises(G.Fp8GmmError) as e:
        G.gmm_mxfp4_fwd(x, codes, scales, sizes, topk=0)
    assert e.value.status == G.ERR_SHAPE
    assert G.gmm_mxfp4_fwd(x[:0], codes, scales, sizes).shape == (0, 256)


# K of 1024 and more with 64 rows an expert and more: the large tiles.  Counts of 128 k: 8, 9, 10, 11, 17, 13.
LARGE = [(700, 1, 3, 1024, 256), (333, 3, 2, 1152, 512), (500, 2, 5, 1280, 768), (64, 1, 1, 1408, 1024),
         (900, 1, 4, 2176, 256), (2600, 1, 7, 1664, 2304)]


@pytest.mark.parametrize("T,k,G_,K,N", LARGE)
@pytest.mark.parametrize("swiglu", [False, True])
def test_product_large_tiles(T, k, G_, K, N, swiglu):
    test_product(T, k, G_, K, N, swiglu)


@pytest.mark.parametrize("M,K,N", [(300, 1024, 128), (700, 1152, 640), (900, 2048, 1152), (200, 640, 1152), (40, 384, 1152)])
def test_product_columns_off_the_tile(M, K, N):
    """N a multiple of 128 that ends inside a tile of 256 columns, in each kind of kernel."""
    import fp8_moe_grouped_amd as G
    x = activations(M, K, 3)
    code, byte = weights(3, N, K, 4)
    codes, scales = P.pack_weights(code, byte)
    sizes = sizes_of(M, 3, 7)
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    G.gmm_mxfp4_fwd(x.cuda(), codes.cuda(), scales.cuda(), sizes.cuda(), out=out)
    check(out, *product(x, code, byte, sizes.tolist(), torch.arange(M)), K, False)


@pytest.mark.parametrize("rows", [[1], [5, 3], [0, 40, 0, 24], [64, 1, 63, 65, 128, 0, 2], [257, 255, 256, 1]])
@pytest.mark.parametrize("K", [256, 1024])
def test_product_row_counts(rows, K):
    """Experts whose rows end at, before and past a tile's edge; more experts than a wave has lanes."""
    import fp8_moe_grouped_amd as G
    N, M = 256, sum(rows)
    for lead in (0, 70):                             # experts without rows before the others
        sizes = [0] * lead + rows
        x = activations(M, K, K)
        code, byte = weights(len(rows), N, K, 2)
        codes, scales = P.pack_weights(code, byte)
        codes = torch.cat((codes[:1].expand(lead, -1, -1), codes)).contiguous()
        scales = torch.cat((scales[:1].expand(lead, -1, -1, -1), scales)).contiguous()
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = G.gmm_mxfp4_fwd(x.cuda(), codes.cuda(), scales.cuda(), torch.tensor(sizes, dtype=torch.int32).cuda(),
                              dev_status=st)
        check(out, *product(x, code, byte, rows, torch.arange(M)), K, False)
        assert int(st) == 0


def test_product_tokens_past_four_gigabytes():
    """Quantized rows of 4 GiB and more: tokens at both ends of them."""
    import fp8_moe_grouped_amd as G
    T, K, N, M = 524_300, 16384, 128, 64
    at = torch.cat((torch.arange(32), T - 32 + torch.arange(32)))
    few = activations(M, K, 1)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    x[at.cuda()] = few.cuda()
    code, byte = weights(1, N, K, 2)
    codes, scales = P.pack_weights(code, byte)
    out = G.gmm_mxfp4_fwd(x, codes.cuda(), scales.cuda(), torch.tensor([M], dtype=torch.int32).cuda(),
                          slot_of_row=at.int().cuda())
    del x
    check(out, *product(few, code, byte, [M], torch.arange(M)), K, False)


# enough tiles of 256 x 256 for the kernel that has them; counts of 128 k: 8, 9, 10, 17, 11, 8
MANY_TILES = [(300, 1, 3, 1024, 15360), (130, 2, 3, 1152, 10240), (500, 2, 5, 1280, 7168), (577, 1, 9, 2176, 6144),
              (900, 1, 1, 1408, 8192), (4700, 1, 70, 1024, 1024)]


@pytest.mark.parametrize("T,k,G_,K,N", MANY_TILES)
@pytest.mark.parametrize("swiglu", [False, True])
def test_product_many_tiles(T, k, G_, K, N, swiglu):
    test_product(T, k, G_, K, N, swiglu)


@pytest.mark.parametrize("rows,N", [([257, 255, 256, 1], 10240), ([64, 1, 63, 65, 300, 0, 200], 10240), ([900], 8320),
                                    ([130, 700, 70], 8320), ([512, 0, 513, 100], 7296)])
def test_product_many_tiles_ragged(rows, N):
    """Rows and columns that end inside the large tiles."""
    import fp8_moe_grouped_amd as G
    K, M = 1152, sum(rows)
    x = activations(M, K, N)
    code, byte = weights(len(rows), N, K, 2)
    codes, scales = P.pack_weights(code, byte)
    out = G.gmm_mxfp4_fwd(x.cuda(), codes.cuda(), scales.cuda(), torch.tensor(rows, dtype=torch.int32).cuda())
    check(out, *product(x, code, byte, rows, torch.arange(M)), K, False)


@pytest.mark.parametrize("M,G_,K,N", [(1500, 3, 2048, 1280), (600, 4, 1152, 1792), (2300, 5, 640, 1536), (700, 20, 512, 384)])
def test_product_between(M, G_, K, N):
    """Sizes at which tiles of 32, 64 and 128 rows are taken."""
    test_product(M, 1, G_, K, N, False)
    test_product(M, 1, G_, K, N, N % 256 == 0)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("lead,M", [(0, 6_000_001), (3, 2 ** 24 - 1)])
def test_product_millions_of_rows_an_expert(lead, M, swiglu):
    """One expert's rows in the large tiles up to the most that a call takes.  Tokens are few: a token's first row
    against the definition, its other rows against that one (the same sums wherever a row stands)."""
    import fp8_moe_grouped_amd as G
    T, K, N = 61, 1024, 256
    g = torch.Generator().manual_seed(M)
    x = activations(T, K, 1)
    code, byte = weights(1 + lead, N, K, 2)
    codes, scales = P.pack_weights(code, byte)
    token = torch.randint(0, T, (M,), generator=g, dtype=torch.int32)
    token[:lead + T] = torch.arange(lead + T, dtype=torch.int32) % T
    sizes = [1] * lead + [M - lead]
    f = G.gmm_silu_mxfp4 if swiglu else G.gmm_mxfp4_fwd
    out = f(x.cuda(), codes.cuda(), scales.cuda(), torch.tensor(sizes, dtype=torch.int32).cuda(), slot_of_row=token.cuda())
    check(out[:lead + T], *product(x, code, byte, [1] * lead + [T], token[:lead + T].long()), K, swiglu)
    first = torch.empty((T, out.shape[1]), dtype=out.dtype, device="cuda")
    first[token[lead:lead + T].cuda().long()] = out[lead:lead + T]
    for at in range(lead, M, 1 << 21):
        rows = slice(at, min(at + (1 << 21), M))
        assert torch.equal(out[rows], first[token[rows].cuda().long()]), at


@pytest.mark.parametrize("M,valid,G_,K,N", [(100, 60, 3, 384, 256), (7, 0, 2, 128, 128), (5000, 3001, 70, 1024, 512), (40, 40, 4, 256, 128)])
def test_product_leaves_stale_rows_alone(M, valid, G_, K, N):
    """Without a map the rows past the valid prefix are neither quantized into the workspace nor in the result."""
    import fp8_moe_grouped_amd as G
    x = activations(M, K, 1)
    x[valid:] = math.nan
    code, byte = weights(G_, N, K, 2)
    codes, scales = P.pack_weights(code, byte)
    sizes = sizes_of(valid, G_, 5)
    ws = torch.full((G.workspace_bytes(G.OP_MXFP4, M, K, N, G_),), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    G.gmm_mxfp4_fwd(x.cuda(), codes.cuda(), scales.cuda(), sizes.cuda(), out=out, workspace=ws)
    assert bool((out[valid:] == 7.0).all())
    held = ws[:M * K // 2].view(M, K // 2)           # the rows' codes come first
    assert bool((held[valid:] == 0xA5).all())
    if valid:
        check(out[:valid], *product(x, code, byte, sizes.tolist(), torch.arange(M)), K, False)


# 120 large tiles and more, at the K, row counts and odd numbers of experts where few columns give the stream kernel
# the work; tests/test_mxfp4_plan.py holds these shapes to the kernel that they are meant for
LARGE_TILES = [(700, 1, 3, 1024, 7680), (333, 3, 2, 1152, 8192), (500, 2, 5, 1280, 5120), (64, 1, 1, 1408, 30976),
               (900, 1, 4, 2176, 6144), (2600, 1, 7, 1664, 2304)]
BETWEEN = [(3092, 5, 640, 1536), (1144, 5, 512, 3328), (697, 4, 512, 1792), (70, 4, 256, 512)]


@pytest.mark.parametrize("T,k,G_,K,N", LARGE_TILES)
@pytest.mark.parametrize("swiglu", [False, True])
def test_product_in_large_tiles(T, k, G_, K, N, swiglu):
    test_product(T, k, G_, K, N, swiglu)


@pytest.mark.parametrize("M,G_,K,N", BETWEEN)
@pytest.mark.parametrize("swiglu", [False, True])
def test_product_in_tiles_of_32_to_128_rows(M, G_, K, N, swiglu):
    test_product(M, 1, G_, K, N, swiglu)


@pytest.mark.parametrize("M,K,N", [(300, 1024, 15488), (700, 1152, 7552), (900, 2048, 7808)])
def test_large_tiles_with_columns_off_the_tile(M, K, N):
    test_product_columns_off_the_tile(M, K, N)


@pytest.mark.parametrize("T", [524_286, 524_287, 524_300])
def test_product_at_four_gigabytes_of_tokens(T):
    """Enough columns for the large tiles: quantized tokens just below 4 GiB go through them, from there on the stream
    kernel takes over.  Tokens at both ends, the last ones and none; 242 copies of 128 columns."""
    import fp8_moe_grouped_amd as G
    K, N, M = 16384, 30976, 64
    at = torch.cat((torch.arange(30), torch.tensor([-1, T]), T - 32 + torch.arange(32)))
    few = activations(M, K, 1)
    few[30:32] = 0                                   # the slots without a token
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    named = (at >= 0) & (at < T)
    x[at[named].cuda()] = few[named].cuda()
    code, byte = weights(1, 128, K, 2)
    codes, scales = P.pack_weights(code, byte)
    out = G.gmm_mxfp4_fwd(x, codes.repeat(1, N // 128, 1).cuda(), scales.repeat(1, 1, N // 128, 1).cuda(),
                          torch.tensor([M], dtype=torch.int32).cuda(), slot_of_row=at.int().cuda())
    del x
    y, mag = product(few, code, byte, [M], torch.arange(M))
    check(out, y.repeat(1, N // 128), mag.repeat(1, N // 128), K, False)


def test_product_of_zero_codes_by_nan_scales():
    """A scale byte of 255 makes values of zero codes NaN too, of weights and of activations; in each kernel."""
    import fp8_moe_grouped_amd as G
    for M, K, N in ((20, 256, 256), (300, 1024, 15360)):
        code, byte = torch.zeros((1, N, K), dtype=torch.uint8), torch.full((1, N, K // 32), 120, dtype=torch.uint8)
        byte[0, 7, K // 32 - 1] = 255
        codes, scales = P.pack_weights(code, byte)
        x = torch.zeros((M, K), dtype=torch.bfloat16)
        x[11, 33] = math.inf
        out = G.gmm_mxfp4_fwd(x.cuda(), codes.cuda(), scales.cuda(), torch.tensor([M], dtype=torch.int32).cuda()).cpu()
        want = torch.zeros((M, N), dtype=torch.bool)
        want[11], want[:, 7] = True, True
        assert torch.equal(torch.isnan(out), want) and bool((out[~want] == 0).all())
