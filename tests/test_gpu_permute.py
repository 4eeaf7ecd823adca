"""GPU tests of dispatch and combine: copies and codes bit for bit, sums within
f32 rounding and half a bf16 step of the plain 64-bit definition."""
import math

import pytest
import torch

from tests import plain_moe as P

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


def routed(T, k, E, seed, masked=0.0):
    """row_of_slot int32 [T, k] of random choices, some masked."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int64)
    ids = ids.masked_fill(torch.rand((T, k), generator=g) < masked, E)
    order = torch.sort(ids.view(-1), stable=True).indices
    rows = torch.full((T * k,), -1, dtype=torch.int32)
    n = int((ids < E).sum())
    rows[order[:n]] = torch.arange(n, dtype=torch.int32)
    return rows.view(T, k), n


def normal(shape, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16)


CASES = [(1, 1, 128, 0.0), (1, 8, 7168, 0.0), (3, 2, 128, 0.5), (37, 6, 2048, 0.1), (129, 3, 1152, 0.2),
         (16, 32, 512, 0.3), (5, 4, 16384, 0.0), (64, 5, 640, 1.0), (700, 8, 384, 0.05)]


@pytest.mark.parametrize("T,k,H,masked", CASES)
def test_permute(T, k, H, masked):
    import fp8_moe_grouped_amd as G
    rows, n = routed(T, k, 9, T + H, masked)
    x = normal((T, H), H)
    x[0, :4] = torch.tensor([math.inf, -math.inf, math.nan, -0.0])
    # exact size, a larger buffer, and one too small for the last rows: those are dropped
    for R in (T * k, T * k + 77, max(1, n - 3)):
        out = torch.full((R, H), 7.0, dtype=torch.bfloat16, device="cuda")
        G.moe_permute(x.cuda(), rows.cuda(), out=out)
        want = torch.full((R, H), 7.0, dtype=torch.bfloat16)
        for j in range(k):
            ok = (rows[:, j] >= 0) & (rows[:, j] < R)
            want[rows[ok, j].long()] = x[ok]
        assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("T,k,H,masked", CASES)
def test_permute_fp8(T, k, H, masked):
    """The same bits as quantize_rows_fp8 on the permuted rows; untouched rows stay."""
    import fp8_moe_grouped_amd as G
    rows, n = routed(T, k, 9, T + H, masked)
    x = normal((T, H), H)
    x[0, 0] = 300.0
    if T > 2:
        x[1] = 0.0
        x[2, 5] = math.inf
    codes = torch.full((T * k + 5, H), 3, dtype=torch.uint8, device="cuda")
    scales = torch.full((T * k + 5,), -1.0, device="cuda")
    G.moe_permute_fp8(x.cuda(), rows.cuda(), codes=codes, scales=scales)
    xs = G.moe_permute(x.cuda(), rows.cuda())
    want_c = torch.full((T * k, H), 3, dtype=torch.uint8, device="cuda")
    want_s = torch.full((T * k,), -1.0, device="cuda")
    G.quantize_rows_fp8(xs, torch.tensor([n], dtype=torch.int32, device="cuda"), codes=want_c, scales=want_s)
    assert torch.equal(codes[:T * k], want_c) and torch.equal(scales[:T * k], want_s)
    assert bool((codes[T * k:] == 3).all()) and bool((scales[n:] == -1).all())


@pytest.mark.parametrize("T,k,H,masked", CASES)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(T, k, H, masked, weighted):
    import fp8_moe_grouped_amd as G
    rows, n = routed(T, k, 9, T + H, masked)
    y = normal((T * k, H), 3)
    y[n:] = math.nan                                 # rows no slot names
    w = torch.softmax(torch.randn((T, k), generator=torch.Generator().manual_seed(9)), 1)
    given = w.masked_fill(rows < 0, math.nan)        # a masked choice's weight is not used
    out = G.moe_combine(y.cuda(), rows.cuda(), given.cuda() if weighted else None).cpu().double()
    want, mag = P.combine(y, rows, w if weighted else None)
    tol = mag * U32 * (k + 1) + want.abs() * 2.0 ** -8 + 2.0 ** -133
    assert bool(((out - want).abs() <= tol).all())


@pytest.mark.parametrize("T,k,H,masked", CASES)
def test_combine_gradient(T, k, H, masked):
    import fp8_moe_grouped_amd as G
    rows, n = routed(T, k, 9, T + H, masked)
    y, dout = normal((T * k + 3, H), 3), normal((T, H), 4, 1e-3)
    y[n:] = math.nan
    w = torch.softmax(torch.randn((T, k), generator=torch.Generator().manual_seed(9)), 1)
    given = w.masked_fill(rows < 0, math.nan)
    dy = torch.full((T * k + 3, H), 7.0, dtype=torch.bfloat16, device="cuda")
    _, dw = G.moe_combine_bwd(dout.cuda(), y.cuda(), rows.cuda(), given.cuda(), dy=dy)
    dy, dw = dy.cpu(), dw.cpu().double()
    assert bool((dy[n:] == 7.0).all())
    for j in range(k):
        r, ok = rows[:, j].long(), rows[:, j] >= 0
        want = dout.double() * w[:, j:j + 1].double()
        # the product rounded to f32, then to bf16
        assert bool(((dy[r[ok]].double() - want[ok]).abs() <= want[ok].abs() * (2.0 ** -8 + 2 * U32) + 2.0 ** -133).all())
        terms = dout.double()[ok] * y[r[ok]].double()
        tol = terms.abs().sum(1) * U32 * (H / 64 + 16)     # one lane's chain of sums, then the lanes'
        assert bool(((dw[ok, j] - terms.sum(1)).abs() <= tol).all())
        assert bool((dw[~ok, j] == 0).all())


def test_gradients_agree_with_differences_and_each_other():
    """combine is linear: <combine(y, w), d> changes with y and w by its gradient;
    permute's gradient is combine without weights."""
    import fp8_moe_grouped_amd as G
    rows, n = routed(40, 4, 5, 1, 0.2)
    y, d = normal((160, 256), 2), normal((40, 256), 3)
    w = torch.rand((40, 4), generator=torch.Generator().manual_seed(4))
    y[n:] = 0
    dy, dw = G.moe_combine_bwd(d.cuda(), y.cuda(), rows.cuda(), w.cuda(), dy=torch.zeros_like(y).cuda())
    f = lambda y, w: float((P.combine(y, rows, w)[0] * d.double()).sum())
    step = normal((160, 256), 5)
    step[n:] = 0
    num = f((y.double() + step.double()), w) - f(y, w)
    exact = float((dy.cpu().double() * step.double()).sum())
    room = float((dy.cpu().double() * step.double()).abs().sum()) * 2.0 ** -7
    assert abs(num - exact) <= room
    sw = torch.rand((40, 4), generator=torch.Generator().manual_seed(6)).double()
    num = f(y, w.double() + sw) - f(y, w)
    terms = dw.cpu().double() * sw
    assert abs(num - float(terms.sum())) <= 1e-4 * float(terms.abs().sum())
    back = G.moe_combine(step.cuda(), rows.cuda()).cpu().double()
    xs = G.moe_permute(d.cuda(), rows.cuda(), out=torch.zeros((160, 256), dtype=torch.bfloat16, device="cuda"))
    a, b = float((xs.cpu().double() * step.double()).sum()), float((back * d.double()).sum())
    assert abs(a - b) <= 2.0 ** -8 * float((back * d.double()).abs().sum()) + 1e-3


def test_refusals():
    import fp8_moe_grouped_amd as G
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    for call in (lambda: G.moe_permute(x, rows[:3]), lambda: G.moe_permute(x, rows.t()),
                 lambda: G.moe_permute(x, rows, out=x[:, :128].contiguous()), lambda: G.moe_permute(x, rows.cpu()),
                 lambda: G.moe_combine(x, rows, torch.zeros((4, 3), device="cuda")),
                 lambda: G.moe_combine_bwd(x, x[:, :128].contiguous(), rows, torch.zeros((4, 2), device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        G.moe_permute(x.float(), rows)
    with pytest.raises(TypeError):
        G.moe_permute(x, rows.long())
    with pytest.raises(G.Fp8GmmError) as e:
        G.moe_permute(x[:, :64].contiguous(), rows)
    assert e.value.status == G.ERR_UNSUPPORTED
    assert G.moe_permute(x[:0], rows[:0]).shape == (0, 256)
    assert G.moe_combine(x[:0], rows[:0]).shape == (0, 256)


def test_rows_past_four_gigabytes():
    """Offsets into a buffer of 2.4e9 values."""
    import fp8_moe_grouped_amd as G
    R, H = 150000, 16384
    y = torch.zeros((R, H), dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([[R - 1, 0], [R - 7, 131073]], dtype=torch.int32, device="cuda")
    x = normal((2, H), 1).cuda()
    G.moe_permute(x, rows, out=y)
    assert torch.equal(y[R - 1], x[0]) and torch.equal(y[131073], x[1]) and int((y != 0).any(1).sum()) == 4
    assert torch.equal(G.moe_combine(y, rows).float(), 2 * x.float())
    dy = torch.zeros_like(y)
    G.moe_combine_bwd(x, y, rows, torch.ones((2, 2), device="cuda"), dy=dy)
    assert torch.equal(dy, y)


def test_more_threads_than_a_launch_dimension():
    """2^24 - 1 tokens in five pieces each: more than 2^32 threads.  All slots but a few are masked."""
    import fp8_moe_grouped_amd as G
    T, H, R = 2 ** 24 - 1, 2176, 8
    rows = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    at = torch.tensor([0, 1, T // 2, 13_421_772, 13_421_773, T - 3, T - 2, T - 1], device="cuda")
    rows[at, 0] = torch.arange(R, dtype=torch.int32, device="cuda")
    small = torch.randn((R, H), device="cuda").to(torch.bfloat16)
    big = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    big[at] = small
    assert torch.equal(G.moe_permute(big, rows, out=torch.empty_like(small)), small)
    big[at - 1] = 7.0
    G.moe_combine(small, rows, out=big)
    assert torch.equal(big[at], small)
    assert not bool(big[T - 5:T - 3].any()) and not bool(big[2:100].any())


def test_permuted_codes_feed_the_forward():
    """moe_permute_fp8's codes and scales in gmm_silu_fp8_q and gmm_fp8_fwd_q: the same bits as the bf16 rows through
    the calls that quantize."""
    import fp8_moe_grouped_amd as G
    T, k, E, H, N = 77, 3, 5, 384, 512
    g = torch.Generator().manual_seed(2)
    x = normal((T, H), 1).cuda()
    r = G.moe_route(torch.randn((T, E), generator=g).masked_fill(torch.rand((T, E), generator=g) < 0.5, -math.inf).cuda(), k)
    n = int(r.group_sizes.sum())
    assert 0 < n < T * k                             # some choices are masked
    codes = torch.randn((E, H, N), generator=g).clamp(-4, 4).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    scale = (0.01 + torch.rand((E, N), generator=g)).cuda()
    aq, ascale = G.moe_permute_fp8(x, r.row_of_slot)
    xs = G.moe_permute(x, r.row_of_slot)
    for from_codes, from_rows in ((G.gmm_silu_fp8_q, G.gmm_silu_fp8), (G.gmm_fp8_fwd_q, G.gmm_fp8_fwd)):
        a, b = from_codes(aq, ascale, codes, scale, r.group_sizes), from_rows(xs, codes, scale, r.group_sizes)
        assert torch.equal(a[:n], b[:n]) and bool(torch.isfinite(a[:n]).all())
