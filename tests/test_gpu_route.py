"""GPU tests of the routing calls against the plain 64-bit definition: chosen
experts, sizes and both maps exactly; weights and gradients within the f32
arithmetic's rounding, a bf16 gradient plus half a step."""
import math

import pytest
import torch

from tests import plain_moe as P

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24     # half a step of f32, relative
INF = math.inf


def logits_of(T, E, dtype, seed, coarse=False, masked=False):
    g = torch.Generator().manual_seed(seed)
    x = 3 * torch.randn((T, E), generator=g)
    if coarse:                                       # few distinct values: ties everywhere
        x = x.round()
    if masked:
        x = x.masked_fill(torch.rand((T, E), generator=g) < 0.3, -INF)
        x[::5] = -INF
        x[1::7] = torch.where(torch.rand((T, E), generator=g)[1::7] < 0.5, torch.finfo(dtype).min, x[1::7])
    return x.to(dtype)


def check_route(x, k, renorm, got):
    ids, w, sizes, rows, slots = P.route(x.cpu(), k, renorm)
    assert torch.equal(got.ids.cpu(), ids)
    assert torch.equal(got.group_sizes.cpu(), sizes)
    assert torch.equal(got.row_of_slot.cpu(), rows)
    assert torch.equal(got.slot_of_row.cpu(), slots)
    # exp: the rounded difference (up to 104 before the result vanishes) and 2 steps; sums of at most
    # 16 + 6 levels; the quotient
    tol = w * U32 * (2 * 104 + 30) + 2.0 ** -140
    g = got.weights.cpu().double()
    assert torch.equal(torch.isnan(g), torch.isnan(w))
    assert bool(((g - w).abs() <= tol)[~torch.isnan(w)].all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (2, 8, 8), (63, 65, 3), (64, 128, 6), (65, 9, 4),
                                   (130, 160, 6), (300, 64, 2), (257, 513, 10), (90, 1024, 32), (1000, 33, 32)])
@pytest.mark.parametrize("kind", ["plain", "ties", "masked"])
def test_route(T, E, k, dtype, kind):
    import fp8_moe_grouped_amd as G
    x = logits_of(T, E, dtype, T * 1000 + E, coarse=kind != "plain", masked=kind == "masked").cuda()
    for renorm in (True, False):
        check_route(x, k, renorm, G.moe_route(x, k, renormalize=renorm))


def test_route_special_values():
    import fp8_moe_grouped_amd as G
    low = torch.finfo(torch.float32).min
    x = torch.tensor([[0.0, -0.0, 0.0, -0.0, -1.0], [math.nan, 1, INF, 2, -INF], [INF, INF, 0, 0, 0],
                      [low, low, -INF, low, -INF], [-INF] * 5, [1e-40, -1e-40, 0, 2e-40, 0],
                      [-math.nan, 0, 0, 0, 0], [3e38, -3e38, 0, 1, 2]])
    for k in (1, 3, 5):
        for renorm in (True, False):
            check_route(x.cuda(), k, renorm, G.moe_route(x.cuda(), k, renormalize=renorm))


@pytest.mark.parametrize("T,E,k", [(16384, 256, 8), (40001, 12, 3), (70000, 1024, 2)])
def test_route_many_tokens(T, E, k):
    """Many blocks, and more than one chunk of tokens a block; the sort against
    torch's stable sort of the same ids."""
    import fp8_moe_grouped_amd as G
    x = logits_of(T, E, torch.bfloat16, 7, masked=E > 32)
    got = G.moe_route(x.cuda(), k)
    f = x.double()
    value, index = torch.sort(f, dim=1, descending=True, stable=True)
    ids = index[:, :k].masked_fill(value[:, :k] == -INF, -1)
    assert torch.equal(got.ids.cpu().long(), ids)
    key = torch.where(ids < 0, E, ids).view(-1)
    order = torch.sort(key, stable=True).indices
    n = int((key < E).sum())
    assert torch.equal(got.slot_of_row.cpu()[:n].long(), order[:n]) and bool((got.slot_of_row[n:] == -1).all())
    rows = torch.full((T * k,), -1)
    rows[order[:n]] = torch.arange(n)
    assert torch.equal(got.row_of_slot.cpu().view(-1).long(), rows)
    assert torch.equal(got.group_sizes.cpu().long(), torch.bincount(key, minlength=E + 1)[:E])


def test_route_empty_and_refusals():
    import fp8_moe_grouped_amd as G
    r = G.moe_route(torch.zeros((0, 8), device="cuda"), 2)
    torch.cuda.synchronize()
    assert r.group_sizes.tolist() == [0] * 8 and r.ids.shape == (0, 2) and r.slot_of_row.numel() == 0
    x = torch.zeros((4, 8), device="cuda")
    with pytest.raises(ValueError):
        G.moe_route(x, 9)
    with pytest.raises(ValueError):
        G.moe_route(x.t(), 2)
    with pytest.raises(TypeError):
        G.moe_route(x.half(), 2)
    with pytest.raises(G.Fp8GmmError) as e:
        G.moe_route(torch.zeros((4, 1025), device="cuda"), 2)
    assert e.value.status == G.ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        G.moe_route(torch.zeros((5000, 8), device="cuda"), 2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 8), (130, 160, 6), (77, 65, 5), (33, 1024, 32), (50, 300, 10)])
def test_route_gradient(T, E, k, dtype, renorm):
    import fp8_moe_grouped_amd as G
    x = logits_of(T, E, dtype, T + E, masked=True).cuda()
    r = G.moe_route(x, k, renormalize=renorm)
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(1))
    sent = dw.clone()
    sent[r.ids.cpu() < 0] = math.nan                 # what a masked choice holds is not read
    got = G.moe_route_bwd(sent.cuda(), x, r.ids, r.weights, renormalize=renorm).cpu()
    assert got.dtype == dtype
    want, mag = P.route_bwd(dw, x.cpu(), r.ids.cpu(), r.weights.cpu(), renorm)
    # p: the rounded difference, exp, a sum of 22 levels, the quotient; the inner sum's 6 levels; three products
    tol = mag * U32 * (2 * 104 + 64) + 2.0 ** -140
    if dtype == torch.bfloat16:
        tol = tol + want.abs() * 2.0 ** -8 + 2.0 ** -133
    assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [5, 64, 1024])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_of_nan_and_inf(renorm, E, dtype):
    """A NaN or +inf among a softmax's logits makes its gradients NaN; a token without experts gets zeros."""
    import fp8_moe_grouped_amd as G
    x = torch.full((6, E), -INF)
    x[0, 1] = math.nan                               # nothing but a NaN
    x[1, 3], x[1, 4] = math.nan, 1.0
    x[2, 0], x[2, 2] = INF, 1.0
    x[3, 2] = 0.5                                    # one expert; row 4: none
    x[5, :] = math.nan
    x = x.to(dtype).cuda()
    r = G.moe_route(x, 2, renormalize=renorm)
    got = G.moe_route_bwd(torch.ones((6, 2), device="cuda"), x, r.ids, r.weights, renormalize=renorm).cpu().float()
    ids = r.ids.cpu()
    for t in (0, 1, 2, 5):
        bad = torch.zeros(E, dtype=torch.bool)
        bad[ids[t][ids[t] >= 0].long()] = True
        assert torch.equal(torch.isnan(got[t]), bad if renorm else torch.ones_like(bad)), t
        assert bool((got[t][~torch.isnan(got[t])] == 0).all())
    assert bool((got[3:5] == 0).all())               # a weight of 1 does not move


def test_route_gradient_by_differences():
    import fp8_moe_grouped_amd as G
    g = torch.Generator().manual_seed(3)
    x = torch.randn((5, 12), generator=g)
    dw = torch.randn((5, 4), generator=g)
    for renorm in (True, False):
        r = G.moe_route(x.cuda(), 4, renormalize=renorm)
        d = G.moe_route_bwd(dw.cuda(), x.cuda(), r.ids, r.weights, renormalize=renorm).cpu().double()
        h = 1e-5
        for e in range(12):
            step = torch.zeros((5, 12), dtype=torch.float64)
            step[:, e] = h
            up, down = P.route(x.double() + step, 4, renorm), P.route(x.double() - step, 4, renorm)
            assert torch.equal(up[0], r.ids.cpu()) and torch.equal(down[0], r.ids.cpu())
            num = ((up[1] - down[1]) * dw.double()).sum(1) / (2 * h)
            # differences: h^2 of the third derivative (at most about 1) and 2^-53 / h; the kernel's f32
            assert bool(((num - d[:, e]).abs() <= 1e-9 + 300 * U32 * dw.abs().double().sum(1)).all())


def test_route_graph_and_stream():
    """Captured, replayed with other inputs and eager work between; and on a side stream."""
    import fp8_moe_grouped_amd as G
    T, E, k = 3000, 96, 5
    xs = [logits_of(T, E, torch.float32, s, masked=True).cuda() for s in range(4)]
    dws = [torch.randn((T, k), device="cuda") for _ in xs]
    eager = []
    for x, dw in zip(xs, dws):
        r = G.moe_route(x, k)
        eager.append(tuple(r) + (G.moe_route_bwd(dw, x, r.ids, r.weights),))
    x, dw = xs[0].clone(), dws[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = G.moe_route(x, k)
        d = G.moe_route_bwd(dw, x, r.ids, r.weights)
    for i in (0, 1, 2, 3, 1):
        x.copy_(xs[i])
        dw.copy_(dws[i])
        graph.replay()
        G.moe_route(xs[(i + 1) % 4], k)
        torch.cuda.synchronize()
        for a, b in zip(tuple(r) + (d,), eager[i]):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s = G.moe_route(xs[2], k)
    side.synchronize()
    for a, b in zip(tuple(s), eager[2]):
        assert torch.equal(a, b)


# every way a token's logits can lie in lanes: rows of 16 or the wave, 4 to 16 logits a lane, whole 16-byte
# chunks or not, and lists of 8 keys or all of a lane's
LANES = [(61, 16, 16), (61, 31, 9), (200, 64, 8), (130, 100, 12), (70, 128, 16), (129, 255, 13), (66, 256, 16),
         (40, 256, 17), (40, 60, 20), (67, 257, 8), (129, 512, 8), (30, 500, 16), (64, 384, 7), (33, 1023, 3),
         (50, 1024, 9)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", LANES)
def test_route_lanes(T, E, k, dtype):
    import fp8_moe_grouped_amd as G
    x = logits_of(T, E, dtype, T + E + k, coarse=k % 2 == 0, masked=E % 2 == 0).cuda()
    g = torch.Generator().manual_seed(k)
    for renorm in (True, False):
        r = G.moe_route(x, k, renormalize=renorm)
        check_route(x, k, renorm, r)
        dw = torch.randn((T, k), generator=g)
        got = G.moe_route_bwd(dw.cuda(), x, r.ids, r.weights, renormalize=renorm).cpu()
        want, mag = P.route_bwd(dw, x.cpu(), r.ids.cpu(), r.weights.cpu(), renorm)
        tol = mag * U32 * (2 * 104 + 64) + 2.0 ** -140       # as in test_route_gradient
        if dtype == torch.bfloat16:
            tol = tol + want.abs() * 2.0 ** -8 + 2.0 ** -133
        assert bool(((got.double() - want).abs() <= tol).all())


def test_route_one_expert_takes_every_token():
    """All tokens prefer the same experts: the longest runs of ranks within waves, blocks and the batch."""
    import fp8_moe_grouped_amd as G
    T, E, k = 9001, 256, 4
    x = torch.zeros((T, E))
    x[:, [200, 3, 77, 150]] = torch.tensor([4.0, 3.0, 2.0, 1.0])
    got = G.moe_route(x.cuda(), k)
    assert torch.equal(got.ids.cpu(), torch.tensor([[200, 3, 77, 150]], dtype=torch.int32).expand(T, k))
    sizes = torch.zeros(E, dtype=torch.int32)
    sizes[[3, 77, 150, 200]] = T
    assert torch.equal(got.group_sizes.cpu(), sizes)
    t = torch.arange(T, dtype=torch.int32)
    rows = torch.stack((3 * T + t, t, T + t, 2 * T + t), dim=1)
    assert torch.equal(got.row_of_slot.cpu(), rows)


def test_route_outputs_of_two_calls_are_apart():
    import fp8_moe_grouped_amd as G
    x = logits_of(100, 32, torch.float32, 1).cuda()
    a = G.moe_route(x, 4)
    kept = [t.clone() for t in a]
    b = G.moe_route(-x, 4)
    for t, old, new in zip(a, kept, b):
        assert torch.equal(t, old) and not torch.equal(t, new)
    assert a.weights.is_contiguous() and a.row_of_slot.is_contiguous() and a.slot_of_row.shape == (400,)


@pytest.mark.parametrize("T", [65, 32768, 32769, 98304, 98305, 140000])
def test_route_tokens_a_block(T):
    """Every size of a block's histogram: one to five chunks of tokens, counts in bytes and in 16 bits."""
    test_route_many_tokens(T, 40, 2)


@pytest.mark.parametrize("E", [5, 17, 250, 600, 1024])
def test_route_every_token_to_one_expert(E):
    """The fullest counts, in the first and the last expert, with 16-bit histograms and with bytes."""
    import fp8_moe_grouped_amd as G
    for T in (20000, 100000):
        for e in (0, E - 1):
            x = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
            x[:, e] = 1
            got = G.moe_route(x, 1)
            assert bool((got.ids == e).all()) and int(got.group_sizes[e]) == T and int(got.group_sizes.sum()) == T
            t = torch.arange(T, dtype=torch.int32, device="cuda")
            assert torch.equal(got.row_of_slot.view(-1), t) and torch.equal(got.slot_of_row, t)
