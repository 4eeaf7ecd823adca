"""GPU tests of the balance losses against the plain 64-bit definition: counts
and tokens exactly, sums and gradients within the f32 arithmetic's rounding, a
bf16 gradient plus half a step."""
import math

import pytest
import torch

from tests import plain_train as P

pytestmark = pytest.mark.gpu
U32 = P.U32
INF = math.inf


def logits_of(T, E, dtype, seed, masked=False, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    x = scale * torch.randn((T, E), generator=g)
    if masked:
        x = x.masked_fill(torch.rand((T, E), generator=g) < 0.3, -INF)
        x[::5] = -INF
        x[1::7] = torch.where(torch.rand((T, E), generator=g)[1::7] < 0.5, torch.finfo(dtype).min, x[1::7])
    return x.to(dtype)


def ids_of(T, E, k, seed):
    """Choices with repeats, masked ones and some outside the experts."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    ids[torch.rand((T, k), generator=g) < 0.1] = -1
    ids[torch.rand((T, k), generator=g) < 0.02] = E
    return ids


def check(got, x, ids=None, counts=None):
    losses, counts, probs, n = P.balance(x, ids, counts)
    relative, z = P.balance_tolerances(x, x.shape[0])
    assert torch.equal(got.counts.cpu().long(), counts.long())
    assert int(got.tokens) == n and got.tokens.shape == (1,)
    for a, want, tol in ((got.probs, probs, probs * relative + 2.0 ** -140),
                         (got.losses[0], losses[0], losses[0] * relative), (got.losses[1], losses[1], z)):
        a = a.cpu().double()
        assert torch.equal(torch.isnan(a), torch.isnan(want))
        past = want > torch.finfo(torch.float32).max            # squares of logits of the type's lowest value
        assert torch.equal(torch.isinf(a), past)
        assert bool(((a - want).abs() <= tol)[~torch.isnan(want) & ~past].all()), (a, want, tol)


def check_grad(got, d, x, counts, n, add=None):
    want, mag = P.balance_bwd(d, x, counts, n, add)
    got = got.cpu().double()
    # exp: the rounded difference (up to 104) for itself and the sum; quotient, dot product over 16 + 6 levels,
    # coefficients, products, sums.  A probability below the smallest normal number is a multiple of 2^-149.
    c = counts.double().clamp(min=0)
    factor = abs(float(d[0])) * x.shape[1] * 2 + (abs(float(d[1])) * 400)
    tol = mag * U32 * (2 * 104 + 80) + 2.0 ** -147 * (1 + factor)
    if x.dtype == torch.bfloat16:
        tol = tol + want.abs() * 2.0 ** -8 + 2.0 ** -133
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert bool(((got - want).abs() <= tol)[~torch.isnan(want)].all())
    assert c.numel() == x.shape[1]


SIZES = [(1, 1, 1), (1, 256, 8), (2, 8, 8), (63, 65, 3), (64, 128, 6), (65, 9, 4), (130, 160, 6), (300, 64, 2),
         (257, 513, 10), (90, 1024, 32), (1000, 33, 32), (129, 255, 13), (66, 500, 1), (30, 12, 2), (1100, 16, 3)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("masked", [False, True])
def test_balance(T, E, k, dtype, masked):
    import fp8_moe_grouped_amd as G
    x, ids = logits_of(T, E, dtype, T + E, masked), ids_of(T, E, k, T)
    got = G.moe_balance_loss(x.cuda(), ids.cuda())
    check(got, x, ids)
    g = torch.Generator().manual_seed(k)
    d = torch.rand(2, generator=g)
    add = torch.randn((T, E), generator=g).to(dtype) * 1e-3
    for a in (None, add):
        grad = G.moe_balance_loss_bwd(d.cuda(), x.cuda(), got.counts, got.tokens, add=None if a is None else a.cuda())
        assert grad.dtype == dtype
        check_grad(grad, d, x, got.counts.cpu(), int(got.tokens), a)


@pytest.mark.parametrize("T,E", [(4096, 40), (16384, 256), (16385, 96), (40000, 16), (70001, 512)])
def test_balance_many_tokens(T, E):
    """One token a lane row and several, the last ones past a whole block."""
    import fp8_moe_grouped_amd as G
    x = logits_of(T, E, torch.float32, E, masked=True).cuda()
    r = G.moe_route(x, 4)
    got = G.moe_balance_loss(x, r.ids)
    assert torch.equal(got.counts, r.group_sizes)
    check(got, x.cpu(), counts=r.group_sizes.cpu())
    d = torch.tensor([0.01, 0.001])
    check_grad(G.moe_balance_loss_bwd(d.cuda(), x, got.counts, got.tokens), d, x.cpu(), got.counts.cpu(),
               int(got.tokens))


@pytest.mark.parametrize("T", [5, 3000])
def test_balance_of_given_counts(T):
    """Loads of several batches, past 2^24 and with a negative one, which counts as none."""
    import fp8_moe_grouped_amd as G
    x = logits_of(T, 24, torch.float32, 3, masked=True)
    counts = torch.randint(0, 1 << 27, (24,), generator=torch.Generator().manual_seed(T), dtype=torch.int32)
    counts[5] = -7
    dev = counts.cuda()
    got = G.moe_balance_loss(x.cuda(), counts=dev)
    assert got.counts.data_ptr() == dev.data_ptr()
    check(got, x, counts=counts)
    d = torch.tensor([1.0, -0.5])
    check_grad(G.moe_balance_loss_bwd(d.cuda(), x.cuda(), dev, got.tokens), d, x, counts, int(got.tokens))


def test_balance_of_nothing():
    import fp8_moe_grouped_amd as G
    none = torch.zeros((0, 8), device="cuda")
    got = G.moe_balance_loss(none, torch.zeros((0, 2), dtype=torch.int32, device="cuda"))
    assert got.losses.tolist() == [0.0, 0.0] and got.counts.tolist() == [0] * 8 and got.tokens.tolist() == [0]
    given = torch.ones(8, dtype=torch.int32, device="cuda")
    got = G.moe_balance_loss(none, counts=given)
    assert got.losses.tolist() == [0.0, 0.0] and got.counts.tolist() == [1] * 8 and got.probs.tolist() == [0.0] * 8
    d = torch.ones(2, device="cuda")
    assert G.moe_balance_loss_bwd(d, none, given, got.tokens).shape == (0, 8)
    for T in (3, 500):                                          # padding alone; tokens without a choice
        x = torch.full((T, 8), -INF, device="cuda")
        ids = torch.full((T, 2), -1, dtype=torch.int32, device="cuda")
        got = G.moe_balance_loss(x, ids)
        assert got.losses.tolist() == [0.0, 0.0] and got.probs.tolist() == [0.0] * 8 and got.tokens.tolist() == [0]
        add = torch.randn((T, 8), device="cuda")
        assert not bool(G.moe_balance_loss_bwd(d, x, got.counts, got.tokens).any())
        assert torch.equal(G.moe_balance_loss_bwd(d, x, got.counts, got.tokens, add=add), add)
        y = torch.randn((T, 8), device="cuda")
        got = G.moe_balance_loss(y, ids)
        check(got, y.cpu(), ids.cpu())
        assert float(got.losses[0]) == 0.0
        check_grad(G.moe_balance_loss_bwd(d, y, got.counts, got.tokens), d.cpu(), y.cpu(), got.counts.cpu(), T)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [math.nan, INF])
def test_balance_nan_and_inf(bad, dtype):
    """One bad token: the losses and probabilities become NaN, other tokens' gradients do not."""
    import fp8_moe_grouped_amd as G
    for T, E, at in ((9, 20, (4, 3)), (700, 300, (650, 299)), (3, 8, (1, 0))):
        x = logits_of(T, E, dtype, 1, masked=True)
        x[at[0]] = -INF if at == (1, 0) else 1.0
        x[at] = bad
        ids = ids_of(T, E, 2, 4)
        got = G.moe_balance_loss(x.cuda(), ids.cuda())
        assert bool(torch.isnan(got.losses).all()) and bool(torch.isnan(got.probs).all())
        check(got, x, ids)
        d = torch.tensor([0.3, 0.1])
        check_grad(G.moe_balance_loss_bwd(d.cuda(), x.cuda(), got.counts, got.tokens), d, x, got.counts.cpu(),
                   int(got.tokens))


def test_balance_far_logits():
    """Logits up to the type's largest, and differences that leave one expert."""
    import fp8_moe_grouped_amd as G
    for scale in (1e3, 1e30, 1e-30):
        x = logits_of(40, 30, torch.float32, 6, scale=scale)
        ids = ids_of(40, 30, 3, 1)
        got = G.moe_balance_loss(x.cuda(), ids.cuda())
        losses, _, probs, _ = P.balance(x, ids)
        check(got, x, ids)
        assert (float(got.losses[1]) == INF) == (scale > 1e18)
        assert float((got.probs.cpu() - probs).abs().max()) < 1e-6


def test_balance_gradient_by_differences():
    """Against differences of the 64-bit losses."""
    import fp8_moe_grouped_amd as G
    x = logits_of(7, 12, torch.float32, 8, masked=False, scale=1.0)
    counts = torch.arange(12, dtype=torch.int32)
    d = torch.tensor([0.6, 0.4])
    grad = G.moe_balance_loss_bwd(d.cuda(), x.cuda(), counts.cuda(), torch.tensor([7], dtype=torch.int32).cuda()).cpu()
    h, loss = 1e-5, lambda y: float((P.balance(y, counts=counts)[0] * d.double()).sum())
    for t in range(7):
        for e in range(12):
            up, down = x.double(), x.double()
            up[t, e] += h
            down[t, e] -= h
            # h^2 / 6 of the third derivative (below 10 for these losses), 2^-53 of the losses / h; f32 arithmetic
            assert abs((loss(up) - loss(down)) / (2 * h) - float(grad[t, e])) < 1e-8 + 300 * U32


def test_balance_into_given_buffers():
    """out is add itself; a workspace of the caller's, whatever it holds, and one that is too small."""
    import fp8_moe_grouped_amd as G
    T, E = 2000, 100
    x, ids = logits_of(T, E, torch.float32, 5, True).cuda(), ids_of(T, E, 4, 5).cuda()
    want = G.moe_balance_loss(x, ids)
    need = G.workspace_bytes(G.OP_BALANCE, T, E, 4, 1, 0)
    got = G.moe_balance_loss(x, ids, workspace=torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(ValueError, match="needed"):
        G.moe_balance_loss(x, ids, workspace=torch.zeros(need - 1, dtype=torch.uint8, device="cuda"))
    d = torch.tensor([0.1, 0.2], device="cuda")
    add = torch.randn((T, E), device="cuda")
    grad = G.moe_balance_loss_bwd(d, x, got.counts, got.tokens, add=add)
    out = torch.full((T, E), 9.0, device="cuda")
    assert G.moe_balance_loss_bwd(d, x, got.counts, got.tokens, add=add, out=out) is out and torch.equal(out, grad)
    assert G.moe_balance_loss_bwd(d, x, got.counts, got.tokens, add=add, out=add) is add and torch.equal(add, grad)


def test_balance_graph_and_stream():
    """Captured, replayed with other inputs and eager work between; two graphs; and on a side stream."""
    import fp8_moe_grouped_amd as G
    T, E, k = 3000, 96, 5
    xs = [logits_of(T, E, torch.float32, s, masked=True).cuda() for s in range(4)]
    ids = [ids_of(T, E, k, s).cuda() for s in range(4)]
    d = torch.tensor([0.01, 0.02], device="cuda")

    def call(x, i):
        b = G.moe_balance_loss(x, i)
        return tuple(b) + (G.moe_balance_loss_bwd(d, x, b.counts, b.tokens),)

    eager = [call(*a) for a in zip(xs, ids)]
    x, i = xs[0].clone(), ids[0].clone()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(x, i))
        graphs.append(graph)
    for turn, n in enumerate((0, 1, 2, 3, 1)):
        x.copy_(xs[n])
        i.copy_(ids[n])
        graphs[turn % 2].replay()
        call(xs[(n + 1) % 4], ids[0])
        torch.cuda.synchronize()
        for a, b in zip(outs[turn % 2], eager[n]):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s = call(xs[2], ids[2])
    side.synchronize()
    for a, b in zip(s, eager[2]):
        assert torch.equal(a, b)


def test_balance_refusals():
    import fp8_moe_grouped_amd as G
    x, ids = torch.zeros((4, 8), device="cuda"), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    counts, tokens, d = ids.view(-1), ids[:1, 0].contiguous(), torch.zeros(2, device="cuda")
    for call in (lambda: G.moe_balance_loss(x), lambda: G.moe_balance_loss(x, ids, counts=counts),
                 lambda: G.moe_balance_loss(x, ids[:3]), lambda: G.moe_balance_loss(x, counts=counts[:7]),
                 lambda: G.moe_balance_loss(x.t(), ids), lambda: G.moe_balance_loss(x, ids.cpu()),
                 lambda: G.moe_balance_loss(x, ids, workspace=torch.zeros(9, dtype=torch.uint8)),
                 lambda: G.moe_balance_loss_bwd(d[:1], x, counts, tokens),
                 lambda: G.moe_balance_loss_bwd(d, x, counts[:7], tokens),
                 lambda: G.moe_balance_loss_bwd(d, x, counts, counts),
                 lambda: G.moe_balance_loss_bwd(d, x, counts, tokens, add=x[:3]),
                 lambda: G.moe_balance_loss_bwd(d, x, counts, tokens, out=x[:3]),
                 lambda: G.moe_balance_loss_bwd(d.cpu(), x, counts, tokens)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: G.moe_balance_loss(x.double(), ids), lambda: G.moe_balance_loss(x, ids.long()),
                 lambda: G.moe_balance_loss_bwd(d, x, counts.long(), tokens),
                 lambda: G.moe_balance_loss_bwd(d, x, counts, tokens, add=x.to(torch.bfloat16))):
        with pytest.raises(TypeError):
            call()
    for bad in (torch.zeros((2, 1025), device="cuda"), torch.zeros((2, 0), device="cuda")):
        with pytest.raises(G.Fp8GmmError):
            G.moe_balance_loss(bad, ids[:2])
    with pytest.raises(G.Fp8GmmError):
        G.moe_balance_loss(x, torch.zeros((4, 33), dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
