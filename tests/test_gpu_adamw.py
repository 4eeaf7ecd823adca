"""GPU tests of the AdamW step against the plain 64-bit definition, with bounds
counted from the f32 arithmetic: states in 32 bits, and in 8 bits where a code
may only be the other neighbour if the rounding's draw is that close."""
import math

import pytest
import torch

from tests import plain_train as P

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def tensors(sizes, dtype, seed, scale):
    """Tensors of any size whose storage goes on behind them, to see what is written there."""
    g = torch.Generator().manual_seed(seed)
    flats, views = [], []
    for n in sizes:
        flat = (scale * torch.randn(n + 64, generator=g)).to(dtype)
        flats.append(flat.cuda())
        views.append(flats[-1][:n])
    return flats, views


def half_step(t, want):
    return want.abs() * 2.0 ** -8 + 2.0 ** -133 if t.dtype == BF16 else 0.0


def near(got, want, tol):
    got = got.detach().cpu().double().reshape(-1)
    assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() - tol).max())


SIZES = [[1], [3, 4, 5], [255, 256, 257], [4095, 4096, 4097, 0, 1], [16385, 7, 1023], [100003], list(range(60))]


@pytest.mark.parametrize("pd,gd", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("sizes", SIZES, ids=[str(s[0]) + "x" + str(len(s)) for s in SIZES])
def test_adamw(sizes, pd, gd):
    import fp8_moe_grouped_amd as G
    (pf, p), (gf, g), (mf, m), (vf, v) = (tensors(sizes, d, i, s) for i, (d, s) in
                                          enumerate(((pd, 0.1), (gd, 1e-2), (F32, 1e-3), (F32, 1e-2))))
    for t in vf:
        t.square_()
    old = [[t.cpu().double() for t in l] for l in (p, g, m, v)]
    behind = [[t[-64:].clone() for t in l] for l in (pf, gf, mf, vf)]
    scale = torch.tensor([0.37], device="cuda") if len(sizes) != 1 else None
    how = dict(lr=3e-3, betas=(0.85, 0.98), eps=1e-7, weight_decay=0.1)
    assert G.adamw_step(p, g, m, v, step=4, grad_scale=scale, **how) is None
    step = P.Step(3e-3, 4, (0.85, 0.98), 1e-7, 0.1, 1.0 if scale is None else float(scale))
    for i in range(len(sizes)):
        (wp, wm, wv), (ep, em, ev) = step(*(l[i] for l in old))
        near(p[i], wp, ep + half_step(p[i], wp))
        near(m[i], wm, em)
        near(v[i], wv, ev)
        assert torch.equal(g[i].cpu().double(), old[1][i])
    for l, kept in zip((pf, gf, mf, vf), behind):
        assert all(torch.equal(t[-64:], b) for t, b in zip(l, kept))


def held_states(sizes, seed, scale, positive):
    g = torch.Generator().manual_seed(seed)
    flats, views = [], []
    for n in sizes:
        codes = torch.randint(0, 127, (n + 64,), generator=g, dtype=torch.uint8)
        codes = codes if positive else codes | (torch.randint(0, 2, (n + 64,), generator=g, dtype=torch.uint8) << 7)
        scales = scale * torch.rand(-(-n // 256) + 8, generator=g)
        flats.append((codes.cuda(), scales.cuda()))
        views.append((flats[-1][0][:n], flats[-1][1][:-(-n // 256)]))
    return flats, views


def check_held(got, x, error, u, positive):
    """Codes and scales of x, each value `error` off."""
    codes, scales = got[0].cpu().reshape(-1), got[1].cpu().double()
    want = P.scales_of(x)
    e = torch.zeros(-(-x.numel() // 256) * 256, dtype=torch.float64)
    e[:x.numel()] = error
    assert bool(((scales - want).abs() <= e.view(-1, 256).amax(1) / 448 + want * 2 * P.U32 + 2.0 ** -149).all())
    low, high = P.held(x, scales, u, positive, error)
    value = P.e4m3(codes)
    mag = value.abs()
    assert bool(((mag == low) | (mag == high)).all())
    assert bool((low == high).double().mean() > 0.99 - 1 / x.numel())   # the bounds leave hardly a choice
    clear = x.abs() > error
    assert bool((torch.signbit(value) == torch.signbit(x))[clear & (mag > 0)].all())


@pytest.mark.parametrize("pd,gd", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("sizes", SIZES[:5] + [list(range(1, 60))], ids=lambda s: str(s[0]) + "x" + str(len(s)))
def test_adamw8(sizes, pd, gd):
    import fp8_moe_grouped_amd as G
    (pf, p), (gf, g) = tensors(sizes, pd, 0, 0.1), tensors(sizes, gd, 1, 1e-2)
    (mf, m), (rf, r) = held_states(sizes, 2, 1e-5, False), held_states(sizes, 3, 1e-5, True)
    old = [[t.cpu().double() for t in l] for l in (p, g)] + [[P.values(c.cpu(), s.cpu()) for c, s in l] for l in (m, r)]
    behind = [[t[-64:].clone() for t in l] for l in (pf, gf)] + [[(c[-64:].clone(), s[-8:].clone()) for c, s in l]
                                                                 for l in (mf, rf)]
    scale = torch.tensor([1.7], device="cuda") if len(sizes) != 1 else None
    seed = (5 << 40) + 77
    how = dict(lr=3e-3, betas=(0.85, 0.98), eps=1e-7, weight_decay=0.1)
    assert G.adamw_step_8bit(p, g, m, r, step=9, grad_scale=scale, seed=seed, **how) is None
    step = P.Step(3e-3, 9, (0.85, 0.98), 1e-7, 0.1, 1.0 if scale is None else float(scale))
    for i, n in enumerate(sizes):
        if n == 0:
            continue
        (wp, wm, wv), (ep, em, ev) = step(old[0][i], old[1][i], old[2][i], old[3][i] ** 2)
        # the old states' own products round once (m) and twice more in the square (v)
        em, ev = em + old[2][i].abs() * P.U32, ev + wv * 4 * P.U32
        near(p[i], wp, 2 * ep + half_step(p[i], wp))
        um, ur = P.noise(seed, 9, i, n)
        check_held(m[i], wm, em, um, False)
        root = torch.sqrt(wv)
        check_held(r[i], root, torch.where(root > 0, ev / (2 * root.clamp(min=1e-300)), 0.0) + root * P.U32, ur, True)
    for l, kept in zip((pf, gf), behind):
        assert all(torch.equal(t[-64:], b) for t, b in zip(l, kept))
    for l, kept in zip((mf, rf), behind[2:]):
        assert all(torch.equal(c[-64:], a) and torch.equal(s[-8:], b) for (c, s), (a, b) in zip(l, kept))


def one(n, seed=0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, generator=g).to(dtype).cuda()


def test_adamw8_rounds_by_chance():
    """The mean of many codes is the value (5 deviations), also where it lies among the smallest codes, and a
    change far below their distance is not lost."""
    import fp8_moe_grouped_amd as G
    n = 256 * 400
    for value in (0.3, 301.7, 0.0011, 0.0071):
        g = torch.full((n,), value, device="cuda")
        g[::256] = 448.0                                        # scale 1 for m' = g
        m, r = G.adamw_8bit_states([g])
        G.adamw_step_8bit([torch.zeros(n, device="cuda")], [g], m, r, lr=1e-3, step=1, betas=(0.0, 0.0), seed=3)
        for codes, scales in (m[0], r[0]):
            assert bool((scales - 1).abs().max() < 1e-6)
            x = P.e4m3(codes.cpu()).view(-1, 256)[:, 1:].reshape(-1)
            d = 2.0 ** (max(math.floor(math.log2(value)), -6) - 3)
            if codes is r[0][0] and value < d:
                assert bool((x == d).all())                     # an r above 0 is never held as 0
                continue
            f = value / d - math.floor(value / d)
            assert set(x.unique().tolist()) <= {math.floor(value / d) * d, (math.floor(value / d) + 1) * d}
            assert abs(float(x.mean()) - value) < 5 * d * (f * (1 - f) / x.numel()) ** 0.5 + 1e-6 * value


def test_adamw8_zeros_and_the_last_block():
    import fp8_moe_grouped_amd as G
    p = torch.ones(600, device="cuda")
    m, r = G.adamw_8bit_states([p])
    G.adamw_step_8bit([p], [torch.zeros_like(p)], m, r, lr=0.1, step=1, weight_decay=0.5)
    assert not m[0][0].any() and not r[0][0].any() and not m[0][1].any() and not r[0][1].any()
    assert torch.allclose(p, torch.full_like(p, 0.95), rtol=1e-6)
    g = torch.zeros_like(p)
    g[590] = 1.0                                                # in the last, shorter block alone
    G.adamw_step_8bit([p], [g], m, r, lr=0.1, step=2)
    assert m[0][1].tolist()[:2] == [0.0, 0.0] and float(m[0][1][2]) > 0 and int(m[0][0].count_nonzero()) == 1


def test_adamw8_tiny_and_huge():
    """Scales that are subnormal or vanish, and states near f32's largest: as the formulas say, no NaN."""
    import fp8_moe_grouped_amd as G
    for value in (1e-44, 1e-40, 1e-36, 1e18):
        g = torch.full((256,), value, device="cuda")
        p = torch.zeros(256, device="cuda")
        m, r = G.adamw_8bit_states([g])
        G.adamw_step_8bit([p], [g], m, r, lr=1e-3, step=1)
        for codes, scales in (m[0], r[0]):
            held = P.values(codes.cpu(), scales.cpu())
            assert bool(torch.isfinite(held).all()) and bool((held >= 0).all())
        assert bool(torch.isfinite(p).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_adamw8_nan_and_inf(bad):
    """A bad gradient spoils its parameter and its block's states, no others."""
    import fp8_moe_grouped_amd as G
    g, p = one(1000, 1), one(1000, 2)
    g[300] = bad
    m, r = G.adamw_8bit_states([p])
    G.adamw_step_8bit([p], [g], m, r, lr=1e-3, step=1)
    assert torch.isnan(p).nonzero().tolist() == [[300]]
    for codes, scales in (m[0], r[0]):
        assert torch.isnan(scales).tolist() == [False, True, False, False]
        held = P.values(codes.cpu(), scales.cpu())
        assert bool(torch.isnan(held[256:512]).all()) and bool(torch.isfinite(held[:256]).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_are_many_calls(bits):
    """More tensors than a launch takes, empty ones among them, against a call for each: the same bits.  (A tensor's
    place in the list is part of its draws: it stays at its place among empty ones.)"""
    import fp8_moe_grouped_amd as G
    sizes = [(37 * i * i) % 5000 if i % 9 else 0 for i in range(131)]
    ps, gs = [one(n, i) for i, n in enumerate(sizes)], [one(n, 1000 + i) for i, n in enumerate(sizes)]
    qs = [p.clone() for p in ps]
    empty = torch.zeros(0, device="cuda")
    if bits == 32:
        s, t = ([[torch.zeros_like(p) for p in ps] for _ in range(2)] for _ in range(2))
        for step in (1, 2):
            G.adamw_step(ps, gs, *s, lr=1e-2, step=step)
            for i in range(len(ps)):
                G.adamw_step([qs[i]], [gs[i]], [t[0][i]], [t[1][i]], lr=1e-2, step=step)
        assert all(torch.equal(a, b) for x, y in zip(s, t) for a, b in zip(x, y))
    else:
        s, t = G.adamw_8bit_states(ps), G.adamw_8bit_states(qs)
        none = G.adamw_8bit_states([empty])[0][0]
        for step in (1, 2):
            G.adamw_step_8bit(ps, gs, *s, lr=1e-2, step=step, seed=8)
            for i in range(len(ps)):
                G.adamw_step_8bit([empty] * i + [qs[i]], [empty] * i + [gs[i]], [none] * i + [t[0][i]],
                                  [none] * i + [t[1][i]], lr=1e-2, step=step, seed=8)
        assert all(torch.equal(a, b) for x, y in zip(s, t) for u, v in zip(x, y) for a, b in zip(u, v))
    assert all(torch.equal(a, b) for a, b in zip(ps, qs))


def test_seed_and_step_decide():
    import fp8_moe_grouped_amd as G
    def codes(seed, step):
        p, g = one(3000, 1), one(3000, 2)
        m, r = G.adamw_8bit_states([p])
        G.adamw_step_8bit([p], [g], m, r, lr=1e-3, step=step, seed=seed)
        return torch.cat((m[0][0], r[0][0]))
    a = codes(1, 1)
    assert torch.equal(a, codes(1, 1))
    for other in ((2, 1), (1, 2), (1 + (1 << 32), 1), ((1 << 64) - 1, 1)):
        assert 0.1 < float((codes(*other) != a).double().mean()) < 0.9, other


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_steps_in_a_graph(bits):
    """Step and learning rate on the device, counted in the graph: the same bits as eager calls with numbers to f32's
    rounding, and the same as eager calls with the device's; eager work between the replays."""
    import fp8_moe_grouped_amd as G
    n, lrs = [5000, 77], [1e-2, 5e-3, 2e-3, 1e-3, 1e-3]
    gs = [[one(k, 10 * t + k) for k in n] for t in range(5)]

    def fresh():
        ps = [one(k, k) for k in n]
        if bits == 8:
            return ps, G.adamw_8bit_states(ps)
        return ps, [[torch.zeros_like(p) for p in ps] for _ in range(2)]

    def call(ps, g, s, lr, step, scale):
        if bits == 8:
            G.adamw_step_8bit(ps, g, *s, lr=lr, step=step, seed=4, grad_scale=scale)
        else:
            G.adamw_step(ps, g, *s, lr=lr, step=step, grad_scale=scale)

    scale = torch.tensor([0.5], device="cuda")
    eager, es = fresh()
    onboard, os_ = fresh()
    for t in range(5):
        call(eager, gs[t], es, lrs[t], t + 1, scale)
        call(onboard, gs[t], os_, torch.tensor(lrs[t], device="cuda"), torch.tensor([t + 1], device="cuda"), scale)
    ps, s = fresh()
    g = [torch.zeros(k, device="cuda") for k in n]
    lr, step = torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        call(ps, g, s, lr, step, scale)
    for t in range(5):
        for a, b in zip(g, gs[t]):
            a.copy_(b)
        lr.fill_(lrs[t])
        graph.replay()
        one(1000, t).sum()
        torch.cuda.synchronize()
    assert int(step) == 5
    for a, b, c in zip(ps, onboard, eager):
        assert torch.equal(a, b)
        if bits == 32:
            # 5 steps, each at most lr * 2 far; their rounding on the host and on the device differ by few U32
            assert float((a - c).abs().max()) < 5 * 64 * P.U32 * (1 + float(c.abs().max()))


def test_step_on_the_device_counts_from_one():
    import fp8_moe_grouped_amd as G
    results = []
    for step in (torch.tensor(1, device="cuda"), torch.tensor(0, device="cuda"), torch.tensor(-9, device="cuda")):
        p, g = one(100, 1), one(100, 2)
        G.adamw_step([p], [g], [torch.zeros_like(p)], [torch.zeros_like(p)], lr=1e-2, step=step)
        results.append(p)
    assert torch.equal(results[0], results[1]) and torch.equal(results[0], results[2])


def test_adamw_far_steps():
    """Bias corrections at large steps, on the host and on the device."""
    import fp8_moe_grouped_amd as G
    for t in (1, 2, 10, 1000, 10 ** 6, (1 << 40) + 3):
        for where in (t, torch.tensor(t, device="cuda")):
            p, g, m, v = one(500, 1), one(500, 2), one(500, 3), one(500, 4).square()
            old = [x.cpu().double() for x in (p, g, m, v)]
            G.adamw_step([p], [g], [m], [v], lr=1e-2, step=where, betas=(0.9, 0.9999))
            (wp, _, _), (ep, _, _) = P.Step(1e-2, t, (0.9, 0.9999))(*old)
            near(p, wp, ep)


def test_adamw_extremes():
    """No rates at all, gradients that are zero or enormous, eps 0 with v above 0."""
    import fp8_moe_grouped_amd as G
    p = one(300, 1)
    kept = p.clone()
    g = torch.zeros_like(p)
    m, v = torch.zeros_like(p), torch.zeros_like(p)
    G.adamw_step([p], [g], [m], [v], lr=0.0, step=1)
    assert torch.equal(p, kept)
    G.adamw_step([p], [g], [m], [v], lr=1.0, step=1, weight_decay=0.0)
    assert torch.equal(p, kept)
    g.fill_(1e30)                                               # v overflows: no step, no NaN
    G.adamw_step([p], [g], [m], [v], lr=1.0, step=1, weight_decay=0.0)
    assert torch.equal(p, kept) and bool(torch.isinf(v).all())
    p, g = torch.ones(8, device="cuda"), torch.full((8,), -2.0, device="cuda")
    G.adamw_step([p], [g], [torch.zeros_like(p)], [torch.zeros_like(p)], lr=0.1, step=1, eps=0.0, weight_decay=0.0)
    assert torch.allclose(p, torch.full_like(p, 1.1), rtol=1e-6)


def test_adamw_shapes_streams_and_leaves():
    """Any shape; parameters that require gradients; a side stream."""
    import fp8_moe_grouped_amd as G
    p = torch.nn.Parameter(one(24, 1).view(2, 3, 4))
    q = p.detach().clone().view(-1)
    s = torch.tensor(2.0, device="cuda")                        # a scalar parameter
    g = one(24, 2)
    zeros = lambda t: torch.zeros_like(t.detach())
    G.adamw_step((p, s), [g.view(2, 3, 4), s.clone()], [zeros(p), zeros(s)], [zeros(p), zeros(s)], lr=0.1, step=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        G.adamw_step([q], [g], [zeros(q)], [zeros(q)], lr=0.1, step=1)
    side.synchronize()
    assert torch.equal(p.detach().view(-1), q) and abs(float(s) - (2.0 - 0.002 - 0.1)) < 1e-5


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pd,gd", [(F32, F32), (BF16, BF16)])
def test_adamw_pieces_of_one_buffer(bits, pd, gd):
    """Tensors that begin at any element of a larger buffer: the bits of tensors of their own, and nothing beside them."""
    import fp8_moe_grouped_amd as G
    step = G.adamw_step_8bit if bits == 8 else G.adamw_step
    sizes = [1, 1000, 257, 4099, 513, 0, 2048, 3, 77]
    _, p = tensors(sizes, pd, 1, 0.1)
    _, g = tensors(sizes, gd, 2, 1e-2)
    if bits == 8:
        m, r = G.adamw_8bit_states(p)
    else:
        m, r = [torch.zeros(n, device="cuda") for n in sizes], [torch.zeros(n, device="cuda") for n in sizes]

    def pieces(l, at, gap):
        flat = torch.full((at + sum(t.numel() + gap for t in l),), 3, dtype=l[0].dtype, device="cuda")
        out = []
        for t in l:
            out.append(flat[at:at + t.numel()])
            out[-1].copy_(t)
            at += t.numel() + gap
        return flat, out

    flats, lists = zip(*(pieces(l, at, gap) for l, at, gap in
                         [(p, 1, 0), (g, 3, 2)] + ([([s[0] for s in x], at, 1) for x, at in ((m, 5), (r, 2))] if bits == 8
                                                   else [(m, 1, 1), (r, 2, 0)])))
    if bits == 8:
        lists = [*lists[:2], [(c, torch.zeros_like(s[1])) for c, s in zip(lists[2], m)],
                 [(c, torch.zeros_like(s[1])) for c, s in zip(lists[3], r)]]
    for t in (1, 2):
        step(p, g, m, r, lr=1e-2, step=t)
        step(*lists, lr=1e-2, step=t)
    for own, part in zip((p, g, m, r), lists):
        for a, b in zip(own, part):
            for x, y in zip(a, b) if isinstance(a, tuple) else ((a, b),):
                assert torch.equal(x, y)
    for flat, l in zip(flats, lists):
        inside = sum(int(((x[0] if isinstance(x, tuple) else x) == 3).sum()) for x in l)
        assert int((flat == 3).sum()) == flat.numel() - sum(sizes) + inside


def test_adamw_past_4_gib():
    """A tensor of bf16 past 2^32 elements: its ends and places around the 32-bit borders."""
    import fp8_moe_grouped_amd as G
    n = (1 << 32) + 5000
    p, g = (torch.zeros(n, dtype=BF16, device="cuda") for _ in range(2))
    spots = [0, 1, (1 << 31) - 1, 1 << 31, (1 << 32) - 1, 1 << 32, (1 << 32) + 257, n - 1]
    g[spots] = 1.0
    p[spots] = 2.0
    m, r = G.adamw_8bit_states([p])
    G.adamw_step_8bit([p], [g], m, r, lr=0.5, step=1, weight_decay=0.0)
    assert p[spots].tolist() == [1.5] * len(spots)
    assert int(p.count_nonzero()) == len(spots) and int(m[0][0].count_nonzero()) == len(spots)
    assert int(m[0][1].count_nonzero()) == len({s // 256 for s in spots})


@pytest.mark.parametrize("way", ["extension", "python"])
def test_adamw_refusals(way, monkeypatch):
    import fp8_moe_grouped_amd as G
    from tests.test_gpu_calls import Nothing
    if way == "python":
        monkeypatch.setattr(G, "_calls", Nothing())
    make = lambda n=100, dtype=F32: torch.ones(n, dtype=dtype, device="cuda")
    how = dict(lr=1e-3, step=1)
    p, g, m, v = make(), make(), make(), make()
    f = lambda *a, **k: G.adamw_step(*a, **{**how, **k})
    for call in (lambda: f([p], [make(99)], [m], [v]), lambda: f([p], [g], [m], []), lambda: f([p], [g.cpu()], [m], [v]),
                 lambda: f([p], [g.view(10, 10)], [m], [v]), lambda: f([make((4, 6)).t()], [make((6, 4))], [m], [v]),
                 lambda: f([p], [g], [m], [v], step=0), lambda: f([p], [g], [m], [v], lr=-1.0),
                 lambda: f([p], [g], [m], [v], lr=math.nan), lambda: f([p], [g], [m], [v], betas=(1.0, 0.9)),
                 lambda: f([p], [g], [m], [v], eps=math.inf), lambda: f([p], [g], [m], [v], step=1 << 64),
                 lambda: f([p], [g], [m], [v], grad_scale=make(2)), lambda: f([p], [g], [m], [v], lr=make(1).cpu()),
                 lambda: f([p], [g], [m], [v], step=torch.tensor([1, 2], device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: f([p], [g], [m.to(BF16)], [v]), lambda: f([p.half()], [g], [m], [v]),
                 lambda: f([p, make(5, BF16)], [g, make(5)], [m, make(5)], [v, make(5)]),
                 lambda: f([p], [g], [m], [v], lr=make(1).double()), lambda: f([p], [g], [m], [v], step=make(1)),
                 lambda: f([p], [g], [m], [v], grad_scale=0.5), lambda: f(p, [g], [m], None)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: f([p, p], [g, g], [m, make()], [v, make()]), lambda: f([p], [g], [m], [m]),
                 lambda: f([p], [p], [m], [v]), lambda: f([p[4:]], [g[4:]], [p[:96]], [v[4:]])):
        with pytest.raises(G.Fp8GmmError) as e:
            call()
        assert e.value.status == G.ERR_OVERLAP
    ms, rs = G.adamw_8bit_states([p])
    h = lambda *a, **k: G.adamw_step_8bit(*a, **{**how, **k})
    for call in (lambda: h([p], [g], ms, [(rs[0][0], make(2))]), lambda: h([p], [g], ms, [(rs[0][0][:50], rs[0][1])]),
                 lambda: h([p], [g], ms, rs, seed=-1), lambda: h([p], [g], ms, rs, seed=1 << 64)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: h([p], [g], ms, [v]), lambda: h([p], [g], ms, [(v, rs[0][1])]), lambda: h([p], [g], [m], rs)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(G.Fp8GmmError) as e:
        h([p], [g], ms, ms)
    assert e.value.status == G.ERR_OVERLAP
    torch.cuda.synchronize()
    # no refused call changed anything
    assert all(torch.equal(t, make()) for t in (p, g, m, v)) and not ms[0][0].any() and not rs[0][1].any()
    assert f([], [], [], []) is None and h([], [], [], []) is None
