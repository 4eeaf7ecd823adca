"""GPU tests of AdamW bit for bit: states against the same f32 operations done
one by one on the CPU, numbers on the device against numbers of the host; and
8-bit states over many steps against unrounded ones."""
import decimal
import math

import pytest
import torch

from tests import plain_train as P

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def f32(v):
    return torch.tensor(v, dtype=torch.float64).to(F32)


def moments(m, v, g, betas, scale=None):
    """m' and v' of f32 tensors on the CPU, each product and sum rounded by itself."""
    b1, c1, b2, c2 = (f32(c) for c in (betas[0], 1 - betas[0], betas[1], 1 - betas[1]))
    g = g.to(F32) if scale is None else g.to(F32) * scale
    return b1 * m + c1 * g, b2 * v + c2 * g * g


def root(x):
    """sqrt in f32, correctly rounded: 64 bits are more than twice f32's and two (the CPU's own in f32 need not be)."""
    return torch.sqrt(x.double()).to(F32)


def spread(n, seed, low=-20, high=4):
    """Numbers of all mantissas over many powers of two."""
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, generator=g) * torch.exp2(torch.randint(low, high, (n,), generator=g).float())


@pytest.mark.parametrize("gd", [F32, BF16])
@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.85, 0.98), (0.0, 0.5)])
@pytest.mark.parametrize("scaled", [False, True])
def test_states_in_32_bits(gd, betas, scaled):
    import fp8_moe_grouped_amd as G
    n = (1 << 20) + 3                                            # lanes of whole chunks, and a tail
    m, v, g = spread(n, 1), spread(n, 2).square(), spread(n, 3).to(gd)
    scale = torch.tensor(0.37) if scaled else None
    dm, dv, p = m.cuda(), v.cuda(), torch.zeros(n, device="cuda")
    G.adamw_step([p], [g.cuda()], [dm], [dv], lr=1e-3, step=5, betas=betas,
                 grad_scale=None if scale is None else scale.cuda())
    wm, wv = moments(m, v, g, betas, scale)
    assert torch.equal(dm.cpu(), wm) and torch.equal(dv.cpu(), wv)


@pytest.mark.parametrize("gd", [F32, BF16])
@pytest.mark.parametrize("n", [256 * 300, 256 * 40 + 77])
def test_states_in_8_bits(n, gd):
    """Scales, and the codes of all values past the smallest normal one: 1/448, the quotient's reciprocal, its product and
    the roots are f32 operations that round once each, the draw's sum is exact."""
    import fp8_moe_grouped_amd as G
    g = torch.Generator().manual_seed(n)
    blocks = -(-n // 256)
    codes = [torch.randint(0, 127, (n,), generator=g, dtype=torch.uint8) for _ in "mr"]
    codes[0] |= torch.randint(0, 2, (n,), generator=g, dtype=torch.uint8) << 7
    scales = [1e-5 * torch.rand(blocks, generator=g) for _ in "mr"]
    grad = (1e-2 * torch.randn(n, generator=g)).to(gd)
    betas, seed, step = (0.9, 0.999), 12345678901, 17
    m, r = ([(c.clone().cuda(), s.clone().cuda())] for c, s in zip(codes, scales))
    G.adamw_step_8bit([torch.zeros(n, device="cuda")], [grad.cuda()], m, r, lr=1e-3, step=step, betas=betas, seed=seed)
    old = [P.e4m3(c).to(F32) * s.repeat_interleave(256)[:n] for c, s in zip(codes, scales)]
    b1, c1, b2, c2 = (f32(c) for c in (betas[0], 1 - betas[0], betas[1], 1 - betas[1]))
    x = grad.to(F32)
    new = b1 * old[0] + c1 * x, root(b2 * old[1] * old[1] + c2 * x * x)
    for (dc, ds), w, u in zip((m[0], r[0]), new, P.noise(seed, step, 0, n)):
        pad = torch.zeros(blocks * 256)
        pad[:n] = w.abs()
        scale = pad.view(-1, 256).amax(1) * f32(1 / 448)
        assert torch.equal(ds.cpu(), scale)
        q = (w * (1 / scale).repeat_interleave(256)[:n]).double().abs()
        d = torch.exp2(torch.floor(torch.log2(q.clamp(min=2.0 ** -6))) - 3)
        want = torch.copysign((torch.floor(q / d + u) * d).clamp(max=448), w.double())
        normal = q >= 2.0 ** -6
        assert float(normal.double().mean()) > 0.9
        assert torch.equal(P.e4m3(dc.cpu())[normal], want[normal])


@pytest.mark.parametrize("low", [0, 1, -1, -47, -48, -49, -70, 50])
def test_roots(low):
    """A block with one root says it in its scale, root * f32(1/448), whose bits part for roots below 1.75 of a power of
    two (the product's steps are then no coarser) and mostly above.  r = s for 2^20 blocks' scales s of every 8th mantissa in
    [2^low, 2^(low + 1)), v' = b2 r^2 of the powers 2 low - 1 to 2 low + 1: both parities, and both sides of the 2^-96 past
    which the root is another one; at 2^-140 v' is subnormal, at 2^100 large."""
    import fp8_moe_grouped_amd as G
    blocks, beta2 = 1 << 20, 0.499
    bits = (127 + low << 23) + 8 * torch.arange(blocks, dtype=torch.int32) + 5
    s = bits.view(F32)
    n = 256 * blocks
    codes = torch.zeros(n, dtype=torch.uint8, device="cuda")
    place = torch.arange(blocks, device="cuda") * 256 + torch.arange(blocks, device="cuda") % 256
    codes[place] = 0x38                                          # 1
    r = [(codes, s.cuda())]
    m = [(torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(blocks, device="cuda"))]
    p, g = (torch.zeros(n, dtype=BF16, device="cuda") for _ in "pg")
    G.adamw_step_8bit([p], [g], m, r, lr=1e-3, step=3, betas=(0.9, beta2))
    want = root(f32(beta2) * s * s) * f32(1 / 448)
    assert torch.equal(r[0][1].cpu(), want)
    largest = codes[place]                                       # 448, or what a rounding up or down leaves of it
    assert bool((largest == 0x7E).all()) or low < -60
    assert int(codes.count_nonzero()) == int((want > 0).sum()) and not p.any()


# --------------------------------------------------------------------------- coefficients

def exact_coefficients(lr, betas, t):
    """lr / (1 - beta1^t) and 1 / sqrt(1 - beta2^t) with 60 digits."""
    with decimal.localcontext() as c:
        c.prec = 60
        c.Emin, c.Emax = -10 ** 15, 10 ** 15
        one, (b1, b2) = decimal.Decimal(1), (decimal.Decimal(b) for b in betas)
        return decimal.Decimal(lr) / (one - b1 ** t), one / (one - b2 ** t).sqrt()


def from_a_tie(x):
    """How far x is from the nearest number between two neighbours in f32, relative to x."""
    mantissa = decimal.Decimal(2) ** 24 * x / decimal.Decimal(2) ** (math.frexp(float(x))[1])
    return float(abs(mantissa % 1 - decimal.Decimal("0.5"))) / 2 ** 24


LR = float(f32(1e-3))
STEPS = [*range(1, 30), 100, 999, 1000, 1001, 12345, 10 ** 5, 10 ** 6 + 1, (1 << 31) + 7]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.95, 0.98), (0.0, 0.9999)])
def test_numbers_on_the_device_are_the_hosts(betas, bits):
    """The coefficients are rounded once, from 64 bits, wherever they are computed: the same bits of p and of the states.
    Two ways in 64 bits differ by a few 2^-53 of beta^t, 2^-53 / (1 - beta) of the difference (2^-39 here): no exact
    coefficient of these steps is that close to a tie."""
    import fp8_moe_grouped_amd as G
    n = 3000
    g = torch.Generator().manual_seed(1)
    p0, g0, m0 = (torch.randn(n, generator=g).cuda() for _ in range(3))
    v0 = torch.randn(n, generator=g).square().cuda()
    step = G.adamw_step_8bit if bits == 8 else G.adamw_step
    for t in STEPS:
        for x in exact_coefficients(LR, betas, t):
            assert from_a_tie(x) > 2.0 ** -36
        ends = []
        for lr, at in ((LR, t), (torch.tensor(LR, device="cuda"), torch.tensor(t, device="cuda")),
                       (LR, torch.tensor([t], device="cuda")), (torch.tensor([LR], device="cuda"), t)):
            p, gs = p0.clone(), g0.clone()
            if bits == 8:
                m, v = G.adamw_8bit_states([p])
                m[0][0].fill_(0x38), m[0][1].copy_(m0[:m[0][1].numel()].abs())
                v[0][0].fill_(0x30), v[0][1].copy_(v0[:v[0][1].numel()])
            else:
                m, v = [m0.clone()], [v0.clone()]
            step([p], [gs], m, v, lr=lr, step=at, betas=betas, weight_decay=0.03)
            ends.append([p] + [y for s in (*m, *v) for y in (s if bits == 8 else [s])])
        for other in ends[1:]:
            assert all(torch.equal(a, b) for a, b in zip(ends[0], other)), t


# --------------------------------------------------------------------------- many steps

def test_second_moment_in_8_bits_over_many_steps():
    """sqrt(v) is rounded by chance to its mean, so v gains the rounding's variance at every step.  With a steady scale (one
    element of a block, the largest, has a constant gradient) an r on a code moves by |r' - r| <= (1 - b2) |g^2 - r^2| / (r (1
    + sqrt(b2))) before it is rounded between codes d <= r / 8 apart: the variance is at most d |r' - r|.  Summed over
    steps with weights b2^k, E v8 <= V + (V + E v8) / (8 (1 + sqrt(b2))) with V = E g^2 = E v, that is 1.13 V for b2 near
    1, and E v8 >= V.  v8's deviation is below 0.4 V: 0.1 of v's own, and 0.36 by those variances, 4 r^2 d |r' - r| a step."""
    import fp8_moe_grouped_amd as G
    blocks, beta2, steps = 256, 0.99, 1000
    gen = torch.Generator(device="cuda").manual_seed(5)
    n = 256 * blocks
    p = torch.zeros(n, device="cuda")
    m, r = G.adamw_8bit_states([p])
    size = torch.exp2(-8 * torch.rand(n, generator=gen, device="cuda"))
    for t in range(1, steps + 1):
        g = size * torch.randn(n, generator=gen, device="cuda")
        g[::256] = 16.0                                          # 2^12 of the smallest: all others are normal codes
        G.adamw_step_8bit([p], [g], m, r, lr=1e-3, step=t, betas=(0.9, beta2), seed=9)
    held = P.values(r[0][0].cpu(), r[0][1].cpu()) ** 2
    ratio = (held / ((1 - beta2 ** steps) * size.cpu().double() ** 2)).view(blocks, 256)[:, 1:]
    off = 5 * 0.4 / ratio.numel() ** 0.5
    a = 1 / (8 * (1 + beta2 ** 0.5))
    assert 1 - off < float(ratio.mean()) < (1 + a) / (1 - a) + off
