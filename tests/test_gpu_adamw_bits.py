"""GPU tests of AdamW bit for bit: numbers on the device against numbers of the
host."""
import decimal
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
F32 = torch.float32


def f32(v):
    return torch.tensor(v, dtype=torch.float64).to(F32)


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
