"""GPU test of AdamW's rates next to the limits of f32, both ways into the
library."""
import pytest
import torch

from tests.test_gpu_calls import Nothing

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("way", ["extension", "python"])
def test_rates_at_the_limits(way, bits, monkeypatch):
    import fp8_moe_grouped_amd as G
    if way == "python":
        monkeypatch.setattr(G, "_calls", Nothing())
    step = G.adamw_step_8bit if bits == 8 else G.adamw_step
    p, g = torch.ones(300, device="cuda"), torch.zeros(300, device="cuda")
    states = G.adamw_8bit_states([p]) if bits == 8 else [[torch.zeros(300, device="cuda")] for _ in "mv"]
    for bad in (dict(lr=1e38), dict(lr=1e39, betas=(0.0, 0.9)), dict(lr=1e30, weight_decay=1e9), dict(lr=1.0, eps=1e38),
                dict(lr=1.0, eps=1e300)):
        with pytest.raises(ValueError):
            step([p], [g], *states, step=1, **bad)
    assert bool((p == 1).all())
    step([p], [g], *states, step=1, lr=1e37, weight_decay=0.0)    # no gradient, no move
    step([p], [g], *states, step=2, lr=1e-3, eps=2.0 ** 126, weight_decay=0.0)
    assert bool((p == 1).all())
    g.fill_(-1.0)                                                 # m' = -1 and v' = 1: 2^127 2^-126
    step([p], [g], *states, step=3, lr=2.0 ** 127, eps=2.0 ** 126, betas=(0.0, 0.0), weight_decay=0.0)
    assert bool(((p - 3).abs() < 3e-6).all())
