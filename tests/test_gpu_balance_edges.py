"""GPU tests of what a caller may do with the balance losses' outputs."""
import io

import pytest
import torch

from tests.test_gpu_balance import ids_of, logits_of
from tests.test_gpu_calls import Nothing

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("way", ["extension", "python"])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("T", [50, 3000])
def test_outputs_can_be_saved(T, given, way, monkeypatch):
    """Together and in pairs, as a checkpoint or a log of a step does."""
    import fp8_moe_grouped_amd as G
    if way == "python":
        monkeypatch.setattr(G, "_calls", Nothing())
    x, ids = logits_of(T, 24, torch.float32, 1).cuda(), ids_of(T, 24, 3, 2).cuda()
    b = G.moe_balance_loss(x, counts=torch.arange(24, dtype=torch.int32, device="cuda")) if given else \
        G.moe_balance_loss(x, ids)
    for names in (b._fields, *((p, q) for p in b._fields for q in b._fields if p < q)):
        f = io.BytesIO()
        torch.save({n: getattr(b, n) for n in names}, f)
        f.seek(0)
        back = torch.load(f, weights_only=True)
        for n in names:
            assert back[n].dtype == getattr(b, n).dtype and torch.equal(back[n], getattr(b, n))
