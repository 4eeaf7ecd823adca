"""GPU tests of the balance losses where sizes or loads are far apart or nearly
alike, and of what a caller may do with their outputs."""
import io

import pytest
import torch

from tests import plain_train as P
from tests.test_gpu_balance import INF, check_grad, ids_of, logits_of
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E", [(7, 8), (40, 24), (300, 160), (33, 1000)])
@pytest.mark.parametrize("base", [1 << 22, (1 << 25) + 1, (1 << 28) + 5, (1 << 31) - 100])
def test_gradient_of_a_nearly_even_load(base, T, E, dtype):
    """Loads of many batches that differ by a few slots: their distances from the mean, not their f32 roundings.  The
    bound is of the distances' magnitudes (see check_grad): a distance is rounded once, and a mean that is off by the
    same for all experts drops out."""
    import fp8_moe_grouped_amd as G
    x = logits_of(T, E, dtype, E)
    counts = base + torch.randint(-50, 51, (E,), generator=torch.Generator().manual_seed(T)).to(torch.int32)
    d = torch.tensor([1.0, 0.0])
    n = torch.tensor([T], dtype=torch.int32)
    check_grad(G.moe_balance_loss_bwd(d.cuda(), x.cuda(), counts.cuda(), n.cuda()), d, x, counts, T)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d1", [(1, 1.0), (1, -0.7), (3, 3.0), (70, 80.0)])
@pytest.mark.parametrize("E", [8, 9, 300])
def test_gradient_of_rows_masked_with_the_lowest_value(E, T, d1, dtype):
    """A token whose logits are the type's lowest value has a log-sum-exp near it, which times 2 d1 / n passes f32: its
    probabilities bring it back, masked experts get 0, and other tokens are as always."""
    import fp8_moe_grouped_amd as G
    x = logits_of(T, E, dtype, 3)
    lowest = torch.full((E,), torch.finfo(dtype).min, dtype=dtype)
    x[0] = torch.where(torch.arange(E) % 2 == 0, lowest, torch.tensor(-INF, dtype=dtype))
    if T > 2:
        x[1], x[T - 1] = lowest, -INF
    counts = torch.arange(E, dtype=torch.int32)
    d = torch.tensor([0.3, d1])
    n = int((x != -INF).any(1).sum())
    for add in (None, torch.ones((T, E), dtype=dtype)):
        got = G.moe_balance_loss_bwd(d.cuda(), x.cuda(), counts.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                                     add=None if add is None else add.cuda())
        want = P.balance_bwd(d, x, counts, n, add)[0]
        assert bool((want.abs() < torch.finfo(dtype).max).all()) and bool(torch.isfinite(want).all())
        check_grad(got, d, x, counts, n, add)
