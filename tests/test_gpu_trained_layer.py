"""The example's layer after updates: what it trains from, and what it decodes with."""
import pytest
import torch

from tests.test_gpu_moe_layer import E, H, I, K

pytestmark = pytest.mark.gpu


def weights(seed):
    g = torch.Generator().manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g)
    router = (normal(H, E) * H ** -0.5).cuda()
    return router, (normal(E, H, 2 * I) * H ** -0.5).to(torch.bfloat16).cuda(), \
        (normal(E, I, H) * I ** -0.5).to(torch.bfloat16).cuda()


def trained(seed, bits=32, steps=2):
    """A layer after a few updates, and its input."""
    from examples.moe_layer import MoeLayer
    layer = MoeLayer(*weights(seed), K)
    g = torch.Generator().manual_seed(seed + 100)
    x, dout = (torch.randn((20, H), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    layer.start_training(bits)
    for _ in range(steps):
        _, saved = layer.forward(x)
        layer.update(layer.backward(dout, saved)[1:], 2e-2)
    return layer, x


def test_masters_are_the_given_weights():
    """Training starts from the weights themselves, not from their codes' values."""
    from examples.moe_layer import MoeLayer
    router, wi, wo = weights(1)
    layer = MoeLayer(router, wi, wo, K)
    layer.start_training()
    assert layer.masters[0] is router
    for master, w in zip(layer.masters[1:], (wi, wo)):
        assert master.dtype == torch.float32 and torch.equal(master, w.float())


def test_training_goes_on_from_the_masters():
    """A second start has fresh states and the masters as they are; the weights first given stay as they were."""
    from examples.moe_layer import MoeLayer
    router, wi, wo = weights(2)
    kept = wi.clone(), wo.clone()
    layer = MoeLayer(router, wi, wo, K)
    layer.start_training()
    layer.update([torch.ones_like(w) for w in layer.masters], 1e-2)
    before = [w.clone() for w in layer.masters]
    layer.start_training(8)
    assert layer.step == 0 and all(torch.equal(a, b) for a, b in zip(layer.masters, before))
    assert not any(bool(codes.any()) for l in layer.states for codes, _ in l)
    assert torch.equal(wi, kept[0]) and torch.equal(wo, kept[1])


@pytest.mark.parametrize("bits", [32, 8])
def test_decoding_after_updates(bits):
    """Decoding reads the updated weights: the bits of a layer made from the masters, and not those of before."""
    from examples.moe_layer import MoeLayer
    layer, x = trained(3, bits)
    old = MoeLayer(layer.router, *weights(3)[1:], K)
    fresh = MoeLayer(layer.router, *(w.to(torch.bfloat16) for w in layer.masters[1:]), K)
    for a, b in zip((*layer.wi4, *layer.wo4), (*fresh.wi4, *fresh.wo4)):
        assert torch.equal(a, b)
    assert torch.equal(layer.decode(x), fresh.decode(x))
    assert not torch.equal(layer.decode(x), old.decode(x))


def test_a_captured_decoding_follows_updates():
    layer, x = trained(4, steps=1)
    layer.decode(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.decode(x)
    for _ in range(3):
        layer.update([torch.ones_like(w) for w in layer.masters], 2e-2)
        graph.replay()
        want = layer.decode(x)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
