"""Training steps of the example's layer on the GPU: routing, products, balance
losses, AdamW and the new codes as they run together."""
import pytest
import torch

from tests import plain_train as P
from tests.test_gpu_moe_layer import E, H, K, layer_and_input

pytestmark = pytest.mark.gpu
COEFFICIENTS = (0.05, 0.01)


def one_step(layer, x, dout):
    _, saved = layer.forward(x)
    balance = layer.balance(saved)
    coefficients = torch.tensor(COEFFICIENTS, device="cuda")
    return saved, balance, layer.backward(dout, saved, balance, coefficients)


def test_gradients_with_the_balance_losses():
    """The router's gradient gains the losses' part, by autograd in 64 bits; the others are as without them."""
    import fp8_moe_grouped_amd as G
    layer, x = layer_and_input(60, 3)
    dout = torch.randn((60, H), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    _, saved = layer.forward(x)
    dx0, drouter0, dwi0, dwo0 = layer.backward(dout, saved)
    saved, balance, (dx, drouter, dwi, dwo) = one_step(layer, x, dout)
    assert torch.equal(dwi, dwi0) and torch.equal(dwo, dwo0)
    assert torch.equal(balance.counts, saved[2].group_sizes)
    router = layer.router.cpu().double().requires_grad_()
    xs = x.cpu().double().requires_grad_()
    logits = xs @ router
    p, c = torch.softmax(logits, 1), balance.counts.cpu().double()
    first = E * (c / c.sum() * p.mean(0)).sum()
    second = (torch.logsumexp(logits, 1) ** 2).mean()
    (COEFFICIENTS[0] * first + COEFFICIENTS[1] * second).backward()
    assert abs(float(balance.losses[0]) - float(first.detach())) < 1e-5
    assert abs(float(balance.losses[1]) - float(second.detach())) < 1e-4
    # drouter is x^T dlogits: each of the two, f32 sums of 60 products in any order, is off by 60 roundings of the sum
    # of magnitudes at most, and dlogits itself by that of its last sum; the losses' own part by 300 of its terms'
    # (the softmax's, see test_gpu_balance)
    _, logits32, r, _, y, _, _ = saved
    _, dweights = G.moe_combine_bwd(dout, y, r.row_of_slot, r.weights)
    dl = G.moe_route_bwd(dweights, logits32, r.ids, r.weights).cpu().double()
    own = P.balance_bwd(torch.tensor(COEFFICIENTS), logits.detach(), balance.counts.cpu(), 60)[1]
    mag = xs.detach().abs().t()
    tol = P.U32 * ((2 * 60 + 2) * (mag @ dl.abs()) + 300 * (mag @ own))
    assert bool((((drouter.double() - drouter0.double()).cpu() - router.grad).abs() <= tol).all())
    # dx is rounded to bf16: half a step of the sum, and of the one without
    off = (dx.double() - dx0.double()).cpu() - xs.grad
    assert float(off.abs().max()) <= float(dx.abs().max()) * 2.0 ** -7


@pytest.mark.parametrize("bits", [32, 8])
def test_updates(bits):
    """Three steps against the plain definition on the gradients that came; the codes are the masters'."""
    layer, x = layer_and_input(40, 7)
    layer.start_training(bits)
    dout = torch.randn((40, H), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    for t in range(1, 4):
        _, _, (_, *gradients) = one_step(layer, x, dout)
        before = [w.cpu().double() for w in layer.masters]
        if bits == 8:
            old = [[P.values(c.cpu(), s.cpu()) for c, s in l] for l in layer.states]
            old[1] = [r ** 2 for r in old[1]]
        else:
            old = [[s.cpu().double().view(-1) for s in l] for l in layer.states]
        layer.update(gradients, 1e-2)
        assert layer.step == t and layer.router is layer.masters[0]
        for i, g in enumerate(gradients):
            (p, _, _), (ep, _, _) = P.Step(1e-2, t)(before[i].view(-1), g.cpu().double().view(-1), old[0][i], old[1][i])
            # twice: an 8-bit state is a product that rounds by itself (m once, r twice in its square)
            assert bool(((layer.masters[i].cpu().double().view(-1) - p).abs() <= 2 * ep).all())
        for (codes, scales), w in zip((layer.wi, layer.wo), layer.masters[1:]):
            value, scale = P.quantize_weights(w.cpu())
            assert torch.equal(scales.cpu(), scale) and torch.equal(P.e4m3(codes.cpu()), value)


def test_a_step_in_a_graph():
    """Forward, losses, backward, update and codes captured once and replayed: the same bits as eager steps."""
    import fp8_moe_grouped_amd as G
    dout = torch.randn((40, H), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    coefficients = torch.tensor(COEFFICIENTS, device="cuda")
    ends = []
    for captured in (False, True):
        layer, x = layer_and_input(40, 9)
        layer.start_training(8)
        step = torch.zeros(1, dtype=torch.int64, device="cuda")

        def run():
            step.add_(1)
            _, saved = layer.forward(x)
            _, *gradients = layer.backward(dout, saved, layer.balance(saved), coefficients)
            G.adamw_step_8bit(layer.masters, gradients, *layer.states, lr=1e-2, step=step)
            for (codes, scales), w in zip((layer.wi, layer.wo), layer.masters[1:]):
                G.quantize_fp8_weights(w, codes=codes, scales=scales)

        start = [t.clone() for t in layer.masters]
        if captured:
            kept = [[t.clone() for t in s] for l in layer.states for s in l]
            codes = [[t.clone() for t in w] for w in (layer.wi, layer.wo)]
            side = torch.cuda.Stream()                       # the library products' own first calls
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                run()
            side.synchronize()
            for a, b in zip(layer.masters, start):
                a.copy_(b)
            for s, k in zip([s for l in layer.states for s in l], kept):
                for a, b in zip(s, k):
                    a.copy_(b)
            for w, k in zip((layer.wi, layer.wo), codes):
                for a, b in zip(w, k):
                    a.copy_(b)
            step.zero_()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                run()
            for _ in range(3):
                graph.replay()
                torch.randn(1000, device="cuda").sum()
                torch.cuda.synchronize()
        else:
            for _ in range(3):
                run()
        assert int(step) == 3
        ends.append([*layer.masters, *layer.wi, *layer.wo] + [t for l in layer.states for s in l for t in s])
    for a, b in zip(*ends):
        assert torch.equal(a, b)


def test_example_prints_the_update(monkeypatch, capsys):
    import examples.moe_layer as M
    monkeypatch.setattr("sys.argv", ["moe_layer.py", "--tokens", "64", "--hidden", "256", "--inner", "128", "--experts",
                                     "8", "--topk", "2"])
    M.main()
    out = capsys.readouterr().out
    assert "update" in out and "decode" in out and K == 3
