"""The extension and the Python path of the balance losses, AdamW and the FP8
weight quantizer: the same results, and what the extension leaves to Python."""
import threading

import pytest
import torch

from tests.test_gpu_calls import Nothing, results

pytestmark = pytest.mark.gpu


def rand(seed, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def adamw(bits, pd=torch.float32, gd=torch.float32, tuples=False, **how):
    """The state after two steps on fresh tensors."""
    import fp8_moe_grouped_amd as G
    kind = tuple if tuples else list
    p, g = kind([rand(1, 300, dtype=pd), rand(2, 4, 70, dtype=pd)]), kind([rand(3, 300, dtype=gd), rand(4, 4, 70, dtype=gd)])
    m, v = (G.adamw_8bit_states(p) if bits == 8 else [[torch.zeros_like(t, dtype=torch.float32) for t in p] for _ in "mv"])
    step = G.adamw_step_8bit if bits == 8 else G.adamw_step
    for t in (1, 2):
        step(p, g, kind(m), kind(v), **{**dict(lr=1e-2, step=t), **how})
    return [*p, *g] + [x for s in (*m, *v) for x in (s if bits == 8 else [s])]


def cases():
    import fp8_moe_grouped_amd as G
    x, ids = rand(5, 300, 12), torch.randint(-1, 12, (300, 3), dtype=torch.int32).cuda()
    counts, tokens = torch.arange(12, dtype=torch.int32).cuda(), torch.tensor([300], dtype=torch.int32).cuda()
    d, w = rand(6, 2), rand(7, 2, 256, 128)
    b16 = lambda t: t.to(torch.bfloat16)
    one = lambda v, t=torch.float32: torch.tensor([v], dtype=t).cuda()
    return {
        "balance": lambda: G.moe_balance_loss(x, ids),
        "balance_large": lambda: G.moe_balance_loss(b16(x).repeat(30, 1), ids.repeat(30, 1)),
        "balance_counts": lambda: G.moe_balance_loss(x, counts=counts),
        "balance_bwd": lambda: G.moe_balance_loss_bwd(d, x, counts, tokens),
        "balance_bwd_add": lambda: G.moe_balance_loss_bwd(d, b16(x), counts, tokens, add=b16(x)),
        "quantize": lambda: G.quantize_fp8_weights(w),
        "quantize_large": lambda: G.quantize_fp8_weights(b16(w).repeat(1, 8, 1)),
        "adamw": lambda: adamw(32),
        "adamw_types": lambda: adamw(32, torch.bfloat16, torch.bfloat16, tuples=True, grad_scale=one(0.5)),
        "adamw_device": lambda: adamw(32, lr=one(0.01), step=one(3, torch.int64), weight_decay=0.0),
        "adamw8": lambda: adamw(8, seed=7, betas=(0.8, 0.9), eps=1e-6),
        "adamw8_types": lambda: adamw(8, torch.float32, torch.bfloat16, tuples=True, seed=(1 << 64) - 1),
        "adamw8_device": lambda: adamw(8, lr=one(0.01), step=one(3, torch.int64), grad_scale=one(2.0)),
    }


NAMES = {"balance": 1, "balance_large": 1, "balance_counts": 1, "balance_bwd": 1, "balance_bwd_add": 1, "quantize": 1,
         "quantize_large": 1, "adamw": 2, "adamw_types": 2, "adamw_device": 2, "adamw8": 2, "adamw8_types": 2,
         "adamw8_device": 2}


@pytest.mark.parametrize("name", NAMES)
def test_both_ways_agree(name, monkeypatch):
    import fp8_moe_grouped_amd as G
    call = cases()[name]
    plain = call()
    monkeypatch.setattr(G, "_calls", Nothing())
    python = call()
    assert type(plain) is type(python)
    for a, b in zip(results(plain), results(python), strict=True):
        assert a.dtype == b.dtype and a.shape == b.shape and a.is_contiguous() and torch.equal(a, b)


def test_the_extension_takes_plain_calls(monkeypatch):
    import fp8_moe_grouped_amd as G
    todo, real, answered = cases(), G._plain(), []

    class Watch:
        def __getattr__(self, name):
            def f(*args):
                out = getattr(real, name)(*args)
                answered.append(out is not None)
                return out
            return f

    monkeypatch.setattr(G, "_calls", Watch())
    for call in todo.values():
        call()
    assert len(answered) == sum(NAMES.values()) and all(answered)


def test_what_is_not_plain_is_left_to_python():
    import fp8_moe_grouped_amd as G
    c = G._plain()
    x, ids = rand(1, 8, 6), torch.zeros((8, 2), dtype=torch.int32, device="cuda")
    counts, tokens, d = ids.view(-1)[:6], ids.view(-1)[:1], rand(2, 2)
    p, w = rand(3, 100), rand(4, 1, 128, 128)
    how = (1e-3, 1, 0.9, 0.999, 1e-8, 0.01, None)
    z = lambda: torch.zeros(100, device="cuda")
    (m,), (r,) = G.adamw_8bit_states([p])
    for out in (c.balance(x, None, None), c.balance(x, ids, counts), c.balance(x[:0], ids[:0], None),
                c.balance(x.half(), ids, None), c.balance(x, ids[:7], None), c.balance(x, None, counts[:5]),
                c.balance(x.t(), ids, None), c.balance(x, ids.cpu(), None), c.balance("x", ids, None),
                c.balance_bwd(d[:1], x, counts, tokens, None), c.balance_bwd(d, x, counts[:5], tokens, None),
                c.balance_bwd(d, x, counts, counts, None), c.balance_bwd(d, x, counts, tokens, x[:7]),
                c.balance_bwd(d, x, counts, tokens, x.to(torch.bfloat16)), c.quantize_fp8(w[0]), c.quantize_fp8(w.half()),
                c.quantize_fp8(w[:, :100].contiguous()), c.quantize_fp8(w.transpose(1, 2)),
                c.adamw([], [], [], [], *how), c.adamw([p], [], [z()], [z()], *how), c.adamw([p], [p], [z()], [z()], *how),
                c.adamw(iter([p]), [z()], [z()], [z()], *how), c.adamw([p], [z()[:50]], [z()], [z()], *how),
                c.adamw([p], [z()], [z()], [z().to(torch.bfloat16)], *how), c.adamw([p], [None], [z()], [z()], *how),
                c.adamw([p], [z()], [z()], [z()], -1.0, *how[1:]), c.adamw([p], [z()], [z()], [z()], 1e-3, 0, *how[2:]),
                c.adamw([p], [z()], [z()], [z()], 1e-3, 1.0, *how[2:]), c.adamw([p], [z()], [z()], [z()], "1", *how[1:]),
                c.adamw([p], [z()], [z()], [z()], 1e-3, 1, 0.9, 0.999, 1e-8, 0.01, 0.5),
                c.adamw([p], [z()], [z()], [z()], 1e-3, 1 << 70, *how[2:]),
                c.adamw([p, p.to(torch.bfloat16)], [z(), z()], [z(), z()], [z(), z()], *how),
                c.adamw8([p], [z()], [m], [r], *how, -1), c.adamw8([p], [z()], [m], [r], *how, 1 << 64),
                c.adamw8([p], [z()], [list(m)], [r], *how, 1), c.adamw8([p], [z()], [m], [(r[0], r[1].repeat(2))], *how, 1),
                c.adamw8([p], [z()], [m], [m], *how, 1), c.adamw8([p], [z()], [m[0]], [r], *how, 1)):
        assert out is None
    assert torch.equal(p, rand(3, 100))
    for f, args in ((c.balance, (x,)), (c.adamw, ([p],)), (c.adamw8, ([p],) * 3), (c.quantize_fp8, ())):
        with pytest.raises(TypeError):
            f(*args)


def test_outputs_share_nothing():
    """The small outputs lie in one allocation: writing one, or dropping the others, leaves each as it was."""
    import fp8_moe_grouped_amd as G
    x, ids = rand(1, 50, 9), torch.randint(0, 9, (50, 2), dtype=torch.int32).cuda()
    a, b = G.moe_balance_loss(x, ids), G.moe_balance_loss(x, ids)
    want = [t.clone() for t in b]
    a.counts.add_(100)
    a.losses.fill_(-1)
    assert torch.equal(a.probs, b.probs) and torch.equal(a.tokens, b.tokens)
    probs = a.probs
    del a
    junk = [torch.full((64,), 7.0, device="cuda") for _ in range(20)]
    torch.cuda.synchronize()
    assert torch.equal(probs, want[2]) and all(torch.equal(t, w) for t, w in zip(b, want)) and len(junk) == 20
    assert all(t.is_contiguous() and not t.requires_grad for t in b)
    assert torch.equal(b.probs.view(3, 3).sum(1).cpu(), want[2].view(3, 3).sum(1).cpu())


@pytest.mark.parametrize("name", ["balance_large", "quantize_large", "adamw8"])
def test_side_streams_and_other_threads(name):
    call = cases()[name]
    want = results(call())
    torch.cuda.synchronize()
    got = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got.append(results(call()))
        s.synchronize()

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 3 and all(torch.equal(a, b) for out in got for a, b in zip(out, want))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("way", ["extension", "python"])
def test_a_graph_notices_the_step(bits, way, monkeypatch):
    """A backward pass that has saved a parameter does not go on with the next step's values."""
    import fp8_moe_grouped_amd as G
    p = [torch.nn.Parameter(rand(1, 300))]
    m, v = G.adamw_8bit_states(p) if bits == 8 else [[torch.zeros(300, device="cuda")] for _ in "mv"]
    G._plain()
    if way == "python":
        monkeypatch.setattr(G, "_calls", Nothing())
    before, loss = p[0]._version, (p[0] * p[0]).sum()
    step = G.adamw_step_8bit if bits == 8 else G.adamw_step
    step(p, [rand(2, 300)], m, v, lr=1e-2, step=1)
    assert p[0]._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():                                 # which counts no versions of what it makes
        step([p[0] + 0.0], [rand(2, 300)], m, v, lr=1e-2, step=2)
