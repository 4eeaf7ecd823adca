"""The binding's extension and its Python path: the same results, and the same
errors for what the extension leaves to Python."""
import pytest
import torch

pytestmark = pytest.mark.gpu


class Nothing:
    """Stands for the extension: leaves every call to Python."""

    def __getattr__(self, name):
        return lambda *args: None


def cases():
    import fp8_moe_grouped_amd as G
    g = torch.Generator().manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g)
    T, H, E, k = 300, 256, 8, 3
    logits = rand(T, E).cuda()
    r = G.moe_route(logits, k)
    x, y = rand(T, H).to(torch.bfloat16).cuda(), rand(T * k, H).to(torch.bfloat16).cuda()
    dw = rand(T, k).cuda()
    w = rand(E, H, 512).to(torch.bfloat16).cuda()
    codes, scales = G.quantize_mxfp4_weights(w)
    return {
        "route": lambda: G.moe_route(logits, k),
        "route_all": lambda: G.moe_route(logits.to(torch.bfloat16), k, renormalize=False),
        "route_large": lambda: G.moe_route(logits.repeat(30, 1), k),
        "route_bwd": lambda: G.moe_route_bwd(dw, logits, r.ids, r.weights),
        "route_bwd_all": lambda: G.moe_route_bwd(dw, logits.to(torch.bfloat16), r.ids, r.weights, renormalize=False),
        "permute": lambda: G.moe_permute(x, r.row_of_slot),
        "permute_fp8": lambda: G.moe_permute_fp8(x, r.row_of_slot),
        "combine": lambda: G.moe_combine(y, r.row_of_slot, r.weights),
        "combine_sum": lambda: G.moe_combine(y, r.row_of_slot),
        "combine_bwd": lambda: G.moe_combine_bwd(x, y, r.row_of_slot, r.weights),
        "quantize": lambda: G.quantize_mxfp4_weights(w),
        "values": lambda: G.dequantize_mxfp4(codes, scales),
        "product": lambda: G.gmm_mxfp4_fwd(x, codes, scales, r.group_sizes, slot_of_row=r.slot_of_row, topk=k),
        "product_silu": lambda: G.gmm_silu_mxfp4(x, codes, scales, r.group_sizes, slot_of_row=r.slot_of_row, topk=k),
        "product_rows": lambda: G.gmm_mxfp4_fwd(y, codes, scales, r.group_sizes),
        "empty": lambda: G.moe_combine(y, r.row_of_slot[:0], r.weights[:0]),
    }


NAMES = ["route", "route_all", "route_large", "route_bwd", "route_bwd_all", "permute", "permute_fp8", "combine",
         "combine_sum", "combine_bwd", "quantize", "values", "product", "product_silu", "product_rows", "empty"]


def results(out):
    return [out] if isinstance(out, torch.Tensor) else list(out)


@pytest.mark.parametrize("name", NAMES)
def test_both_ways_agree(name, monkeypatch):
    import fp8_moe_grouped_amd as G
    call = cases()[name]
    plain = call()
    monkeypatch.setattr(G, "_calls", Nothing())
    python = call()
    assert type(plain) is type(python)
    for a, b in zip(results(plain), results(python), strict=True):
        assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b)


def test_the_extension_takes_plain_calls(monkeypatch):
    """Every plain call is answered by the extension itself."""
    import fp8_moe_grouped_amd as G
    todo = cases()
    real = G._plain()
    answered = []

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
    assert len(answered) == len(NAMES) and all(answered)


def test_what_is_not_plain_is_left_to_python():
    import fp8_moe_grouped_amd as G
    c = G._plain()
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((4, 2), device="cuda")
    codes = torch.zeros((2, 128, 64), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((2, 1, 128, 4), dtype=torch.uint8, device="cuda")
    sizes = torch.zeros(2, dtype=torch.int32, device="cuda")
    for out in (c.permute(x.cpu(), rows), c.permute(x, rows.long()), c.permute(x[:3], rows), c.permute("x", rows),
                c.permute(x[:, :96].contiguous(), rows), c.permute(x[:, ::2], rows), c.permute(x, rows[:, 0]),
                c.combine(x, rows, w[:3]), c.combine(x, rows, rows), c.combine(x, rows, w.cpu()), c.combine(None, rows, w),
                c.combine_bwd(x[:3], x, rows, w), c.combine_bwd(x[:, :64].contiguous(), x, rows, w),
                c.route(w, 3, True), c.route(w, 0, True), c.route(w, -1, True), c.route(w.half(), 1, True),
                c.route(torch.zeros((2, 1025), device="cuda"), 1, True),
                c.route_bwd(w, w, rows, w[:, :1].contiguous(), True), c.quantize_weights(codes), c.values(codes, scales[:1]),
                c.values(codes, scales[:, :, :64].contiguous()), c.product(x, codes, scales, sizes[:1], None, 1, False),
                c.product(x, codes, scales, sizes, None, 0, False), c.product(x, codes, scales, sizes, None, 1, True),
                c.product(x, codes, scales, sizes, sizes.long(), 1, False)):
        assert out is None
    with pytest.raises(TypeError):
        c.permute(x)
    with pytest.raises(TypeError):
        c.route(w, "k", True)


def test_side_stream_and_other_threads():
    import threading

    import fp8_moe_grouped_amd as G
    call = cases()["product"]
    want = call()
    torch.cuda.synchronize()
    got = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got.append(call())
        s.synchronize()

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 3 and all(torch.equal(o, want) for o in got)


@pytest.mark.parametrize("way", ["extension", "python"])
def test_refusals_of_either_way(way, monkeypatch):
    """Flags without a truth, integers past 32 bits, scratch in host memory: errors, before any launch."""
    import fp8_moe_grouped_amd as G
    if way == "python":
        monkeypatch.setattr(G, "_calls", Nothing())
    logits = torch.zeros((4, 8), device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((4, 2), device="cuda")
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros((2, 128, 64), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((2, 1, 128, 4), dtype=torch.uint8, device="cuda")
    sizes = torch.zeros(2, dtype=torch.int32, device="cuda")
    two = torch.zeros(2)
    for call in (lambda: G.moe_route(logits, 2, renormalize=two),
                 lambda: G.moe_route_bwd(w, logits, ids, w, renormalize=two)):
        with pytest.raises(RuntimeError, match="ambiguous"):
            call()
    for k in ((1 << 32) + 2, 1 << 70, -(1 << 70)):
        with pytest.raises(ValueError):
            G.moe_route(logits, k)
    for k in ((1 << 32) + 1, 1 << 70):
        with pytest.raises(ValueError, match="topk"):
            G.gmm_mxfp4_fwd(x, codes, scales, sizes, topk=k)
    for bad in (dict(dev_status=torch.zeros(1, dtype=torch.int32)), dict(dev_status=sizes[:0]),
                dict(workspace=torch.zeros(1 << 16, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            G.gmm_mxfp4_fwd(x, codes, scales, sizes, **bad)
    for bad in (dict(dev_status=sizes.long()), dict(workspace=torch.zeros(1 << 16, device="cuda"))):
        with pytest.raises(TypeError):
            G.gmm_mxfp4_fwd(x, codes, scales, sizes, **bad)
    with pytest.raises(ValueError):
        G.moe_route(logits, 2, workspace=torch.zeros(1 << 16, dtype=torch.uint8))
    torch.cuda.synchronize()
