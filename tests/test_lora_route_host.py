"""Refusals of the adapters', the routing's and the routed layer's entry points, on the CPU: no call here validates, so none launches."""
import ctypes

import pytest
import torch

from weight_only_quantized_int8_amd import LoraAdapters, Mxfp4Weight, lora_add, moe_layer_routed, moe_route
from weight_only_quantized_int8_amd import binding as B

A = 1 << 24  # fake, 256-byte aligned "device" addresses, never dereferenced


def err(rc):
    assert rc != B.INT8W_OK
    return rc, B.load_library().int8w_last_error().decode()


def pool(a=A, b=2 * A, scales=3 * A, ranks=None, num=4, rank=16, k=64, n=96):
    return B.LoraDesc(a, b, scales, ranks, num, rank, k, n)


def out(base=4 * A, y=5 * A, bs=96, ys=96):
    return B.LoraOut(base, y, bs, ys)


def add(pools=None, outs=None, count=None, x=6 * A, xs=64, ids=7 * A, m=8, ws=8 * A, nbytes=1 << 20):
    pools = [pool()] if pools is None else pools
    outs = [out()] * len(pools) if outs is None else outs
    parr, oarr = (B.LoraDesc * max(1, len(pools)))(*pools), (B.LoraOut * max(1, len(outs)))(*outs)
    return B.int8w_lora_add(parr, oarr, len(pools) if count is None else count, x, xs, ids, m, ws, nbytes, 0)


NULL, SHAPE, UNSUPPORTED, ALIGN, ALIAS = (B.INT8W_ERR_NULL, B.INT8W_ERR_SHAPE, B.INT8W_ERR_UNSUPPORTED, B.INT8W_ERR_ALIGN,
                                          B.INT8W_ERR_ALIAS)


@pytest.mark.parametrize("kw,code,text", [
    (dict(count=0), SHAPE, "count"),
    (dict(count=5), SHAPE, "count"),
    (dict(pools=[pool(a=0)]), NULL, "missing a tensor"),
    (dict(pools=[pool(b=0)]), NULL, "missing a tensor"),
    (dict(pools=[pool(num=0)]), SHAPE, "zero dimension"),
    (dict(pools=[pool(k=0)]), SHAPE, "zero dimension"),
    (dict(pools=[pool(n=0)]), SHAPE, "zero dimension"),
    (dict(pools=[pool(rank=0)]), SHAPE, "rank 0"),
    (dict(pools=[pool(rank=12)]), SHAPE, "rank 12"),
    (dict(pools=[pool(rank=264)]), SHAPE, "rank 264"),
    (dict(pools=[pool(k=60)]), SHAPE, "in_features 60"),
    (dict(pools=[pool(k=1 << 20)]), SHAPE, "below 2^20"),
    (dict(pools=[pool(n=1 << 20)]), SHAPE, "below 2^20"),
    (dict(pools=[pool(num=1 << 24)]), SHAPE, "below 2^24"),
    (dict(pools=[pool(a=A + 8)]), ALIGN, "a or b"),
    (dict(pools=[pool(b=2 * A + 2)]), ALIGN, "a or b"),
    (dict(pools=[pool(scales=3 * A + 2)]), ALIGN, "scales or ranks"),
    (dict(pools=[pool(ranks=3 * A + 2)]), ALIGN, "scales or ranks"),
    (dict(pools=[pool(), pool(num=5)]), SHAPE, "pools differ"),
    (dict(pools=[pool(), pool(k=128)]), SHAPE, "pools differ"),
    (dict(m=(1 << 20) + 1), SHAPE, "more than 2^20"),
    (dict(x=0), NULL, "x, ids"),
    (dict(ids=0), NULL, "x, ids"),
    (dict(pools=[pool(rank=72)], ws=0), NULL, "workspace"),
    (dict(xs=56), SHAPE, "x_stride"),
    (dict(xs=68), SHAPE, "x_stride"),
    (dict(xs=(1 << 32) + 8), SHAPE, "x_stride"),
    (dict(x=6 * A + 8), ALIGN, "x is not"),
    (dict(ids=7 * A + 2), ALIGN, "ids"),
    (dict(ws=8 * A + 128), ALIGN, "workspace"),
    (dict(pools=[pool(rank=72)], nbytes=64), SHAPE, "workspace of 64"),
    (dict(outs=[out(y=0)]), NULL, "y is NULL"),
    (dict(outs=[out(y=5 * A + 1)]), ALIGN, "y/base"),
    (dict(outs=[out(base=4 * A + 1)]), ALIGN, "y/base"),
    (dict(outs=[out(ys=95)]), SHAPE, "y_stride"),
    (dict(outs=[out(bs=95)]), SHAPE, "base_stride"),
    (dict(outs=[out(y=6 * A)]), ALIAS, "input x"),
    (dict(outs=[out(y=7 * A)]), ALIAS, "input ids"),
    (dict(outs=[out(y=A + 64)]), ALIAS, "input a"),
    (dict(outs=[out(y=3 * A)]), ALIAS, "input scales"),
    (dict(outs=[out(y=4 * A + 2)]), ALIAS, "input base"),
    (dict(outs=[out(base=4 * A, y=4 * A, bs=96, ys=104)]), ALIAS, "input base"),
    (dict(pools=[pool(rank=72)], outs=[out(y=8 * A + 16)]), ALIAS, "workspace"),
    (dict(pools=[pool(rank=72)], outs=[out(base=8 * A + 16)]), ALIAS, "workspace"),
    (dict(pools=[pool(rank=72)], ws=6 * A), ALIAS, "input x"),
    (dict(pools=[pool(), pool()], outs=[out(ys=200), out(y=5 * A + 2 * 95, ys=200)]), ALIAS, "two outputs"),
    (dict(pools=[pool(), pool()], outs=[out(ys=200), out(y=5 * A + 2 * 105, ys=200)]), ALIAS, "two outputs"),
    (dict(pools=[pool(), pool()], outs=[out(ys=200), out(y=5 * A + 2 * 96, ys=208)]), ALIAS, "two outputs"),
    (dict(pools=[pool(), pool()], outs=[out(base=None, ys=200), out(base=5 * A, y=9 * A, bs=200)]), ALIAS, "input base"),
])
def test_adapter_calls_are_refused(kw, code, text):
    rc, msg = err(add(**kw))
    assert rc == code and text in msg, (rc, msg)


def test_workspace_of_bad_pools_is_zero_and_of_no_rows():
    assert B.int8w_lora_workspace_bytes(pool(rank=12), 1, 8) == 0
    assert B.int8w_lora_workspace_bytes(pool(), 1, 0) == 0
    for m in (1, 16, 200, 256, 257, 4096, 1 << 20):
        p = pool(rank=72)
        one, two = B.int8w_lora_workspace_bytes(p, 1, m), B.int8w_lora_workspace_bytes((B.LoraDesc * 2)(p, p), 2, m)
        assert one >= m * 72 * 4 and one % 256 == 0 and two >= 2 * m * 72 * 4


def test_few_rows_of_small_matrices_need_no_workspace():
    assert [B.int8w_lora_workspace_bytes(pool(), 1, m) for m in (1, 8, 16)] == [0, 0, 0]
    # refused for its output, so past the workspace, which is neither needed nor looked at
    for kw in (dict(ws=0, nbytes=0), dict(ws=6 * A), dict(nbytes=64)):
        rc, msg = err(add(outs=[out(y=0)], **kw))
        assert rc == NULL and "y is NULL" in msg, (kw, msg)
    rc, msg = err(add(ws=8 * A + 128))  # its alignment is looked at all the same
    assert rc == ALIGN and "workspace" in msg


@pytest.mark.parametrize("m", [65, 4096, 70001, 1 << 20])
def test_many_rows_of_tiny_matrices_are_planned(m):
    assert B.int8w_lora_workspace_bytes(pool(k=8, rank=8, n=40), 1, m) >= m * 8 * 4  # a row a workgroup would pass the grid


def test_no_rows_are_nothing_to_do():
    assert add(m=0, x=0, ids=0, ws=0) == B.INT8W_OK
    assert B.int8w_moe_route(route(tokens=0, logits=0), 0) == B.INT8W_OK


def route(logits=A, bias=None, ids=2 * A, weights=3 * A, tokens=5, experts=16, topk=4, fmt=1, scoring=0, groups=4, topk_groups=2, group_score=0):
    return B.RouteCall(logits, bias, ids, weights, tokens, experts, topk, fmt, scoring, groups, topk_groups, group_score, 1, 1.0)


@pytest.mark.parametrize("kw,code,text", [
    (dict(experts=0), SHAPE, "num_experts"), (dict(experts=513), SHAPE, "num_experts"), (dict(topk=0), SHAPE, "topk"),
    (dict(topk=17), SHAPE, "topk"), (dict(experts=3, groups=1, topk_groups=1), SHAPE, "topk"), (dict(fmt=2), UNSUPPORTED, "logits_format"),
    (dict(scoring=2), UNSUPPORTED, "scoring"), (dict(group_score=2), UNSUPPORTED, "group_score"), (dict(groups=0), SHAPE, "groups"),
    (dict(groups=5), SHAPE, "groups"), (dict(experts=128, groups=128), SHAPE, "groups"), (dict(topk_groups=0), SHAPE, "topk_groups"),
    (dict(topk_groups=5), SHAPE, "topk_groups"), (dict(topk=9), SHAPE, "topk 9 of 2 groups"), (dict(logits=0), NULL, "NULL"),
    (dict(ids=0), NULL, "NULL"), (dict(weights=0), NULL, "NULL"), (dict(logits=A + 2), ALIGN, "logits"), (dict(fmt=0, logits=A + 1), ALIGN, "logits"),
    (dict(bias=4 * A + 2), ALIGN, "bias"), (dict(ids=2 * A + 2), ALIGN, "ids"), (dict(ids=A + 16), ALIAS, "input logits"),
    (dict(bias=3 * A + 16), ALIAS, "input bias"), (dict(weights=2 * A + 16), ALIAS, "ids"),
])
def test_routings_are_refused(kw, code, text):
    rc, msg = err(B.int8w_moe_route(route(**kw), 0))
    assert rc == code and text in msg, (rc, msg)
    rc, msg = err(B.int8w_moe_route(ctypes.POINTER(B.RouteCall)(), 0))
    assert rc == NULL and "call is NULL" in msg


E, I, H = 4, 96, 64


def layer():
    def mx(rows, k, at):
        return B.Mxfp4Desc(at * A, (at + 1) * A, rows, k)
    return mx(E * I, H, 10), mx(E * I, H, 12), mx(E * H, I, 14)


def routed(x=20 * A, ids=21 * A, weights=22 * A, resid=None, y=23 * A, tokens=3, topk=2):
    return B.MoeRoutedCall(x, ids, weights, resid, y, tokens, topk)


@pytest.mark.parametrize("call,code,text", [
    (routed(topk=0), SHAPE, "topk"), (routed(topk=17), SHAPE, "topk"), (routed(x=0), NULL, "NULL"), (routed(ids=0), NULL, "ids"),
    (routed(weights=0), NULL, "weights"), (routed(y=0), NULL, "NULL"), (routed(ids=21 * A + 2), ALIGN, "ids/weights"),
    (routed(weights=22 * A + 2), ALIGN, "ids/weights"), (routed(y=20 * A), ALIAS, "input x"), (routed(y=21 * A), ALIAS, "input ids"),
    (routed(y=22 * A), ALIAS, "input weights"), (routed(resid=23 * A + 2), ALIAS, "x_resid"),
    (ctypes.POINTER(B.MoeRoutedCall)(), NULL, "call is NULL"),
])
def test_routed_layers_are_refused(call, code, text):
    rc, msg = err(B.int8w_mxfp4_moe_layer_routed(*layer(), E, call, 30 * A, 1 << 19, 0))
    assert rc == code and text in msg, (rc, msg)


def test_a_routed_layer_takes_more_choices_than_experts_and_checks_the_workspace():
    rc, msg = err(B.int8w_mxfp4_moe_layer_routed(*layer(), E, routed(topk=6), 30 * A, 100, 0))
    assert rc == SHAPE and "workspace of 100" in msg
    rc, msg = err(B.int8w_mxfp4_moe_layer_routed(*layer(), 3, routed(), 30 * A, 1 << 19, 0))
    assert rc == SHAPE and "not 3 experts" in msg
    assert B.int8w_mxfp4_moe_layer_routed(*layer(), E, routed(tokens=0), 0, 0, 0) == B.INT8W_OK


def test_python_checks():
    bf = torch.bfloat16
    with pytest.raises(ValueError, match="3-D bfloat16"):
        LoraAdapters(torch.zeros(2, 8, 16), torch.zeros(2, 4, 8, dtype=bf))
    with pytest.raises(ValueError, match="b must be"):
        LoraAdapters(torch.zeros(2, 8, 16, dtype=bf), torch.zeros(2, 4, 16, dtype=bf))
    with pytest.raises(ValueError, match="rank 12"):
        LoraAdapters(torch.zeros(2, 12, 16, dtype=bf), torch.zeros(2, 4, 12, dtype=bf))
    with pytest.raises(ValueError, match="contiguous"):
        LoraAdapters(torch.zeros(2, 16, 8, dtype=bf).transpose(1, 2), torch.zeros(2, 4, 8, dtype=bf))
    with pytest.raises(ValueError, match="on one GPU"):
        LoraAdapters(torch.zeros(2, 8, 16, dtype=bf), torch.zeros(2, 4, 8, dtype=bf))
    with pytest.raises(ValueError, match="at least one"):
        LoraAdapters.from_list([])
    with pytest.raises(ValueError, match="adapters must be"):
        LoraAdapters.from_list([(torch.zeros(4, 16, dtype=bf), torch.zeros(8, 5, dtype=bf), 1.0)])
    with pytest.raises(B.Int8wError, match="1..4 pools"):
        lora_add([], torch.zeros(1, 16, dtype=bf), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU tensor"):
        moe_route(torch.zeros(2, 4), 2)
    with pytest.raises(TypeError, match="three Int8Weight or three Mxfp4Weight"):
        moe_layer_routed(None, None, None, 4, torch.zeros(1, 64, dtype=bf), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 2))


@pytest.mark.parametrize("topk", [0, 17])
def test_a_wrong_topk_is_refused_before_it_sizes_the_scratch(topk, monkeypatch):
    def host(rows, k):
        codes, scales = torch.zeros(rows, k // 2, dtype=torch.uint8), torch.zeros(rows, k // 32, dtype=torch.uint8)
        w = Mxfp4Weight.__new__(Mxfp4Weight)
        w._set(codes, scales, rows, k, codes.device, codes.data_ptr(), scales.data_ptr())
        return w
    monkeypatch.setattr(B, "int8w_moe_workspace_bytes", lambda *a: pytest.fail(f"scratch sized for topk {topk}"))
    with pytest.raises(B.Int8wError, match="topk"):
        moe_layer_routed(host(E * I, H), host(E * I, H), host(E * H, I), E, torch.zeros(3, H, dtype=torch.bfloat16),
                         torch.zeros(3, topk, dtype=torch.int32), torch.zeros(3, topk))


def test_another_device_is_made_current_for_the_launch(monkeypatch):
    seen = []

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            seen.append(self.device)

        def __exit__(self, *exc):
            seen.append("back")
    monkeypatch.setattr(B, "_current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "device", Device)
    for here in (torch.device("cuda", 1), torch.device("cuda"), torch.device("cpu")):
        B._call(here, lambda *a: B.INT8W_OK, 1, 2)
    assert seen == []
    B._call(torch.device("cuda", 0), lambda *a: B.INT8W_OK)
    assert seen == [torch.device("cuda", 0), "back"]
    with pytest.raises(B.Int8wError):
        B._call(torch.device("cuda", 0), lambda *a: B.INT8W_ERR_SHAPE)
    assert seen[2:] == [torch.device("cuda", 0), "back"]


def test_packed_arguments_are_the_structures():
    c = route(bias=9 * A, tokens=7, experts=60, topk=3, scoring=1, groups=6, topk_groups=2, group_score=1)
    packed = B._ROUTE_CALL.pack(A, 9 * A, 2 * A, 3 * A, 7, 60, 3, 1, 1, 6, 2, 1, 1, 1.0)
    assert bytes(B.RouteCall.from_buffer_copy(packed))[:72] == bytes(c)[:72]
    assert B._LORA_OUT.pack(4 * A, 5 * A, 96, 97) == bytes(out(ys=97))


def fake_pool(a, b, scales=None):
    p = LoraAdapters.__new__(LoraAdapters)
    p.a, p.b, p.scales, p.ranks, p.device = a, b, scales, None, a.device
    p.trained = a.requires_grad or b.requires_grad or (scales is not None and scales.requires_grad)
    (p.num_adapters, p.rank, p.in_features), p.out_features = a.shape, b.shape[1]
    p.desc = B.LoraDesc(a.data_ptr(), b.data_ptr(), None, None, p.num_adapters, p.rank, p.in_features, p.out_features)
    p.packed = bytes(p.desc)
    return p


def test_inputs_that_require_a_gradient_are_refused(monkeypatch):
    bf = torch.bfloat16
    zeros = {"x": (2, 16), "a": (3, 8, 16), "b": (3, 24, 8), "scales": (3,), "base": (2, 24)}
    ids = torch.zeros(2, dtype=torch.int32)
    launched = []
    monkeypatch.setattr(B, "_call", lambda dev, entry, *args: launched.append(entry))
    monkeypatch.setattr(B, "_stream_of", lambda dev: 0)

    class Projection:  # what gemm_lora asks of its weight
        in_features = k = 16
        out_features = rows = 24
        device = torch.device("cpu")

        def gemm(self, x, y):
            launched.append("gemm")
            return torch.zeros(2, 24, dtype=bf)
    for trained in ("x", "a", "b", "scales", "base", None):
        t = {k: torch.zeros(s, dtype=torch.float32 if k == "scales" else bf, requires_grad=k == trained) for k, s in zeros.items()}
        pool, other = fake_pool(t["a"], t["b"], t["scales"]), fake_pool(*(torch.zeros(zeros[k], dtype=bf) for k in "ab"))
        calls = [lambda: lora_add(pool, t["x"], ids, t["base"]), lambda: lora_add([other, pool], t["x"], ids, [None, t["base"]])]
        if trained != "base":
            calls += [lambda: B.Int8Weight.gemm_lora(Projection(), t["x"], pool, ids), lambda: Mxfp4Weight.gemm_lora(Projection(), t["x"], pool, ids)]
        for call in calls:
            del launched[:]
            if trained:
                with pytest.raises(B.Int8wError, match="has no backward") as e:
                    call()
                assert e.value.code == UNSUPPORTED and not launched
            with torch.no_grad():
                call()
            assert launched
            if not trained:
                call()

    class Logits(torch.Tensor):  # as if on a GPU
        device = torch.device("cuda", 0)
    monkeypatch.setattr(B, "_need_slots", lambda *a: None)
    slots = dict(ids=torch.zeros(2, 2, dtype=torch.int32), weights=torch.zeros(2, 2))
    for trained in ("logits", "bias", None):
        logits = torch.zeros(2, 4).as_subclass(Logits).requires_grad_(trained == "logits")
        bias = torch.zeros(4).as_subclass(Logits).requires_grad_(trained == "bias") if trained != "logits" else None
        if trained:
            with pytest.raises(B.Int8wError, match="moe_route has no backward"):
                moe_route(logits, 2, "sigmoid", bias, **slots)
        with torch.no_grad():
            moe_route(logits, 2, "sigmoid", bias, **slots)

    def host(rows, k):
        codes, scales = torch.zeros(rows, k // 2, dtype=torch.uint8), torch.zeros(rows, k // 32, dtype=torch.uint8)
        w = Mxfp4Weight.__new__(Mxfp4Weight)
        w._set(codes, scales, rows, k, codes.device, codes.data_ptr(), scales.data_ptr())
        return w
    weights = host(E * I, H), host(E * I, H), host(E * H, I)
    for trained in ("x", "weights", "x_resid", None):
        t = {"x": torch.zeros(2, H, dtype=bf), "weights": torch.zeros(2, 2), "x_resid": torch.zeros(2, H, dtype=bf)}
        if trained:
            t[trained].requires_grad_()
        call = lambda: moe_layer_routed(*weights, E, t["x"], torch.zeros(2, 2, dtype=torch.int32), t["weights"], t["x_resid"])  # noqa: E731
        if trained:
            with pytest.raises(B.Int8wError, match="moe_layer_routed has no backward"):
                call()
        with torch.no_grad():
            call()


def test_gemm_lora_makes_the_weights_device_current_for_its_product(monkeypatch):
    seen = []

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            seen.append(self.device)

        def __exit__(self, *exc):
            seen.append("back")
    monkeypatch.setattr(B, "_current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(B, "_need_pool", lambda *a: None)
    monkeypatch.setattr(B, "_add_in_place", lambda pool, x, ids, y: seen.append("adapters") or y)

    class Projection:
        in_features = k = out_features = rows = 16

        def __init__(self, index):
            self.device = torch.device("cuda", index)

        def gemm(self, x, y):
            seen.append("gemm")
            return y
    for cls in (B.Int8Weight, Mxfp4Weight):
        for index, want in ((0, [torch.device("cuda", 0), "gemm", "back", "adapters"]), (1, ["gemm", "adapters"])):
            del seen[:]
            assert cls.gemm_lora(Projection(index), None, None, None, "y") == "y"
            assert seen == want


def test_gemm_lora_refuses_rows_before_its_product():
    class Projection:
        in_features = k = 8
        out_features = rows = 8
        device = torch.device("cpu")

        def gemm(self, x, y):
            pytest.fail("the product was launched")
    bf, m = torch.bfloat16, (1 << 20) + 1
    pool = fake_pool(torch.zeros(1, 8, 8, dtype=bf), torch.zeros(1, 8, 8, dtype=bf))
    for cls in (B.Int8Weight, Mxfp4Weight):
        with pytest.raises(B.Int8wError, match="more than 2\\^20") as e:
            cls.gemm_lora(Projection(), torch.zeros(m, 8, dtype=bf), pool, torch.zeros(m, dtype=torch.int32))
        assert e.value.code == SHAPE


@pytest.mark.parametrize("num,k,n,shift,code,text", [
    (0, 16, 24, 0, NULL, "missing a tensor"), (2, 1 << 20, 24, 0, SHAPE, "below 2^20"), (2, 16, 1 << 20, 0, SHAPE, "below 2^20"),
    (2, 16, 24, 4, ALIGN, "a or b"), (2, 16, 24, 0, None, ""),
])
def test_a_pool_that_no_call_takes_is_not_made(num, k, n, shift, code, text):
    class Gpu(torch.Tensor):  # as if on a GPU
        device = torch.device("cuda", 0)

    def zeros(*shape):
        count = shape[0] * shape[1] * shape[2]
        return torch.zeros(count + 16, dtype=torch.bfloat16)[shift:shift + count].view(shape).as_subclass(Gpu)
    if code is None:
        assert LoraAdapters(zeros(num, 8, k), zeros(num, n, 8)).num_adapters == num
        return
    with pytest.raises(B.Int8wError) as e:
        LoraAdapters(zeros(num, 8, k), zeros(num, n, 8))
    assert e.value.code == code and text in str(e.value)
