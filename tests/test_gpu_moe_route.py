"""The routing to experts by itself, and the expert layer from a given routing, against their 64-bit definitions
(tests/adapter_reference.py).  Every test prints its case first."""
import numpy as np
import pytest
import torch

import adapter_reference as A
import mx_reference as R
from helpers import bits_to_dev, dev_to_bits
from test_gpu_moe_layer import Layer, bits_of, check, inputs
from weight_only_quantized_int8_amd import Int8wError, Mxfp4Weight, moe_gemv, moe_layer, moe_layer_routed, moe_route

pytestmark = pytest.mark.gpu


def log(msg):
    print(msg, flush=True)


def same(got, want, what):
    ids, w = got[0].cpu().numpy(), got[1].double().cpu().numpy()
    assert np.array_equal(ids, want[0]), f"{what}: rows {np.flatnonzero((ids != want[0]).any(1))[:5]}"
    # fp32: a score is off by its exponential (2^-23, and 2^-24 of the argument's size where a difference was rounded),
    # sum, quotient: 2^-21 together; the sum that divides it by as much again and an addition for each of up to 512
    # values, in 14 steps; quotient and factor: 2^-23.  Arguments here are below 2^4 where the weight is above
    # 2^-30 of the largest; what is far below that may be lost.
    lim = (2.0 ** -20 + 2.0 ** -19 + 2.0 ** -20) * np.abs(want[1]) + 2.0 ** -30 * np.abs(want[1]).max(initial=0.0, where=~np.isnan(want[1]))
    assert np.array_equal(np.isnan(w), np.isnan(want[1])), what
    assert ((np.abs(w - want[1]) <= lim) | np.isnan(w)).all(), what


SIZES = [  # T, E, topk, groups, topk_groups
    (1, 1, 1, 1, 1), (1, 8, 2, 1, 1), (3, 2, 2, 2, 2), (5, 60, 4, 1, 1), (4, 60, 6, 6, 3), (9, 64, 16, 1, 1), (1, 65, 8, 1, 1), (7, 64, 6, 64, 9),
    (130, 128, 8, 8, 4), (6, 160, 6, 8, 3), (33, 200, 5, 8, 1), (64, 256, 8, 8, 4), (5, 500, 10, 20, 7), (17, 512, 16, 16, 16), (2, 512, 3, 2, 1),
]


@pytest.mark.parametrize("T,E,topk,groups,topk_groups", SIZES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_against_the_definition(T, E, topk, groups, topk_groups, scoring, biased):
    log(f"route T={T} E={E} topk={topk} groups={groups}/{topk_groups} {scoring} biased={biased}")
    for i, group_score in enumerate(("max", "top2")):
        for bf16, mask in ((False, 0.0), (True, 0.0), (False, 0.4), (True, 0.9)):
            _, ld, l = inputs(T + E + i, T, 8, E, bf16, mask)
            rng = np.random.default_rng(E)
            bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if biased else None
            renorm, scale = bool((T + i) % 2), 1.0 if bf16 else 2.5
            got = moe_route(ld, topk, scoring, torch.from_numpy(bias).cuda() if biased else None, groups, topk_groups, group_score,
                            renorm, scale)
            same(got, A.route(l, topk, scoring, bias, groups, topk_groups, group_score, renorm, scale), (group_score, bf16, mask))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_rows_with_nothing_ties_and_odd_values(scoring, groups):
    log(f"odd rows {scoring} groups={groups}")
    E, inf, nan = 12, np.inf, np.nan
    rows = [np.full(E, -inf), np.zeros(E), np.full(E, np.finfo(np.float32).min), np.full(E, np.finfo(np.float32).max),
            np.array([0, nan] + [0] * (E - 2)), np.array([nan] * E), np.array([-inf] * (E - 1) + [nan]), np.array([inf] + [0] * (E - 1)),
            np.array([0, inf, -inf, inf] + [1] * (E - 4)), np.array([-inf] * (E - 1) + [2.0]), np.array([-inf] * (E - 1) + [-3000.0]),
            np.array([500.0] + [-500.0] * (E - 1)), np.arange(E) % 3 * 1.0, np.array([-0.0, 0.0] * (E // 2)), np.array([-200.0] * E),
            np.array([30.0, 40.0, 50.0, 60.0] * (E // 4))]
    l = np.array(rows, np.float32)
    ld = torch.from_numpy(l).cuda()
    for bias in (None, np.zeros(E, np.float32), np.array([0.25, -0.5] * (E // 2), np.float32), np.array([inf] + [0] * (E - 2) + [-inf], np.float32),
                 np.array([0, nan] + [0] * (E - 2), np.float32), np.full(E, -inf, np.float32)):
        for group_score in ("max", "top2"):
            for renorm in (True, False):
                got = moe_route(ld, 5, scoring, None if bias is None else torch.from_numpy(bias).cuda(), groups, max(1, groups // 2 + 1),
                                group_score, renorm, 0.5)
                same(got, A.route(l.astype(np.float64), 5, scoring, bias, groups, max(1, groups // 2 + 1), group_score, renorm, 0.5),
                     (bias, group_score, renorm))


def test_choices_do_not_hang_on_a_rounding():
    # scores one unit of fp32 and less apart once biased: fp32 sums would tie or swap them
    log("close scores")
    rng = np.random.default_rng(3)
    T, E = 500, 64
    l = (0.5 + 2.0 ** -22 * rng.integers(0, 40, (T, E))).astype(np.float32)
    bias = (16.0 + 2.0 ** -19 * rng.integers(0, 2, E)).astype(np.float32)
    got = moe_route(torch.from_numpy(l).cuda(), 8, "sigmoid", torch.from_numpy(bias).cuda(), 8, 4)
    same(got, A.route(l.astype(np.float64), 8, "sigmoid", bias, 8, 4), "close")


def test_many_tokens_outputs_given_and_their_extent():
    log("extent")
    T, E, topk = 1003, 64, 3
    _, ld, l = inputs(1, T, 8, E, mask=0.2)
    ids = torch.full((T + 1, topk), 7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, topk), 7.0, device="cuda")
    got = moe_route(ld, topk, ids=ids[:T], weights=w[:T])
    assert got[0].data_ptr() == ids.data_ptr() and got[1].data_ptr() == w.data_ptr()
    same(got, A.route(l, topk), "given outputs")
    assert (ids[T] == 7).all() and (w[T] == 7).all()
    empty = moe_route(ld[:0], topk)
    assert empty[0].shape == (0, topk) and empty[1].shape == (0, topk)
    ids16 = moe_route(ld, topk, ids=ids[:T].view(torch.uint32))[0]
    assert ids16.dtype == torch.uint32


def routed_want(L, xb, ids, w, resid=None):
    return A.experts(R.bf16_values(xb), *L.ref, L.mag, ids.cpu().numpy().astype(np.int64), w.double().cpu().numpy(), resid)


@pytest.mark.parametrize("fmt", ["mxfp4", "gs32", "gs64"])
@pytest.mark.parametrize("T,E,topk,I,H", [(1, 1, 1, 128, 128), (1, 8, 3, 256, 384), (1, 70, 16, 128, 256), (2, 4, 2, 256, 384), (9, 60, 6, 128, 256),
                                          (65, 8, 2, 128, 256), (130, 5, 4, 192, 320), (1, 3, 2, 192, 320)])
def test_router_then_experts(fmt, T, E, topk, I, H):
    log(f"routed layer {fmt} T={T} E={E} topk={topk} I={I} H={H}")
    L = Layer(T + E + I, fmt, E, I, H)
    xb, ld, _ = inputs(T + E, T, H, E, mask=0.3)
    bias = torch.from_numpy((0.1 * np.random.default_rng(E).standard_normal(E)).astype(np.float32)).cuda()
    ids, w = moe_route(ld, topk, "sigmoid", bias, routed_scale=2.0)
    x = bits_to_dev(xb)
    y = moe_layer_routed(*L.gpu, E, x, ids, w)
    check(y, *routed_want(L, xb, ids, w), "routed")
    assert torch.equal(y.view(torch.int16), moe_layer_routed(*L.gpu, E, x, ids, w).view(torch.int16))
    rb = bits_of(np.random.default_rng(9).standard_normal((T, H)))
    r = bits_to_dev(rb)
    moe_layer_routed(*L.gpu, E, x, ids, w, x_resid=r, y=r)
    check(r, *routed_want(L, xb, ids, w, R.bf16_values(rb)), "in place")
    # the softmax routing from outside: the layer's own limits
    ids, w = moe_route(ld, topk)
    ref, lim = L.want(R.bf16_values(xb), ld.double().cpu().numpy(), topk)
    check(moe_layer_routed(*L.gpu, E, x, ids, w), ref, lim, "softmax")


@pytest.mark.parametrize("fmt", ["mxfp4", "gs64"])
@pytest.mark.parametrize("T", [1, 12, 70])
def test_given_routings_of_any_kind(fmt, T):
    # holes, one expert twice and three times, weights of both signs, sums of 0, NaN and ids far outside
    log(f"given routings {fmt} T={T}")
    E, I, H, topk = 6, 128, 192, 7
    L = Layer(4, fmt, E, I, H)
    rng = np.random.default_rng(T)
    xb = bits_of(rng.standard_normal((T, H)))
    special = [([-1, 2, -1, 0, 6, 2, 5], [1.0, 0.5, 2.0, -0.75, 9.0, 0.25, 0.0]), ([3] * 7, [0.5, -0.25, 1.0, 0.0, 0.0, 0.125, 2.0]),
               ([1, 4, 1, 4, 1, 4, -1], [0.5, 0.5, -0.5, 0.25, 0.0, -0.75, 1.0]), ([-1] * 7, [1.0] * 7), ([0, 1, 2, 3, 4, 5, 6], [0.0] * 7),
               ([0, 1, 2, 3, 4, 5, -1], [0.1, 0.2, 0.3, 0.4, 0.5, 0.6, np.nan]), ([5, 1, 2, 3, 4, 0, -(1 << 31)], [1.0] * 7)]
    for shift in range(len(special) if T == 1 else 1):
        ids = rng.integers(-1, E + 1, (T, topk)).astype(np.int32)
        w = rng.standard_normal((T, topk)).astype(np.float32)
        for t, (i, v) in enumerate(special[shift:shift + T]):
            ids[t], w[t] = i, v
        di, dw = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
        y = moe_layer_routed(*L.gpu, E, bits_to_dev(xb), di, dw)
        check(y, *routed_want(L, xb, di, dw), f"shift {shift}")


def test_route_then_expert_products():
    # the ids as moe_gemv takes them: a slot without an expert is NaN there
    log("route, then moe_gemv")
    from weight_only_quantized_int8_amd import Int8Weight
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    E, N, K, T, topk = 6, 64, 256, 5, 3
    W = Int8Weight.quantize(torch.randn((E * N, K), generator=g, device="cuda").bfloat16(), 64)
    x = torch.randn((T, 1, K), generator=g, device="cuda").bfloat16()
    logits = torch.randn((T, E), generator=g, device="cuda")
    logits[2, 1:] = -float("inf")
    ids, w = moe_route(logits, topk, "sigmoid")
    y = moe_gemv(W, E, x, ids).double()
    dense = W.dequantize_to().double().view(E, N, K)
    for t in range(T):
        for j in range(topk):
            e = int(ids[t, j])
            if e < 0:
                assert torch.isnan(y[t, j]).all() and float(w[t, j]) == 0
            else:  # the weight's own BF16 rounding apart, within the product's rounding: 2^-8 each
                ref, mag = dense[e] @ x[t, 0].double(), dense[e].abs() @ x[t, 0].double().abs()
                assert ((y[t, j] - ref).abs() <= 2.0 ** -7 * ref.abs() + 2.0 ** -8 * mag).all()
    assert (ids[2] >= 0).sum() == 1


def test_another_stream_and_a_graph():
    log("route and layer: stream and graph")
    E, I, H, topk = 8, 256, 256, 3
    for fmt, T in (("mxfp4", 1), ("gs64", 20), ("mxfp4", 70)):
        L = Layer(30, fmt, E, I, H)
        xb, ld, _ = inputs(T, T, H, E)
        x, bias = bits_to_dev(xb), torch.linspace(-0.1, 0.1, E, device="cuda")

        def step():
            ids, w = moe_route(ld, topk, "sigmoid", bias, 4, 2, routed_scale=2.5)
            return moe_layer_routed(*L.gpu, E, x, ids, w, x_resid=x)
        want = step()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = step()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                gy = step()
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        for i in range(4):
            xb, l2, _ = inputs(100 + i, T, H, E, mask=0.3)
            x.copy_(bits_to_dev(xb))
            ld.copy_(l2)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(gy.view(torch.int16), step().view(torch.int16)), (fmt, T, i)


def test_wrong_arguments_raise():
    log("refusals")
    E, I, H, T = 4, 128, 128, 2
    L = Layer(33, "mxfp4", E, I, H)
    xb, ld, _ = inputs(1, T, H, E)
    x = bits_to_dev(xb)
    ids, w = moe_route(ld, 2)
    for bad in (ld.double(), ld.t().contiguous().t(), ld.cpu(), ld[0]):
        with pytest.raises(ValueError, match="logits"):
            moe_route(bad, 2)
    with pytest.raises(ValueError, match="scoring"):
        moe_route(ld, 2, "tanh")
    with pytest.raises(ValueError, match="bias"):
        moe_route(ld, 2, bias=torch.zeros(3, device="cuda"))
    for kw in (dict(groups=3), dict(groups=4, topk_groups=5), dict(groups=4, topk_groups=1)):
        with pytest.raises(Int8wError):
            moe_route(ld, 2, **kw)
    for k in (0, 5, 17):
        with pytest.raises(Int8wError, match="topk"):
            moe_route(ld, k)
    with pytest.raises(ValueError, match="ids must be"):
        moe_layer_routed(*L.gpu, E, x, ids.long(), w)
    with pytest.raises(ValueError, match="weights must be"):
        moe_layer_routed(*L.gpu, E, x, ids, w[:1])
    with pytest.raises(Int8wError, match="not 2 experts"):
        moe_layer_routed(*L.gpu, 2, x, ids, w)
    with pytest.raises(Int8wError, match="overlaps"):
        moe_layer_routed(*L.gpu, E, x, ids, w, y=x)
    with pytest.raises(TypeError):
        moe_layer_routed(L.gpu[0], L.gpu[1], None, E, x, ids, w)
    assert moe_layer_routed(*L.gpu, E, x[:0], ids[:0], w[:0]).shape == (0, H)
    assert torch.isfinite(moe_layer(*L.gpu, E, x, ld, 2).float()).all() and isinstance(L.gpu[0], Mxfp4Weight)
    assert dev_to_bits(x).shape == (T, H)
