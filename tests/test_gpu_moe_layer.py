"""The mixture-of-experts layer against its 64-bit definition, within limits counted from the fp32 arithmetic and
the BF16 rounding of the inner product (tests/mx_reference.py).  Every test prints its case first."""
import numpy as np
import pytest
import torch

import mx_reference as R
from helpers import bits_to_dev, dev_to_bits
from weight_only_quantized_int8_amd import Int8Weight, Int8wError, Mxfp4Weight, moe_layer

pytestmark = pytest.mark.gpu


def log(msg):
    print(msg, flush=True)


def bits_of(x):
    return R.bf16_bits(np.asarray(x, np.float32))


class Layer:
    """Random experts in one of the formats, on the GPU and in float64."""

    def __init__(self, seed, fmt, E, I, H):
        rng = np.random.default_rng(seed)
        self.E, self.I, self.H = E, I, H
        self.gpu, self.ref, self.mag = [], [], []
        for n, k in ((E * I, H), (E * I, H), (E * H, I)):
            if fmt == "mxfp4":
                codes = rng.integers(0, 256, (n, k // 2), np.uint8)
                scales = rng.integers(117, 122, (n, k // 32), np.uint8)
                self.gpu.append(Mxfp4Weight(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()))
                w = R.decode(codes, scales)
                mag = np.abs(w)
            else:
                gs = int(fmt[2:])
                codes = rng.integers(0, 256, (n, k), np.uint8)
                s = bits_of(rng.uniform(1e-4, 4e-4, (n, k // gs)))
                b = bits_of(-128 * R.bf16_values(s) * (1 + rng.uniform(-0.05, 0.05, s.shape)))
                self.gpu.append(Int8Weight.from_arrays(codes.view(np.uint32), s, b, gs))
                w, mag = R.affine_weight(codes, s, b, gs)
            self.ref.append(w.reshape(E, n // E, k))
            self.mag.append(mag.reshape(E, n // E, k))

    def run(self, x, logits, topk, **kw):
        return moe_layer(*self.gpu, self.E, x, logits, topk, **kw)

    def want(self, x, logits, topk, renormalize=True, routed_scale=1.0, x_resid=None):
        return R.moe(x, *self.ref, self.mag, logits, topk, renormalize, routed_scale, x_resid)


def inputs(seed, T, H, E, bf16_logits=False, mask=0.0):
    rng = np.random.default_rng(seed)
    xb = bits_of(rng.standard_normal((T, H)))
    l = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    l[rng.random((T, E)) < mask] = -np.inf
    if bf16_logits:
        lb = np.where(np.isinf(l), np.uint16(0xFF80), bits_of(np.where(np.isinf(l), 0, l)))
        return xb, bits_to_dev(lb), np.where(lb == 0xFF80, -np.inf, R.bf16_values(lb))
    return xb, torch.from_numpy(l).cuda(), l.astype(np.float64)


def check(y, ref, lim, what):
    y = R.bf16_values(dev_to_bits(y))
    assert np.array_equal(np.isnan(y), np.isnan(ref)), what
    ok = (np.abs(y - ref) <= lim) | np.isnan(ref)
    assert ok.all(), f"{what}: {np.count_nonzero(~ok)} of {ok.size} outside; first {np.argwhere(~ok)[0]} " \
                     f"got {y[~ok][0]} want {ref[~ok][0]} within {lim[~ok][0]}"


FORMATS = ["mxfp4", "gs32", "gs64", "gs128"]

CASES = [  # T, E, topk, I, H
    (1, 1, 1, 128, 128), (1, 4, 2, 256, 384), (1, 8, 8, 384, 128), (1, 70, 6, 128, 256), (1, 200, 4, 128, 128),
    (1, 4, 2, 1152, 2176), (2, 4, 2, 256, 384), (3, 60, 6, 128, 256), (8, 4, 4, 128, 640), (17, 2, 2, 128, 256),
    (13, 130, 8, 128, 128), (64, 5, 3, 256, 128), (65, 8, 2, 128, 256), (130, 3, 1, 128, 128), (5, 512, 16, 128, 128),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,topk,I,H", CASES)
def test_layer(fmt, T, E, topk, I, H):
    log(f"layer {fmt} T={T} E={E} topk={topk} I={I} H={H}")
    L = Layer(T + E + I + H, fmt, E, I, H)
    xb, ld, l = inputs(T * 3 + E, T, H, E)
    renorm = (T + E) % 2 == 0
    y = L.run(bits_to_dev(xb), ld, topk, renormalize=renorm)
    ref, lim = L.want(R.bf16_values(xb), l, topk, renorm)
    check(y, ref, lim, "layer")
    again = L.run(bits_to_dev(xb), ld, topk, renormalize=renorm)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("fmt,I,H", [("mxfp4", 96, 160), ("mxfp4", 32, 32), ("mxfp4", 544, 1056), ("gs32", 96, 160),
                                     ("gs32", 32, 32), ("gs64", 192, 320), ("gs32", 1056, 2080)])
@pytest.mark.parametrize("T", [1, 2, 6, 40])
def test_odd_sizes(fmt, I, H, T):
    log(f"odd sizes {fmt} I={I} H={H} T={T}")
    L = Layer(I + H, fmt, 6, I, H)
    xb, ld, l = inputs(T, T, H, 6, bf16_logits=True)
    ref, lim = L.want(R.bf16_values(xb), l, 3)
    check(L.run(bits_to_dev(xb), ld, 3), ref, lim, "layer")


@pytest.mark.parametrize("fmt", ["mxfp4", "gs64"])
@pytest.mark.parametrize("T", [1, 7, 33])
def test_masks_ties_and_rows_with_nothing(fmt, T):
    log(f"masks {fmt} T={T}")
    E, I, H = 9, 128, 256
    L = Layer(5, fmt, E, I, H)
    xb, ld, l = inputs(T, T, H, E, mask=0.5)
    rows = [np.full(E, -np.inf), np.zeros(E), np.full(E, np.finfo(np.float32).min), np.array([0.0, np.nan] + [0.0] * (E - 2)),
            np.array([np.inf] + [0.0] * (E - 1)), np.array([-np.inf] * (E - 1) + [2.0]), np.array([500.0] + [-500.0] * (E - 1))]
    for shift in range(0, len(rows), T if T < len(rows) else len(rows)):
        l2 = l.copy()
        for t, r in enumerate(rows[shift:shift + T]):
            l2[t] = r
        for renorm in (True, False):
            ref, lim = L.want(R.bf16_values(xb), l2, 4, renorm)
            y = L.run(bits_to_dev(xb), torch.from_numpy(l2.astype(np.float32)).cuda(), 4, renormalize=renorm)
            check(y, ref, lim, f"shift {shift} renorm {renorm}")
            empty = (l2 == -np.inf).all(1)
            assert (dev_to_bits(y)[empty] == 0).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "gs32"])
@pytest.mark.parametrize("T", [1, 5, 70])
def test_residual_scale_and_in_place(fmt, T):
    log(f"residual {fmt} T={T}")
    E, I, H = 6, 128, 192
    L = Layer(8, fmt, E, I, H)
    xb, ld, l = inputs(T, T, H, E, mask=0.3)
    l[T // 2] = -np.inf  # this row gives the residual itself
    ld = torch.from_numpy(l.astype(np.float32)).cuda()
    rb = bits_of(np.random.default_rng(9).standard_normal((T, H)))
    for scale in (2.5, -1.0):
        ref, lim = L.want(R.bf16_values(xb), l, 2, True, scale, R.bf16_values(rb))
        r = bits_to_dev(rb)
        y = L.run(bits_to_dev(xb), ld, 2, routed_scale=scale, x_resid=r)
        check(y, ref, lim, f"residual, scale {scale}")
        assert np.array_equal(dev_to_bits(y)[T // 2], rb[T // 2])
        L.run(bits_to_dev(xb), ld, 2, routed_scale=scale, x_resid=r, y=r)
        assert torch.equal(r.view(torch.int16), y.view(torch.int16))
    y = L.run(bits_to_dev(xb), ld, 2, routed_scale=0.0, x_resid=bits_to_dev(rb))
    assert np.array_equal(dev_to_bits(y), rb)


def test_every_token_to_one_expert():
    # 64 tokens of one expert: four segments of it; the others idle
    log("one expert takes all")
    E, I, H, T = 8, 256, 128, 64
    for fmt in ("mxfp4", "gs64"):
        L = Layer(12, fmt, E, I, H)
        xb, _, l = inputs(1, T, H, E)
        l[:, 5] = 50.0
        ref, lim = L.want(R.bf16_values(xb), l, 1)
        check(L.run(bits_to_dev(xb), torch.from_numpy(l.astype(np.float32)).cuda(), 1), ref, lim, fmt)


def test_nan_weights_reach_only_their_tokens():
    log("nan weights")
    E, I, H, T = 4, 128, 128, 6
    rng = np.random.default_rng(3)
    mats = []
    for n, k in ((E * I, H), (E * I, H), (E * H, I)):
        c = torch.from_numpy(rng.integers(0, 256, (n, k // 2), np.uint8)).cuda()
        s = torch.full((n, k // 32), 119, dtype=torch.uint8, device="cuda")
        mats.append((c, s))
    mats[1][1][2 * I:3 * I] = 255  # expert 2's up projection is NaN
    W = [Mxfp4Weight(*m) for m in mats]
    l = torch.zeros(T, E, device="cuda")
    l[:, 0] = 3.0
    l[1, 2] = l[4, 2] = 9.0
    x = bits_to_dev(bits_of(rng.standard_normal((T, H))))
    for rows in (range(T), [0], [1]):
        rows = list(rows)
        y = moe_layer(*W, E, x[rows].contiguous(), l[rows].contiguous(), 1)
        assert torch.isnan(y.float()).all(1).tolist() == [r in (1, 4) for r in rows]


def test_long_rows_fall_back_from_the_one_token_form():
    # eight chosen experts' inner products do not fit the LDS of the one-token kernels
    log("one token, long rows")
    E, I, H = 8, 16384, 64
    L = Layer(21, "mxfp4", E, I, H)
    xb, ld, l = inputs(2, 1, H, E)
    ref, lim = L.want(R.bf16_values(xb), l, 8)
    check(L.run(bits_to_dev(xb), ld, 8), ref, lim, "layer")


@pytest.mark.parametrize("T", [1, 5, 24])
def test_expert_values_about_2_to_the_128(T):
    # the first block of every row under scale byte 254, against activations of about 2^-130: finite below 2^128;
    # expert 2's up projection has a value of 2^128 there, which is an infinity
    log(f"largest scales T={T}")
    E, I, H = 4, 128, 128
    rng = np.random.default_rng(50)
    gpu, ref = [], []
    for n, k, big in ((E * I, H, True), (E * I, H, True), (E * H, I, False)):
        q = rng.integers(0, 16, (n, k))
        scales = rng.integers(117, 122, (n, k // 32)).astype(np.uint8)
        if big:
            q[:, :32] = (q[:, :32] & 8) | rng.integers(1, 4, (n, 32))  # 0.5, 1, 1.5: up to 1.5 * 2^127
            scales[:, 0] = 254
        if len(gpu) == 1:
            q[2 * I + 5, 7] = 4  # 2 * 2^127
        codes = (q[:, 0::2] | q[:, 1::2] << 4).astype(np.uint8)
        gpu.append(Mxfp4Weight(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()))
        ref.append(R.decode(codes, scales).reshape(E, n // E, k))
    x = rng.standard_normal((T, H))
    x[:, :32] *= 2.0 ** -130
    xb = bits_of(x)
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[:, 2] = -np.inf
    for infinite in ([], [T // 2]):
        l[infinite, 2] = 9.0
        y = moe_layer(*gpu, E, bits_to_dev(xb), torch.from_numpy(l).cuda(), 2)
        want, lim = R.moe(R.bf16_values(xb), *ref, [np.abs(w) for w in ref], l.astype(np.float64), 2)
        y = R.bf16_values(dev_to_bits(y))
        keep = np.array([t not in infinite for t in range(T)])
        assert (np.abs(y - want)[keep] <= lim[keep]).all()
        assert not np.isfinite(y[~keep]).any()


@pytest.mark.parametrize("I", [2048, 2080, 4096, 4128])
@pytest.mark.parametrize("H", [96, 2048])
def test_one_token_about_64_kib_of_lds(I, H):
    # the chosen experts' inner products take 32, 64, 64 and 96 KiB, and the kernel has an array of its own
    log(f"one token I={I} H={H}")
    L = Layer(22, "mxfp4", 8, I, H)
    xb, ld, l = inputs(3, 1, H, 8)
    ref, lim = L.want(R.bf16_values(xb), l, 8)
    check(L.run(bits_to_dev(xb), ld, 8), ref, lim, "layer")


def test_experts_past_32_bits():
    # gate of 40 experts x 16384 x 8192: 5.4 GB of codes; the last experts are the ones taken
    log("large experts")
    E, I, H = 40, 16384, 8192
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    W = []
    for n, k in ((E * I, H), (E * I, H), (E * H, I)):
        codes = torch.randint(0, 256, (n, k), generator=g, device="cuda", dtype=torch.uint8)
        s = torch.full((n, k // 128), 2e-4, dtype=torch.bfloat16, device="cuda")
        W.append(Int8Weight(codes.view(torch.int32), s, -128 * s, 128))

    def deq(w, e, rows):
        c = w.packed[e * rows:(e + 1) * rows].contiguous().view(torch.uint8).double()
        return (c - 128) * float(torch.tensor(2e-4).bfloat16())
    for T in (1, 2):
        xb = bits_of(np.random.default_rng(T).standard_normal((T, H)))
        l = torch.full((T, E), -5.0, device="cuda")
        l[:, 38], l[:, 39] = 1.0, 2.0
        log(f"  T={T}")
        y = moe_layer(*W, E, bits_to_dev(xb), l, 2)
        x = torch.from_numpy(R.bf16_values(xb)).cuda()
        p = torch.softmax(torch.tensor([1.0, 2.0], dtype=torch.float64), 0).tolist()
        want = 0
        for r, e in zip(p, (38, 39)):
            a, u = x @ deq(W[0], e, I).t(), x @ deq(W[1], e, I).t()
            want = want + r * (a * torch.sigmoid(a) * u) @ deq(W[2], e, H).t()
        # the sum's rounding (2^-8 of y) and h's, which averages: 4 sigma of 2^-9 |h| |w| in quadrature, far below 2^-6 rms
        rms = want.square().mean().sqrt()
        assert ((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -6 * rms).all()


def test_another_stream_and_a_graph():
    log("stream and graph")
    E, I, H = 6, 256, 256
    for fmt, T in (("mxfp4", 1), ("gs64", 1), ("mxfp4", 20), ("gs32", 3)):
        L = Layer(30, fmt, E, I, H)
        xb, ld, _ = inputs(T, T, H, E)
        x = bits_to_dev(xb)
        want = L.run(x, ld, 2)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = L.run(x, ld, 2)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                gy = L.run(x, ld, 2)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        for i in range(4):
            xb, l2, _ = inputs(100 + i, T, H, E, mask=0.3)
            x.copy_(bits_to_dev(xb))
            ld.copy_(l2)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(gy.view(torch.int16), L.run(x, ld, 2).view(torch.int16)), (fmt, T, i)


def test_workspace_that_must_grow_during_capture(monkeypatch):
    log("capture without a cached workspace")
    from weight_only_quantized_int8_amd import binding
    L = Layer(31, "mxfp4", 4, 128, 128)
    xb, ld, _ = inputs(1, 3, 128, 4)
    x = bits_to_dev(xb)
    want = L.run(x, ld, 2)
    monkeypatch.setattr(binding, "_workspaces", {})
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            y = L.run(x, ld, 2)
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))


def test_graph_keeps_its_scratch_when_later_calls_need_more():
    log("a graph, then larger calls, then replays")
    E, I, H = 6, 256, 256
    L = Layer(32, "mxfp4", E, I, H)
    xb, ld, _ = inputs(1, 20, H, E)
    x = bits_to_dev(xb)
    want = L.run(x, ld, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            y = L.run(x, ld, 2)
    torch.cuda.synchronize()
    big = Layer(33, "mxfp4", 16, 8192, 128)
    xb2, ld2, _ = inputs(2, 64, 128, 16)
    keep = []
    for _ in range(3):
        keep.append(big.run(bits_to_dev(xb2), ld2, 16))
        keep.append(torch.full((40 << 20,), 7, dtype=torch.uint8, device="cuda"))
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))
        assert all((k == 7).all() for k in keep[1::2])
        assert torch.equal(keep[0].view(torch.int16), keep[-2].view(torch.int16))


def test_calls_that_overlap_on_streams():
    log("two streams at a time")
    E, I, H = 6, 512, 512
    layers = [Layer(34 + i, "mxfp4", E, I, H) for i in range(2)]
    data = [inputs(40 + i, 48, H, E) for i in range(2)]
    xs = [bits_to_dev(d[0]) for d in data]
    want = [L.run(x, d[1], 3) for L, x, d in zip(layers, xs, data)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(layers[i].run(xs[i], data[i][1], 3))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y.view(torch.int16), want[i].view(torch.int16)) for y in got[i])


def test_outputs_stay_inside_their_buffer_and_no_tokens():
    log("extent")
    E, I, H, T = 4, 128, 160, 3
    L = Layer(32, "gs32", E, I, H)
    xb, ld, _ = inputs(1, T, H, E)
    buf = torch.full((T * H + 64,), 77.0, dtype=torch.bfloat16, device="cuda")
    L.run(bits_to_dev(xb), ld, 2, y=buf[:T * H].view(T, H))
    torch.cuda.synchronize()
    assert (buf[T * H:] == 77.0).all()
    assert L.run(bits_to_dev(xb)[:0], ld[:0], 2).shape == (0, H)


def test_wrong_arguments_raise():
    log("refusals")
    E, I, H, T = 4, 128, 128, 2
    L = Layer(33, "mxfp4", E, I, H)
    Q = Layer(34, "gs64", E, I, H)
    xb, ld, _ = inputs(1, T, H, E)
    x = bits_to_dev(xb)
    with pytest.raises(TypeError):
        moe_layer(L.gpu[0], L.gpu[1], Q.gpu[2], E, x, ld, 2)
    for bad in (ld[:1], ld.double(), ld.t().contiguous().t(), ld.cpu()):
        with pytest.raises(ValueError):
            L.run(x, bad, 2)
    with pytest.raises(ValueError):
        L.run(x[:, :96], ld, 2)
    with pytest.raises(Int8wError, match="topk"):
        L.run(x, ld, 5)
    with pytest.raises(Int8wError, match="not 2 experts"):
        moe_layer(*L.gpu, 2, x, ld[:, :2].contiguous(), 1)
    with pytest.raises(Int8wError, match="overlaps"):
        L.run(x, ld, 2, y=x)
