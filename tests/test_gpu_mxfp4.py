"""MXFP4 on the GPU against the 64-bit definition: quantization bit for bit, products within limits counted from
the fp32 arithmetic (tests/mx_reference.py).  Every test prints its case first."""
import numpy as np
import pytest
import torch

import mx_reference as R
from helpers import bits_to_dev, dev_to_bits
from weight_only_quantized_int8_amd import Mxfp4Weight
from weight_only_quantized_int8_amd import binding as B

pytestmark = pytest.mark.gpu


def log(msg):
    print(msg, flush=True)


def bits_of(x):
    return R.bf16_bits(x.astype(np.float32))


def to_dev(x, dtype):
    if dtype == "f32":
        return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()
    return bits_to_dev(bits_of(x))


def rounded(x, dtype):
    return x.astype(np.float32).astype(np.float64) if dtype == "f32" else R.bf16_values(bits_of(x))


def matrix(seed, rows, k, lo=110, hi=140):
    """Random codes and scales; every tenth block zero scale byte region is left to other tests."""
    rng = np.random.default_rng(seed)
    return rng.integers(0, 256, (rows, k // 2), np.uint8), rng.integers(lo, hi, (rows, k // 32), np.uint8)


def weight(codes, scales):
    return Mxfp4Weight(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())


def check(y, ref, lim, what):
    y = R.bf16_values(dev_to_bits(y))
    assert (np.isnan(y) == np.isnan(ref)).all(), what
    ok = np.abs(y - ref) <= lim + 1e-300
    ok |= np.isnan(ref)
    assert ok.all(), f"{what}: {np.count_nonzero(~ok)} of {ok.size} outside; first {np.argwhere(~ok)[0]} " \
                     f"got {y[~ok][0]} want {ref[~ok][0]} within {lim[~ok][0]}"


# ---- quantize, dequantize ---------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 32), (3, 96), (16, 4096), (5, 2080), (257, 1056), (1, 28672), (1000, 64)])
def test_quantize_bit_exact(rows, k, dtype):
    log(f"quantize {rows}x{k} {dtype}")
    rng = np.random.default_rng(rows * 7 + k)
    x = rng.standard_normal((rows, k)) * 2.0 ** rng.integers(-20, 20, (rows, 1))
    x[rows // 2, :32] = 0
    x[0, :8] = [1.0, -0.25, 0.75, 2.5, -3.5, 5.0, 7.0, -0.0]
    codes, scales = R.encode(rounded(x, dtype))
    q = Mxfp4Weight.quantize(to_dev(x, dtype))
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    back = dev_to_bits(q.dequantize_to())
    assert np.array_equal(R.bf16_values(back), R.decode(codes, scales))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_special_blocks(dtype):
    log(f"quantize special blocks {dtype}")
    inf, nan = np.inf, np.nan
    rows = []
    for v in (0.0, -0.0, 2.0 ** -133, 2.0 ** -126, -2.0 ** -124, 1.5 * 2.0 ** -123, 2.0 ** 127, -1.9921875 * 2.0 ** 127,
              inf, -inf, nan):
        r = np.zeros(64)
        r[17] = v
        r[40:] = -1.5  # the second block, untouched by the first
        rows.append(r)
    for e in range(-126, 128, 11):  # every code's midpoints under this scale
        r = np.zeros(64)
        r[:15] = np.array([4, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 7, 0.249, 0.251, 4.99, 5.01, -5, -.75]) * 2.0 ** (e - 2)
        rows.append(r)
    x = np.array(rows)
    codes, scales = R.encode(np.where(np.isfinite(x), rounded(np.where(np.isfinite(x), x, 0), dtype), x))
    if dtype == "f32":
        d = torch.from_numpy(x.astype(np.float32)).cuda()
    else:
        b = bits_of(np.where(np.isfinite(x), x, 0))
        b[x == inf], b[x == -inf], b[np.isnan(x)] = 0x7F80, 0xFF80, 0x7FC0
        d = bits_to_dev(b)
    q = Mxfp4Weight.quantize(d)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)


def test_dequantize_every_byte_and_scale():
    log("dequantize all codes and scales")
    codes = np.tile(np.repeat(np.arange(256, dtype=np.uint8)[None], 1, 0), (256, 1))  # [256, 256] -> k = 512
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    got = R.bf16_values(dev_to_bits(weight(codes, scales).dequantize_to()))
    want = R.decode(codes, scales)
    want = np.where(np.abs(want) >= 2.0 ** 128, np.sign(want) * np.inf, want)  # beyond BF16
    assert np.array_equal(got, want, equal_nan=True)


def test_outputs_stay_inside_their_buffers():
    log("output extents")
    rows, k, m = 37, 160, 3
    codes, scales = matrix(1, rows, k)
    w = weight(codes, scales)
    x = bits_to_dev(bits_of(np.random.default_rng(2).standard_normal((m, k))))
    for n, run in ((rows * k, lambda b: w.dequantize_to(b.view(rows, k))), (m * rows, lambda b: w.gemm(x, b.view(m, rows))),
                   (m * rows, lambda b: w.gemm_mx(Mxfp4Weight.quantize(x), b.view(m, rows)))):
        buf = torch.full((n + 64,), 77.0, dtype=torch.bfloat16, device="cuda")
        run(buf[:n])
        torch.cuda.synchronize()
        assert (buf[n:] == 77.0).all() and not (buf[:n] == 77.0).all()


# ---- products ---------------------------------------------------------------------------------

# every kernel and both sides of each switch: one row, few rows (1, 2, 4 loads of activations), 17..64 rows, tiles;
# K below a piece, off the 128- and 512-k steps; N off the 16-row tiles
SHAPES = [(1, 1, 32), (1, 77, 64), (1, 4096, 4096), (1, 1025, 4128), (1, 300, 28672), (1, 33, 36896), (1, 8, 90016),
          (2, 50, 96), (4, 1024, 4096), (5, 130, 544), (8, 4096, 1024), (9, 77, 2080), (16, 513, 4096), (16, 40, 14336),
          (17, 100, 1056), (32, 260, 4096), (64, 1000, 608), (33, 7, 8192), (65, 70, 96), (96, 300, 2080), (128, 1024, 1024),
          (130, 259, 4128), (300, 1024, 512), (513, 129, 672), (700, 2304, 256),
          # 64 x 32 tiles, and 64 x 64 / 64 x 128, with every edge ragged: K off 128 and off 512, one to nine groups
          (130, 1501, 4128), (100, 1790, 608), (513, 513, 2080), (70, 2501, 32), (700, 2301, 1056)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm(m, n, k):
    log(f"gemm m={m} n={n} k={k}")
    codes, scales = matrix(m + n + k, n, k)
    x = np.random.default_rng(k).standard_normal((m, k)) * 3
    xb = bits_of(x)
    w, xd = weight(codes, scales), bits_to_dev(xb)
    y = w.gemm(xd)
    ref, lim = R.product(R.bf16_values(xb), R.decode(codes, scales))
    check(y, ref, lim, f"gemm {m}x{n}x{k}")
    assert torch.equal(y.view(torch.int16), w.gemm(xd).view(torch.int16))


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm_mx(m, n, k):
    log(f"gemm_mx m={m} n={n} k={k}")
    codes, scales = matrix(m + n + k, n, k)
    xc, xs = matrix(m * n + 1, m, k)
    w, x = weight(codes, scales), weight(xc, xs)
    y = w.gemm_mx(x)
    ref, lim = R.product(R.decode(xc, xs), R.decode(codes, scales))
    check(y, ref, lim, f"gemm_mx {m}x{n}x{k}")
    assert torch.equal(y.view(torch.int16), w.gemm_mx(x).view(torch.int16))


@pytest.mark.parametrize("m,n,k", [(1000, 2700, 1024), (520, 14336, 256)])
def test_large_tiles(m, n, k):
    log(f"large tiles m={m} n={n} k={k}")
    codes, scales = matrix(9, n, k)
    xb = bits_of(np.random.default_rng(3).standard_normal((m, k)))
    w = weight(codes, scales)
    W = R.decode(codes, scales)
    ref, lim = R.product(R.bf16_values(xb), W)
    check(w.gemm(bits_to_dev(xb)), ref, lim, "gemm")
    q = Mxfp4Weight.quantize(bits_to_dev(xb))
    qx = R.decode(*R.encode(R.bf16_values(xb)))
    ref, lim = R.product(qx, W)
    check(w.gemm_mx(q), ref, lim, "gemm_mx")


@pytest.mark.parametrize("m", [1, 3, 9, 20, 70, 300])
def test_nan_scale_stays_in_its_row(m):
    log(f"nan scale m={m}")
    n, k = 90, 736
    codes, scales = matrix(4, n, k)
    scales[17, 5] = 255
    scales[88, 22] = 255  # the last block of a row: the next row's must not see it
    xb = bits_of(np.random.default_rng(5).standard_normal((m, k)))
    w = weight(codes, scales)
    ref, lim = R.product(R.bf16_values(xb), R.decode(codes, scales))
    check(w.gemm(bits_to_dev(xb)), ref, lim, "gemm")
    xc, xs = matrix(6, m, k)
    xs[m // 2, 3] = 255
    ref, lim = R.product(R.decode(xc, xs), R.decode(codes, scales))
    check(w.gemm_mx(weight(xc, xs)), ref, lim, "gemm_mx")


@pytest.mark.parametrize("m", [1, 4, 40, 200])
def test_extreme_scales_and_activations(m):
    # scale bytes 0 and 250, activations near the ends of BF16: products stay exact, sums finite
    log(f"extremes m={m}")
    n, k = 48, 256
    codes, scales = matrix(7, n, k, 0, 3)
    xb = bits_of(np.random.default_rng(8).standard_normal((m, k)) * 2.0 ** 100)
    ref, lim = R.product(R.bf16_values(xb), R.decode(codes, scales))
    check(weight(codes, scales).gemm(bits_to_dev(xb)), ref, lim, "small scales")
    codes, scales = matrix(7, n, k, 245, 250)
    xb = bits_of(np.random.default_rng(8).standard_normal((m, k)) * 2.0 ** -60)
    ref, lim = R.product(R.bf16_values(xb), R.decode(codes, scales))
    check(weight(codes, scales).gemm(bits_to_dev(xb)), ref, lim, "large scales")


def largest_scales(seed, n, k):
    """Scale bytes 253 and 254 with magnitudes below 2^128 in the even rows, any in the odd ones."""
    rng = np.random.default_rng(seed)
    scales = rng.integers(253, 255, (n, k // 32)).astype(np.uint8)
    q = rng.integers(0, 8, (n, k))
    most = np.where(np.repeat(scales, 32, 1) == 253, 6, 4)  # codes of 4 and of 2: the first that are not below
    q = np.where((np.arange(n) % 2 == 0)[:, None], q % most, q) + 8 * rng.integers(0, 2, (n, k))
    return (q[:, 0::2] | q[:, 1::2] << 4).astype(np.uint8), scales


@pytest.mark.parametrize("m", [1, 2, 7, 16, 30, 100, 600])
def test_values_about_2_to_the_128(m):
    # with X in BF16 a value from 2^128 on is infinity, as fp32 and dequantize_to have it; with X in MXFP4 it is exact
    log(f"largest scales m={m}")
    n, k = 120, 320
    codes, scales = largest_scales(41, n, k)
    w, exact = weight(codes, scales), R.decode(codes, scales)
    W = np.where(np.abs(exact) >= 2.0 ** 128, np.copysign(np.inf, exact), exact)
    assert np.isfinite(W[::2]).all() and np.isinf(W[1::2]).any(1).all()
    assert np.array_equal(R.bf16_values(dev_to_bits(w.dequantize_to())), W)
    x = np.random.default_rng(m).standard_normal((m, k)) * 2.0 ** -40
    x[m // 2, ::3] = 0.0  # 0 times infinity
    x[0] = np.abs(x[0]) * np.where(exact[1] < 0, -1, 1)  # row 1: infinities of one sign
    xb = bits_of(x)
    X = R.bf16_values(xb)
    with np.errstate(invalid="ignore"):
        inf = np.array([[np.sum(a * b) for b in W] for a in X])
    ref, lim = R.product(X, np.where(np.isinf(W), 0.0, W))
    y = R.bf16_values(dev_to_bits(w.gemm(bits_to_dev(xb))))
    assert np.array_equal(np.isnan(y), np.isnan(inf)) and np.array_equal(np.isinf(y), np.isinf(inf))
    assert np.array_equal(np.sign(y[np.isinf(y)]), np.sign(inf[np.isinf(inf)]))
    ok = np.isfinite(inf)
    assert ok[:, ::2].all() and np.isnan(inf).any() and (m == 1 or np.isinf(inf).any())
    assert (np.abs(y - ref)[ok] <= lim[ok]).all()
    xc, xs = matrix(42, m, k, 80, 90)
    ref, lim = R.product(R.decode(xc, xs), exact)
    check(w.gemm_mx(weight(xc, xs)), ref, lim, "gemm_mx")


@pytest.mark.parametrize("m", [1, 2, 12, 30, 100])
def test_scales_of_any_alignment(m):
    log(f"unaligned scales m={m}")
    n, k = 70, 1024
    codes, scales = matrix(11, n, k)
    buf = torch.zeros(n * (k // 32) + 3, dtype=torch.uint8, device="cuda")
    for off in (1, 2, 3):
        s = buf[off:off + scales.size].view(n, k // 32)
        s.copy_(torch.from_numpy(scales))
        w = Mxfp4Weight(torch.from_numpy(codes).cuda(), s)
        xb = bits_of(np.random.default_rng(12).standard_normal((m, k)))
        ref, lim = R.product(R.bf16_values(xb), R.decode(codes, scales))
        check(w.gemm(bits_to_dev(xb)), ref, lim, f"offset {off}")
        q = Mxfp4Weight.quantize(bits_to_dev(xb))
        xs = torch.zeros(q.scales.numel() + 3, dtype=torch.uint8, device="cuda")[off:off + q.scales.numel()].view_as(q.scales)
        xs.copy_(q.scales)
        a, b = w.gemm_mx(q), w.gemm_mx(Mxfp4Weight(q.codes, xs))
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("off", [0, 1, 2])
@pytest.mark.parametrize("m,n", [(130, 1501), (700, 2301), (1000, 2700)])
def test_tiles_with_nan_scales_of_any_alignment(m, n, off):
    # 64 x 32, 64 x 64 (64 x 128) and large tiles; K = 736: 23 scale bytes a row, so every row's start differs
    log(f"tiles m={m} n={n} offset {off}")
    k = 736
    codes, scales = matrix(31, n, k)
    scales[n // 3, 5] = 255
    scales[n - 2, 22] = 255  # the last block of a row
    s = torch.zeros(scales.size + 3, dtype=torch.uint8, device="cuda")[off:off + scales.size].view(n, k // 32)
    s.copy_(torch.from_numpy(scales))
    w = Mxfp4Weight(torch.from_numpy(codes).cuda(), s)
    W = R.decode(codes, scales)
    xb = bits_of(np.random.default_rng(32).standard_normal((m, k)))
    ref, lim = R.product(R.bf16_values(xb), W)
    check(w.gemm(bits_to_dev(xb)), ref, lim, "gemm")
    xc, xsc = matrix(33, m, k)
    xsc[m // 2, 3] = 255
    xs = torch.zeros(xsc.size + 3, dtype=torch.uint8, device="cuda")[off:off + xsc.size].view(m, k // 32)
    xs.copy_(torch.from_numpy(xsc))
    ref, lim = R.product(R.decode(xc, xsc), W)
    check(w.gemm_mx(Mxfp4Weight(torch.from_numpy(xc).cuda(), xs)), ref, lim, "gemm_mx")


def test_no_rows():
    log("no rows")
    w = weight(*matrix(13, 40, 64))
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert w.gemm(x).shape == (0, 40)
    q = Mxfp4Weight.quantize(x)
    assert q.rows == 0 and w.gemm_mx(q).shape == (0, 40)


def test_offsets_past_32_bits():
    # 2^21 + 40 rows of 4352: 4.6 GB of codes; the last rows against the definition
    log("large weight")
    n, k = (1 << 21) + 40, 4352
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(115, 125, (n, k // 32), generator=g, device="cuda", dtype=torch.uint8)
    w = Mxfp4Weight(codes, scales)
    W = R.decode(codes[-50:].cpu().numpy(), scales[-50:].cpu().numpy())
    for m in (1, 3, 70):
        xb = bits_of(np.random.default_rng(m).standard_normal((m, k)))
        ref, lim = R.product(R.bf16_values(xb), W)
        log(f"  m={m}")
        check(w.gemm(bits_to_dev(xb))[:, -50:], ref, lim, f"m={m}")
    xc, xs = matrix(1, 70, k)
    ref, lim = R.product(R.decode(xc, xs), W)
    check(w.gemm_mx(weight(xc, xs))[:, -50:], ref, lim, "gemm_mx")


@pytest.mark.parametrize("k", [30720, 30752, 32768, 32800])
@pytest.mark.parametrize("n", [9, 1500, 2100])
def test_one_row_about_64_kib_of_lds(n, k):
    # X takes 60, 64, 64 and 68 KiB; the kernel's own array makes the second and third more than 64
    log(f"one row n={n} k={k}")
    codes, scales = matrix(n + k, n, k)
    xb = bits_of(np.random.default_rng(k).standard_normal((1, k)))
    ref, lim = R.product(R.bf16_values(xb), R.decode(codes, scales))
    check(weight(codes, scales).gemm(bits_to_dev(xb)), ref, lim, f"{n}x{k}")


def test_rows_past_the_threads_of_a_launch():
    # 2^28 + 48 rows: 16 threads a row are more than a launch counts in 32 bits
    log("longest weights")
    n, k = (1 << 28) + 48, 32
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(115, 125, (n, 1), generator=g, device="cuda", dtype=torch.uint8)
    w = Mxfp4Weight(codes, scales)
    for m in (1, 2, 5, 9):
        xb = bits_of(np.random.default_rng(m).standard_normal((m, k)))
        xc, xs = matrix(m, m, k)
        for what, x, run in (("gemm", R.bf16_values(xb), lambda: w.gemm(bits_to_dev(xb))),
                             ("gemm_mx", R.decode(xc, xs), lambda: w.gemm_mx(weight(xc, xs)))):
            log(f"  m={m} {what}")
            y = run()
            for a in (0, n // 2, n - 50):  # the first rows, some in the middle, the last
                ref, lim = R.product(x, R.decode(codes[a:a + 50].cpu().numpy(), scales[a:a + 50].cpu().numpy()))
                check(y[:, a:a + 50], ref, lim, f"{what} m={m} rows from {a}")
            del y


def test_another_stream_and_a_graph():
    log("stream and graph")
    n, k, m = 512, 2048, 5
    codes, scales = matrix(14, n, k)
    w = weight(codes, scales)
    xb = bits_of(np.random.default_rng(15).standard_normal((m, k)))
    x = bits_to_dev(xb)
    want, wantq = w.gemm(x), w.gemm_mx(Mxfp4Weight.quantize(x))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = w.gemm(x)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            gy, gq = w.gemm(x), w.gemm_mx(Mxfp4Weight.quantize(x))
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    for i in range(4):  # replays with other inputs, and the program's own work between them
        xb = bits_of(np.random.default_rng(20 + i).standard_normal((m, k)))
        x.copy_(bits_to_dev(xb))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(gy.view(torch.int16), w.gemm(x).view(torch.int16))
        assert torch.equal(gq.view(torch.int16), w.gemm_mx(Mxfp4Weight.quantize(x)).view(torch.int16))


def test_wrong_arguments_raise():
    log("refusals")
    w = weight(*matrix(16, 64, 128))
    x = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    for bad in (x[:, :96], x.float(), x.t().contiguous().t(), x.cpu()):
        with pytest.raises((ValueError, TypeError)):
            w.gemm(bad)
    with pytest.raises(ValueError):
        w.gemm(x, torch.empty(100, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        w.gemm_mx(weight(*matrix(17, 4, 64)))
    buf = torch.zeros(129 * 2, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(B.Int8wError, match="16-byte"):
        w.gemm(buf[1:257].view(2, 128))
    with pytest.raises(B.Int8wError, match="overlaps"):
        w.gemm(x, x.view(-1)[:128].view(2, 64))
