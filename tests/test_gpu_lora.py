"""Low-rank adapters against their 64-bit definition, within limits counted from the roundings (tests/adapter_reference.py).
Every test prints its case first."""
import numpy as np
import pytest
import torch

import adapter_reference as R
from weight_only_quantized_int8_amd import Int8Weight, Int8wError, LoraAdapters, Mxfp4Weight, lora_add

pytestmark = pytest.mark.gpu


def log(msg):
    print(msg, flush=True)


def randn(g, *shape, gain=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * gain).bfloat16()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def pool_of(g, num, rank, k, n, scales=True):
    return LoraAdapters(randn(g, num, rank, k, gain=k ** -0.5), randn(g, num, n, rank, gain=0.3),
                        0.5 + torch.rand(num, generator=g, device="cuda") if scales else None)


def ids_of(kind, m, num, seed):
    rng = np.random.default_rng(seed)
    if kind == "own":  # a row each
        ids = rng.permutation(max(m, num))[:m] % num
    elif kind == "one":
        ids = np.full(m, num - 1)
    elif kind == "none":
        ids = np.full(m, -1)
    elif kind == "runs":
        ids = np.sort(rng.integers(0, num, m))[::-1].copy()
    else:
        ids = rng.integers(-1, num, m)
    return torch.from_numpy(ids.astype(np.int32)).cuda()


def f64(t):
    return t.double().cpu().numpy()


def bits(t):
    return t.contiguous().view(torch.int16)


def check(y, pool, x, ids, base, what):
    scales = f64(pool.scales) if pool.scales is not None else np.ones(pool.num_adapters)
    ref, lim = R.lora(f64(x), f64(pool.a), f64(pool.b), scales, ids.cpu().numpy().astype(np.int64),
                      f64(base) if base is not None else None)
    got = f64(y)
    assert got.shape == ref.shape
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    ok = (np.abs(got - ref) <= lim) | np.isnan(ref)
    assert ok.all(), f"{what}: {np.count_nonzero(~ok)} of {ok.size} outside; first {np.argwhere(~ok)[0]} got {got[~ok][0]} " \
                     f"want {ref[~ok][0]} within {lim[~ok][0]}"


SIZES = [  # m, K, N, rank, adapters
    (1, 8, 1, 8, 1), (1, 256, 320, 16, 3), (1, 4096, 64, 8, 2), (2, 72, 7, 24, 2), (3, 520, 250, 64, 5), (15, 128, 96, 40, 4),
    (16, 64, 64, 16, 3), (17, 320, 257, 32, 2), (33, 1032, 130, 72, 40), (64, 128, 256, 128, 9), (65, 200, 100, 16, 70),
    (130, 96, 600, 256, 3), (256, 64, 72, 8, 20), (257, 64, 72, 8, 20), (300, 264, 514, 48, 7), (513, 72, 40, 136, 3),
    (700, 128, 1027, 64, 11), (3, 16392, 40, 8, 2), (5, 128, 96, 128, 3), (2, 2056, 1500, 64, 3), (1, 24, 513, 56, 2), (63, 16384, 24, 16, 30),
    (1100, 64, 264, 24, 9), (2500, 72, 136, 8, 300),
]


@pytest.mark.parametrize("kind", ["own", "one", "runs", "mixed", "none"])
@pytest.mark.parametrize("m,K,N,rank,num", SIZES)
def test_against_the_definition(m, K, N, rank, num, kind):
    log(f"lora m={m} K={K} N={N} rank={rank} num={num} ids={kind}")
    g = gen(m + K + N)
    pool, x, ids = pool_of(g, num, rank, K, N, scales=(m + N) % 3 != 0), randn(g, m, K), ids_of(kind, m, num, m)
    base = randn(g, m, N) if (m + K) % 4 else None
    y = lora_add(pool, x, ids, base)
    check(y, pool, x, ids, base, kind)
    assert torch.equal(bits(y), bits(lora_add(pool, x, ids, base)))
    if base is not None:
        lora_add(pool, x, ids, base, base)
        assert torch.equal(bits(y), bits(base))


@pytest.mark.parametrize("m", [1, 5, 64, 300])
@pytest.mark.parametrize("odd", [0, 1, 8])
def test_fused_projections_in_place(m, odd):
    # q, k and v as columns of one matrix, `odd` columns before them and after: alignment and strides
    log(f"fused projections m={m} odd={odd}")
    g = gen(m)
    K, ns, num = 264, (320, 72, 73), 5
    pools = [pool_of(g, num, r, K, n, scales=n != 72) for n, r in zip(ns, (16, 40, 8))]
    wide = randn(g, m, odd + sum(ns) + odd)
    x = randn(g, m, K + 16)[:, 8:8 + K]
    ids = ids_of("mixed", m, num, m)
    before = wide.clone()
    at = np.cumsum([odd] + list(ns))
    views = [wide[:, int(a):int(a) + n] for a, n in zip(at, ns)]
    bases = [v.clone() for v in views]
    apart = lora_add(pools, x, ids, [before[:, int(a):int(a) + n] for a, n in zip(at, ns)])
    out = lora_add(pools, x, ids, views, views)
    for y, v, p, b in zip(apart, out, pools, bases):
        assert torch.equal(bits(y), bits(v))
        check(y, p, x, ids, b, "fused")
        alone = lora_add(p, x, ids, b)
        check(alone, p, x, ids, b, "alone")
    assert torch.equal(bits(wide[:, :odd]), bits(before[:, :odd]))
    assert torch.equal(bits(wide[:, odd + sum(ns):]), bits(before[:, odd + sum(ns):]))


@pytest.mark.parametrize("m", [1, 40, 270])
def test_own_ranks(m):
    log(f"own ranks m={m}")
    g = gen(m)
    K, N, made = 136, 200, []
    for i, r in enumerate((1, 4, 8, 13, 64, 33, 100)):
        made.append((randn(g, r, K, gain=K ** -0.5), randn(g, N, r, gain=0.3), 0.25 * (i + 1)))
    pool = LoraAdapters.from_list(made)
    assert pool.rank == 104 and pool.ranks.tolist() == [1, 4, 8, 13, 64, 33, 100]
    x, ids, base = randn(g, m, K), ids_of("mixed", m, len(made), m), randn(g, m, N)
    y = lora_add(pool, x, ids, base)
    check(y, pool, x, ids, base, "ranks")
    full = LoraAdapters(pool.a, pool.b, pool.scales)  # the same with the zeros read
    assert torch.equal(bits(y), bits(lora_add(full, x, ids, base)))


@pytest.mark.parametrize("m", [1, 20, 64, 400])
def test_own_ranks_of_nothing_and_beyond_the_pool(m):
    # rank 0: base itself in value; above the pool's: the pool's
    log(f"rank 0 and large ranks m={m}")
    for rank, K in ((16, 64), (72, 520)):
        g = gen(m + rank)
        pool, x, base = pool_of(g, 4, rank, K, 300), randn(g, m, K), randn(g, m, 300)
        pool.a[1], pool.b[1] = 0, 0
        own = LoraAdapters(pool.a, pool.b, pool.scales, torch.tensor([rank, 0, rank + 9, -1], dtype=torch.int32, device="cuda"))
        for kind in ("mixed", "runs"):
            ids = ids_of(kind, m, 4, m)
            ids[0] = 1
            y = lora_add(own, x, ids, base)
            check(y, pool, x, ids, base, kind)
            assert torch.equal(y[0], base[0]) and torch.equal(bits(y), bits(lora_add(pool, x, ids, base)))


@pytest.mark.parametrize("m", [20, 70, 400])
def test_what_one_row_holds_stays_in_it(m):
    log(f"infinities and NaN m={m}")
    g = gen(m)
    K, N, num = 128, 150, 6
    pool, x, ids, base = pool_of(g, num, 24, K, N), randn(g, m, K), ids_of("mixed", m, num, 1), randn(g, m, N)
    ids[3], ids[4], ids[5], ids[6], ids[7] = 1, -1, 2, 0, 3
    want = lora_add(pool, x, ids, base)
    x[3, 5], x[4, 0], x[5, 100] = float("nan"), float("nan"), float("inf")
    base[6, 2], base[7, 3] = float("-inf"), float("nan")
    pool.a[4, 3, 7] = float("inf")
    pool.b[5, 17, 2] = float("nan")
    y = lora_add(pool, x, ids, base)
    host = ids.cpu().numpy()
    touched = (host == 4) | (host == 5)
    touched[[3, 5, 6, 7]] = True
    same = (bits(y) == bits(want)).all(1).cpu().numpy()
    assert same[~touched].all()
    assert torch.equal(bits(y[4]), bits(base[4]))  # no adapter: x is not looked at
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[5]).any()
    assert torch.isnan(y[7, 3]) and not torch.isfinite(y[6, 2])
    fives = np.flatnonzero(host == 5)
    fives = fives[~np.isin(fives, [3, 5, 6, 7])]
    nan = torch.isnan(y[fives.tolist()])
    assert nan[:, 17].all() and int(nan.sum()) == len(fives)


@pytest.mark.parametrize("m", [9, 300])
def test_ids_outside_the_pool(m):
    log(f"bad ids m={m}")
    g = gen(m)
    pool, x, base = pool_of(g, 4, 16, 64, 300), randn(g, m, 64), randn(g, m, 300)
    ids = ids_of("mixed", m, 4, m)
    good = lora_add(pool, x, ids, base)
    for bad in (4, 1 << 20, -2, -(1 << 31)):
        other = ids.clone()
        other[m // 2] = bad
        for b in (base, None):
            y = lora_add(pool, x, other, b)
            assert (bits(y[m // 2]) == 0x7FC0).all()
            if b is not None:
                keep = [t for t in range(m) if t != m // 2]
                assert torch.equal(bits(y[keep]), bits(good[keep]))
    none = lora_add(pool, x, torch.full_like(ids, -1))
    assert (bits(none) == 0).all()


def test_outputs_stay_inside_their_rows():
    log("extent")
    g = gen(1)
    for m in (3, 290):
        pool, x, ids = pool_of(g, 4, 8, 64, 90), randn(g, m, 64), ids_of("mixed", m, 4, 2)
        buf = torch.full((m + 2, 101), 77.0, dtype=torch.bfloat16, device="cuda")
        y = buf[1:m + 1, 5:95]
        lora_add(pool, x, ids, None, y)
        check(y, pool, x, ids, None, "view")
        assert (buf[0] == 77).all() and (buf[m + 1] == 77).all() and (buf[:, :5] == 77).all() and (buf[:, 95:] == 77).all()
        assert lora_add(pool, x[:0], ids[:0]).shape == (0, 90)


def test_a_pool_past_32_bits():
    # 5000 adapters of 16 x 32768: 5.2 GB of A; the last ones are named
    log("large pool")
    num, rank, K, N = 5000, 16, 32768, 96
    g = gen(4)
    a = torch.zeros((num, rank, K), dtype=torch.bfloat16, device="cuda")
    b = torch.zeros((num, N, rank), dtype=torch.bfloat16, device="cuda")
    a[-3:], b[-3:] = randn(g, 3, rank, K, gain=K ** -0.5), randn(g, 3, N, rank)
    pool = LoraAdapters(a, b)
    for m in (2, 300):
        x = randn(g, m, K)
        ids = torch.tensor([num - 1 - i % 3 for i in range(m)], dtype=torch.int32, device="cuda")
        y = lora_add(pool, x, ids)
        last = LoraAdapters(a[-3:].contiguous(), b[-3:].contiguous())
        check(y, last, x, ids - (num - 3), None, f"m={m}")


@pytest.mark.parametrize("m", [70000, (1 << 16) + 1])
def test_more_rows_than_one_round_of_groups(m):
    # more than 64 pieces of 1024 rows; the rows about the ends of pieces and of rounds are looked at
    log(f"many rows m={m}")
    g = gen(5)
    pool, x, base = pool_of(g, 7, 8, 72, 40), randn(g, m, 72), randn(g, m, 40)
    for kind in ("mixed", "runs"):
        ids = ids_of(kind, m, 7, 3)
        y = lora_add(pool, x, ids, base)
        at = torch.tensor(sorted({t for e in range(0, m + 1024, 1024) for t in (e - 2, e - 1, e, e + 1) if 0 <= t < m} | {m - 1}))
        check(y[at], pool, x[at], ids[at], base[at], kind)
        e = ids.long().clamp(min=0)  # all rows, to what BF16 tells
        u = torch.matmul(pool.a.double()[e], x.double().unsqueeze(2))
        ref = base.double() + torch.where(ids >= 0, pool.scales.double()[e], 0.0).unsqueeze(1) * torch.matmul(pool.b.double()[e], u).squeeze(2)
        assert ((y.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -12).all()


@pytest.mark.parametrize("m", [64, 65, 70001])
def test_many_rows_of_tiny_matrices(m):
    log(f"tiny matrices m={m}")
    g = gen(m + 3)
    pool, x, base = pool_of(g, 3, 8, 8, 40), randn(g, m, 8), randn(g, m, 40)
    ids = ids_of("mixed", m, 3, 7)
    check(lora_add(pool, x, ids, base), pool, x, ids, base, m)


def test_the_same_call_gives_the_same_bits():
    # where groups lie in the plan depends on the order of atomics; no result may
    log("repeats")
    g = gen(8)
    for m, num in ((700, 90), (300, 3), (2000, 400)):
        pool, x, ids, base = pool_of(g, num, 24, 520, 136), randn(g, m, 520), ids_of("mixed", m, num, 1), randn(g, m, 136)
        want = lora_add(pool, x, ids, base)
        for _ in range(20):
            assert torch.equal(bits(want), bits(lora_add(pool, x, ids, base)))


def test_rows_far_apart():
    # the last rows of x and y begin beyond 2^32 bytes
    log("wide strides")
    g = gen(6)
    m, K, N, stride = 40, 64, 32, 1 << 26
    wide = torch.zeros(m * stride, dtype=torch.bfloat16, device="cuda")
    x, y = wide.as_strided((m, K), (stride, 1), 0), wide.as_strided((m, N), (stride, 1), 1024)
    x.copy_(randn(g, m, K))
    pool, ids = pool_of(g, 3, 8, K, N), ids_of("mixed", m, 3, 1)
    lora_add(pool, x, ids, None, y)
    check(y, pool, x, ids, None, "wide strides")


def test_another_stream_a_graph_and_calls_at_a_time():
    log("streams and graphs")
    for m in (1, 30, 300):
        g = gen(m)
        pools = [pool_of(g, 5, 16, 256, n) for n in (192, 64)]
        x, ids = randn(g, m, 256), ids_of("mixed", m, 5, m)
        base = [randn(g, m, n) for n in (192, 64)]
        want = lora_add(pools, x, ids, base)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        graphs, outs = [], []
        for s in streams:
            with torch.cuda.stream(s):
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=s):
                    outs.append(lora_add(pools, x, ids, base))
                graphs.append(graph)
        torch.cuda.synchronize()
        for i in range(4):  # two graphs replayed at a time, new inputs, eager calls between
            x.copy_(randn(g, m, 256))
            ids.copy_(ids_of("mixed", m, 5, 100 + i))
            torch.cuda.synchronize()
            for s, graph in zip(streams, graphs):
                with torch.cuda.stream(s):
                    graph.replay()
            eager = lora_add(pools, x, ids, base)
            torch.cuda.synchronize()
            for out in outs:
                assert all(torch.equal(bits(a), bits(b)) for a, b in zip(out, eager)), (m, i)
        got = [[], []]
        for _ in range(10):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    got[i].append(lora_add(pools, x, ids, base))
        torch.cuda.synchronize()
        assert all(torch.equal(bits(a), bits(b)) for ys in got[0] + got[1] for a, b in zip(ys, eager))
        assert len(want) == 2


@pytest.mark.parametrize("m", [1, 7, 48, 280])
def test_beside_a_projection(m):
    log(f"gemm_lora m={m}")
    g = gen(m)
    N, K = 320, 256
    pool, x, ids = pool_of(g, 4, 16, K, N), randn(g, m, K), ids_of("mixed", m, 4, m)
    dense = randn(g, N, K, gain=K ** -0.5)
    for W in (Int8Weight.quantize(dense, 64), Mxfp4Weight.quantize(dense)):
        plain = W.gemm(x)
        y = W.gemm_lora(x, pool, ids)
        check(y, pool, x, ids, plain, type(W).__name__)
        out = torch.full((m * N + 8,), 3.0, dtype=torch.bfloat16, device="cuda")
        assert W.gemm_lora(x, pool, ids, out) is out
        assert torch.equal(bits(out[:m * N].view(m, N)), bits(y)) and (out[m * N:] == 3).all()


def test_wrong_arguments_raise():
    log("refusals")
    g = gen(1)
    pool, x, ids = pool_of(g, 3, 8, 64, 40), randn(g, 4, 64), ids_of("mixed", 4, 3, 0)
    for bad in (ids[:3], ids.long(), ids.cpu(), ids.view(2, 2)):
        with pytest.raises(ValueError, match="ids"):
            lora_add(pool, x, bad)
    with pytest.raises(ValueError, match="x must be"):
        lora_add(pool, x[:, :56], ids)
    with pytest.raises(TypeError, match="bfloat16"):
        lora_add(pool, x.float(), ids)
    with pytest.raises(ValueError, match="base must be"):
        lora_add(pool, x, ids, randn(g, 4, 41))
    with pytest.raises(ValueError, match="contiguous"):
        lora_add(pool, x, ids, randn(g, 40, 4).t())
    with pytest.raises(Int8wError, match="multiple of 8"):
        lora_add(pool, randn(g, 4, 68)[:, :64], ids)
    with pytest.raises(Int8wError, match="16-byte"):
        lora_add(pool, randn(g, 4, 72)[:, 4:68], ids)
    wide = randn(g, 4, 100)
    with pytest.raises(Int8wError, match="overlaps input base"):
        lora_add(pool, x, ids, wide[:, :40], wide[:, 8:48])
    with pytest.raises(Int8wError, match="two outputs"):
        lora_add([pool, pool], x, ids, None, [wide[:, :40], wide[:, 32:72]])
    with pytest.raises(Int8wError, match="pools differ"):
        lora_add([pool, pool_of(g, 2, 8, 64, 40)], x, ids)
    with pytest.raises(Int8wError, match="1..4 pools"):
        lora_add([pool] * 5, x, ids)
    with pytest.raises(ValueError, match="one base and one output"):
        lora_add([pool, pool], x, ids, [None])
    with pytest.raises(ValueError, match="in_features 64 and out_features 48"):
        Mxfp4Weight.quantize(randn(g, 48, 64)).gemm_lora(x, pool, ids)
