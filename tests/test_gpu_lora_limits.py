"""Low-rank adapters at the ends of their ranges: own ranks beside infinities, large factors, values beyond BF16's largest; against
their 64-bit definition (tests/adapter_reference.py), in each of the forms a call can take.  Every test prints its case first."""
import numpy as np
import pytest
import torch

import adapter_reference as R
from test_gpu_lora import bits, f64, gen, ids_of, pool_of, randn
from weight_only_quantized_int8_amd import LoraAdapters, lora_add

pytestmark = pytest.mark.gpu

# rows, K, N, rank: one launch; a workgroup a row; groups of up to 16 and of up to 64 rows
FORMS = [(1, 64, 96, 16), (7, 72, 300, 8), (40, 520, 130, 48), (1, 520, 96, 72), (30, 136, 600, 136), (64, 256, 96, 256), (65, 64, 96, 16),
         (90, 136, 300, 72), (400, 520, 130, 16), (700, 136, 96, 64), (600, 72, 264, 136)]


def log(msg):
    print(msg, flush=True)


def check(y, ref, lim, what):
    """Finite values within their limits, NaN where NaN is wanted, infinities of the wanted sign."""
    got = f64(y)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in rows {np.flatnonzero((np.isnan(got) != np.isnan(ref)).any(1))[:8]}"
    with np.errstate(invalid="ignore"):
        ok = np.isnan(ref) | (got == ref) | (np.isfinite(ref) & (np.abs(got - ref) <= lim))
    assert ok.all(), f"{what}: {np.count_nonzero(~ok)} outside; first {np.argwhere(~ok)[0]} got {got[~ok][0]} want {ref[~ok][0]}"


@pytest.mark.parametrize("m,K,N,rank", FORMS)
@pytest.mark.parametrize("kind", ["mixed", "runs"])
def test_an_own_rank_beside_infinities(m, K, N, rank, kind):
    # an adapter of rank r is a sum over r: what x holds meets no padding, and of rank 0 nothing at all
    log(f"own ranks and infinities m={m} K={K} N={N} rank={rank} {kind}")
    g = gen(m + rank)
    num = 6
    own = [0, 1, min(rank, 3), 8, rank, min(rank, 17)]
    pool, x, base = pool_of(g, num, rank, K, N), randn(g, m, K), randn(g, m, N)
    for e, r in enumerate(own):
        pool.a[e, r:] = 0
        pool.b[e, :, r:] = 0
    pool = LoraAdapters(pool.a, pool.b, pool.scales, torch.tensor(own, dtype=torch.int32, device="cuda"))
    for first in range(num) if m == 1 else (0,):
        ids = ids_of(kind, m, num, m)
        ids[0] = first
        wrong = x.clone()
        wrong[0::3, 5] = float("inf")
        wrong[0::6, K - 1] = -float("inf")
        if m > 4:
            wrong[4, 9] = float("nan")
        y = lora_add(pool, wrong, ids, base)
        host, xs, bs = ids.cpu().numpy(), f64(wrong), f64(base)
        ref, lim = np.empty((m, N)), np.zeros((m, N))
        for e in range(-1, num):
            at, r = np.flatnonzero(host == e), own[e] if e >= 0 else 1
            if not len(at):
                continue
            if r == 0:  # base itself
                ref[at] = bs[at]
                continue
            with np.errstate(invalid="ignore"):
                ref[at], lim[at] = R.lora(xs[at], f64(pool.a)[max(e, 0):max(e, 0) + 1, :r], f64(pool.b)[max(e, 0):max(e, 0) + 1, :, :r],
                                          f64(pool.scales)[max(e, 0):max(e, 0) + 1], np.zeros(len(at), int) if e >= 0 else np.full(len(at), -1), bs[at])
        check(y, ref, lim, (kind, first))
        assert first != 0 or torch.equal(bits(y[0]), bits(base[0]))


@pytest.mark.parametrize("m,K,N,rank", FORMS)
def test_a_large_factor_of_small_products(m, K, N, rank):
    # the factor comes last: times u alone it would pass fp32's range, B u it does not
    log(f"large factors m={m} K={K} N={N} rank={rank}")
    g = gen(m + K)
    pool, x, base, ids = pool_of(g, 3, rank, K, N), randn(g, m, K, gain=2.0 ** 20), randn(g, m, N, gain=2.0 ** 12), ids_of("mixed", m, 3, 2)
    ids[0] = 1
    pool = LoraAdapters(pool.a, pool.b * 2.0 ** -100, torch.tensor([2.0 ** 118, 1.5 * 2.0 ** 112, 2.0 ** 96], device="cuda"))
    for b in (base, None):
        y = lora_add(pool, x, ids, b)
        ref, lim = R.lora(f64(x), f64(pool.a), f64(pool.b), f64(pool.scales), ids.cpu().numpy(), f64(b) if b is not None else None)
        assert np.isfinite(ref).all() and (np.abs(ref) < 2.0 ** 120).all()
        check(y, ref, lim, b is None)


@pytest.mark.parametrize("m,K,N,rank", FORMS)
def test_values_between_the_largest_of_bf16_and_of_fp32(m, K, N, rank):
    # u is BF16's largest value and half a unit of it: finite, though its rounding to BF16 is not
    log(f"u beyond BF16 m={m} K={K} N={N} rank={rank}")
    g = gen(m + N)
    a, b = torch.zeros(2, rank, K, dtype=torch.bfloat16, device="cuda"), randn(g, 2, N, rank, gain=2.0 ** -120)
    most = torch.finfo(torch.bfloat16).max
    a[:, :, 3], a[:, :, 11] = 1.0, torch.tensor([1.0, -1.0], device="cuda").repeat(rank // 2)
    x = torch.zeros(m, K, dtype=torch.bfloat16, device="cuda")
    x[:, 3], x[:, 11] = most, 2.0 ** 119
    x[1::2] = -x[1::2]
    pool, ids = LoraAdapters(a, b), ids_of("runs", m, 2, 1)
    base = randn(g, m, N)
    y = lora_add(pool, x, ids, base)
    ref, lim = R.lora(f64(x), f64(a), f64(b), np.ones(2), ids.cpu().numpy(), f64(base))
    assert np.isfinite(ref).all()
    check(y, ref, lim, "u beyond BF16")
    x[0, 3], x[m - 1, 5] = float("inf"), float("nan")  # these stay what they are
    a[:, :, 5] = 1.0
    y = lora_add(pool, x, ids, base)
    assert not torch.isfinite(y[0]).any() and torch.isnan(y[m - 1]).all()


@pytest.mark.parametrize("m,N,rank,num", [(700, 4200, 8, 90), (1600, 4100, 64, 24), (1300, 5000, 16, 1300), (400, 4097, 136, 30), (2600, 130, 16, 30),
                                          (3100, 4104, 32, 26)])
def test_groups_on_an_xcd_of_their_own_and_spread(m, N, rank, num):
    # from 24 groups on an XCD has whole groups where u is much or columns are few; wide outputs of small u are spread
    log(f"groups m={m} N={N} rank={rank} num={num}")
    g = gen(m + N)
    K = 64
    pool, x, base = pool_of(g, num, rank, K, N), randn(g, m, K), randn(g, m, N)
    for kind in ("runs", "mixed"):
        ids = ids_of(kind, m, num, 4)
        y = lora_add(pool, x, ids, base)
        at = np.unique(np.concatenate([np.arange(0, m, max(1, m // 100)), [m - 1]]))
        ref, lim = R.lora(f64(x)[at], f64(pool.a), f64(pool.b), f64(pool.scales), ids.cpu().numpy()[at], f64(base)[at])
        check(y[torch.from_numpy(at).cuda()], ref, lim, kind)
        e = ids.long().clamp(min=0)  # all rows, to what BF16 tells
        u = torch.matmul(pool.a.double()[e], x.double().unsqueeze(2)).squeeze(2)
        for t in range(0, m, 200):
            own = torch.matmul(pool.b.double()[e[t:t + 200]], u[t:t + 200].unsqueeze(2)).squeeze(2) * pool.scales.double()[e[t:t + 200]].unsqueeze(1)
            ref = base[t:t + 200].double() + torch.where(ids[t:t + 200, None] >= 0, own, 0.0)
            assert ((y[t:t + 200].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -12).all()
