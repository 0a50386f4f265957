"""The statistical limits of mx_limits.py: they accept what the definition's roundings make, and reject the mistakes
that the worst-case limits are too wide for on long rows (a lost block, scales of another group, a lost choice).
Mistakes are planted in the 64-bit reference, on the CPU."""
import numpy as np
import pytest

import mx_limits as L
import mx_reference as R


def fp32_product(x, w):
    """y in fp32 sums of 32 terms a step, rounded to BF16."""
    acc = np.zeros((x.shape[0], w.shape[0]), np.float32)
    for k in range(0, x.shape[1], 32):
        acc = acc + (x[:, k:k + 32] @ w[:, k:k + 32].T).astype(np.float32)
    return L.rounded(acc)


@pytest.mark.parametrize("m,n,k", [(1, 8, 90016), (1, 33, 36896), (5, 40, 14336), (64, 50, 4096), (3, 100, 96)])
def test_products_as_rounded_are_accepted(m, n, k):
    w = R.decode(*L.mx_matrix(k, n, k))
    x = L.rounded(np.random.default_rng(m).standard_normal((m, k)))
    assert L.product_faults(fp32_product(x, w), x @ w.T, k) == []


@pytest.mark.parametrize("m,n,k", [(1, 8, 90016), (1, 33, 36896), (5, 40, 14336)])
def test_products_with_a_mistake_are_rejected(m, n, k):
    codes, scales = L.mx_matrix(k, n, k)
    w = R.decode(codes, scales)
    x = L.rounded(np.random.default_rng(m).standard_normal((m, k)))
    ref = x @ w.T
    worst = R.product(x, w)[1]
    missed = 0
    for block in range(0, k // 32, 11):  # one block of 32 not added
        ks = slice(32 * block, 32 * block + 32)
        y = L.rounded(ref - x[:, ks] @ w[:, ks].T)
        assert L.product_faults(y, ref, k), f"block {block}"
        missed += (np.abs(y - ref) <= worst).all()
    print(f"the worst case misses {missed} of {(k // 32 + 10) // 11} lost blocks")
    y = L.rounded(x[:, :-2048] @ w[:, :-2048].T)
    assert L.product_faults(y, ref, k)
    shifted = scales.copy()
    shifted[:, 32:] = scales[:, :-32]  # past k = 1024 the scales of k - 1024
    assert L.product_faults(L.rounded(x @ R.decode(codes, shifted).T), ref, k)
    one = w.copy()
    one[n // 2, 64:96] = 0  # a block of a single weight row
    assert L.product_faults(L.rounded(x @ one.T), ref, k)


CASES = [("gs32", 2, 1152, 2176, 1), ("gs64", 2, 1152, 2176, 1), ("gs128", 2, 1152, 2176, 3), ("gs32", 3, 1056, 2080, 6),
         ("mxfp4", 8, 16384, 64, 1), ("mxfp4", 4, 544, 1056, 5)]


@pytest.mark.parametrize("fmt,E,I,H,T", CASES)
def test_layers(fmt, E, I, H, T):
    topk = min(E, 8)
    ex = L.Experts(E + I, fmt, E, I, H)
    W = [ex.values(i) for i in range(3)]
    xb, l = L.layer_inputs(T, T, H, E)
    x, l = R.bf16_values(xb), l.astype(np.float64)
    ref = L.layer(x, W, l, topk)
    assert L.layer_faults(L.rounded(L.layer(x, W, l, topk, round_h=True)), ref, I, H) == []

    def rejected(what, V, l=l):
        y = L.rounded(L.layer(x, V, l, topk, round_h=True))
        assert L.layer_faults(y, ref, I, H), what

    for i, k in ((0, H), (1, H), (2, I)):
        for block in sorted({0, k // 64, k // 32 - 1}):  # a block of 32 lost in every expert, and in the second alone
            for experts in (slice(None), slice(1, 2)):
                V = list(W)
                V[i] = W[i].copy()
                V[i][experts, :, 32 * block:32 * block + 32] = 0
                rejected(f"matrix {i} block {block} {experts}", V)
        if k > 1024 + ex.gs and (fmt != "mxfp4" or i == 2):
            raw, g = ex.raw[i], 1024 // ex.gs
            ex.raw[i] = [raw[0]] + [np.concatenate((a[:, :g], a[:, :-g]), 1) for a in raw[1:]]
            V = list(W)
            V[i] = ex.values(i)  # past k = 1024 the scales and biases of k - 1024
            ex.raw[i] = raw
            rejected(f"matrix {i}: groups", V)
    lost = l.copy()
    lost[np.arange(T), np.argsort(-l, 1)[:, topk - 1]] = -np.inf  # each token's last choice
    rejected("a lost choice", W, lost)
