"""Long rows of the MXFP4 products and of the expert layer on the GPU within the statistical limits of mx_limits.py,
which notice a lost block of 32 or the scales of another group.  Every test prints its case first."""
import numpy as np
import pytest
import torch

import mx_limits as L
import mx_reference as R
from helpers import bits_to_dev, dev_to_bits
from weight_only_quantized_int8_amd import Int8Weight, Mxfp4Weight, moe_layer

pytestmark = pytest.mark.gpu


def log(msg):
    print(msg, flush=True)


def values(y):
    return R.bf16_values(dev_to_bits(y))


# one row: both sides of the one-row kernel's LDS limit, segments shared by one, two and four waves; few rows: one,
# two and four loads of activations, four and eight waves; more rows on small weights; the small and the large tiles
SHAPES = [(1, 8, 90016), (1, 33, 36896), (1, 700, 14336), (1, 1500, 8192), (1, 2500, 4128), (3, 70, 28672), (7, 50, 36896),
          (16, 300, 14336), (9, 4200, 2080), (40, 100, 14336), (200, 1600, 4096), (300, 2304, 2080), (1000, 4100, 1056)]


def weight(codes, scales):
    return Mxfp4Weight(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_products(m, n, k):
    log(f"products m={m} n={n} k={k}")
    codes, scales = L.mx_matrix(k + n, n, k)
    w, W = weight(codes, scales), R.decode(codes, scales)
    xb = R.bf16_bits(np.random.default_rng(m).standard_normal((m, k)).astype(np.float32))
    assert L.product_faults(values(w.gemm(bits_to_dev(xb))), R.bf16_values(xb) @ W.T, k) == []
    xc, xs = L.mx_matrix(m, m, k)
    assert L.product_faults(values(w.gemm_mx(weight(xc, xs))), R.decode(xc, xs) @ W.T, k) == []


# rows of several segments and of a part of one in every format; MXFP4 inner products that do not fit the one-token form
LAYERS = [(f, 2, 1152, 2176, 2, T) for f in ("gs32", "gs64", "gs128") for T in (1, 2, 6, 40)]
LAYERS += [("gs32", 3, 1056, 2080, 2, T) for T in (1, 2, 6, 40)]
LAYERS += [("mxfp4", 8, 16384, 64, 8, T) for T in (1, 3)]
LAYERS += [("mxfp4", 4, 2080, 4128, 3, T) for T in (1, 2, 20)]


@pytest.mark.parametrize("fmt,E,I,H,topk,T", LAYERS)
def test_layers(fmt, E, I, H, topk, T):
    log(f"layer {fmt} E={E} I={I} H={H} topk={topk} T={T}")
    ex = L.Experts(E + I, fmt, E, I, H)
    xb, l = L.layer_inputs(T, T, H, E)
    y = values(moe_layer(*ex.upload(), E, bits_to_dev(xb), torch.from_numpy(l).cuda(), topk))
    ref = L.layer(R.bf16_values(xb), [ex.values(i) for i in range(3)], l.astype(np.float64), topk)
    assert L.layer_faults(y, ref, I, H) == []


@pytest.mark.parametrize("gs", [32, 64])
def test_experts_past_32_bits_with_scales_of_their_own(gs):
    # gate of 40 experts x 16384 x 8192: 5.4 GB of codes; the last experts are taken
    log(f"large experts, groups of {gs}")
    E, I, H = 40, 16384, 8192
    g = torch.Generator(device="cuda")
    g.manual_seed(gs)
    W = []
    for n, k in ((E * I, H), (E * I, H), (E * H, I)):
        codes = torch.randint(0, 256, (n, k), generator=g, device="cuda", dtype=torch.uint8)
        s = (torch.rand(n, k // gs, generator=g, device="cuda") * 3e-4 + 1e-4).bfloat16()
        b = (-128.0 * s.float() * (1.0 + 0.1 * (torch.rand(n, k // gs, generator=g, device="cuda") - 0.5))).bfloat16()
        W.append(Int8Weight(codes.view(torch.int32), s, b, gs))

    def expert(w, e, rows):
        part = slice(e * rows, (e + 1) * rows)
        q = w.packed[part].view(torch.uint8).double().reshape(rows, -1, gs)
        return (q * w.scales[part].double().unsqueeze(-1) + w.biases[part].double().unsqueeze(-1)).reshape(rows, -1)

    for T in (1, 2):
        log(f"  T={T}")
        xb, _ = L.layer_inputs(T, T, H, E)
        l = torch.full((T, E), -50.0, device="cuda")
        l[:, 38], l[:, 39] = 0.25, 0.0
        y = moe_layer(*W, E, bits_to_dev(xb), l, 2)
        x = torch.from_numpy(R.bf16_values(xb)).cuda()
        want = 0
        for r, e in zip(torch.softmax(torch.tensor([0.25, 0.0], dtype=torch.float64), 0).tolist(), (38, 39)):
            a, u = x @ expert(W[0], e, I).t(), x @ expert(W[1], e, I).t()
            want = want + (r * a * torch.sigmoid(a) * u) @ expert(W[2], e, H).t()
        assert L.layer_faults(values(y), want.cpu().numpy(), I, H) == []
