"""The routing to experts where values are equal, too near to tell, infinite or at the end of fp32's range, against its 64-bit
definition (tests/adapter_reference.py), with one to eight experts a lane.  Every test prints its case first."""
import numpy as np
import pytest
import torch

import adapter_reference as A
from test_gpu_moe_route import same
from weight_only_quantized_int8_amd import moe_route

pytestmark = pytest.mark.gpu

LOW = float(np.finfo(np.float32).min)


def log(msg):
    print(msg, flush=True)


def run(l, topk, bf16=False, scoring="softmax", bias=None, groups=1, topk_groups=None, group_score="top2", renorm=True, what=None):
    ld = torch.from_numpy(l).cuda()
    if bf16:
        ld = ld.bfloat16()
        assert np.array_equal(ld.float().cpu().numpy(), l)
    got = moe_route(ld, topk, scoring, None if bias is None else torch.from_numpy(bias).cuda(), groups, topk_groups, group_score, renorm)
    same(got, A.route(l.astype(np.float64), topk, scoring, bias, groups, topk_groups, group_score, renorm), what)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E", [12, 60, 128, 256, 500, 512])
def test_zeros_of_both_signs_are_equal(E, bf16):
    log(f"signed zeros E={E} bf16={bf16}")
    rng = np.random.default_rng(E)
    step = 2.0 ** -133 if bf16 else 2.0 ** -149  # the smallest value
    rows = [np.full(E, -1.0) for _ in range(4)]
    for row, (a, b) in zip(rows, ((0, 1), (1, 2), (3, E - 1), (E // 2 - 1, E // 2))):
        row[a], row[b] = -0.0, 0.0
    rows += [np.resize([-0.0, 0.0], E), np.resize([0.0, -0.0], E), np.full(E, -0.0)]
    rows += [np.where(rng.random(E) < 0.5, -0.0, 0.0) for _ in range(4)]
    rows += [np.where(rng.random(E) < 0.2, np.where(rng.random(E) < 0.5, -0.0, 0.0), -2.0) for _ in range(4)]
    rows += [step * rng.integers(-9, 10, E) * rng.choice([-1.0, 1.0], E) for _ in range(4)]  # about zero, many of them equal
    l = np.array(rows, np.float32)
    assert np.signbit(l[0, 0]) and l[0, 0] == 0 and (l[-1] != 0).any()
    for topk in (1, 5):
        for scoring in ("softmax", "sigmoid"):
            for groups, topk_groups, group_score in ((1, 1, "max"), (4, 2, "max"), (4, 2, "top2")):
                run(l, topk, bf16, scoring, None, groups, topk_groups, group_score, what=(topk, scoring, groups, group_score))


@pytest.mark.parametrize("E", [12, 128, 256, 512])
def test_infinities_are_equal(E):
    # more and fewer of them than are taken, at all places in their lanes
    log(f"infinities E={E}")
    inf, rng = np.inf, np.random.default_rng(E)
    rows = []
    for at in ((1, 2), (2, 5), (3, 4, E - 1), tuple(range(1, 9)), tuple(range(E - 9, E, 2)), tuple(range(E))):
        rows.append(rng.standard_normal(E))
        rows[-1][list(at)] = inf
    rows += [np.where(rng.random(E) < p, inf, rng.standard_normal(E)) for p in (0.02, 0.1, 0.5)]
    rows += [np.where(rng.random(E) < 0.1, inf, -inf), np.where(rng.random(E) < 0.3, inf, 1.0), rng.standard_normal(E)]
    l = np.array(rows, np.float32)
    biases = [None, 0.1 * rng.standard_normal(E), np.zeros(E), np.zeros(E), np.where(rng.random(E) < 0.2, inf, 0.0), np.full(E, inf)]
    biases[2][[3, 4]] = inf
    biases[3][[5, E - 2, 7]] = inf
    for bias in biases:
        for topk in (1, 5):
            for groups, topk_groups in ((1, 1), (4, 2)):
                for group_score in ("max", "top2"):
                    for bf16 in (False, True):
                        for scoring in ("softmax", "sigmoid"):
                            v = np.where(l == inf, 3.0, l).astype(np.float32) if scoring == "softmax" else l
                            if bf16:
                                v = torch.from_numpy(v).bfloat16().float().numpy()
                            run(v, topk, bf16, scoring, None if bias is None else bias.astype(np.float32), groups, topk_groups, group_score,
                                what=(bias, topk, groups, group_score, bf16, scoring))


@pytest.mark.parametrize("E,groups", [(64, 8), (256, 8), (512, 16), (500, 20)])
def test_near_values_with_several_experts_a_lane(E, groups):
    # a unit of fp32 and less apart: cut off in a candidate, lost in a biased score
    log(f"near values E={E}")
    rng = np.random.default_rng(E)
    T = 150
    l = (0.5 + 2.0 ** -24 * rng.integers(0, 40, (T, E))).astype(np.float32)
    few = np.where(rng.random((T, E)) < 0.03, l, -4.0).astype(np.float32)
    bias = (16.0 + 2.0 ** -19 * rng.integers(0, 2, E)).astype(np.float32)
    for v in (l, -l, few):
        for scoring in ("softmax", "sigmoid"):
            run(v, 8, False, scoring, None, what=("alone", scoring))
            run(v, 8, False, scoring, None, groups, groups // 2, "max", what=("groups", scoring))
            run(v, 8, False, scoring, bias, groups, groups // 2, "max", what=("biased", scoring))
            run(v, 1, False, scoring, bias, what=("one", scoring))


@pytest.mark.parametrize("E", [16, 60, 64, 128, 256])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_group_sums_past_the_range_of_fp32(E, scoring):
    # the sum of two biases is no infinity where it is compared
    log(f"large group sums E={E} {scoring}")
    inf, rng = np.inf, np.random.default_rng(E)
    l = rng.standard_normal((6, E)).astype(np.float32)
    l[5, E // 2:] = -inf
    for groups in (4, 2) if E != 60 else (6, 12):
        size = E // groups
        for pairs in (((3e38, 1e38), (3e38, 3e38), (2.5e38, 2.5e38), (0, 0)), ((LOW, LOW), (-2e38, -2e38), (-3e38, -1e38), (LOW, -3e38)),
                      ((-inf, -inf), (LOW, LOW), (-inf, -inf), (-inf, LOW)), ((inf, 1), (3e38, 3e38), (inf, inf), (3.4e38, 3.4e38)),
                      ((-inf, -inf), (LOW, LOW), (1, LOW), (-inf, 3e38))):
            bias = np.empty(E, np.float32)
            for g in range(groups):
                two = pairs[g % 4]
                low = min(two) if min(two) < 0 else -1.0
                bias[g * size:(g + 1) * size] = low
                bias[g * size + g % 2], bias[(g + 1) * size - 1] = two
            for topk_groups in (1, groups // 2, groups):
                for topk in (1, min(3, size)):
                    run(l, topk, False, scoring, bias, groups, topk_groups, "top2", what=(groups, pairs, topk_groups, topk))


def test_more_tokens_than_one_launch_has_threads_for():
    # 64 threads a token; a launch has fewer than 2^32
    T = (1 << 26) + 5
    log(f"many tokens T={T}")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    l = torch.randint(-9, 9, (T, 2), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    ids = torch.full((T + 1, 1), 7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, 1), 7.0, device="cuda")
    moe_route(l, 1, ids=ids[:T], weights=w[:T])
    assert torch.equal(ids[:T, 0], (l[:, 1] > l[:, 0]).int()) and (w[:T] == 1).all()
    assert int(ids[T]) == 7 and float(w[T]) == 7


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_slots_without_an_expert_weigh_nothing_whatever_the_factor(scoring, renorm):
    log(f"factor {scoring} renorm={renorm}")
    l = torch.full((4, 6), -float("inf"), device="cuda")
    l[1, 2], l[2, 0], l[2, 5], l[3] = 0.5, -60.0, -61.0, 0.25
    for factor in (float("inf"), float("nan"), -float("inf")):
        ids, w = moe_route(l, 3, scoring, renormalize=renorm, routed_scale=factor)
        assert torch.equal(ids.cpu(), torch.tensor([[-1, -1, -1], [2, -1, -1], [0, 5, -1], [0, 1, 2]], dtype=torch.int32))
        none = ids < 0
        assert (w[none] == 0).all() and not torch.isfinite(w[~none]).any(), factor
