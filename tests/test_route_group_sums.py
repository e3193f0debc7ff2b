"""Group scores that cancel: the two largest score + bias of a group are of
opposite sign and far larger than their sum, so the sum's fp32 error is that of
its terms.  The experts must still be those of 64-bit arithmetic."""
import numpy as np
import pytest
import torch

import activation_sparsity_prep_b200 as sq
import oracle.ops as ref

gpu = pytest.mark.gpu
LOWEST, LARGEST = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max


def two_groups_of_two(seed, T, B):
    """Logits near 0 and biases +B, -B in each group: the groups' sums lie
    within about 1e-3 of 1."""
    g = np.random.default_rng(seed)
    l = (0.002 * g.standard_normal((T, 4))).astype(np.float32)
    return l, np.array([B, -B, -B, B], dtype=np.float32)


def check(l, b, k, **kw):
    r = sq.moe_route(torch.from_numpy(l).cuda(), k, bias=torch.from_numpy(b).cuda(), **kw)
    ids, w = ref.route(l, k, bias=b, **kw)
    wrong = np.nonzero((r.ids.cpu().numpy() != ids).any(1))[0]
    assert not len(wrong), f"{len(wrong)} of {len(l)} tokens, the first {wrong[:5]}"
    # tests/test_route.py derives 2^-17
    assert np.all(np.abs(r.weights.cpu().numpy() - w) <= 2.0 ** -17 * np.abs(w) + 1e-37)
    ri, off, pos = ref.dispatch(ids, l.shape[1])
    assert np.array_equal(r.row_index.cpu().numpy(), ri) and np.array_equal(r.position.cpu().numpy(), pos)


def test_these_biases_mislead_a_sum_of_rounded_terms():
    """The groups of a plain fp32 evaluation differ from those of 64 bits where
    the gap of the rounded sums is beyond any multiple of their own step."""
    l, b = two_groups_of_two(1, 20000, 1000.0)
    s = 1.0 / (1.0 + np.exp(-l.astype(np.float64)))
    c = s + b
    exact = c[:, 2:].sum(1) > c[:, :2].sum(1)
    f = s.astype(np.float32) + b
    gap = f[:, 2:].sum(1) - f[:, :2].sum(1)
    wrong = (gap > 0) != exact
    assert wrong.sum() > 20 and np.abs(gap[wrong]).max() > 100 * 2.0 ** -24


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("B", [1.0, 64.0, 100.0, 1000.0, 1e6, 1e20])
def test_sums_that_cancel(B, score):
    l, b = two_groups_of_two(7, 20000, B)
    check(l, b, 1, score=score, groups=2, group_score="top2")


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,topk_groups,k", [(64, 8, 3, 6), (60, 20, 5, 4), (96, 4, 2, 8), (256, 8, 4, 8), (512, 16, 4, 8),
                                                    (24, 12, 4, 3)])
@pytest.mark.parametrize("B", [100.0, 3000.0])
def test_cancelling_groups_of_every_layout(E, groups, topk_groups, k, B, score):
    """One expert of a group at +B, the others at -B: groups of whole lanes and
    others, few candidates and, where the -B ones are not told apart, many."""
    g = np.random.default_rng(E)
    size = E // groups
    l = (0.01 * g.standard_normal((500, E))).astype(np.float32)
    b = np.full(E, -B, dtype=np.float32)
    b[np.arange(groups) * size + g.integers(0, size, groups)] = B
    check(l, b, k, score=score, groups=groups, topk_groups=topk_groups, group_score="top2")


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("E,groups,topk_groups,k", [(8, 4, 3, 5), (64, 8, 5, 30), (60, 20, 9, 20), (256, 8, 7, 32)])
def test_the_lowest_and_the_largest_biases(E, groups, topk_groups, k, group_score, score):
    """Two of them pass the range of fp32 as a sum; an expert at the lowest
    value is still one, and comes before none."""
    g = np.random.default_rng(E + k)
    l = g.standard_normal((50, E)).astype(np.float32)
    size = E // groups
    for low, high in ((LOWEST, 0.0), (0.0, LARGEST), (LOWEST, LARGEST)):
        b = (0.1 * g.standard_normal(E)).astype(np.float32)
        b[size:4 * size] = low if low else b[size:4 * size]
        if high:
            b[:size] = high
        check(l, b, k, score=score, groups=groups, topk_groups=topk_groups, group_score=group_score)


@gpu
def test_large_biases_without_groups():
    l, b = two_groups_of_two(9, 4000, 1000.0)
    check(l, b, 3, score="sigmoid")
    check(l, b, 3, score="softmax")
