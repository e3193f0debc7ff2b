"""Weights far below a token's others: the chosen scores underflow in fp32 where
their share of the sum does not.  Tolerance: an fp32 result of values evaluated
in double, half a step of 2^-24; 2^-17 (tests/test_route.py) where the fp32
evaluation decides, which reaches arguments of 64, and 2^-24 of the argument
beyond; a result below fp32's normal range may be 0."""
import numpy as np
import pytest
import torch

import activation_sparsity_prep_b200 as sq
import oracle.ops as ref

pytestmark = pytest.mark.gpu


def check(l, k, bias=None, **kw):
    r = sq.moe_route(torch.from_numpy(l).cuda(), k, bias=None if bias is None else torch.from_numpy(bias).cuda(), **kw)
    ids, w = ref.route(l, k, bias=bias, **kw)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    tol = 2.0 ** -17 + 2.0 ** -22 * np.abs(l).max()
    got = r.weights.cpu().numpy().astype(np.float64)
    off = np.abs(got - w) > tol * w + 2.0 ** -126
    assert not off.any(), (got[off][:4], w[off][:4])
    return w


def test_sigmoid_scores_of_very_unlikely_experts():
    g = np.random.default_rng(1)
    l = np.array([[-60.0, -92.0, -500.0], [-88.5, -87.5, -300.0], [-20.0, -95.0, -100.0], [-0.5, -75.0, -88.6]], dtype=np.float32)
    w = check(l, 2, score="sigmoid")
    assert (w[0] > 1e-15).all() and w[0, 1] < 1e-13          # e^-32
    for E, k in ((40, 3), (256, 8), (400, 32)):
        l = (-70.0 + 15.0 * g.standard_normal((200, E))).astype(np.float32)
        check(l, k, score="sigmoid")
        check(l, k, score="sigmoid", groups=4, topk_groups=2, group_score="top2")
        check(l, k, bias=g.standard_normal(E).astype(np.float32), score="sigmoid")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(100, 18), (256, 8), (512, 20)])
def test_experts_chosen_by_their_bias(E, k, score):
    """Biases that fall along the experts choose neighbours, many of which lie
    in the same lanes, whatever their scores."""
    g = np.random.default_rng(E)
    l = (40.0 * g.standard_normal((300, E))).astype(np.float32)
    b = np.linspace(20.0, 0.0, E).astype(np.float32)
    check(l, k, bias=b, score=score)
    check(l, k, bias=b, score=score, groups=4, topk_groups=2, group_score="max")
    check(l, k, bias=b, score=score, renormalize=False)
