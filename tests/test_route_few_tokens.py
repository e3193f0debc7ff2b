"""Few tokens, around the bound up to which one launch makes the choice and the
dispatch order: every number of experts a lane, with and without a bias and
groups; a token has the same experts and weights alone as in a batch."""
import numpy as np
import pytest
import torch

import activation_sparsity_prep_b200 as sq
from tests.test_route import NEG, check, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 65])
@pytest.mark.parametrize("E,k,groups,topk_groups", [(20, 4, 4, 2), (60, 6, 6, 3), (128, 8, 8, 4), (200, 8, 8, 3), (256, 8, 8, 4), (400, 32, 10, 4)])
@pytest.mark.parametrize("biased", [False, True])
def test_around_one_launch(T, E, k, groups, topk_groups, biased):
    l = logits_of(T * E, T, E)
    if T > 1:
        l[T // 2] = NEG
        l[0, k - 1:] = NEG
    b = torch.from_numpy((0.1 * np.random.default_rng(E).standard_normal(E)).astype(np.float32)) if biased else None
    for kw in (dict(score="sigmoid"), dict(score="softmax", groups=groups, topk_groups=topk_groups, group_score="top2")):
        r = check(l, k, bias=b, **kw)
        one = sq.moe_route(l[-1:].cuda(), k, bias=None if b is None else b.cuda(), **kw)
        assert torch.equal(one.ids[0], r.ids[-1]) and torch.equal(one.weights[0], r.weights[-1])
