"""Routing to experts: the choice, the dispatch order and the weighted sum
back, against the 64-bit reference.

Tolerances.  ids and the dispatch order are equal.  An fp32 weight: the
exponential is within 2 ulp (2^-22), its argument's rounding adds up to
|l - max| 2^-24 (|l - max| <= 64 here: 2^-18), the sums and quotients add at
most (16 + 5 + 5 + 4) 2^-24; in all below 2^-17.  A combined element: k
products and additions in fp32, (k + 2) 2^-24 of the terms' magnitudes, and
half a step of the output's type."""
import numpy as np
import pytest
import torch

import activation_sparsity_prep_b200 as sq
import oracle.ops as ref

gpu = pytest.mark.gpu
NEG = -float("inf")


def logits_of(seed, T, E, dtype=torch.float32):
    g = np.random.default_rng(seed)
    l = torch.from_numpy((2.0 * g.standard_normal((T, E)) + g.standard_normal(E)).astype(np.float32))
    return l.to(dtype)


def check(l, k, bias=None, **kw):
    """Route on the GPU and compare everything with the reference."""
    E = l.shape[1]
    r = sq.moe_route(l if l.is_cuda else l.cuda(), k, bias=None if bias is None else bias.cuda(), **kw)
    torch.cuda.synchronize()
    ids, w = ref.route(l.float().cpu().numpy(), k, bias=None if bias is None else bias.numpy(), **kw)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    got = r.weights.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - w) <= 2.0 ** -17 * np.abs(w) + 1e-37)
    ri, off, pos = ref.dispatch(ids, E)
    assert np.array_equal(r.row_index.cpu().numpy(), ri)
    assert np.array_equal(r.offsets.cpu().numpy(), off)
    assert np.array_equal(r.position.cpu().numpy(), pos)
    return r


# ------------------------------------------------------- reference (CPU) --

def test_reference_route_by_hand():
    l = np.log(np.array([[1.0, 4.0, 2.0, 1.0]]))
    ids, w = ref.route(l, 2)
    assert ids.tolist() == [[1, 2]] and np.allclose(w, [[2 / 3, 1 / 3]])
    ids, w = ref.route(l, 2, renormalize=False, scale=2.0)
    assert np.allclose(w, [[1.0, 0.5]])
    # ties to the lower index; a bias moves the choice and not the weight
    ids, w = ref.route(np.zeros((1, 4)), 2)
    assert ids.tolist() == [[0, 1]]
    ids, w = ref.route(l, 1, bias=np.array([0.9, 0, 0, 0.0]), renormalize=False)
    assert ids.tolist() == [[0]] and np.allclose(w, 1 / 8)
    # groups {0, 1} and {2, 3}: by their largest, then by their two largest
    l = np.array([[1.0, -9, 0.9, 0.8]])
    assert ref.route(l, 1, "sigmoid", groups=2)[0].tolist() == [[0]]
    assert ref.route(l, 1, "sigmoid", groups=2, group_score="top2")[0].tolist() == [[2]]
    # masked experts are never chosen
    ids, w = ref.route(np.array([[NEG, 1.0, np.nan], [NEG, NEG, NEG]]), 2)
    assert ids.tolist() == [[1, -1], [-1, -1]] and w.tolist() == [[1, 0], [0, 0]]


def test_reference_dispatch_is_a_stable_sort():
    ids = np.random.default_rng(1).integers(-1, 6, (50, 3))
    ri, off, pos = ref.dispatch(ids, 5)
    order = [(e, i) for i, e in enumerate(ids.reshape(-1)) if 0 <= e < 5]
    order.sort()
    assert off[5] == len(order)
    assert ri[:len(order)].tolist() == [i // 3 for _, i in order] and not ri[len(order):].any()
    assert all(pos.reshape(-1)[i] == n for n, (_, i) in enumerate(order))
    assert (pos.reshape(-1)[(ids.reshape(-1) < 0) | (ids.reshape(-1) >= 5)] == -1).all()


# ----------------------------------------------------------------- route --

@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (2, 8, 8), (7, 33, 3), (300, 60, 6), (130, 128, 8),
                                   (65, 257, 9), (40, 512, 32), (1100, 16, 2)])
def test_route_plain(T, E, k, score, dtype):
    check(logits_of(T + E, T, E, dtype), k, score=score)


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,E,k,groups,topk_groups", [(200, 256, 8, 8, 4), (33, 64, 6, 8, 3), (50, 60, 4, 20, 5),
                                                      (50, 32, 3, 32, 7), (9, 512, 8, 2, 1), (64, 96, 8, 4, 4)])
def test_route_groups(T, E, k, groups, topk_groups, score, group_score, biased):
    b = torch.from_numpy((0.1 * np.random.default_rng(E).standard_normal(E)).astype(np.float32)) if biased else None
    check(logits_of(T * E, T, E), k, bias=b, score=score, groups=groups, topk_groups=topk_groups,
          group_score=group_score)


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize,scale", [(False, 1.0), (True, 2.5), (False, 0.5)])
def test_route_weights(score, renormalize, scale):
    check(logits_of(3, 64, 40), 5, score=score, renormalize=renormalize, scale=scale)


@gpu
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_masks(score, groups, biased):
    """Rows with no expert, with fewer than k, NaN, whole groups masked, the
    lowest finite value, a bias of -inf, logits of both zeros."""
    E, k = 32, 4
    l = logits_of(5, 40, E)
    l[0] = NEG
    l[1, 3:] = NEG
    l[2, ::2] = float("nan")
    l[3] = float("nan")
    l[4, 8:] = NEG
    l[5, :31] = NEG
    l[6, 4:] = torch.finfo(torch.float32).min
    l[7] = torch.finfo(torch.float32).min
    l[8] = 0.0
    l[9] = torch.where(torch.arange(E) % 2 == 0, 0.0, -0.0)
    l[10] = 60.0
    b = None
    if biased:
        b = torch.linspace(-0.2, 0.2, E)
        b[30] = NEG
    check(l, k, bias=b, score=score, groups=groups, topk_groups=min(groups, 2), group_score="top2")


@gpu
def test_route_lowest_of_bf16():
    l = logits_of(8, 6, 24, torch.bfloat16)
    l[:, 5:] = torch.finfo(torch.bfloat16).min
    check(l, 6)
    check(l, 6, score="sigmoid")


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_near_ties_are_decided_in_64_bits(score):
    """Every expert's score + bias lies within a few 1e-9 of the others: far
    below an fp32 step, above 64-bit rounding."""
    g = np.random.default_rng(11)
    T, E, k = 64, 64, 8
    l = g.standard_normal((T, E)).astype(np.float32)
    l[:] = l[0]                                             # one row of logits, biases that level its scores
    s = 1.0 / (1.0 + np.exp(-l[0].astype(np.float64)))
    if score == "softmax":
        s = np.exp(l[0].astype(np.float64))
        s /= s.sum()
    b = (0.75 - s).astype(np.float32)
    c = s + b.astype(np.float64)
    assert np.ptp(c) < 1e-7 and np.diff(np.sort(c)).min() > 1e-14
    check(torch.from_numpy(l), k, bias=torch.from_numpy(b), score=score)
    check(torch.from_numpy(l), k, bias=torch.from_numpy(b), score=score, groups=8, topk_groups=3, group_score="top2")


@gpu
def test_route_equal_scores_go_to_the_lower_index():
    l = torch.zeros((5, 100))
    l[2, 50:] = 1.0
    b = torch.zeros(100)
    for bias in (None, b):
        for groups, group_score in ((1, "max"), (10, "max"), (10, "top2")):
            check(l, 7, bias=bias, groups=groups, topk_groups=min(2, groups), group_score=group_score)


@gpu
def test_route_strided_logits_and_no_tokens():
    wide = logits_of(13, 50, 200).cuda()
    l = wide[:, 7:47]
    assert not l.is_contiguous()
    check(l, 4)
    check(wide[::3, 100:], 3, score="sigmoid")
    r = sq.moe_route(wide[:0], 4)
    torch.cuda.synchronize()
    assert r.ids.shape == (0, 4) and r.offsets.cpu().tolist() == [0] * 201


@gpu
def test_route_large_batch():
    check(logits_of(17, 9001, 128, torch.bfloat16), 8)


# -------------------------------------------------------------- dispatch --

@gpu
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 128), (5, 3, 7), (127, 8, 60), (512, 8, 512), (513, 8, 512),
                                   (4097, 8, 128), (3000, 3, 256), (20001, 2, 5), (33000, 8, 256)])
def test_dispatch(T, k, E):
    g = np.random.default_rng(T + E)
    ids = g.integers(-2, E + 2, (T, k)).astype(np.int32)
    ids[ids == E + 1] = 2 ** 31 - 1
    d = sq.moe_dispatch(torch.from_numpy(ids).cuda(), E)
    torch.cuda.synchronize()
    ri, off, pos = ref.dispatch(ids, E)
    assert np.array_equal(d.offsets.cpu().numpy(), off)
    assert np.array_equal(d.row_index.cpu().numpy(), ri)
    assert np.array_equal(d.position.cpu().numpy(), pos)


@gpu
@pytest.mark.parametrize("T", [10, 5000])
def test_dispatch_one_expert_takes_all_or_none(T):
    for value, E in ((3, 9), (-1, 9), (9, 9)):
        ids = np.full((T, 2), value, dtype=np.int32)
        d = sq.moe_dispatch(torch.from_numpy(ids).cuda(), E)
        ri, off, pos = ref.dispatch(ids, E)
        assert np.array_equal(d.offsets.cpu().numpy(), off)
        assert np.array_equal(d.row_index.cpu().numpy(), ri)
        assert np.array_equal(d.position.cpu().numpy(), pos)


# --------------------------------------------------------------- combine --

@gpu
@pytest.mark.parametrize("ydt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rdt", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,N", [(1, 1, 8), (3, 8, 2048), (50, 6, 264), (129, 10, 2056), (20, 33, 40), (700, 2, 5120)])
def test_combine(T, k, N, ydt, rdt):
    g = np.random.default_rng(T * N)
    rows = T * k + 3
    Y = torch.from_numpy(g.standard_normal((rows, N)).astype(np.float32)).to(ydt)
    pos = g.permutation(rows)[:T * k].reshape(T, k).astype(np.int32)
    pos[g.random((T, k)) < 0.2] = -1
    pos[0, 0] = rows + 5                                    # outside: adds nothing
    if T > 2:
        pos[2] = -1
        pos[1, :] = pos[1, 0]                               # the same row k times
    w = g.random((T, k)).astype(np.float32)
    w[pos < 0] = np.nan                                     # not read into the sum
    res = None if rdt is None else torch.from_numpy(g.standard_normal((T, N)).astype(np.float32)).to(rdt)
    out = sq.moe_combine(Y.cuda(), torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda(),
                         residual=None if res is None else res.cuda())
    dt = rdt or ydt
    assert out.dtype == dt
    y, mag = ref.combine(Y.float().numpy(), pos, np.nan_to_num(w), None if res is None else res.float().numpy())
    err = np.abs(out.float().cpu().numpy() - y)
    half = torch.finfo(dt).eps / 2
    assert np.all(err <= (k + 2) * 2.0 ** -24 * mag * 1.01 + half * np.abs(y) * 1.01 + 1e-37)


@gpu
def test_combine_into_the_residual():
    g = torch.Generator().manual_seed(3)
    Y = torch.randn((64, 128), generator=g).bfloat16().cuda()
    pos = torch.randperm(64, generator=g).int().view(16, 4).cuda()
    w = torch.rand((16, 4), generator=g).cuda()
    res = torch.randn((16, 128), generator=g).cuda()
    want = sq.moe_combine(Y, pos, w, residual=res)
    got = sq.moe_combine(Y, pos, w, residual=res, out=res)
    assert got is res and torch.equal(got, want)


@gpu
@pytest.mark.parametrize("offset", [0, 1, 2, 4])
@pytest.mark.parametrize("T,E,groups", [(5, 128, 1), (300, 256, 8), (70, 200, 1), (70, 100, 5), (66, 60, 4), (9, 512, 16),
                                        (80, 510, 1)])
def test_route_bias_of_any_alignment(T, E, groups, offset):
    l = logits_of(T + E, T, E)
    g = np.random.default_rng(offset)
    room = torch.from_numpy(0.2 * g.standard_normal(E + 4).astype(np.float32))
    room[offset + E // 2], room[offset + E - 1] = NEG, float("nan")
    bias = room.cuda()[offset:offset + E]
    assert bias.data_ptr() % 16 == offset * 4 % 16
    kw = dict(score="sigmoid", groups=groups, topk_groups=max(1, groups // 2), group_score="top2")
    r = sq.moe_route(l.cuda(), 4, bias=bias, **kw)
    ids, w = ref.route(l.numpy(), 4, bias=bias.cpu().numpy(), **kw)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.all(np.abs(r.weights.cpu().numpy() - w) <= 2.0 ** -17 * np.abs(w) + 1e-37)
