"""Refused calls of the operators around the linears: the C ABI rejects bad
arguments on the host before it touches a device (CPU), the binding raises
ValueError before it hands over a pointer (GPU)."""
import ctypes

import pytest
import torch

import activation_sparsity_prep_b200 as sq
from activation_sparsity_prep_b200 import ops

P, INVALID = 0x1000, 1
gpu = pytest.mark.gpu


def lib():
    L = sq.load_sharq_ops()
    ops._declare(L)
    return L


def route(T=4, k=2, E=8, ids=P, weights=P, row_index=P, offsets=P, position=P, logits=P, ld=8, fp32=0, bias=None,
          score=0, groups=1, topk_groups=1, group_score=0, scale=1.0):
    o = ops._RouteOptions(score, groups, topk_groups, group_score, 1, scale)
    r = ops._Routing(ids, weights, row_index, offsets, position, T, k, E)
    return lib().sharq_moe_route(logits, ld, fp32, bias, ctypes.byref(o), ctypes.byref(r), None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(k=0), dict(k=33, E=64, ld=64), dict(k=9), dict(E=0), dict(E=513, ld=513), dict(T=2 ** 31),
    dict(T=2 ** 30, k=2), dict(score=2), dict(score=-1), dict(groups=0), dict(groups=3), dict(groups=33, E=66, ld=66),
    dict(groups=4, topk_groups=0), dict(groups=4, topk_groups=5), dict(groups=4, topk_groups=1, k=3),
    dict(group_score=2), dict(scale=float("nan")), dict(scale=float("inf")), dict(logits=None), dict(ids=None),
    dict(weights=None), dict(logits=P + 1), dict(logits=P + 2, fp32=1), dict(bias=P + 2), dict(ids=P + 1),
    dict(weights=P + 2), dict(ld=7), dict(ld=-8, T=1), dict(row_index=None), dict(offsets=None), dict(position=None),
    dict(row_index=P + 2), dict(offsets=P + 1), dict(position=P + 3)])
def test_route_refusals(kw):
    assert route(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(T=-1), dict(k=0), dict(E=0), dict(E=513), dict(T=2 ** 31), dict(ids=None),
                                dict(row_index=None), dict(offsets=None), dict(position=None), dict(ids=P + 2),
                                dict(offsets=P + 1), dict(row_index=P + 1), dict(position=P + 1)])
def test_dispatch_refusals(kw):
    f = dict(ids=P, weights=None, row_index=P, offsets=P, position=P, T=4, k=2, E=8)
    f.update(kw)
    assert lib().sharq_moe_dispatch(ctypes.byref(ops._Routing(*f.values())), None) == INVALID
    assert lib().sharq_moe_dispatch(None, None) == INVALID


@pytest.mark.parametrize("kw", [dict(N=0), dict(N=12), dict(N=-8), dict(N=(1 << 24) + 8), dict(rows=-1), dict(T=-1), dict(T=2 ** 31), dict(k=0),
                                dict(Y=None), dict(position=None), dict(weights=None), dict(out=None), dict(Y=P + 8),
                                dict(residual=P + 2), dict(out=P + 4), dict(position=P + 2), dict(weights=P + 1)])
def test_combine_refusals(kw):
    f = dict(Y=P, yf=0, rows=8, N=16, position=P, weights=P, T=4, k=2, residual=P, out=P, of=0)
    f.update(kw)
    assert lib().sharq_moe_combine(*f.values(), None) == INVALID


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(K=0), dict(K=12), dict(K=32776), dict(M=-1), dict(M=2 ** 31), dict(norm=3), dict(norm=-1),
    dict(eps=-1.0), dict(eps=float("nan")), dict(alpha=float("inf")), dict(G=0), dict(G=3), dict(x=P + 2), dict(h=P + 8),
    dict(h=None, post_gamma=P), dict(h=None, gate=P, ld_gate=64), dict(norm=0, gamma=P), dict(norm=0, shift=P, ld_shift=64),
    dict(ld_x=63), dict(ld_x=65), dict(ld_h=32), dict(ld_out=60), dict(gate=P, ld_gate=68), dict(scale=P, G=2, ld_scale=8),
    dict(shift=P, ld_shift=-8), dict(gamma=P + 2), dict(beta=P + 4), dict(y=P + 2), dict(out_x=P + 2),
    dict(q=(None, P, 4, 64)), dict(q=(P, None, 4, 64)), dict(q=(P, P, 5, 64)), dict(q=(P, P, 4, 128)), dict(q=(P + 8, P, 4, 64)),
    dict(q=(P, P + 2, 4, 64))])
def test_residual_norm_refusals(kw):
    f = dict(x=P, h=P, out_x=P, y=P, ld_x=64, ld_h=64, ld_out=64, M=4, G=1, K=64, norm=1, alpha=1.0, eps=1e-6)
    f.update(kw)
    q = f.pop("q", None)
    a = ops._ResidualNorm(**f)
    if q:
        rows = ops._RowsInt8(*q)
        a.q = ctypes.pointer(rows)
    assert lib().sharq_residual_norm(ctypes.byref(a), None) == INVALID


@pytest.mark.parametrize("kw", [dict(X=None), dict(X=P + 2), dict(gamma=P + 2), dict(eps=-1.0), dict(M=-1), dict(K=4),
                                dict(K=32776), dict(codes=None), dict(scales=None), dict(codes=P + 4), dict(scales=P + 1)])
def test_quantise_refusals(kw):
    f = dict(X=P, gamma=None, eps=1e-6, codes=P, scales=P, M=4, K=64)
    f.update(kw)
    o = ops._RowsInt8(f["codes"], f["scales"], f["M"], f["K"])
    assert lib().sharq_prepare_int8(f["X"], f["gamma"], f["eps"], ctypes.byref(o), None) == INVALID
    if "gamma" not in kw and "eps" not in kw:
        w = ops._WeightInt8(f["codes"], f["scales"], f["M"], f["K"])
        assert lib().sharq_quantize_weight_int8(f["X"], ctypes.byref(w), None) == INVALID


@pytest.mark.parametrize("kw", [dict(M=-1), dict(M=2 ** 30 + 1), dict(N=2 ** 30 + 1), dict(N=0), dict(K=24), dict(K=0), dict(K=65552), dict(wK=128),
                                dict(xc=None), dict(xs=None), dict(wc=None), dict(ws=None), dict(Y=None), dict(xc=P + 8),
                                dict(wc=P + 1), dict(xs=P + 2), dict(ws=P + 1), dict(Y=P + 8), dict(bias=P + 1),
                                dict(bias=P + 2, bf=1)])
def test_linear_int8_refusals(kw):
    f = dict(xc=P, xs=P, wc=P, ws=P, M=4, N=32, K=64, Y=P, bias=None, bf=0)
    f.update(kw)
    x = ops._RowsInt8(f["xc"], f["xs"], f["M"], f["K"])
    w = ops._WeightInt8(f["wc"], f["ws"], f["N"], f.get("wK", f["K"]))
    assert lib().sharq_linear_int8(ctypes.byref(x), ctypes.byref(w), f["bias"], f["bf"], f["Y"], 0, None) == INVALID


def test_null_structs_are_refused():
    L = lib()
    r = ctypes.byref(ops._Routing(P, P, P, P, P, 1, 1, 1))
    assert L.sharq_moe_route(P, 8, 0, None, None, r, None) == INVALID
    o = ops._RouteOptions(0, 1, 1, 0, 1, 1.0)
    assert L.sharq_moe_route(P, 8, 0, None, ctypes.byref(o), None, None) == INVALID
    assert L.sharq_residual_norm(None, None) == INVALID
    assert L.sharq_prepare_int8(P, None, 0.0, None, None) == INVALID
    assert L.sharq_quantize_weight_int8(P, None, None) == INVALID
    assert L.sharq_linear_int8(None, None, None, 0, P, 0, None) == INVALID


def test_host_tensors_are_refused():
    z = torch.zeros((4, 8))
    for call in (lambda: sq.moe_route(z, 2), lambda: sq.moe_dispatch(z.int(), 4), lambda: sq.moe_combine(z, z, z),
                 lambda: sq.residual_norm(z), lambda: sq.prepare_int8(z), lambda: sq.quantize_weight_int8(z),
                 lambda: sq.linear_int8(sq.PreparedInt8(z, z, 4, 8), None)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@gpu
def test_binding_refusals_on_the_device():
    dev = torch.device("cuda")
    bf = dict(dtype=torch.bfloat16, device=dev)
    l = torch.zeros((4, 8), device=dev)
    ids = torch.zeros((4, 2), dtype=torch.int32, device=dev)
    x = torch.zeros((4, 64), **bf)
    q = sq.PreparedInt8.empty(4, 64)
    w = sq.WeightInt8.empty(32, 64)
    bad = [
        ("2-D", lambda: sq.moe_route(l[0], 2)), ("dtype", lambda: sq.moe_route(l.half(), 2)),
        ("k=9", lambda: sq.moe_route(l, 9)), ("k=0", lambda: sq.moe_route(l, 0)), ("score", lambda: sq.moe_route(l, 2, "relu")),
        ("groups", lambda: sq.moe_route(l, 2, groups=3)), ("topk_groups", lambda: sq.moe_route(l, 2, groups=4, topk_groups=5)),
        ("unit stride", lambda: sq.moe_route(l.t(), 2)), ("bias", lambda: sq.moe_route(l, 2, bias=torch.zeros(7, device=dev))),
        ("bias", lambda: sq.moe_route(l, 2, bias=torch.zeros(8, **bf))), ("row stride", lambda: sq.moe_route(l[:1].expand(4, 8), 2)),
        ("out.ids", lambda: sq.moe_route(l, 2, out=sq.Routing.empty(4, 3, 8))),
        ("dtype", lambda: sq.moe_dispatch(ids.long(), 8)), ("E=0", lambda: sq.moe_dispatch(ids, 0)),
        ("contiguous", lambda: sq.moe_dispatch(ids.t(), 8)),
        ("N=12", lambda: sq.moe_combine(torch.zeros((8, 12), **bf), ids, l[:, :2].contiguous())),
        ("weights", lambda: sq.moe_combine(x, ids, l)), ("residual", lambda: sq.moe_combine(x, ids, l[:, :2].contiguous(), residual=x[:3])),
        ("out", lambda: sq.moe_combine(x, ids, l[:, :2].contiguous(), residual=x, out=x.float())),
        ("K=60", lambda: sq.residual_norm(torch.zeros((4, 60), **bf))), ("norm", lambda: sq.residual_norm(x, norm="batch")),
        ("need h", lambda: sq.residual_norm(x, gate=x[:1])), ("nothing", lambda: sq.residual_norm(x, norm=None)),
        ("need a norm", lambda: sq.residual_norm(x, x, norm=None, gamma=x[0])),
        ("need a norm", lambda: sq.residual_norm(x, x, norm=None, int8=True)),
        ("divide", lambda: sq.residual_norm(x, x, gate=x[:3])), ("is torch", lambda: sq.residual_norm(x, x, post_gamma=x[0], gamma=x[0].float())),
        ("is torch", lambda: sq.residual_norm(x, x, gate=x[:1], shift=x[:1].float())),
        ("boundary", lambda: sq.residual_norm(torch.zeros((4, 65), **bf)[:, 1:], x)), ("another layout", lambda: sq.residual_norm(*_aliased(dev))),
        ("out_y", lambda: sq.residual_norm(x, x, int8=True, out_y=sq.PreparedInt8.empty(3, 64))),
        ("dtype", lambda: sq.prepare_int8(x.float())), ("gamma", lambda: sq.prepare_int8(x, x[0].float())),
        ("out describes", lambda: sq.prepare_int8(x, out=sq.PreparedInt8.empty(4, 72))),
        ("contiguous", lambda: sq.prepare_int8(torch.zeros((4, 128), **bf)[:, :64])),
        ("out describes", lambda: sq.quantize_weight_int8(x, out=w)),
        ("K=", lambda: sq.linear_int8(q, sq.WeightInt8.empty(32, 128))), ("WeightInt8", lambda: sq.linear_int8(q, q)),
        ("bias", lambda: sq.linear_int8(q, w, bias=torch.zeros(31, device=dev))),
        ("out", lambda: sq.linear_int8(q, w, out=torch.zeros((4, 31), **bf))),
        ("dtype", lambda: sq.linear_int8(q, w, out_fp32=True, out=torch.zeros((4, 32), **bf))),
    ]
    for match, call in bad:
        with pytest.raises(ValueError, match=match):
            call()


def _aliased(dev):
    """x with a row stride of 128 and an out_x that starts where it does."""
    wide = torch.zeros((4, 128), dtype=torch.bfloat16, device=dev)
    x = wide[:, :64]
    return x, x.clone(), "rms", None, None, 1.0, None, None, None, None, 1e-6, False, wide.view(-1)[:256].view(4, 64)


def test_first_argument_by_keyword_and_signature():
    import inspect
    z = torch.zeros((4, 8))
    for call in (lambda: sq.moe_route(logits=z, k=2), lambda: sq.residual_norm(h=z, x=z), lambda: sq.prepare_int8(X=z),
                 lambda: sq.linear_int8(w=None, x=sq.PreparedInt8(z, z, 4, 8)), lambda: sq.moe_route()):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    assert "stream" in inspect.signature(sq.moe_combine).parameters


@gpu
def test_calls_by_keyword():
    x = torch.randn((4, 64), device="cuda").bfloat16()
    q, s = sq.prepare_int8(x), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    by_name = sq.prepare_int8(X=x, stream=s)
    y = sq.residual_norm(h=x, x=x)[1]
    torch.cuda.synchronize()
    assert torch.equal(q.codes, by_name.codes) and torch.equal(q.scales, by_name.scales)
    assert torch.equal(y, sq.residual_norm(x, x)[1])
    w = sq.quantize_weight_int8(W=x)
    assert torch.equal(sq.linear_int8(x=q, w=w), sq.linear_int8(q, w))
    with pytest.raises(ValueError, match="PreparedInt8"):
        sq.linear_int8(x, w)
