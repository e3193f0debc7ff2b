"""The operators around the linears on no rows, with every optional part."""
import ctypes

import pytest
import torch

import activation_sparsity_prep_b200 as sq
from activation_sparsity_prep_b200 import ops

gpu = pytest.mark.gpu
B, F = torch.bfloat16, torch.float32
P = 0x1000


@pytest.mark.parametrize("parts", [("post_gamma",), ("gate",), ("post_gamma", "gate")])
def test_no_rows_are_no_error(parts):
    """Tensors without rows have no address: h is null there."""
    L = sq.load_sharq_ops()
    ops._declare(L)
    f = dict(x=None, h=None, out_x=None, y=None, gamma=P, ld_x=64, ld_h=64, ld_out=64, ld_gate=64, M=0, G=1, K=64, norm=1,
             alpha=1.0, eps=1e-6)
    f.update({p: P for p in parts})
    assert L.sharq_residual_norm(ctypes.byref(ops._ResidualNorm(**f)), None) == 0


@gpu
@pytest.mark.parametrize("norm", ["rms", "layer", None])
def test_no_rows_with_every_part(norm):
    x = torch.zeros((0, 64), dtype=F, device="cuda")
    v = torch.ones(64, device="cuda", dtype=B)
    mod = torch.ones((2, 3, 64), device="cuda", dtype=B)
    kw = dict(post_gamma=v, gate=mod[:, 0])
    if norm:
        kw.update(gamma=v, beta=v, scale=mod[:, 1], shift=mod[:, 2])
    xo, y = sq.residual_norm(x, x.to(B), norm=norm, **kw)
    assert xo.shape == (0, 64) and (y is None if norm is None else y.shape == (0, 64))
    if norm:
        _, q = sq.residual_norm(x, x.to(B), norm=norm, int8=True, **kw)
        w = sq.quantize_weight_int8(torch.ones((8, 64), device="cuda", dtype=B))
        assert sq.linear_int8(q, w).shape == (0, 8)
        assert sq.linear_int8(sq.prepare_int8(x.to(B), v), w).shape == (0, 8)
    ids = torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    d = sq.moe_dispatch(ids, 7)
    assert d.offsets.tolist() == [0] * 8
    assert sq.moe_combine(x, ids, ids.float()).shape == (0, 64)
