"""Rows that hold NaN or infinities on their way through the 8-bit operators:
what is not finite must not come out as a finite value."""
import pytest
import torch

import activation_sparsity_prep_b200 as sq

pytestmark = pytest.mark.gpu
B = torch.bfloat16


@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("M,K", [(5, 64), (5, 272), (7, 4096), (3, 18944), (3000, 1024)])
@pytest.mark.parametrize("form", ["plain", "norm", "residual"])
def test_a_row_that_is_not_finite_stays_so_in_8_bits(form, M, K, value):
    """Its scale, and with it every element of the product, is not finite; the
    rows beside it are as without it."""
    g = torch.Generator(device="cuda").manual_seed(M + K)
    X = torch.randn((M, K), generator=g, device="cuda").to(B)
    gm = (0.5 + torch.rand(K, generator=g, device="cuda")).to(B)

    def quantised(x):
        if form == "residual":
            return sq.residual_norm(x.float(), x, norm="layer", gamma=gm, int8=True)[1]
        return sq.prepare_int8(x, gm if form == "norm" else None)

    good = quantised(X)
    bad = X.clone()
    hit = [1, M - 1]
    bad[1, K - 3] = float(value)                             # one element of a row, and a whole row
    bad[M - 1] = float(value)
    q = quantised(bad)
    w = sq.quantize_weight_int8(torch.randn((24, K), generator=g, device="cuda").to(B))
    bias = torch.ones(24, device="cuda")
    y = sq.linear_int8(q, w, bias=bias, out_fp32=True)
    assert not torch.isfinite(q.scales[hit]).any()
    assert not torch.isfinite(y[hit]).any()
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[hit] = False
    assert torch.equal(q.codes[rest], good.codes[rest]) and torch.equal(q.scales[rest], good.scales[rest])
    assert torch.equal(y[rest], sq.linear_int8(good, w, bias=bias, out_fp32=True)[rest])
