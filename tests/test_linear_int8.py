"""The 8-bit integer linear against exact integer sums.

Tolerance: the int32 sum is exact; its rounding to fp32, the two scale
products and the bias addition are each half a step of 2^-24, so an fp32
element is within 4 2^-24 of the product's magnitude plus 2^-24 of the bias
and the result; bf16 adds half a step, 2^-8."""
import numpy as np
import pytest
import torch

import activation_sparsity_prep_b200 as sq
import oracle.ops as ref

pytestmark = pytest.mark.gpu


def operands(seed, M, N, K, full=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lo = -128 if full else -127
    x = torch.randint(lo, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(lo, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.rand(M, generator=g, device="cuda") * 0.1 + 1e-3
    ws = torch.rand(N, generator=g, device="cuda") * 0.01 + 1e-4
    return sq.PreparedInt8(x, xs, M, K), sq.WeightInt8(w, ws, N, K)


def exact(x, w, bias, rows):
    """fp64 result for some rows; integer sums below 2^53 are exact in fp64."""
    acc = x.codes[rows].double() @ w.codes.double().t()
    y = acc * x.scales[rows].double()[:, None] * w.scales.double()
    mag = y.abs()
    return (y if bias is None else y + bias.double()), mag


def check(x, w, bias=None, rows=None):
    rows = torch.arange(x.M, device="cuda") if rows is None else rows
    y64, mag = exact(x, w, bias, rows)
    b = 0 if bias is None else bias.double().abs()
    out = {}
    for fp32 in (True, False):
        y = sq.linear_int8(x, w, bias=bias, out_fp32=fp32)
        assert y.shape == (x.M, w.N) and y.dtype == (torch.float32 if fp32 else torch.bfloat16)
        tol = 4 * 2.0 ** -24 * mag + 2.0 ** -24 * (b + y64.abs()) + 1e-37
        if not fp32:
            tol = tol + 2.0 ** -8 * y64.abs() * 1.01
        err = (y[rows].double() - y64).abs()
        assert bool((err <= tol).all()), float((err / tol).max())
        out[fp32] = y
    assert torch.equal(out[True].bfloat16(), out[False])
    torch.cuda.synchronize()
    assert sq.last_device_status() == 0
    return out[False]


def test_reference_by_hand():
    y, mag = ref.linear_int8([[1, -2]], [0.5], [[3, 4], [-128, 127]], [1.0, 2.0], [10, 0])
    assert y.tolist() == [[7.5, -382.0]] and mag.tolist() == [[2.5, 382.0]]


MS = [1, 2, 3, 5, 8, 9, 16, 17, 31, 48, 64, 65, 100, 128, 129, 200, 256, 257, 400]


@pytest.mark.parametrize("M", MS)
@pytest.mark.parametrize("N,K", [(256, 256), (1000, 528), (136, 2064)])
def test_shapes(M, N, K):
    check(*operands(M * N, M, N, K))


@pytest.mark.parametrize("M", [1, 4, 7, 33, 130, 300])
@pytest.mark.parametrize("N,K", [(1, 16), (7, 48), (33, 160), (129, 1040), (2050, 272), (515, 16)])
def test_odd_extents(M, N, K):
    check(*operands(M + N, M, N, K))


@pytest.mark.parametrize("M", [1, 6, 40, 150, 1030])
@pytest.mark.parametrize("bdt", [torch.bfloat16, torch.float32])
def test_bias(M, bdt):
    x, w = operands(3, M, 648, 320)
    check(x, w, bias=torch.randn(648, device="cuda").to(bdt))
    # a bias that starts off a 16-byte boundary
    check(x, w, bias=torch.randn(649, device="cuda").to(bdt)[1:])


@pytest.mark.parametrize("M,N,K", [(1, 4096, 14336), (16, 28672, 4096), (48, 4096, 14336), (128, 6144, 4096),
                                   (512, 4608, 3584), (2041, 4608, 3584), (1, 37888, 3584), (64, 512, 65536),
                                   (300, 3584, 18944)])
def test_model_sizes(M, N, K):
    x, w = operands(5, M, N, K)
    rows = torch.arange(M, device="cuda") if M <= 64 else torch.randperm(M, device="cuda")[:64].sort().values
    check(x, w, rows=rows)


@pytest.mark.parametrize("M", [1, 5, 20, 200])
def test_extreme_codes(M):
    """All codes -128 at the longest K: sums of 2^30 must not wrap."""
    K, N = 65536, 160
    x = sq.PreparedInt8(torch.full((M, K), -128, dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda"), M, K)
    w = sq.WeightInt8(torch.full((N, K), -128, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda"), N, K)
    w.codes[1::2] = 127
    y = sq.linear_int8(x, w, out_fp32=True)
    assert bool((y[:, ::2] == 2.0 ** 30).all()) and bool((y[:, 1::2] == -128.0 * 127 * K).all())
    check(*operands(9, M, N, 1024, full=True))


@pytest.mark.parametrize("M", [1, 9, 70, 333])
def test_rows_do_not_depend_on_their_batch(M):
    x, w = operands(21, 400, 520, 784)
    y = sq.linear_int8(x, w)
    part = sq.PreparedInt8(x.codes[7:7 + M].clone(), x.scales[7:7 + M].clone(), M, x.K)
    assert torch.equal(sq.linear_int8(part, w), y[7:7 + M])


def test_no_rows_and_repeated_calls():
    x, w = operands(1, 0, 64, 64)
    assert sq.linear_int8(x, w).shape == (0, 64)
    for M in (1, 20, 90, 700):
        x, w = operands(M, M, 384, 4112)
        y = sq.linear_int8(x, w)
        for _ in range(5):
            assert torch.equal(sq.linear_int8(x, w), y)


def test_quantised_linear_end_to_end():
    """prepare_int8 + quantize_weight_int8 + linear_int8 against the unquantised
    product: each operand is off by at most half a step of its row."""
    M, N, K = 70, 512, 1024
    X = torch.randn((M, K), device="cuda").bfloat16()
    W = (0.02 * torch.randn((N, K), device="cuda")).bfloat16()
    x, w = sq.prepare_int8(X), sq.quantize_weight_int8(W)
    y = sq.linear_int8(x, w, out_fp32=True).double()
    want = X.double() @ W.double().t()
    hx, hw = 0.5001 * x.scales.double()[:, None], 0.5001 * w.scales.double()
    bound = hx * W.double().abs().sum(1) + X.double().abs().sum(1)[:, None] * hw + K * hx * hw
    assert bool(((y - want).abs() <= bound + 1e-5 * want.abs().max()).all())


@pytest.mark.parametrize("M", [3, 40, 64])
@pytest.mark.parametrize("N,K", [(130, 65536), (1024, 4096), (3584, 3584), (6144, 4096), (10240, 8192), (12288, 4096),
                                 (5000, 1040), (37000, 2064)])
def test_every_split_of_k(M, N, K):
    x, w = operands(M + N, M, N, K, full=True)
    check(x, w)
