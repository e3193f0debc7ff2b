"""The grouped linears where some choices take no row: rows from offsets[E]
on belong to no expert and come back as zeros, so that the prepare behind them,
whose tensor scales span all rows, sees nothing of what the memory held."""
import pytest
import torch

import activation_sparsity_prep_b200 as sq
from tests.test_layer_ops import MoeBlock, gen, randn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
NEG = -float("inf")


def routed(blk, T, live, seed):
    """A prepared norm output and a routing whose last T - live tokens, and a
    choice of the first, are masked."""
    g = gen(seed)
    x, y = sq.residual_norm(randn(g, T, blk.D), randn(g, T, blk.D), gamma=blk.gamma)
    logits = randn(g, T, blk.E)
    logits[live:] = NEG
    if live:
        logits[0, 1:] = NEG
    return x, y, sq.moe_route(logits, blk.k, score="sigmoid")


def junk(shape, dtype):
    """Memory as an allocation may find it: NaN, infinities and large values."""
    t = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    t[::3] = float("inf")
    t[1::3] = 3e38
    return t


def experts(blk, P, x, r, H0=None, Y0=None):
    H, amax = sq.moe_linear_swiglu(P, r.row_index, r.offsets, blk.up, out=H0)
    Y = sq.moe_linear(sq.prepare_amax(H, amax), None, r.offsets, blk.down, out=Y0)
    return H, amax, Y, sq.moe_combine(Y, r.position, r.weights, residual=x)


@pytest.mark.parametrize("T,live", [(1, 0), (1, 1), (9, 5), (40, 0), (130, 90), (700, 33)])
def test_masked_tokens_leave_nothing_behind(T, live):
    blk = MoeBlock()
    x, y, r = routed(blk, T, live, T + live)
    n, rows = int(r.offsets[-1]), T * blk.k
    assert n == (live - 1) * blk.k + 1 if live else n == 0
    P = sq.prepare(y)
    zeros = lambda c: torch.zeros((rows, c), dtype=BF, device="cuda")  # noqa: E731
    want = experts(blk, P, x, r, zeros(blk.I), zeros(blk.D))
    got = experts(blk, P, x, r, junk((rows, blk.I), BF), junk((rows, blk.D), BF))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not got[0][n:].any() and not got[2][n:].any()
    assert float(got[1]) == float(got[0].abs().max())
    assert torch.equal(got[3][live:], x[live:])               # a masked token keeps its residual
    # and with the call's own allocations, over memory left by others
    for _ in range(3):
        left = [junk((rows, c), BF) for c in (blk.I, blk.D, blk.I, blk.D)]
        del left
        own = experts(blk, P, x, r)
        assert all(torch.equal(a, b) for a, b in zip(own, want))
    torch.cuda.synchronize()
    assert sq.last_device_status() == 0


@pytest.mark.parametrize("residual_scale", ["own", "shared"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_rows_of_no_expert_are_zeros_in_every_form(fmt, residual_scale):
    """Both types of the result; the experts' rows as without dropped ones."""
    g = gen(3)
    T, E, N, K, n = 300, 5, 384, 256, 201
    P = sq.prepare(randn(g, T, K), None, fmt=fmt, residual_scale=residual_scale)
    off = torch.tensor([0, 3, 3, 140, 141, n], dtype=torch.int32, device="cuda")
    ri = torch.randint(0, T, (T,), generator=g, device="cuda", dtype=torch.int32)
    w = sq.Weight.empty(N, K, fmt, E=E)
    sb = sq.scale_bytes(N, K, fmt)
    for e in range(E):
        we = sq.Weight(w.codes[e], w.scales[e * sb:(e + 1) * sb], w.tensor_scale[e:e + 1], N, K, w.fmt)
        sq.quantize_weight(randn(g, N, K, scale=0.05), fmt, out=we)
    for fp32 in (False, True):
        dt = torch.float32 if fp32 else BF
        want = sq.moe_linear(P, ri[:n].contiguous(), off, w, out_fp32=fp32)
        got = sq.moe_linear(P, ri, off, w, out_fp32=fp32, out=junk((T, N), dt))
        assert torch.equal(got[:n], want) and not got[n:].any()
        # dispatched row t is prepared row t
        own = sq.moe_linear(P, None, off, w, out_fp32=fp32, out=junk((T, N), dt))
        rows = torch.arange(T, dtype=torch.int32, device="cuda")
        assert torch.equal(own, sq.moe_linear(P, rows, off, w, out_fp32=fp32)) and not own[n:].any()
    H, amax = sq.moe_linear_swiglu(P, ri, off, w, out=junk((T, N // 2), BF))
    want, a = sq.moe_linear_swiglu(P, ri[:n].contiguous(), off, w)
    assert torch.equal(H[:n], want) and torch.equal(amax, a) and not H[n:].any()
    torch.cuda.synchronize()
    assert sq.last_device_status() == 0


def test_captured_with_other_masks():
    """A graph replayed with other masks: rows that were an expert's before."""
    blk = MoeBlock()
    g = gen(8)
    T = 50
    x, y = sq.residual_norm(randn(g, T, blk.D), randn(g, T, blk.D), gamma=blk.gamma)
    P = sq.prepare(y)
    logits = randn(g, T, blk.E)
    fixed = logits.clone()

    def run():
        r = sq.moe_route(fixed, blk.k, score="sigmoid")
        return experts(blk, P, x, r)

    run()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = run()
    for live in (50, 7, 0, 31):
        fixed.copy_(logits)
        fixed[live:] = NEG
        gr.replay()
        r = sq.moe_route(fixed, blk.k, score="sigmoid")
        zeros = [torch.zeros((T * blk.k, c), dtype=BF, device="cuda") for c in (blk.I, blk.D)]
        want = experts(blk, P, x, r, *zeros)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_block_of_no_tokens():
    blk = MoeBlock()
    e = torch.zeros((0, blk.D), dtype=BF, device="cuda")
    out = blk(e, e.clone())
    torch.cuda.synchronize()
    assert out.shape == (0, blk.D) and sq.last_device_status() == 0
