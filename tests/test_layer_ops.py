"""The operators around the linears together, as a layer uses them: a
mixture-of-experts block from the residual stream back to it, an attention
projection in 8 bits, both captured into graphs and on other streams, with
guarded outputs."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import activation_sparsity_prep_b200 as sq
from activation_sparsity_prep_b200 import workloads as wl
import oracle.ops as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, scale=1.0, dtype=BF):
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def stacked(g, E, N, K):
    w = sq.Weight.empty(N, K, E=E)
    sb = sq.scale_bytes(N, K)
    for e in range(E):
        we = sq.Weight(w.codes[e], w.scales[e * sb:(e + 1) * sb], w.tensor_scale[e:e + 1], N, K, w.fmt)
        sq.quantize_weight(randn(g, N, K, scale=0.05), out=we)
    return w


class MoeBlock:
    """Residual addition and norm, router, SwiGLU experts, weighted sum."""

    def __init__(self, E=16, k=4, D=512, I=256, seed=1):
        g = gen(seed)
        self.E, self.k, self.D, self.I = E, k, D, I
        self.gamma = (0.5 + torch.rand(D, generator=g, device="cuda")).to(BF)
        self.router = randn(g, D, E, scale=0.1)
        self.bias = 0.05 * torch.randn(E, generator=g, device="cuda")
        self.up, self.down = stacked(g, E, 2 * I, D), stacked(g, E, D, I)

    def __call__(self, x, h, padded=None, keep=None):
        x2, y = sq.residual_norm(x, h, gamma=self.gamma)
        logits = y @ self.router
        if padded is not None:
            logits = logits.masked_fill(padded[:, None], -float("inf"))
        r = sq.moe_route(logits, self.k, score="sigmoid", bias=self.bias, groups=4, topk_groups=2, group_score="top2",
                         scale=1.5)
        T = r.row_index.numel()
        # rows of dropped choices stay as they are: zeros
        H0 = torch.zeros((T, self.I), dtype=BF, device="cuda")
        Y0 = torch.zeros((T, self.D), dtype=BF, device="cuda")
        H, amax = sq.moe_linear_swiglu(sq.prepare(y), r.row_index, r.offsets, self.up, out=H0)
        Y = sq.moe_linear(sq.prepare_amax(H, amax), None, r.offsets, self.down, out=Y0)
        out = sq.moe_combine(Y, r.position, r.weights, residual=x2)
        if keep is not None:
            keep.update(x2=x2, y=y, logits=logits, r=r, H=H, Y=Y)
        return out


@pytest.mark.parametrize("T", [1, 7, 65, 300])
@pytest.mark.parametrize("pad", [False, True])
def test_moe_block(T, pad):
    blk = MoeBlock()
    g = gen(T)
    x, h = randn(g, T, blk.D, scale=2.0), randn(g, T, blk.D)
    padded = torch.rand(T, generator=g, device="cuda") < 0.3 if pad else None
    if pad:
        padded[0] = T > 1
    k = {}
    out = blk(x, h, padded, k)
    torch.cuda.synchronize()
    assert sq.last_device_status() == 0
    ids, w = ref.route(k["logits"].float().cpu().numpy(), blk.k, "sigmoid", blk.bias.cpu().numpy(), 4, 2, "top2", True, 1.5)
    r = k["r"]
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    live = ids >= 0
    assert np.array_equal(live.all(1), ~padded.cpu().numpy()) if pad else live.all()
    # the grouped linears take this order as they take one made on the host
    n = int(live.sum())
    rows, off = wl.group_by_expert(np.where(live, ids, blk.E), blk.E + 1)
    assert np.array_equal(r.row_index.cpu().numpy()[:n], rows[:n])
    assert np.array_equal(r.offsets.cpu().numpy(), off[:blk.E + 1])
    if n:
        P = sq.prepare(k["y"])
        Hr, ar = sq.moe_linear_swiglu(P, torch.from_numpy(rows[:n].copy()).cuda(), r.offsets, blk.up)
        assert torch.equal(Hr, k["H"][:n]) and not k["H"][n:].any()
        Yr = sq.moe_linear(sq.prepare_amax(Hr, ar), None, r.offsets, blk.down)
        assert torch.equal(Yr, k["Y"][:n]) and not k["Y"][n:].any()
    want, mag = ref.combine(k["Y"].float().cpu().numpy(), r.position.cpu().numpy(), r.weights.cpu().numpy(),
                            k["x2"].float().cpu().numpy())
    err = np.abs(out.float().cpu().numpy() - want)
    assert np.all(err <= (blk.k + 2) * 2.0 ** -24 * mag * 1.01 + 2.0 ** -8 * np.abs(want) * 1.01)
    if pad:                                                 # a padded token keeps its residual
        assert torch.equal(out[padded], k["x2"][padded])


class Projection:
    """The 8-bit q/k/v projection behind a block."""

    def __init__(self, D=640, N=776, seed=3):
        g = gen(seed)
        self.gamma = (0.5 + torch.rand(D, generator=g, device="cuda")).to(BF)
        self.W = randn(g, N, D, scale=0.05)
        self.w = sq.quantize_weight_int8(self.W)
        self.bias = randn(g, N)

    def __call__(self, x, h):
        x2, q = sq.residual_norm(x, h, gamma=self.gamma, int8=True)
        return x2, q, sq.linear_int8(q, self.w, bias=self.bias)


@pytest.mark.parametrize("T", [1, 3, 40, 70, 515])
def test_projection_in_8_bits(T):
    p = Projection()
    g = gen(T)
    x, h = randn(g, T, 640, dtype=torch.float32), randn(g, T, 640)
    x2, q, y = p(x, h)
    assert x2.dtype == torch.float32
    want, mag = ref.linear_int8(q.codes.cpu().numpy(), q.scales.cpu().numpy(), p.w.codes.cpu().numpy(),
                                p.w.scales.cpu().numpy(), p.bias.float().cpu().numpy())
    err = np.abs(y.float().cpu().numpy() - want)
    assert np.all(err <= 4 * 2.0 ** -24 * mag + 2.0 ** -8 * np.abs(want) * 1.01 + 2.0 ** -24 * 16)
    # and near the product that was not quantised: half a step of each operand
    _, n = ref.residual_norm(x.cpu().numpy(), h.float().cpu().numpy(), gamma=p.gamma.float().cpu().numpy())
    W = p.W.float().cpu().numpy().astype(np.float64)
    hx = 0.5001 * q.scales.cpu().numpy()[:, None] + 1e-4 * np.abs(n).max()
    hw = 0.5001 * p.w.scales.cpu().numpy()
    bound = hx * np.abs(W).sum(1) + np.abs(n).sum(1)[:, None] * hw + 640 * hx * hw
    full = n @ W.T + p.bias.float().cpu().numpy()
    assert np.all(np.abs(y.float().cpu().numpy() - full) <= bound + 2.0 ** -8 * np.abs(full) * 1.01)


def everything(blk, proj, a):
    out = blk(a["x"], a["h"])
    return (out,) + tuple(proj(a["px"], a["ph"])[i] for i in (0, 2))


def inputs(T, seed):
    g = gen(seed)
    return {"x": randn(g, T, 512), "h": randn(g, T, 512), "px": randn(g, T, 640), "ph": randn(g, T, 640)}


@pytest.mark.parametrize("T", [1, 33, 150])
def test_captured_and_replayed(T):
    """Two graphs of the same calls, replayed in turn on new inputs."""
    blk, proj = MoeBlock(), Projection()
    states = [inputs(T, 5), inputs(T, 6)]
    everything(blk, proj, states[0])
    graphs = []
    for a in states:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = everything(blk, proj, a)
        graphs.append((gr, outs))
    for turn in range(3):
        for i, (gr, outs) in enumerate(graphs):
            fresh = inputs(T, 100 + 10 * turn + i)
            for n, v in states[i].items():
                v.copy_(fresh[n])
            want = everything(blk, proj, fresh)
            gr.replay()
            assert all(torch.equal(p, q) for p, q in zip(outs, want))
    torch.cuda.synchronize()
    assert sq.last_device_status() == 0


def test_streams_joined_by_events_eager_and_captured():
    """Work forked to a side stream and joined again: a call after the join
    sees what both wrote, also where it is placed early."""
    g = gen(31)
    w = sq.quantize_weight_int8(randn(g, 1040, 512, scale=0.05))
    w2 = sq.quantize_weight_int8(randn(g, 512, 1040, scale=0.05))
    x, h = randn(g, 300, 512), randn(g, 300, 512)
    side = torch.cuda.Stream()
    big = torch.randn((4096, 4096), device="cuda")

    def forked():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            slow = big @ big                                  # the side stream's result comes late
            hs = h * (1.0 + 0.0 * slow[0, 0]).to(BF)
            y = sq.linear_int8(sq.prepare_int8(hs), w)
        a, q = sq.residual_norm(x, h, int8=True)
        z = sq.linear_int8(q, w)
        main.wait_stream(side)
        _, q2 = sq.residual_norm(y, z, int8=True)
        out, _ = sq.residual_norm(a, sq.linear_int8(q2, w2))
        return a, y, z, out

    a, q = sq.residual_norm(x, h, int8=True)
    z = sq.linear_int8(q, w)
    y = sq.linear_int8(sq.prepare_int8(h), w)
    torch.cuda.synchronize()
    _, q2 = sq.residual_norm(y, z, int8=True)
    want = (a, y, z, sq.residual_norm(a, sq.linear_int8(q2, w2))[0])
    for _ in range(5):
        got = forked()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = forked()
    for _ in range(5):
        for t in got:
            t.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_first_calls_inside_a_capture():
    """A process whose first call of every operator is captured."""
    code = """
import torch, activation_sparsity_prep_b200 as sq
x = torch.randn(200, 512, device="cuda").bfloat16(); h = x.flip(0).contiguous(); l = torch.randn(5000, 64, device="cuda")
w = sq.WeightInt8(torch.ones(264, 512, dtype=torch.int8, device="cuda"), torch.ones(264, device="cuda"), 264, 512)
def run():
    out = []
    for n in (1, 50, 200):
        x2, q = sq.residual_norm(x[:n], h[:n], int8=True)
        out += [x2, sq.linear_int8(q, w)]
    for n in (3, 5000):
        r = sq.moe_route(l[:n], 4, bias=l[0].contiguous(), score="sigmoid")
        out += [r.ids, r.row_index, sq.moe_combine(x[:n * 4 if n < 50 else 200], r.position, r.weights)]
    return out
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = run()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, run()))
assert sq.last_device_status() == 0
print("captured")
"""
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert p.returncode == 0 and "captured" in p.stdout, p.stderr[-2000:]


def test_other_streams_at_once():
    """The same calls on two side streams at once, through `stream` and through
    the current stream, with temporaries freed under them."""
    blk, proj = MoeBlock(), Projection()
    a, b = inputs(200, 8), inputs(90, 9)
    want_a, want_b = everything(blk, proj, a), everything(blk, proj, b)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s):
            got_a = everything(blk, proj, a)
        with torch.cuda.stream(t):
            got_b = everything(blk, proj, b)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got_a, want_a))
        assert all(torch.equal(p, q) for p, q in zip(got_b, want_b))
    # stream=: outputs and temporaries belong to it
    x2, q = sq.residual_norm(a["px"], a["ph"], gamma=proj.gamma, int8=True, stream=s)
    y = sq.linear_int8(q, proj.w, bias=proj.bias, stream=s)
    logits = a["x"][:, :16]
    torch.cuda.current_stream().synchronize()
    r = sq.moe_route(logits, 3, stream=s)
    d = sq.moe_dispatch(r.ids, 16, stream=s)
    c = sq.moe_combine(want_a[0], r.position.clamp(max=0), r.weights, stream=s)
    s.synchronize()
    assert torch.equal(x2, want_a[1]) and torch.equal(y, want_a[2])
    assert torch.equal(d.position, r.position) and torch.equal(d.row_index, r.row_index)
    assert c.shape == (200, 512)


@pytest.mark.slow
def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: their last rows against the same
    rows alone."""
    g = gen(41)
    M, K = 540000, 4096                                      # 2.2e9 elements
    x, h = torch.zeros((M, K), dtype=BF, device="cuda"), torch.zeros((M, K), dtype=BF, device="cuda")
    x[-3:], h[-3:] = randn(g, 3, K), randn(g, 3, K)
    gm = (0.5 + torch.rand(K, generator=g, device="cuda")).to(BF)
    xo, y = sq.residual_norm(x, h, gamma=gm)
    x1, y1 = sq.residual_norm(x[-3:], h[-3:], gamma=gm)
    assert torch.equal(xo[-3:], x1) and torch.equal(y[-3:], y1) and not y[:5].any()
    del xo, y
    _, q = sq.residual_norm(x, h, gamma=gm, int8=True)
    _, q1 = sq.residual_norm(x[-3:], h[-3:], gamma=gm, int8=True)
    assert torch.equal(q.codes[-3:], q1.codes) and torch.equal(q.scales[-3:], q1.scales)
    # experts' rows behind 2^31 elements
    pos = torch.tensor([[M - 1, M - 3], [M - 2, 0]], dtype=torch.int32, device="cuda")
    w = torch.rand((2, 2), generator=g, device="cuda")
    near = torch.cat((x[:1], x[-3:]))
    assert torch.equal(sq.moe_combine(x, pos, w), sq.moe_combine(near, torch.tensor([[3, 1], [2, 0]], dtype=torch.int32,
                                                                                    device="cuda"), w))
    # a product whose operand and whose result pass it
    w8 = sq.quantize_weight_int8(randn(g, 264, K, scale=0.05))
    assert torch.equal(sq.linear_int8(q, w8)[-3:], sq.linear_int8(q1, w8))
    del x, h, q
    a = sq.prepare_int8(randn(g, 36000, 32))
    b = sq.quantize_weight_int8(randn(g, 60008, 32))
    out = sq.linear_int8(a, b)                               # 2.2e9 elements
    tail = sq.PreparedInt8(a.codes[-2:].clone(), a.scales[-2:].clone(), 2, 32)
    assert torch.equal(out[-2:], sq.linear_int8(tail, b))
    wt = sq.WeightInt8(b.codes[-8:].clone(), b.scales[-8:].clone(), 8, 32)
    assert torch.equal(out[:, -8:], sq.linear_int8(a, wt))
    del out
    # a long weight for one token
    one = sq.prepare_int8(randn(g, 1, 4096))
    big = sq.WeightInt8(torch.zeros((540000, 4096), dtype=torch.int8, device="cuda"), torch.ones(540000, device="cuda"), 540000, 4096)
    big.codes[-1] = 1
    y = sq.linear_int8(one, big, out_fp32=True)
    assert float(y[0, -1]) != 0 and not y[0, :-1].any()
    want = float(one.codes.double().sum()) * float(one.scales[0])
    assert abs(float(y[0, -1]) - want) <= 4 * 2.0 ** -24 * abs(want)
    torch.cuda.synchronize()
    assert sq.last_device_status() == 0


# ------------------------------------------------------------- guarded ----

GUARD = 4096


class Guarded:
    """Buffers inside larger ones whose margins must keep their bytes."""

    def __init__(self):
        self.held = []

    def __call__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        raw = torch.full((n + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.held.append((raw, n))
        return raw[GUARD:GUARD + n].view(dtype).view(shape)

    def intact(self):
        return all(bool((r[:GUARD] == 0xA5).all()) and bool((r[GUARD + n:] == 0xA5).all()) for r, n in self.held)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 60, 6), (64, 128, 8), (65, 16, 3), (1500, 256, 8), (5000, 40, 8)])
def test_guarded_routing(T, E, k):
    g, G = gen(T), Guarded()
    l = torch.randn((T, E), generator=g, device="cuda")
    l[torch.rand(T, generator=g, device="cuda") < 0.2] = -float("inf")
    want = sq.moe_route(l, k)
    i32 = torch.int32
    out = sq.Routing(G((T, k), i32), G((T, k), torch.float32), G((T * k,), i32), G((E + 1,), i32), G((T, k), i32))
    assert sq.moe_route(l, k, out=out) is out
    for n in ("ids", "weights", "row_index", "offsets", "position"):
        assert torch.equal(getattr(out, n), getattr(want, n)), n
    for N in (8, 264, 2056):
        Y = torch.randn((T * k, N), generator=g, device="cuda").to(BF)
        res = torch.randn((T, N), generator=g, device="cuda")
        o = G((T, N), torch.float32)
        sq.moe_combine(Y, out.position, out.weights, residual=res, out=o)
        assert torch.equal(o, sq.moe_combine(Y, want.position, want.weights, residual=res))
    assert G.intact()


@pytest.mark.parametrize("M,K", [(1, 8), (5, 264), (3, 4104), (700, 520), (2500, 264), (1300, 3584), (700, 4104), (400, 18944)])
@pytest.mark.parametrize("xdt", [BF, torch.float32])
def test_guarded_residual_norm(M, K, xdt):
    """Few rows and many, whole and ragged chunks; a row of a large batch has
    the bits of the row alone."""
    g, G = gen(M + K), Guarded()
    x, h = randn(g, M, K, dtype=xdt), randn(g, M, K)
    gm = (0.5 + torch.rand(K, generator=g, device="cuda")).to(BF)
    mod = randn(g, 1, 6, K, scale=0.3)
    for kw in (dict(gamma=gm), dict(post_gamma=gm, norm="layer"), dict(gate=mod[:, 0], scale=mod[:, 1], shift=mod[:, 2], norm="layer"),
               dict(post_gamma=gm, gate=mod[:, 0], gamma=gm, scale=mod[:, 1], alpha=0.5), dict(norm=None)):
        ox = G((M, K), xdt)
        oy = None if kw.get("norm", "rms") is None else G((M, K), BF)
        sq.residual_norm(x, h, out_x=ox, out_y=oy, **kw)
        at = M // 2
        x1, y1 = sq.residual_norm(x[at:at + 1], h[at:at + 1], **kw)
        assert torch.equal(ox[at], x1[0]) and (oy is None or torch.equal(oy[at], y1[0]))
        assert torch.isfinite(ox.float()).all()
    q = sq.PreparedInt8(G((M, K), torch.int8), G((M,), torch.float32), M, K)
    sq.residual_norm(x, h, gamma=gm, int8=True, out_y=q)
    _, q1 = sq.residual_norm(x[-1:], h[-1:], gamma=gm, int8=True)
    assert torch.equal(q.codes[-1], q1.codes[0]) and torch.equal(q.scales[-1:], q1.scales)
    if xdt == BF:
        sq.prepare_int8(x, out=q)
        codes, scales = ref.quantize_rows_int8(x.float().cpu().numpy())
        assert np.array_equal(q.codes.cpu().numpy(), codes) and np.array_equal(q.scales.cpu().numpy(), scales)
        w = sq.WeightInt8(q.codes, q.scales, M, K)
        q.codes.zero_()
        sq.quantize_weight_int8(x, out=w)
        assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert G.intact()


@pytest.mark.parametrize("M", [1, 2, 3, 16, 50, 64, 65, 200, 300, 1025])
@pytest.mark.parametrize("N,K", [(8, 1040), (36, 2064), (1000, 512), (515, 1152), (4100, 2064)])
@pytest.mark.parametrize("fp32", [False, True])
def test_guarded_linear_int8(M, N, K, fp32):
    g, G = gen(M + N), Guarded()
    x = sq.PreparedInt8.empty(M, K)
    w = sq.WeightInt8.empty(N, K)
    for t in (x, w):
        t.codes.copy_(torch.randint(-127, 128, t.codes.shape, generator=g, device="cuda", dtype=torch.int8))
        t.scales.copy_(torch.rand(t.scales.shape, generator=g, device="cuda"))
    out = G((M, N), torch.float32 if fp32 else BF)
    sq.linear_int8(x, w, out_fp32=fp32, out=out)
    want = (x.codes.double() @ w.codes.double().t()) * x.scales.double()[:, None] * w.scales.double()
    tol = 4 * 2.0 ** -24 if fp32 else 4 * 2.0 ** -24 + 2.0 ** -8 * 1.01
    assert bool(((out.double() - want).abs() <= tol * want.abs()).all())
    assert G.intact()
    torch.cuda.synchronize()
    assert sq.last_device_status() == 0
