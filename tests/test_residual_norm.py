"""The residual addition with its norms, gate and modulation, against the
64-bit reference.

Tolerances, before the last rounding.  Sums over K run as K / threads <= 64
terms a thread, then 10 butterfly steps: a statistic is within 80 2^-24
relative, its root and quotient add 4 steps; each factor or addition after it
one step of the value it makes.  So |y - y64| <= c 2^-24 (magnitudes added
into y), c = 100, where the magnitudes are those of every term: x and the
gated block output divided by the deviation, the mean (layer norm), beta and
shift.  The last rounding is half a step of the output's type."""
import numpy as np
import pytest
import torch

import activation_sparsity_prep_b200 as sq
import oracle.ops as ref

gpu = pytest.mark.gpu
C = 100 * 2.0 ** -24


def make(seed, M, K, G, dt, mdt, xdt, hdt, names, offset=0.0):
    g = np.random.default_rng(seed)

    def t(a, d):
        return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(d).cuda()

    kw = {}
    x = t(3 * g.standard_normal((M, K)) * np.exp(g.standard_normal((M, 1))) + offset, xdt)
    if "h" in names:
        kw["h"] = t(g.standard_normal((M, K)), hdt)
    for n in ("post_gamma", "gamma"):
        if n in names:
            kw[n] = t(0.5 + g.random(K), dt)
    if "beta" in names:
        kw["beta"] = t(0.1 * g.standard_normal(K), dt)
    if {"gate", "scale", "shift"} & set(names):
        mod = t(0.3 * g.standard_normal((G, 6, K)), mdt)
        for i, n in enumerate(("shift", "scale", "gate")):
            if n in names:
                kw[n] = mod[:, i]                            # strided chunks of one tensor
    return x, kw


def as64(kw):
    return {n: v.double().cpu().numpy() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}


def bounds(x, kw, norm, eps):
    """fp64 x', y and the magnitudes that their fp32 errors scale with."""
    kw64 = as64(kw)
    x64 = x.double().cpu().numpy()
    xp, y = ref.residual_norm(x64, norm=norm, eps=eps, **kw64)
    xmag = np.abs(x64) + np.abs(xp - x64)
    if y is None:
        return xp, None, xmag, None
    d = xp - xp.mean(1, keepdims=True) if norm == "layer" else xp
    r = 1 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    mag = xmag + (np.abs(xp).mean(1, keepdims=True) if norm == "layer" else 0)
    mag = mag * r
    M = len(x64)

    def rows(v):
        return np.repeat(v, M // len(v), axis=0)

    if "gamma" in kw64:
        mag = mag * np.abs(kw64["gamma"])
    if "beta" in kw64:
        mag = mag + np.abs(kw64["beta"])
    if "scale" in kw64:
        mag = mag * (1 + np.abs(rows(kw64["scale"])))
    if "shift" in kw64:
        mag = mag + np.abs(rows(kw64["shift"]))
    return xp, y, xmag, mag


def check(x, norm, eps=1e-6, **kw):
    xo, y = sq.residual_norm(x, norm=norm, eps=eps, **kw)
    torch.cuda.synchronize()
    xp, y64, xmag, mag = bounds(x, kw, norm, eps)
    if "h" in kw:
        half = torch.finfo(x.dtype).eps / 2
        assert xo.dtype == x.dtype
        assert np.all(np.abs(xo.double().cpu().numpy() - xp) <= C * xmag + half * np.abs(xp) * 1.01 + 1e-37)
    else:
        assert xo is x
    if norm is None:
        assert y is None
    else:
        assert y.dtype == torch.bfloat16
        assert np.all(np.abs(y.double().cpu().numpy() - y64) <= C * mag * 1.01 + 2.0 ** -8 * np.abs(y64) * 1.01 + 1e-37)
    return xo, y


def test_reference_by_hand():
    x, y = ref.residual_norm([[3.0, 4.0]], [[1.0, -1.0]], norm="rms", alpha=2.0, gate=[[1.0, 2.0]], eps=0.0)
    assert x.tolist() == [[5.0, 0.0]] and np.allclose(y, [[np.sqrt(2), 0]])
    x, y = ref.residual_norm([[1.0, 3.0]], norm="layer", gamma=[2, 2], beta=[1, 1], scale=[[1, 1]], shift=[[0, 5]], eps=0.0)
    assert np.allclose(y, [[-2, 11]])
    x, y = ref.residual_norm([[0.0, 0.0]], [[3.0, 4.0]], norm=None, post_gamma=[1, 2], eps=0.0)
    assert y is None and np.allclose(x, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])
    c, s = ref.quantize_rows_int8([[1.0, -2.0, 0.5], [0, 0, 0]])
    assert c.tolist() == [[64, -127, 32], [0, 0, 0]] and s.tolist() == [np.float32(2) / np.float32(127), 0]


B, F = torch.bfloat16, torch.float32


@gpu
@pytest.mark.parametrize("M,K", [(1, 8), (3, 264), (1, 4096), (5, 4104), (7, 8192), (2, 8200), (3, 18944), (2, 32768),
                                 (300, 1000), (64, 256)])
@pytest.mark.parametrize("norm", ["rms", "layer", None])
def test_sizes(M, K, norm):
    names = {"h", "post_gamma"} | ({"gamma"} if norm else set()) | ({"beta"} if norm == "layer" else set())
    x, kw = make(M + K, M, K, 1, B, B, B, B, names)
    check(x, norm, **kw)


@gpu
@pytest.mark.parametrize("xdt", [B, F])
@pytest.mark.parametrize("hdt", [B, F])
@pytest.mark.parametrize("dt,mdt", [(B, B), (F, B), (B, F)])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_types_and_modulation(xdt, hdt, dt, mdt, norm):
    names = {"h", "post_gamma", "gate", "gamma", "beta", "scale", "shift"}
    x, kw = make(7, 12, 520, 3, dt, mdt, xdt, hdt, names)
    check(x, norm, alpha=0.7, **kw)


@gpu
@pytest.mark.parametrize("names", [set(), {"h"}, {"h", "gate"}, {"gamma"}, {"beta"}, {"scale"}, {"shift"},
                                   {"h", "scale", "shift"}, {"h", "post_gamma", "gate"}])
@pytest.mark.parametrize("norm", ["rms", "layer", None])
def test_optional_parts(names, norm):
    if norm is None:
        names = names & {"h", "post_gamma", "gate"}
        if not names:
            return
    x, kw = make(9, 10, 1048, 5, B, B, F, B, names)
    check(x, norm, **kw)


@gpu
def test_a_row_for_each_modulation_row_and_large_offsets():
    x, kw = make(10, 33, 512, 33, B, F, F, B, {"h", "gate", "scale", "shift"}, offset=200.0)
    check(x, "layer", **kw)
    check(x, "rms", **kw)


@gpu
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_zero_and_constant_rows(norm):
    x = torch.zeros((4, 640), dtype=F).cuda()
    x[1] = 3.0
    x[2] = 1e-20
    x[3, 5] = 1.0
    _, y = sq.residual_norm(x, norm=norm)
    assert torch.isfinite(y.float()).all() and not y[0].any()
    if norm == "layer":
        assert not y[1].any()
    check(x[3:], norm)


@gpu
def test_strided_rows_in_place_and_batch_invariance():
    wide = torch.randn((40, 3 * 512), device="cuda").bfloat16()
    x, h = wide[:, 512:1024], wide[:, 1024:]
    gm = torch.rand(512, device="cuda").bfloat16()
    xo, y = check(x, "rms", h=h, gamma=gm)
    # one row alone gives the same bits
    x1, y1 = sq.residual_norm(x[17:18], h[17:18], gamma=gm)
    assert torch.equal(x1[0], xo[17]) and torch.equal(y1[0], y[17])
    # into x, and into h, with strided rows
    for target in ("x", "h"):
        w2 = wide.clone()
        xx, hh = w2[:, 512:1024], w2[:, 1024:]
        o, y2 = sq.residual_norm(xx, hh, gamma=gm, out_x=xx if target == "x" else hh)
        assert torch.equal(o, xo) and torch.equal(y2, y)
        assert torch.equal(w2[:, :512], wide[:, :512])       # its neighbours stay
        assert torch.equal((hh if target == "x" else xx), (h if target == "x" else x))


@gpu
def test_no_rows():
    x = torch.zeros((0, 64), dtype=B, device="cuda")
    xo, y = sq.residual_norm(x, x.clone())
    assert xo.shape == (0, 64) and y.shape == (0, 64)


# ----------------------------------------------------------------- 8 bits --

@gpu
@pytest.mark.parametrize("M,K", [(1, 16), (5, 264), (33, 4096), (3, 18944), (2, 32768)])
def test_quantised_rows_without_a_norm_are_bit_exact(M, K):
    g = np.random.default_rng(K)
    X = torch.from_numpy((g.standard_normal((M, K)) * np.exp(3 * g.standard_normal((M, 1)))).astype(np.float32)).bfloat16()
    X[0, :8] = torch.tensor([1.0, -1.0, 0.5, 0.25, -0.5, 0.0, -0.0, 1.0])
    if M > 1:
        X[1] = 0
    if M > 2:
        X[2] *= 1e-30
    if M > 4:
        X[4] = 1e-38
        X[3, 0] = torch.finfo(torch.bfloat16).max
    codes, scales = ref.quantize_rows_int8(X.float().numpy())
    for q in (sq.prepare_int8(X.cuda()), sq.quantize_weight_int8(X.cuda())):
        assert np.array_equal(q.codes.cpu().numpy(), codes)
        assert np.array_equal(q.scales.cpu().numpy(), scales)


@gpu
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("M,K", [(1, 8), (40, 4096), (6, 14336)])
def test_quantised_norm(M, K, norm):
    """A code is the nearest to y's quotient up to y's own error: at most half
    a step plus C times the magnitudes in steps."""
    x, kw = make(M * K, M, K, 1, B, B, F, B, {"h", "gamma", "scale", "shift"})
    _, q = sq.residual_norm(x, norm=norm, int8=True, **kw)
    _, y, _, mag = bounds(x, kw, norm, 1e-6)
    a = np.abs(y).max(1, keepdims=True)
    amag = mag.max(1, keepdims=True)
    s = q.scales.cpu().numpy().astype(np.float64)[:, None]
    assert np.all(np.abs(s - a / 127) <= C * 2 * amag / 127 + 2.0 ** -24 * a / 127)
    v = q.codes.cpu().numpy() * s
    assert np.all(np.abs(v - y) <= 0.5 * s * (1 + 2.0 ** -20) + 3 * C * amag)
    # the RMS form equals prepare_int8 on the same rows
    if norm == "rms":
        X = x.bfloat16()
        g = kw["gamma"]
        p = sq.prepare_int8(X, g)
        _, p2 = sq.residual_norm(X, gamma=g, int8=True)
        assert torch.equal(p.codes, p2.codes) and torch.equal(p.scales, p2.scales)
