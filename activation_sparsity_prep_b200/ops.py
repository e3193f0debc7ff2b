"""The rest of a layer around its linears: routing to experts and back, the
residual addition with its norms, and linears in 8-bit integers.

Python binding of the second half of ``include/sharq.h``, where the formulas
stand.  As in the rest of the package every call checks its tensors first
(ValueError, nothing enqueued), returns without synchronising, and has no CPU
fallback.  A call runs on the device of its tensors; with ``stream`` it runs
there, and what it allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

_P, _I, _I64, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float


class _Routing(ctypes.Structure):
    _fields_ = [("ids", _P), ("weights", _P), ("row_index", _P), ("offsets", _P), ("position", _P),
                ("T", _I64), ("k", _I), ("E", _I)]


class _RouteOptions(ctypes.Structure):
    _fields_ = [("score", _I), ("groups", _I), ("topk_groups", _I), ("group_score", _I),
                ("renormalize", _I), ("scale", _F)]


class _RowsInt8(ctypes.Structure):
    _fields_ = [("codes", _P), ("scales", _P), ("M", _I64), ("K", _I)]


class _WeightInt8(ctypes.Structure):
    _fields_ = [("codes", _P), ("scales", _P), ("N", _I), ("K", _I)]


class _ResidualNorm(ctypes.Structure):
    _fields_ = ([(n, _P) for n in ("x", "h", "post_gamma", "gate", "gamma", "beta", "scale", "shift", "out_x", "y")]
                + [("q", ctypes.POINTER(_RowsInt8))]
                + [(n, _I64) for n in ("ld_x", "ld_h", "ld_gate", "ld_scale", "ld_shift", "ld_out", "M", "G")]
                + [(n, _I) for n in ("K", "norm", "x_is_fp32", "h_is_fp32", "norm_is_fp32", "mod_is_fp32")]
                + [("alpha", _F), ("eps", _F)])


def _declare(L: ctypes.CDLL) -> None:
    """Argument types of the entry points this module calls."""
    R = ctypes.POINTER(_Routing)
    for name, args in (
            ("sharq_moe_route", [_P, _I64, _I, _P, ctypes.POINTER(_RouteOptions), R, _P]),
            ("sharq_moe_dispatch", [R, _P]),
            ("sharq_moe_combine", [_P, _I, _I64, _I, _P, _P, _I64, _I, _P, _P, _I, _P]),
            ("sharq_residual_norm", [ctypes.POINTER(_ResidualNorm), _P]),
            ("sharq_prepare_int8", [_P, _P, _F, ctypes.POINTER(_RowsInt8), _P]),
            ("sharq_quantize_weight_int8", [_P, ctypes.POINTER(_WeightInt8), _P]),
            ("sharq_linear_int8", [ctypes.POINTER(_RowsInt8), ctypes.POINTER(_WeightInt8), _P, _I, _P, _I, _P])):
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, _I


_lib = None


def _load() -> ctypes.CDLL:
    global _lib
    from . import load_sharq_ops
    L = load_sharq_ops()
    _declare(L)
    _lib = L
    return L


def _call(name: str, *args) -> None:
    st = getattr(_lib or _load(), name)(*args)
    if st != 0:
        from . import SharqError
        raise SharqError(name, st)


def _stream(dev) -> int:
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _placed(fn):
    """Run a call on its first tensor's device and, when given, on `stream`:
    kernels, allocations and frees then all belong to that stream."""
    sig = inspect.signature(fn)
    name = next(iter(sig.parameters))

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = args[0] if args else kw.get(name)
        t = first.codes if isinstance(first, (PreparedInt8, WeightInt8)) else first
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{fn.__name__} needs CUDA tensors")
        if stream is None and t.device.index == torch._C._cuda_getDevice():
            return fn(*args, **kw)
        if stream is not None and stream.device != t.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
        with torch.cuda.device(t.device), torch.cuda.stream(stream):
            return fn(*args, **kw)
    call.__signature__ = sig.replace(parameters=[*sig.parameters.values(), inspect.Parameter(
        "stream", inspect.Parameter.KEYWORD_ONLY, default=None)])
    return call


_BF16_FP32 = (torch.bfloat16, torch.float32)


def _flat(name: str, t, shape: Tuple[int, ...], dtypes, dev, align: int = 16):
    """t: a contiguous tensor of `shape` and one of `dtypes` on `dev`."""
    _kind(name, t, shape, dtypes, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.data_ptr() % align:
        raise ValueError(f"{name} must start on a {align}-byte boundary")


def _kind(name: str, t, shape, dtypes, dev):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is required")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _rows(name: str, t, shape: Tuple[int, int], dtypes, dev, align: int = 16) -> int:
    """t: [rows, K] with unit stride along K, any row stride of whole
    `align` bytes; returns that stride in elements."""
    _kind(name, t, shape, dtypes, dev)
    ld, unit = t.stride()
    if unit != 1 and shape[1] != 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    if shape[0] <= 1:
        ld = shape[1]
    elif ld < shape[1]:
        raise ValueError(f"{name} must not overlap itself (row stride {ld})")
    if t.data_ptr() % align or (shape[0] > 1 and ld * t.element_size() % align):
        raise ValueError(f"every row of {name} must start on a {align}-byte boundary")
    return ld


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------- routing --

_SCORE = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORE = {"max": 0, "top2": 1}
_I32 = (torch.int32,)
_FP32 = (torch.float32,)


@dataclass
class Routing:
    """Each token's experts and the order a grouped linear takes them in."""
    ids: "object"            # int32 [T, k], -1 for none
    weights: "object"        # fp32 [T, k] (None when built by moe_dispatch)
    row_index: "object"      # int32 [T * k], token of each dispatched row
    offsets: "object"        # int32 [E + 1]
    position: "object"       # int32 [T, k], dispatched row of each choice, -1 for none

    @staticmethod
    def empty(T: int, k: int, E: int, device="cuda") -> "Routing":
        # one allocation; every part starts on a 16-byte boundary
        n = T * k
        pad, off = (n + 3) // 4 * 4, (E + 4) // 4 * 4
        b = torch.empty((4 * pad + off,), dtype=torch.int32, device=device)
        grid, rows = (T, k), (k, 1)
        return Routing(b.as_strided(grid, rows, 0), b.view(torch.float32).as_strided(grid, rows, pad),
                       b.as_strided((n,), (1,), 2 * pad), b.as_strided((E + 1,), (1,), 3 * pad),
                       b.as_strided(grid, rows, 3 * pad + off))


def _check_routing(r: Routing, T: int, k: int, E: int, dev) -> None:
    _flat("out.ids", r.ids, (T, k), _I32, dev, 4)
    _flat("out.weights", r.weights, (T, k), _FP32, dev, 4)
    _flat("out.row_index", r.row_index, (T * k,), _I32, dev, 4)
    _flat("out.offsets", r.offsets, (E + 1,), _I32, dev, 4)
    _flat("out.position", r.position, (T, k), _I32, dev, 4)


@_placed
def moe_route(logits, k: int, score: str = "softmax", bias=None, groups: int = 1, topk_groups: int = 1,
              group_score: str = "max", renormalize: bool = True, scale: float = 1.0,
              out: Optional[Routing] = None) -> Routing:
    """Choose k experts for each token and build the dispatch order.

    logits: [T, E] bf16 or fp32 (any row stride), -inf or NaN where an expert
    is masked; score: "softmax" or "sigmoid"; bias: fp32 [E], added for the
    choice only; groups / topk_groups / group_score ("max" or "top2"): keep
    the best groups of neighbouring experts first.  A token with fewer than k
    experts left has ids of -1 and weights of 0 behind them; those choices take
    no dispatched row, and the grouped linears return zeros in the rows behind
    the last live one.  The result's row_index and offsets go to moe_linear (up
    to 256 experts, where E may be 512 here), position and weights to
    moe_combine."""
    if logits.dim() != 2:
        raise ValueError("logits must be a 2-D tensor [T, E]")
    T, E = logits.shape
    dev = logits.device
    if score not in _SCORE:
        raise ValueError(f"score is {score!r}, expected 'softmax' or 'sigmoid'")
    if group_score not in _GROUP_SCORE:
        raise ValueError(f"group_score is {group_score!r}, expected 'max' or 'top2'")
    if not 1 <= E <= 512:
        raise ValueError(f"E={E} experts, expected 1 to 512")
    if not 1 <= groups <= 32 or E % groups:
        raise ValueError(f"groups={groups} must divide E={E} and be at most 32")
    if not 1 <= topk_groups <= groups:
        raise ValueError(f"topk_groups={topk_groups}, expected 1 to {groups}")
    if not 1 <= k <= min(32, E // groups * topk_groups):
        raise ValueError(f"k={k}, expected 1 to {min(32, E // groups * topk_groups)}")
    if T * k >= 2 ** 31:
        raise ValueError(f"T * k = {T * k} choices, expected below 2^31")
    ld = _rows("logits", logits, (T, E), _BF16_FP32, dev, 2)
    if bias is not None:
        _flat("bias", bias, (E,), _FP32, dev, 4)
    if out is not None:
        _check_routing(out, T, k, E, dev)
    r = out if out is not None else Routing.empty(T, k, E, dev)
    opt = _RouteOptions(_SCORE[score], groups, topk_groups, _GROUP_SCORE[group_score], 1 if renormalize else 0, scale)
    c = _Routing(r.ids.data_ptr(), r.weights.data_ptr(), r.row_index.data_ptr(), r.offsets.data_ptr(),
                 r.position.data_ptr(), T, k, E)
    _call("sharq_moe_route", logits.data_ptr(), ld, 1 if logits.dtype == torch.float32 else 0, _ptr(bias),
          ctypes.byref(opt), ctypes.byref(c), _stream(dev))
    return r


@_placed
def moe_dispatch(ids, E: int) -> Routing:
    """Dispatch order of given expert ids (int32 [T, k]; outside 0 .. E-1:
    dropped), as moe_route builds it.  The result's weights are None."""
    if ids.dim() != 2:
        raise ValueError("ids must be a 2-D tensor [T, k]")
    T, k = ids.shape
    dev = ids.device
    if not 1 <= E <= 512:
        raise ValueError(f"E={E} experts, expected 1 to 512")
    if k < 1 or T * k >= 2 ** 31:
        raise ValueError(f"T * k = {T * k} choices of k={k}, expected k >= 1 and below 2^31")
    _flat("ids", ids, (T, k), _I32, dev, 4)
    i32 = dict(dtype=torch.int32, device=dev)
    r = Routing(ids, None, torch.empty((T * k,), **i32), torch.empty((E + 1,), **i32), torch.empty((T, k), **i32))
    c = _Routing(ids.data_ptr(), None, r.row_index.data_ptr(), r.offsets.data_ptr(), r.position.data_ptr(), T, k, E)
    _call("sharq_moe_dispatch", ctypes.byref(c), _stream(dev))
    return r


@_placed
def moe_combine(Y, position, weights, residual=None, out=None):
    """Expert outputs back to the tokens: sum_j weights[t, j] *
    Y[position[t, j]] (+ residual[t]).  Y: [rows, N] in dispatch order, bf16
    or fp32; position int32 and weights fp32 [T, k]; residual [T, N] bf16 or
    fp32, which is then the result's type (else Y's).  out may be residual."""
    if Y.dim() != 2:
        raise ValueError("Y must be a 2-D tensor [rows, N]")
    rows, N = Y.shape
    dev = Y.device
    _flat("Y", Y, (rows, N), _BF16_FP32, dev)
    if N < 8 or N % 8 or N > 2 ** 24:
        raise ValueError(f"N={N} must be a multiple of 8 from 8 to 2^24")
    if not isinstance(position, torch.Tensor) or position.dim() != 2:
        raise ValueError("position must be a 2-D tensor [T, k]")
    T, k = position.shape
    if k < 1:
        raise ValueError("position must have k >= 1 columns")
    _flat("position", position, (T, k), _I32, dev, 4)
    _flat("weights", weights, (T, k), _FP32, dev, 4)
    dt = Y.dtype
    if residual is not None:
        _flat("residual", residual, (T, N), _BF16_FP32, dev)
        dt = residual.dtype
    if out is not None:
        _flat("out", out, (T, N), (dt,) if residual is not None else _BF16_FP32, dev)
    else:
        out = torch.empty((T, N), dtype=dt, device=dev)
    _call("sharq_moe_combine", Y.data_ptr(), 1 if Y.dtype == torch.float32 else 0, rows, N, position.data_ptr(),
          weights.data_ptr(), T, k, _ptr(residual), out.data_ptr(), 1 if out.dtype == torch.float32 else 0,
          _stream(dev))
    return out


# ------------------------------------------------- 8-bit integer operands --

@dataclass
class PreparedInt8:
    """8-bit tokens with one scale each."""
    codes: "object"          # int8 [M, K]
    scales: "object"         # fp32 [M]
    M: int
    K: int

    @staticmethod
    def empty(M: int, K: int, device="cuda") -> "PreparedInt8":
        return PreparedInt8(torch.empty((M, K), dtype=torch.int8, device=device),
                            torch.empty((M,), dtype=torch.float32, device=device), M, K)


@dataclass
class WeightInt8:
    """8-bit weight with one scale for each output channel."""
    codes: "object"          # int8 [N, K]
    scales: "object"         # fp32 [N]
    N: int
    K: int

    @staticmethod
    def empty(N: int, K: int, device="cuda") -> "WeightInt8":
        return WeightInt8(torch.empty((N, K), dtype=torch.int8, device=device),
                          torch.empty((N,), dtype=torch.float32, device=device), N, K)


_I8 = (torch.int8,)


def _check_rows8(name: str, q, rows: int, K: int, dev) -> None:
    _flat(f"{name} codes", q.codes, (rows, K), _I8, dev)
    _flat(f"{name} scales", q.scales, (rows,), _FP32, dev, 4)


def _check_extent(K: int) -> None:
    if not 8 <= K <= 32768 or K % 8:
        raise ValueError(f"K={K}, expected a multiple of 8 from 8 to 32768")


@_placed
def prepare_int8(X, gamma=None, eps: float = 1e-6, out: Optional[PreparedInt8] = None) -> PreparedInt8:
    """X bf16 [M, K] -> 8-bit codes and a scale for each row, after RMSNorm
    with gamma (bf16 [K]) when it is given.  K: a multiple of 8 up to 32768
    (of 16 where linear_int8 follows).  A row with NaN or infinities gets a
    scale that is not finite."""
    if X.dim() != 2:
        raise ValueError("X must be a 2-D tensor [M, K]")
    M, K = X.shape
    dev = X.device
    _check_extent(K)
    _flat("X", X, (M, K), (torch.bfloat16,), dev)
    if gamma is not None:
        _flat("gamma", gamma, (K,), (torch.bfloat16,), dev)
    if out is not None:
        if (out.M, out.K) != (M, K):
            raise ValueError(f"out describes M={out.M}, K={out.K}; the call needs M={M}, K={K}")
        _check_rows8("out", out, M, K, dev)
    q = out if out is not None else PreparedInt8(torch.empty_like(X, dtype=torch.int8),
                                                 torch.empty((M,), dtype=torch.float32, device=dev), M, K)
    c = _RowsInt8(q.codes.data_ptr(), q.scales.data_ptr(), M, K)
    _call("sharq_prepare_int8", X.data_ptr(), _ptr(gamma), eps, ctypes.byref(c), _stream(dev))
    return q


@_placed
def quantize_weight_int8(W, out: Optional[WeightInt8] = None) -> WeightInt8:
    """W bf16 [N, K] -> 8-bit codes and a scale for each output channel; K as
    prepare_int8."""
    if W.dim() != 2:
        raise ValueError("W must be a 2-D tensor [N, K]")
    N, K = W.shape
    dev = W.device
    if N < 1:
        raise ValueError("W must have at least one row")
    _check_extent(K)
    _flat("W", W, (N, K), (torch.bfloat16,), dev)
    if out is not None:
        if (out.N, out.K) != (N, K):
            raise ValueError(f"out describes N={out.N}, K={out.K}; the call needs N={N}, K={K}")
        _check_rows8("out", out, N, K, dev)
    w = out if out is not None else WeightInt8.empty(N, K, dev)
    c = _WeightInt8(w.codes.data_ptr(), w.scales.data_ptr(), N, K)
    _call("sharq_quantize_weight_int8", W.data_ptr(), ctypes.byref(c), _stream(dev))
    return w


@_placed
def linear_int8(x: PreparedInt8, w: WeightInt8, bias=None, out_fp32: bool = False, out=None):
    """Linear in 8-bit integers: Y[i, j] = x.scales[i] * w.scales[j] *
    sum_k x.codes[i, k] * w.codes[j, k] (+ bias[j]), the sum exact.  K: a
    multiple of 16 up to 65536; bias: bf16 or fp32 [N]; Y: bf16, or fp32 with
    out_fp32."""
    if not isinstance(x, PreparedInt8) or not isinstance(w, WeightInt8):
        raise ValueError("linear_int8 takes a PreparedInt8 and a WeightInt8")
    dev = x.codes.device
    if w.K != x.K:
        raise ValueError(f"weight K={w.K} does not match the activations' K={x.K}")
    if not 16 <= x.K <= 65536 or x.K % 16:
        raise ValueError(f"K={x.K}, expected a multiple of 16 from 16 to 65536")
    if not 1 <= w.N <= 2 ** 30 or x.M > 2 ** 30:
        raise ValueError(f"M={x.M}, N={w.N}, expected M up to 2^30 and N from 1 to 2^30")
    _check_rows8("x", x, x.M, x.K, dev)
    _check_rows8("weight", w, w.N, w.K, dev)
    if bias is not None:
        _flat("bias", bias, (w.N,), _BF16_FP32, dev, bias.element_size())
    dt = torch.float32 if out_fp32 else torch.bfloat16
    if out is not None:
        _flat("out", out, (x.M, w.N), (dt,), dev)
    else:
        out = torch.empty((x.M, w.N), dtype=dt, device=dev)
    cx = _RowsInt8(x.codes.data_ptr(), x.scales.data_ptr(), x.M, x.K)
    cw = _WeightInt8(w.codes.data_ptr(), w.scales.data_ptr(), w.N, w.K)
    _call("sharq_linear_int8", ctypes.byref(cx), ctypes.byref(cw), _ptr(bias),
          1 if bias is not None and bias.dtype == torch.float32 else 0, out.data_ptr(), 1 if out_fp32 else 0,
          _stream(dev))
    return out


# ------------------------------------------------------ residual stream --

_NORM = {None: 0, "rms": 1, "layer": 2}


@_placed
def residual_norm(x, h=None, norm: Optional[str] = "rms", post_gamma=None, gate=None, alpha: float = 1.0,
                  gamma=None, beta=None, scale=None, shift=None, eps: float = 1e-6, int8: bool = False,
                  out_x=None, out_y=None):
    """The residual addition with the norms, gate and modulation around it:

        u  = h, or RMSNorm(h) * post_gamma
        x' = x + alpha * gate * u
        y  = norm(x') * gamma + beta, then y * (1 + scale) + shift

    norm: "rms", "layer" or None (no y).  x: [M, K] bf16 or fp32, h: [M, K]
    bf16 or fp32 (rows may be strided); gate, scale, shift: [G, K] (rows may be
    strided: the chunks of one modulation tensor), row r of M using row
    r // (M / G).  Returns (x', y): x' in x's type (x itself when h is None),
    y bf16, or a PreparedInt8 with int8=True, or None.  out_x may be x or h."""
    if x.dim() != 2:
        raise ValueError("x must be a 2-D tensor [M, K]")
    M, K = x.shape
    dev = x.device
    _check_extent(K)
    if norm not in _NORM:
        raise ValueError(f"norm is {norm!r}, expected 'rms', 'layer' or None")
    a = _ResidualNorm()
    a.ld_x = _rows("x", x, (M, K), _BF16_FP32, dev)
    if h is not None:
        a.ld_h = _rows("h", h, (M, K), _BF16_FP32, dev)
        a.h, a.h_is_fp32 = h.data_ptr(), h.dtype == torch.float32
    elif post_gamma is not None or gate is not None:
        raise ValueError("post_gamma and gate need h")
    elif norm is None:
        raise ValueError("without h and without a norm there is nothing to compute")
    if norm is None:
        if gamma is not None or beta is not None or scale is not None or shift is not None:
            raise ValueError("gamma, beta, scale and shift need a norm")
        if int8 or out_y is not None:
            raise ValueError("int8 and out_y need a norm")
    if post_gamma is not None or gamma is not None or beta is not None:
        first = None
        for name, v in (("post_gamma", post_gamma), ("gamma", gamma), ("beta", beta)):
            if v is not None:
                _flat(name, v, (K,), _BF16_FP32, dev)
                first = first or (name, v.dtype)
                if v.dtype != first[1]:
                    raise ValueError(f"{name} is {v.dtype}, {first[0]} is {first[1]}")
                setattr(a, name, v.data_ptr())
        a.norm_is_fp32 = first[1] == torch.float32
    a.G = 1
    if gate is not None or scale is not None or shift is not None:
        first = None
        for name, v in (("gate", gate), ("scale", scale), ("shift", shift)):
            if v is not None:
                if first is None:
                    if not isinstance(v, torch.Tensor) or v.dim() != 2:
                        raise ValueError(f"{name} must be a 2-D tensor [G, K]")
                    first, G = (name, v.dtype), v.shape[0]
                    if G < 1 or M % G:
                        raise ValueError(f"G={G} rows of {name} must divide M={M}")
                setattr(a, "ld_" + name, _rows(name, v, (G, K), _BF16_FP32, dev))
                if v.dtype != first[1]:
                    raise ValueError(f"{name} is {v.dtype}, {first[0]} is {first[1]}")
                setattr(a, name, v.data_ptr())
        a.G, a.mod_is_fp32 = G, first[1] == torch.float32
    if out_x is not None:
        a.ld_out = _rows("out_x", out_x, (M, K), (x.dtype,), dev)
        for name, v, ld in (("x", x, a.ld_x), ("h", h, a.ld_h)):
            if v is not None and v.data_ptr() == out_x.data_ptr() and (ld != a.ld_out or v.dtype != x.dtype):
                raise ValueError(f"out_x starts where {name} does but has another layout")
        a.out_x = out_x.data_ptr()
    elif h is not None:
        out_x = torch.empty_like(x, memory_format=torch.contiguous_format)
        a.out_x, a.ld_out = out_x.data_ptr(), K
    y, q = None, None
    if norm is not None:
        if int8:
            if out_y is not None:
                if not isinstance(out_y, PreparedInt8) or (out_y.M, out_y.K) != (M, K):
                    raise ValueError(f"out_y must be a PreparedInt8 of M={M}, K={K}")
                _check_rows8("out_y", out_y, M, K, dev)
            y = out_y if out_y is not None else PreparedInt8.empty(M, K, dev)
            q = _RowsInt8(y.codes.data_ptr(), y.scales.data_ptr(), M, K)
            a.q = ctypes.pointer(q)
        else:
            if out_y is not None:
                _flat("out_y", out_y, (M, K), (torch.bfloat16,), dev)
            y = out_y if out_y is not None else torch.empty_like(x, dtype=torch.bfloat16,
                                                                 memory_format=torch.contiguous_format)
            a.y = y.data_ptr()
    a.x, a.x_is_fp32 = x.data_ptr(), x.dtype == torch.float32
    a.M, a.K, a.norm, a.alpha, a.eps = M, K, _NORM[norm], alpha, eps
    _call("sharq_residual_norm", ctypes.byref(a), _stream(dev))
    return out_x if out_x is not None else x, y
