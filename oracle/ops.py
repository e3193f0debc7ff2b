"""Plain 64-bit reference of the operators around the linears (routing to
experts, the residual addition with its norms, 8-bit integer linears), from
the formulas in include/sharq.h.  Test infrastructure only."""
import numpy as np


def route(logits, k, score="softmax", bias=None, groups=1, topk_groups=1, group_score="max",
          renormalize=True, scale=1.0):
    """logits [T, E] -> (ids int64 [T, k], weights fp64 [T, k]), token by token."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    ids = np.full((T, k), -1, dtype=np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        live = [e for e in range(E) if logits[t, e] > -np.inf and b[e] > -np.inf]
        s = np.zeros(E)
        if live and score == "softmax":
            m = max(logits[t, e] for e in live)
            for e in live:
                s[e] = np.exp(logits[t, e] - m)
            s /= s.sum()
        elif score == "sigmoid":
            with np.errstate(over="ignore"):
                for e in live:
                    s[e] = 1.0 / (1.0 + np.exp(-logits[t, e]))
        # without a bias the order of the scores is that of the logits
        c = {e: s[e] + b[e] for e in live}
        order = c if bias is not None else {e: logits[t, e] for e in live}
        if groups > 1:
            size = E // groups
            of = {}
            for g in range(groups):
                inside = sorted((e for e in live if e // size == g), key=lambda e: -c[e])
                if inside:
                    of[g] = (max(order[e] for e in inside) if group_score == "max"
                             else sum(c[e] for e in inside[:2]))
            best = sorted(of, key=lambda g: (-of[g], g))[:topk_groups]
            live = [e for e in live if e // size in best]
        chosen = sorted(live, key=lambda e: (-order[e], e))[:k]
        ids[t, :len(chosen)] = chosen
        w[t, :len(chosen)] = s[chosen]
        if renormalize:
            total = w[t].sum()
            w[t] = w[t] / total if total > 0 else 0.0
    return ids, w * scale


def dispatch(ids, E):
    """ids [T, k] -> (row_index [T * k], offsets [E + 1], position [T, k])."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    row_index = np.zeros(T * k, dtype=np.int32)
    position = np.full(T * k, -1, dtype=np.int32)
    offsets = np.zeros(E + 1, dtype=np.int32)
    at = 0
    for e in range(E):
        mine = np.nonzero(flat == e)[0]
        row_index[at:at + len(mine)] = mine // k
        position[mine] = np.arange(at, at + len(mine))
        at += len(mine)
        offsets[e + 1] = at
    return row_index, offsets, position.reshape(T, k)


def combine(Y, position, weights, residual=None):
    """(fp64 result, sum of the terms' magnitudes) of the weighted sum."""
    Y, weights = np.asarray(Y, dtype=np.float64), np.asarray(weights, dtype=np.float64)
    T, k = position.shape
    out = np.zeros((T, Y.shape[1]))
    mag = np.zeros_like(out)
    for j in range(k):
        live = np.nonzero((position[:, j] >= 0) & (position[:, j] < Y.shape[0]))[0]
        term = weights[live, j][:, None] * Y[position[live, j]]
        out[live] += term
        mag[live] += np.abs(term)
    if residual is not None:
        out += residual
        mag += np.abs(residual)
    return out, mag


def residual_norm(x, h=None, norm="rms", post_gamma=None, gate=None, alpha=1.0, gamma=None, beta=None,
                  scale=None, shift=None, eps=1e-6):
    """(x', y) in fp64; y is None without a norm."""
    x = np.asarray(x, dtype=np.float64)
    M, K = x.shape

    def rows(v):
        v = np.asarray(v, dtype=np.float64)
        return np.repeat(v, M // v.shape[0], axis=0)

    if h is not None:
        u = np.asarray(h, dtype=np.float64)
        if post_gamma is not None:
            u = u / np.sqrt((u * u).mean(1, keepdims=True) + eps) * np.asarray(post_gamma, dtype=np.float64)
        if gate is not None:
            u = u * rows(gate)
        x = x + alpha * u
    if norm is None:
        return x, None
    y = x - x.mean(1, keepdims=True) if norm == "layer" else x
    y = y / np.sqrt((y * y).mean(1, keepdims=True) + eps)
    if gamma is not None:
        y = y * np.asarray(gamma, dtype=np.float64)
    if beta is not None:
        y = y + np.asarray(beta, dtype=np.float64)
    if scale is not None:
        y = y * (1.0 + rows(scale))
    if shift is not None:
        y = y + rows(shift)
    return x, y


def quantize_rows_int8(y):
    """Codes and scales of fp32 rows, each operation rounded to fp32 as
    stated; bit-exact for rows that need no norm."""
    y = np.asarray(y, dtype=np.float32)
    a = np.abs(y).max(1) if y.shape[1] else np.zeros(len(y), np.float32)
    live = a >= np.float32(2.0 ** -100)
    safe = np.where(live, a, np.float32(1))
    inv = np.where(live, np.float32(127) / safe, np.float32(0)).astype(np.float32)
    codes = np.rint((y * inv[:, None]).astype(np.float32)).astype(np.int8)
    return codes, np.where(live, safe / np.float32(127), np.float32(0)).astype(np.float32)


def linear_int8(xc, xs, wc, ws, bias=None):
    """(fp64 result, magnitude of the product) of the 8-bit linear."""
    acc = np.asarray(xc, dtype=np.int64) @ np.asarray(wc, dtype=np.int64).T
    y = acc.astype(np.float64) * np.asarray(xs, np.float64)[:, None] * np.asarray(ws, np.float64)[None]
    return (y if bias is None else y + np.asarray(bias, np.float64)), np.abs(y)
