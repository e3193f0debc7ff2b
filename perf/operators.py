"""The operators around the FP4 linears and the cases they are measured on.

Three families: routing to experts with its dispatch order and the weighted
sum back to tokens (moe_route, moe_combine), the residual addition with the
norms, gate and modulation around a block (residual_norm), and the 8-bit
integer linear with a scale for each token and channel (prepare_int8,
linear_int8).  run() computes a case in plain torch operations, or, where
`own` is set, through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one decoded token through the router of a 128-expert layer, top 8
        {"name": "route_decode_E128", "op": "route", "T": 1, "E": 128, "k": 8, "score": "softmax", "bias": False,
         "groups": 1, "topk_groups": 1, "group_score": "max", "renormalize": True, "dtype": "bf16", "padded": 0.0},
        # the same layer's prefill of 4096 tokens
        {"name": "route_prefill_E128", "op": "route", "T": 4096, "E": 128, "k": 8, "score": "softmax", "bias": False,
         "groups": 1, "topk_groups": 1, "group_score": "max", "renormalize": True, "dtype": "bf16", "padded": 0.0},
        # a large padded batch, sigmoid scores with a balance bias, 4 of 8 groups, fp32 logits
        {"name": "route_groups_E256", "op": "route", "T": 16383, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "topk_groups": 4, "group_score": "top2", "renormalize": True, "dtype": "fp32", "padded": 0.03},
        # expert outputs of a few decoded tokens back to their rows
        {"name": "combine_decode", "op": "combine", "T": 5, "k": 8, "N": 2048, "dtype": "bf16", "residual": True,
         "padded": 0.0},
        # expert outputs of a 4096-token prefill
        {"name": "combine_prefill", "op": "combine", "T": 4096, "k": 8, "N": 2048, "dtype": "bf16", "residual": True,
         "padded": 0.0},
        # residual addition and the next RMSNorm for one decoded token
        {"name": "norm_decode", "op": "norm", "M": 1, "K": 4096, "post": False, "pre": "rms", "mod": False, "G": 1,
         "x": "bf16"},
        # norms after and before a block at prefill
        {"name": "norm_sandwich", "op": "norm", "M": 4096, "K": 3584, "post": True, "pre": "rms", "mod": False, "G": 1,
         "x": "bf16"},
        # a video DiT block: gate, LayerNorm, scale and shift for each of two samples, fp32 residual stream
        {"name": "norm_dit", "op": "norm", "M": 8190, "K": 5120, "post": False, "pre": "layer", "mod": True, "G": 2,
         "x": "fp32"},
        # one decoded token through a gate+up projection
        {"name": "int8_decode", "op": "int8", "M": 1, "N": 28672, "K": 4096, "norm": True, "bias": False},
        # a small batch through a down projection
        {"name": "int8_batch", "op": "int8", "M": 48, "N": 4096, "K": 14336, "norm": False, "bias": False},
        # ragged prefill through a biased q/k/v projection
        {"name": "int8_prefill", "op": "int8", "M": 2041, "N": 4608, "K": 3584, "norm": True, "bias": True},
        # prefill through the widest projection
        {"name": "int8_large", "op": "int8", "M": 4096, "N": 37888, "K": 3584, "norm": True, "bias": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "combine", "norm", "int8"])
    if op == "route":
        E, groups, topk_groups = rng.choice([(8, 1, 1), (16, 1, 1), (60, 1, 1), (64, 1, 1), (64, 8, 3), (96, 4, 2),
                                             (128, 1, 1), (160, 8, 3), (256, 8, 4), (256, 1, 1), (384, 1, 1)])
        score = rng.choice(["softmax", "sigmoid"])
        T = _log(rng, 1, 16384)
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(8, E // groups * topk_groups)),
                "score": score, "bias": rng.random() < 0.5, "groups": groups, "topk_groups": topk_groups,
                "group_score": rng.choice(["max", "top2"]), "renormalize": rng.random() < 0.7,
                "dtype": rng.choice(["bf16", "fp32"]), "padded": rng.choice([0.0, 0.1]) if T > 16 else 0.0}
    if op == "combine":
        T = _log(rng, 1, 8192)
        return {"op": op, "T": T, "k": rng.randint(1, 8), "N": 8 * _log(rng, 32, 640),
                "dtype": rng.choice(["bf16", "bf16", "fp32"]), "residual": rng.random() < 0.5,
                "padded": rng.choice([0.0, 0.1]) if T > 16 else 0.0}
    if op == "norm":
        G = rng.choice([1, 1, 2, 3])
        return {"op": op, "M": G * _log(rng, 1, 2700), "K": 8 * _log(rng, 32, 1792), "post": rng.random() < 0.5,
                "pre": rng.choice(["rms", "layer", "none"]), "mod": rng.random() < 0.5, "G": G,
                "x": rng.choice(["bf16", "fp32"])}
    M = _log(rng, 1, 4096)
    return {"op": op, "M": M, "N": 8 * _log(rng, 64, 3584), "K": 16 * _log(rng, 32, 896),
            "norm": rng.random() < 0.5, "bias": rng.random() < 0.5}


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _uniform(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, op = case, case["op"]
    if op == "route":
        # logits of a trained router: a spread of about 1.5 a token, experts of uneven popularity
        logits = 1.5 * _rand(g, c["T"], c["E"]) + 0.5 * _rand(g, c["E"])
        logits[_uniform(g, c["T"]) < c["padded"]] = -math.inf
        bias = 0.05 * _rand(g, c["E"]) if c["bias"] else None
        return {"case": c, "logits": logits.to(DT[c["dtype"]]), "bias": bias}
    if op == "combine":
        n = c["T"] * c["k"]
        position = torch.randperm(n, generator=g, device="cuda").to(torch.int32).view(c["T"], c["k"])
        position[_uniform(g, c["T"]) < c["padded"]] = -1
        weights = _uniform(g, c["T"], c["k"]) + 0.05
        weights = weights / weights.sum(1, keepdim=True)
        res = _rand(g, c["T"], c["N"]).to(DT[c["dtype"]]) if c["residual"] else None
        return {"case": c, "Y": _rand(g, n, c["N"]).to(DT[c["dtype"]]), "position": position, "weights": weights,
                "residual": res}
    if op == "norm":
        M, K, G = c["M"], c["K"], c["G"]
        spread = torch.exp(0.5 * _rand(g, M, 1))
        s = {"case": c, "x": (3.0 * spread * _rand(g, M, K)).to(DT[c["x"]]),
             "h": (spread * _rand(g, M, K)).to(torch.bfloat16), "post_gamma": None, "gate": None, "gamma": None,
             "beta": None, "scale": None, "shift": None}
        if c["post"]:
            s["post_gamma"] = (0.5 + _uniform(g, K)).to(torch.bfloat16)
        if c["mod"]:
            # the chunks of one modulation tensor [G, 6, K], as its linear gives it
            mod = (0.3 * _rand(g, G, 6, K)).to(torch.bfloat16)
            s["gate"] = mod[:, 2]
            if c["pre"] != "none":
                s["shift"], s["scale"] = mod[:, 0], mod[:, 1]
        if c["pre"] != "none" and not c["mod"]:
            s["gamma"] = (0.5 + _uniform(g, K)).to(torch.bfloat16)
            if c["pre"] == "layer":
                s["beta"] = (0.1 * _rand(g, K)).to(torch.bfloat16)
        return s
    M, N, K = c["M"], c["N"], c["K"]
    X = _rand(g, M, K) * torch.exp(0.5 * _rand(g, M, 1))
    X[:, torch.randint(0, K, (max(1, K // 200),), generator=g, device="cuda")] *= 20.0   # outlier channels
    W = 0.02 * _rand(g, N, K)
    amax = W.abs().amax(1)
    return {"case": c, "X": X.to(torch.bfloat16), "gamma": (0.5 + _uniform(g, K)).to(torch.bfloat16) if c["norm"] else None,
            "codes": (W * (127.0 / amax)[:, None]).round().to(torch.int8), "scales": amax / 127.0,
            "bias": _rand(g, N).to(torch.bfloat16) if c["bias"] else None}


# ------------------------------------------------------------ plain forms --

def _route_plain(c, logits, bias):
    T, E, k = c["T"], c["E"], c["k"]
    l = logits.double()                                       # scores next to one another decide the choice
    ok = l > -math.inf
    if c["score"] == "softmax":
        m = l.amax(1, keepdim=True)
        e = torch.where(ok, torch.exp(l - m), 0.0)
        s = e / e.sum(1, keepdim=True)
    else:
        s = torch.where(ok, 1.0 / (1.0 + torch.exp(-l)), 0.0)
    key = torch.where(ok, s + bias.double() if bias is not None else s, -math.inf)
    if c["groups"] > 1:
        by = key.view(T, c["groups"], E // c["groups"])
        if c["group_score"] == "max":
            of = by.amax(2)
        else:
            two = by.sort(dim=2, descending=True).values[:, :, :2]
            of = torch.where(two[:, :, 0] > -math.inf, torch.where(two > -math.inf, two, 0.0).sum(2), -math.inf)
        order = of.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        keep = torch.zeros_like(of, dtype=torch.bool).scatter_(1, order, True)
        key = torch.where(keep[:, :, None], by, -math.inf).reshape(T, E)
    top = key.sort(dim=1, descending=True, stable=True)
    chosen = top.values[:, :k] > -math.inf
    ids = torch.where(chosen, top.indices[:, :k], -1)
    w = torch.where(chosen, s.gather(1, top.indices[:, :k]), 0.0)
    if c["renormalize"]:
        t = w.sum(1, keepdim=True)
        w = torch.where(t > 0, w / t, 0.0)
    # dispatch: by expert, tokens ascending inside one
    flat = torch.where(chosen, ids, E).reshape(-1)
    by_expert = flat.sort(dim=0, stable=True)
    offsets = torch.searchsorted(by_expert.values, torch.arange(E + 1, device=flat.device))
    at = torch.arange(T * k, device=flat.device)
    row_index = torch.where(at < offsets[E], by_expert.indices // k, 0)
    position = torch.empty_like(at).scatter_(0, by_expert.indices, at)
    position = torch.where(flat < E, position, -1).view(T, k)
    return {"ids": ids.int(), "weights": w.float(), "row_index": row_index.int(), "offsets": offsets.int(),
            "position": position.int()}


def _combine_plain(s):
    at = s["position"]
    rows = s["Y"][at.clamp(min=0).long()].float()
    w = torch.where(at < 0, 0.0, s["weights"])
    y = (rows * w[:, :, None]).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["Y"].dtype)


def _rows(v, M):
    """[G, K] for M rows: row r of the rows has v[r // (M / G)]."""
    return v.float().repeat_interleave(M // v.shape[0], 0)


def _norm_plain(s):
    c, x, u = s["case"], s["x"], s["h"].float()
    if s["post_gamma"] is not None:
        u = u * torch.rsqrt(u.square().mean(1, keepdim=True) + EPS) * s["post_gamma"].float()
    if s["gate"] is not None:
        u = u * _rows(s["gate"], c["M"])
    t = x.float() + u
    out = {"x": t.to(x.dtype)}
    if c["pre"] == "none":
        return out
    if c["pre"] == "rms":
        y = t * torch.rsqrt(t.square().mean(1, keepdim=True) + EPS)
    else:
        d = t - t.mean(1, keepdim=True)
        y = d * torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    if s["gamma"] is not None:
        y = y * s["gamma"].float()
    if s["beta"] is not None:
        y = y + s["beta"].float()
    if s["scale"] is not None:
        y = y * (1.0 + _rows(s["scale"], c["M"])) + _rows(s["shift"], c["M"])
    out["y"] = y.to(torch.bfloat16)
    return out


def _int8_plain(s):
    y = s["X"].float()
    if s["gamma"] is not None:
        y = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) * s["gamma"].float()
    amax = y.abs().amax(1, keepdim=True)
    q = (y * (127.0 / amax)).round()
    out = (q @ s["codes"].float().t()) * (amax / 127.0) * s["scales"]
    if s["bias"] is not None:
        out = out + s["bias"].float()
    return out.to(torch.bfloat16)


def run(s):
    c = s["case"]
    if own:
        import activation_sparsity_prep_b200 as sq
        if c["op"] == "route":
            r = sq.moe_route(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                             topk_groups=c["topk_groups"], group_score=c["group_score"], renormalize=c["renormalize"])
            return {"ids": r.ids, "weights": r.weights, "row_index": r.row_index, "offsets": r.offsets,
                    "position": r.position}
        if c["op"] == "combine":
            return sq.moe_combine(s["Y"], s["position"], s["weights"], residual=s["residual"])
        if c["op"] == "norm":
            x, y = sq.residual_norm(s["x"], s["h"], norm=None if c["pre"] == "none" else c["pre"],
                                    post_gamma=s["post_gamma"], gate=s["gate"], gamma=s["gamma"], beta=s["beta"],
                                    scale=s["scale"], shift=s["shift"], eps=EPS)
            return {"x": x} if y is None else {"x": x, "y": y}
        w = sq.WeightInt8(s["codes"], s["scales"], c["N"], c["K"])
        return sq.linear_int8(sq.prepare_int8(s["X"], s["gamma"], EPS), w, bias=s["bias"])
    if c["op"] == "route":
        return _route_plain(c, s["logits"], s["bias"])
    return {"combine": _combine_plain, "norm": _norm_plain, "int8": _int8_plain}[c["op"]](s)


def work(case):
    c, op = case, case["op"]
    size = {"bf16": 2, "fp32": 4}
    if op == "route":
        n = c["T"] * c["k"]
        return {"bytes": c["T"] * c["E"] * size[c["dtype"]] + 16 * n + 4 * (c["E"] + 1), "flops": 4 * c["T"] * c["E"]}
    if op == "combine":
        b = size[c["dtype"]]
        rows = c["T"] * c["k"] + c["T"] * (2 if c["residual"] else 1)
        return {"bytes": rows * c["N"] * b + 8 * c["T"] * c["k"], "flops": 2 * c["T"] * c["k"] * c["N"]}
    if op == "norm":
        one = 2 * size[c["x"]] + 2 + (2 if c["pre"] != "none" else 0)
        return {"bytes": c["M"] * c["K"] * one, "flops": 10 * c["M"] * c["K"]}
    M, N, K = c["M"], c["N"], c["K"]
    return {"bytes": 2 * M * K + N * K + 4 * N + 2 * M * N, "flops": 2 * M * N * K}


# ------------------------------------------- the definitions, in 64 bits --

def _route_exact(c, s):
    l = s["logits"].float().cpu().numpy().astype(np.float64)
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    live = np.isfinite(l)
    with np.errstate(over="ignore", invalid="ignore"):
        if c["score"] == "softmax":
            p = np.where(live, np.exp(np.where(live, l, 0.0) - np.where(live, l, -np.inf).max(1, initial=-1e30)[:, None]), 0.0)
            total = p.sum(1)[:, None]
            p = np.divide(p, total, out=np.zeros_like(p), where=total > 0)
        else:
            p = np.where(live, 1.0 / (1.0 + np.exp(-np.where(live, l, 0.0))), 0.0)
    b = np.zeros(E) if s["bias"] is None else s["bias"].cpu().numpy().astype(np.float64)
    key = np.where(live, p + b, -np.inf)
    if G > 1:
        part = -np.sort(-key.reshape(T, G, -1), axis=2)
        of = part[:, :, 0].copy()
        if c["group_score"] == "top2" and part.shape[2] > 1:
            of += np.where(np.isfinite(part[:, :, 1]), part[:, :, 1], 0.0)
        rank = np.argsort(np.argsort(-of, axis=1, kind="stable"), axis=1, kind="stable")
        key = np.where(np.repeat(rank < c["topk_groups"], E // G, axis=1), key, -np.inf)
    at = np.argsort(-key, axis=1, kind="stable")[:, :k]
    w = np.where(np.isfinite(np.take_along_axis(key, at, 1)), np.take_along_axis(p, at, 1), 0.0)
    if c["renormalize"]:
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return {"ids": None, "weights": w, "row_index": None, "offsets": None, "position": None}


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "route":
        return _route_exact(c, s)
    if c["op"] == "combine":
        out = torch.zeros((c["T"], c["N"]), dtype=torch.float64, device="cuda")
        if s["residual"] is not None:
            out += s["residual"].double()
        rows = s["Y"].double()
        for j in range(c["k"]):
            at = s["position"][:, j].long()
            live = torch.nonzero(at >= 0)[:, 0]
            out[live] += rows[at[live]] * s["weights"][live, j].double()[:, None]
        return out
    if c["op"] == "norm":
        each = c["M"] // c["G"]
        x, h = s["x"].double(), s["h"].double()
        if s["post_gamma"] is not None:
            h = h / ((h * h).sum(1, keepdim=True) / c["K"] + EPS).sqrt() * s["post_gamma"].double()
        if s["gate"] is not None:
            h = (h.view(c["G"], each, c["K"]) * s["gate"].double()[:, None]).view(c["M"], c["K"])
        t = x + h
        if c["pre"] == "none":
            return {"x": t}
        y = t - t.sum(1, keepdim=True) / c["K"] if c["pre"] == "layer" else t
        y = y / ((y * y).sum(1, keepdim=True) / c["K"] + EPS).sqrt()
        if s["gamma"] is not None:
            y = y * s["gamma"].double()
        if s["beta"] is not None:
            y = y + s["beta"].double()
        if s["scale"] is not None:
            y = y.view(c["G"], each, c["K"])
            y = (y + y * s["scale"].double()[:, None] + s["shift"].double()[:, None]).view(c["M"], c["K"])
        return {"x": t, "y": y}
    y = s["X"].double()
    if s["gamma"] is not None:
        y = y / ((y * y).sum(1, keepdim=True) / c["K"] + EPS).sqrt() * s["gamma"].double()
    step = y.abs().max(1, keepdim=True).values / 127.0
    out = torch.round(y / step) @ s["codes"].double().t()
    out = out * step * s["scales"].double()[None]
    return out + s["bias"].double() if s["bias"] is not None else out
