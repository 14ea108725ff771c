"""Cases of the expert-routing operators: route, expert_plan, dispatch, combine and grad_clip.

`run` computes each in plain torch operations, or, where `own` is true, by the
package's calls.  Shapes follow the MoE layer of this repository (16384 tokens,
32 experts, top 4, 2880 features, segments of 128 rows) and ranges around it.
"""
import math

import numpy as np
import torch

own = False

ALIGN = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases
def _route(tokens, experts, top_k, score, dtype, bias=False, masked=False, groups=1, top_groups=1, group_best=1,
           renormalise=True, scale=1.0, backward=False):
    return {"op": "route", "tokens": tokens, "experts": experts, "top_k": top_k, "score": score, "dtype": dtype,
            "bias": bias, "masked": masked, "groups": groups, "top_groups": top_groups, "group_best": group_best,
            "renormalise": renormalise, "scale": scale, "backward": backward}


def _plan(tokens, experts, top_k):
    return {"op": "plan", "tokens": tokens, "experts": experts, "top_k": top_k}


def _rows(op, tokens, experts, top_k, cols, dtype, out_dtype):
    return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "cols": cols, "dtype": dtype,
            "out_dtype": out_dtype}


def _clip(tensors, smallest, largest, dtype, ratio):
    return {"op": "clip", "tensors": tensors, "smallest": smallest, "largest": largest, "dtype": dtype, "ratio": ratio}


def listed():
    return [
        # one token of one request: only latency counts
        {"name": "route one token", **_route(1, 32, 4, "softmax", "bf16")},
        # the training layer's tokens, scores from the router's bf16 product
        {"name": "route layer", **_route(16384, 32, 4, "softmax", "bf16")},
        # many experts in groups with a balance bias, a batch padded to an odd length
        {"name": "route grouped", **_route(8191, 256, 8, "sigmoid", "f32", bias=True, masked=True, groups=8,
                                           top_groups=4, group_best=2, scale=2.0)},
        # the router's gradient where every expert's logit gets one
        {"name": "route gradient", **_route(16384, 128, 6, "softmax", "bf16", renormalise=False, backward=True)},
        # a small decoding batch
        {"name": "plan decode", **_plan(48, 32, 4)},
        # a long batch over many experts
        {"name": "plan long", **_plan(65536, 256, 8)},
        # a decoding batch's rows into mostly empty segments
        {"name": "dispatch decode", **_rows("dispatch", 48, 32, 4, 2880, "bf16", "bf16")},
        # the training layer's activations
        {"name": "dispatch layer", **_rows("dispatch", 16384, 32, 4, 2880, "bf16", "bf16")},
        # the down projection's binary32 rows back to tokens
        {"name": "combine layer", **_rows("combine", 16384, 32, 4, 2880, "f32", "bf16")},
        # its gradient, with the bf16 rows that the fused product keeps
        {"name": "combine gradient", **_rows("combine_bwd", 16384, 32, 4, 2880, "bf16", "bf16")},
        # biases and norms: many small tensors of odd sizes, a launch-bound step
        {"name": "clip small", **_clip(48, 1, 66001, "bf16", 0.5)},
        # a layer's weight gradients, from biases to the matrices of eight experts
        {"name": "clip layer", **_clip(24, 33, 132710400, "f32", 0.5)},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "plan", "dispatch", "combine", "combine_bwd", "clip"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 2, 512 // groups)
        tokens = _log(rng, 1, 32768)
        top_groups = rng.randint(1, groups)
        top_k = min(rng.randint(1, 8), experts // groups * top_groups)
        return _route(tokens, experts, top_k, rng.choice(["softmax", "sigmoid"]), rng.choice(["bf16", "f32"]),
                      bias=rng.random() < 0.5, masked=rng.random() < 0.3, groups=groups, top_groups=top_groups,
                      group_best=rng.choice([1, 2]), renormalise=rng.random() < 0.6,
                      scale=rng.choice([1.0, 2.0, 1.5]), backward=rng.random() < 0.4)
    if op == "plan":
        experts = _log(rng, 2, 512)
        return _plan(_log(rng, 1, 65536), experts, min(experts, rng.randint(1, 8)))
    if op == "clip":
        largest = _log(rng, 1000, 100000000)
        tensors = rng.randint(1, 60) if largest < 1000000 else rng.randint(1, 12)
        return _clip(tensors, rng.randint(1, 900), largest, rng.choice(["bf16", "f32"]), rng.choice([0.5, 0.1, 2.0]))
    experts = _log(rng, 2, 256)
    cols = rng.choice([2880, 5760, _log(rng, 16, 5760), _log(rng, 16, 5760)])
    dtype = rng.choice(["bf16", "f32"])
    return _rows(op, _log(rng, 1, 12000), experts, min(experts, rng.randint(1, 8)), cols, dtype,
                 dtype if op == "dispatch" else rng.choice(["bf16", "f32"]))


def _capacity(c):
    """Rows that hold every split of the slots over the experts."""
    slots = c["tokens"] * c["top_k"]
    return (slots + min(c["experts"], slots) * (ALIGN - 1)) // ALIGN * ALIGN


def _sizes(c):
    n = c["tensors"]
    r = c["largest"] / c["smallest"]
    return [c["largest"]] if n == 1 else [int(round(c["smallest"] * r ** (i / (n - 1)))) for i in range(n)]


# ------------------------------------------------------------------ inputs
def _zipf_ids(g, c):
    """Distinct experts of each token, expert i with probability proportional
    to (i + 1)^-1.1 (Gumbel top-k)."""
    u = torch.rand((c["tokens"], c["experts"]), generator=g, device="cuda").clamp_(1e-20, 1 - 1e-7)
    logp = -1.1 * torch.log(torch.arange(1, c["experts"] + 1, device="cuda", dtype=torch.float32))
    return torch.topk(logp - torch.log(-torch.log(u)), c["top_k"], dim=1).indices.to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def empty(*shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    s = {"case": c}
    if c["op"] == "clip":
        s["grads"] = [normal(n, dtype=DTYPES[c["dtype"]], std=1e-3) for n in _sizes(c)]
        s["max_norm"] = c["ratio"] * 1e-3 * math.sqrt(sum(_sizes(c)))
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
        s["norm"] = empty(1, dtype=torch.float32)
        if own:
            from fp4_precision_numerics_b200 import mxfp4
            s["list"] = mxfp4.GradList(s["grads"], out=s["out"])
        return s
    T, E, k = c["tokens"], c["experts"], c["top_k"]
    if c["op"] == "route":
        s["logits"] = normal(T, E, dtype=DTYPES[c["dtype"]], std=1.5)
        s["bias"] = normal(E, std=0.05) if c["bias"] else None
        s["mask"] = torch.rand(T, generator=g, device="cuda") < 0.9 if c["masked"] else None
        if c["backward"]:
            s["ids"] = _plain_route(s)["ids"]
            s["d_weights"] = normal(T, k)
            s["out"] = torch.empty_like(s["logits"])
        else:
            s["out"] = {"ids": empty(T, k, dtype=torch.int32), "weights": empty(T, k, dtype=torch.float32)}
        return s
    ids = _zipf_ids(g, c)
    rows = _capacity(c)
    if c["op"] == "plan":
        s["ids"] = ids
        s["out"] = {"counts": empty(E, dtype=torch.int32), "offsets": empty(E + 1, dtype=torch.int32),
                    "row_of_slot": empty(T, k, dtype=torch.int32), "slot_of_row": empty(rows, dtype=torch.int32)}
        return s
    s["plan"] = _plain_plan({"case": c, "ids": ids})
    dt, odt, C = DTYPES[c["dtype"]], DTYPES[c["out_dtype"]], c["cols"]
    if c["op"] == "dispatch":
        s["x"] = normal(T, C, dtype=dt)
        s["out"] = empty(rows, C, dtype=dt)
        return s
    s["y"] = normal(rows, C, dtype=dt)
    w = torch.softmax(normal(T, k), dim=1)
    s["weights"] = w
    if c["op"] == "combine":
        s["out"] = empty(T, C, dtype=odt)
    else:
        s["d_out"] = normal(T, C, dtype=odt, std=1e-3)
        s["out"] = {"dy": empty(rows, C, dtype=odt), "d_weights": empty(T, k, dtype=torch.float32)}
    return s


# ------------------------------------------------------------------ plain forms
def _scores(logits, score, dtype):
    l = logits.to(dtype)
    if score == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True)
    return 1 / (1 + torch.exp(-l))


def _plain_route(s):
    c = s["case"]
    k, G = c["top_k"], c["groups"]
    # the choice is made in 64 bits: values next to each other decide it
    z = _scores(s["logits"], c["score"], torch.float64)
    if s["bias"] is not None:
        z = z + s["bias"].double()
    if G > 1:
        T, E = z.shape
        best = torch.sort(z.view(T, G, E // G), dim=2, descending=True).values
        of_group = best[:, :, :min(c["group_best"], E // G)].sum(2)
        kept = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        stays = torch.zeros((T, G), dtype=torch.bool, device=z.device).scatter_(1, kept, True)
        z = torch.where(stays.repeat_interleave(E // G, dim=1), z, -math.inf)
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    w = _scores(s["logits"], c["score"], torch.float32).gather(1, ids)
    if c["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    w = w * c["scale"]
    ids = ids.to(torch.int32)
    if s["mask"] is not None:
        ids = torch.where(s["mask"][:, None], ids, -1)
        w = torch.where(s["mask"][:, None], w, 0.0)
    return {"ids": ids, "weights": w}


def _plain_route_bwd(s):
    c = s["case"]
    live = s["ids"] >= 0
    ids = s["ids"].clamp_min(0).long()
    dw = torch.where(live, s["d_weights"] * c["scale"], 0.0)
    p = _scores(s["logits"], c["score"], torch.float32)
    q = p.gather(1, ids)
    if c["renormalise"]:
        w = q / q.sum(1, keepdim=True)
        dq = (dw - (w * dw).sum(1, keepdim=True)) / q.sum(1, keepdim=True)
    else:
        dq = dw
    dp = torch.zeros_like(p).scatter_(1, ids, torch.where(live, dq, 0.0))
    if c["score"] == "softmax":
        dl = p * (dp - (p * dp).sum(1, keepdim=True))
    else:
        dl = p * (1 - p) * dp
    return dl.to(s["logits"].dtype)


def _plain_plan(s):
    c = s["case"]
    E, rows = c["experts"], _capacity(c)
    flat = s["ids"].reshape(-1).long()
    counts = torch.zeros(E, dtype=torch.int64, device=flat.device).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.cumsum((counts + ALIGN - 1) // ALIGN * ALIGN, 0)
    by_expert = torch.sort(flat, stable=True).indices
    expert = flat[by_expert]
    first = torch.cumsum(counts, 0) - counts
    row = offsets[expert] + torch.arange(flat.numel(), device=flat.device) - first[expert]
    row_of_slot = torch.empty_like(flat)
    row_of_slot[by_expert] = row
    slot_of_row = torch.full((rows,), -1, dtype=torch.int64, device=flat.device)
    slot_of_row[row] = by_expert
    i32 = torch.int32
    return {"counts": counts.to(i32), "offsets": offsets.to(i32), "row_of_slot": row_of_slot.view_as(s["ids"]).to(i32),
            "slot_of_row": slot_of_row.to(i32)}


def _plain_dispatch(s):
    slot = s["plan"]["slot_of_row"].long()
    rows = s["x"][slot.clamp_min(0) // s["case"]["top_k"]]
    return torch.where((slot >= 0)[:, None], rows, torch.zeros((), dtype=rows.dtype, device=rows.device))


def _plain_combine(s):
    y = s["y"][s["plan"]["row_of_slot"].long()].float()
    return (s["weights"][:, :, None] * y).sum(1).to(DTYPES[s["case"]["out_dtype"]])


def _plain_combine_bwd(s):
    rows = s["plan"]["row_of_slot"].long()
    d = s["d_out"].float()
    dw = (d[:, None, :] * s["y"][rows].float()).sum(2)
    dy = torch.zeros(s["y"].shape, dtype=s["d_out"].dtype, device=d.device)
    dy[rows] = (s["weights"][:, :, None] * d[:, None, :]).to(dy.dtype)
    return {"dy": dy, "d_weights": dw}


def _plain_clip(s):
    squares = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]])
    norm = squares.sum().sqrt()
    over = (norm > s["max_norm"]) & torch.isfinite(norm)
    coef = torch.where(over, s["max_norm"] / norm, 1.0).float()
    return {"norm": norm.float().view(1), "grads": [(t.float() * coef).to(t.dtype) for t in s["grads"]]}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"route": _plain_route_bwd if c.get("backward") else _plain_route, "plan": _plain_plan,
                "dispatch": _plain_dispatch, "combine": _plain_combine, "combine_bwd": _plain_combine_bwd,
                "clip": _plain_clip}[c["op"]](s)
    from fp4_precision_numerics_b200 import mxfp4
    if c["op"] == "route" and c["backward"]:
        return mxfp4.route_bwd(s["logits"], s["ids"], s["d_weights"], score=c["score"], renormalise=c["renormalise"],
                               scale=c["scale"], out=s["out"])
    if c["op"] == "route":
        return mxfp4.route(s["logits"], c["top_k"], score=c["score"], bias=s["bias"], mask=s["mask"],
                           groups=c["groups"], top_groups=c["top_groups"], group_best=c["group_best"],
                           renormalise=c["renormalise"], scale=c["scale"], out=s["out"])
    if c["op"] == "plan":
        return mxfp4.expert_plan(s["ids"], c["experts"], align=ALIGN, out=s["out"])
    if c["op"] == "dispatch":
        return mxfp4.dispatch(s["x"], s["plan"], out=s["out"])
    if c["op"] == "combine":
        return mxfp4.combine(s["y"], s["plan"], s["weights"], out=s["out"])
    if c["op"] == "combine_bwd":
        return mxfp4.combine_bwd(s["d_out"], s["y"], s["plan"], s["weights"], out=s["out"])
    mxfp4.grad_clip(s["list"], s["max_norm"], norm=s["norm"])
    return {"norm": s["norm"], "grads": s["out"]}


# ------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "clip":
        n = sum(_sizes(c))
        return {"bytes": 2 * n * BYTES[c["dtype"]] + 4, "flops": 3 * n}
    T, E, k = c["tokens"], c["experts"], c["top_k"]
    N, rows = T * k, _capacity(c)
    if c["op"] == "route":
        es = BYTES[c["dtype"]]
        if c["backward"]:
            whole = c["score"] == "softmax" and not c["renormalise"]
            return {"bytes": T * E * es + (T * E if whole else N) * es + N * 8, "flops": (6 * T * E if whole else 8 * N)}
        return {"bytes": T * E * es + (4 * E if c["bias"] else 0) + (T if c["masked"] else 0) + N * 8, "flops": 6 * T * E}
    if c["op"] == "plan":
        return {"bytes": 8 * N + 4 * rows + 8 * E + 4, "flops": 2 * N}
    es, eo, C = BYTES[c["dtype"]], BYTES[c["out_dtype"]], c["cols"]
    if c["op"] == "dispatch":
        return {"bytes": T * C * es + rows * C * es + 4 * rows, "flops": 0}
    if c["op"] == "combine":
        return {"bytes": N * C * es + T * C * eo + 8 * N, "flops": 2 * N * C}
    return {"bytes": T * C * eo + N * C * es + rows * C * eo + 12 * N, "flops": 3 * N * C}


# ------------------------------------------------------------------ exact values
def _host(t):
    return t.cpu().numpy() if t.dtype != torch.bfloat16 else t.float().cpu().numpy()


def _exact_scores(l, score):
    l = l.astype(np.float64)
    if score == "sigmoid":
        return np.where(l >= 0, 1.0 / (1.0 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1.0 + np.exp(-np.abs(l))))
    e = np.exp(l - l.max(axis=1, keepdims=True))
    return e / e.sum(axis=1, keepdims=True)


def _exact_route(s):
    c = s["case"]
    p = _exact_scores(_host(s["logits"]), c["score"])
    z = p + _host(s["bias"]).astype(np.float64)[None, :] if s["bias"] is not None else p.copy()
    T, E = p.shape
    G = c["groups"]
    if G > 1:
        n = E // G
        of_group = np.empty((T, G))
        for i in range(G):
            part = np.sort(z[:, i * n:(i + 1) * n], axis=1)
            of_group[:, i] = part[:, -1] + (part[:, -2] if c["group_best"] > 1 and n > 1 else 0.0)
        kept = np.argsort(-of_group, axis=1, kind="stable")[:, :c["top_groups"]]
        out = np.ones((T, G), dtype=bool)
        np.put_along_axis(out, kept, False, axis=1)
        z[np.repeat(out, n, axis=1)] = -np.inf
    ids = np.argsort(-z, axis=1, kind="stable")[:, :c["top_k"]]
    w = np.take_along_axis(p, ids, axis=1)
    if c["renormalise"]:
        w = w / w.sum(axis=1, keepdims=True)
    w = w * c["scale"]
    if s["mask"] is not None:
        live = _host(s["mask"])[:, None]
        ids, w = np.where(live, ids, -1), np.where(live, w, 0.0)
    return {"ids": ids.astype(np.int32), "weights": w}


def _exact_route_bwd(s):
    c = s["case"]
    p = _exact_scores(_host(s["logits"]), c["score"])
    ids, dw = _host(s["ids"]), _host(s["d_weights"]).astype(np.float64) * c["scale"]
    T, E = p.shape
    t = np.arange(T)
    live = ids[:, 0] >= 0
    dl = np.zeros((T, E))
    cols = [np.maximum(ids[:, j], 0) for j in range(c["top_k"])]
    q = [p[t, e] for e in cols]
    total = sum(q) if c["renormalise"] else np.ones(T)
    mean = sum(a / total * dw[:, j] for j, a in enumerate(q)) if c["renormalise"] else np.zeros(T)
    grads = [(dw[:, j] - mean) / total for j in range(c["top_k"])]
    if c["score"] == "softmax":
        dl -= p * sum(a * b for a, b in zip(q, grads))[:, None]
        for e, a, b in zip(cols, q, grads):
            dl[t, e] += a * b
    else:
        for e, a, b in zip(cols, q, grads):
            dl[t, e] += a * (1.0 - a) * b
    dl[~live] = 0.0
    return dl


def _exact_plan(s):
    c = s["case"]
    ids = _host(s["ids"]).reshape(-1)
    counts = np.bincount(ids, minlength=c["experts"])
    offsets = np.concatenate([[0], np.cumsum(-(-counts // ALIGN) * ALIGN)])
    row_of_slot = np.empty(ids.size, dtype=np.int32)
    slot_of_row = np.full(_capacity(c), -1, dtype=np.int32)
    for e in range(c["experts"]):
        slots = np.nonzero(ids == e)[0]
        at = offsets[e] + np.arange(slots.size)
        row_of_slot[slots] = at
        slot_of_row[at] = slots
    return {"counts": counts.astype(np.int32), "offsets": offsets.astype(np.int32),
            "row_of_slot": row_of_slot.reshape(c["tokens"], c["top_k"]), "slot_of_row": slot_of_row}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "route":
        return _exact_route_bwd(s) if c["backward"] else _exact_route(s)
    if c["op"] == "plan":
        return _exact_plan(s)
    if c["op"] == "clip":
        total = 0.0
        for t in s["grads"]:
            for part in t.split(1 << 26):
                total += float((part.double() ** 2).sum())
        norm = math.sqrt(total)
        coef = min(1.0, s["max_norm"] / norm)
        return {"norm": np.array([norm]), "grads": [t.double() * coef for t in s["grads"]]}
    k, rows = c["top_k"], s["plan"]["row_of_slot"].long()
    if c["op"] == "dispatch":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for j in range(k):
            out[rows[:, j]] = s["x"].double()
        return out
    w = s["weights"].double()
    if c["op"] == "combine":
        out = torch.zeros((c["tokens"], c["cols"]), dtype=torch.float64, device="cuda")
        for j in range(k):
            out += w[:, j, None] * s["y"][rows[:, j]].double()
        return out
    d = s["d_out"].double()
    dy = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    dw = torch.empty((c["tokens"], k), dtype=torch.float64, device="cuda")
    for j in range(k):
        dy[rows[:, j]] = w[:, j, None] * d
        dw[:, j] = (s["y"][rows[:, j]].double() * d).sum(1)
    return {"dy": dy, "d_weights": dw}
