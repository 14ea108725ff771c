"""Plain binary64 forms of the routing calls of include/mxfp4.h (numpy),
written from the declarations there and independently of the kernels."""
import numpy as np

HALF_F32 = 2.0 ** -24       # half a step of binary32, relative


def half_step(dtype) -> float:
    """Largest relative error of one rounding to a torch dtype."""
    import torch
    return torch.finfo(dtype).eps / 2


def f64(t) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def scores(l, score):
    l = np.asarray(l, dtype=np.float64)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        m = l.max(axis=1, keepdims=True)
        e = np.where(m == -np.inf, 0.0, np.exp(l - m))
        z = e.sum(axis=1, keepdims=True)
        return np.where(z == 0, 0.0, e / np.where(z == 0, 1.0, z))


def _order(z):
    """Indices by descending value, ties to the lowest index, NaN last."""
    nan = np.isnan(z)
    return np.lexsort((np.arange(z.size), -np.where(nan, 0.0, z), nan))


def route(l, k, score="softmax", bias=None, mask=None, groups=1, top_groups=None, group_best=1, renormalise=True,
          scale=1.0):
    l = np.asarray(l, dtype=np.float64)
    T, E = l.shape
    top_groups = groups if top_groups is None else top_groups
    s = scores(l, score)
    by_logit = bias is None and (groups == top_groups or group_best == 1)
    z = l.copy() if by_logit else s + (0.0 if bias is None else np.asarray(bias, dtype=np.float64)[None])
    ids = np.full((T, k), -1, dtype=np.int32)
    w = np.zeros((T, k))
    n = E // groups
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        allowed = np.arange(E)
        if groups != top_groups:
            of = np.empty(groups)
            for g in range(groups):
                part = z[t, g * n:(g + 1) * n]
                best = part[_order(part)][:min(group_best, n)]
                of[g] = best.sum()
            kept = _order(of)[:top_groups]
            allowed = np.nonzero(np.isin(np.arange(E) // n, kept))[0]
        ids[t] = allowed[_order(z[t, allowed])][:k]
        w[t] = s[t, ids[t]]
        if renormalise:
            total = w[t].sum()
            w[t] = w[t] / total if total != 0 else 0.0
    return ids, w * scale


def route_bwd(l, ids, dw, score="softmax", renormalise=True, scale=1.0):
    """(gradient, magnitude): the gradient by the chain rule through the
    scores, and the sum of the magnitudes of the terms that make it up."""
    s = scores(l, score)
    T, E = s.shape
    g = np.zeros((T, E))
    mag = np.zeros((T, E))
    for t in range(T):
        live = (ids[t] >= 0) & (ids[t] < E)
        idx, d = ids[t][live], dw[t][live] * scale
        if not idx.size:
            continue
        q = s[t, idx]
        ds, dm = np.zeros(E), np.zeros(E)
        if renormalise:
            total = q.sum()
            if total == 0:
                continue
            mean, mean_m = (q * d).sum() / total, (q * abs(d)).sum() / total
            np.add.at(ds, idx, (d - mean) / total)
            np.add.at(dm, idx, (abs(d) + mean_m) / total)
        else:
            np.add.at(ds, idx, d)
            np.add.at(dm, idx, abs(d))
        if score == "softmax":
            g[t] = s[t] * (ds - (s[t] * ds).sum())
            mag[t] = s[t] * (dm + (s[t] * dm).sum())
            if renormalise:      # the sum over the scores is zero: only the chosen get a gradient
                rest = np.ones(E, dtype=bool)
                rest[idx] = False
                g[t, rest], mag[t, rest] = 0.0, 0.0
        else:
            g[t] = s[t] * (1 - s[t]) * ds
            mag[t] = s[t] * (1 - s[t]) * dm
    return g, mag


def plan(ids, experts, align, rows, fill=False):
    flat = np.asarray(ids).reshape(-1)
    good = (flat >= 0) & (flat < experts)
    counts = np.bincount(flat[good], minlength=experts)
    offsets = np.concatenate([[0], np.cumsum(-(-counts // align) * align)])
    row_of_slot = np.full(flat.size, -1, dtype=np.int64)
    slot_of_row = np.full(rows, -1, dtype=np.int64)
    order = np.argsort(np.where(good, flat, experts), kind="stable")[:counts.sum()]
    first = np.cumsum(counts) - counts
    e = flat[order]
    at = offsets[e] + np.arange(order.size) - first[e]
    row_of_slot[order] = at
    slot_of_row[at] = order
    if fill:
        offsets[-1] = rows
    return dict(counts=counts, offsets=offsets, row_of_slot=row_of_slot.reshape(np.shape(ids)), slot_of_row=slot_of_row)


def combine(y, row_of_slot, weights):
    """(sum, sum of magnitudes) per token."""
    T, k = row_of_slot.shape
    out, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for j in range(k):
        r = row_of_slot[:, j]
        live = (r >= 0) & (r < y.shape[0])
        v = (1.0 if weights is None else weights[live, j, None]) * y[r[live]]
        out[live] += v
        mag[live] += abs(v)
    return out, mag


def combine_bwd(d, y, row_of_slot, weights):
    T, k = row_of_slot.shape
    dy, dw, mag = np.zeros(y.shape), np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        r = row_of_slot[:, j]
        live = np.nonzero((r >= 0) & (r < y.shape[0]))[0]
        dy[r[live]] = weights[live, j, None] * d[live]
        dw[live, j] = (d[live] * y[r[live]]).sum(1)
        mag[live, j] = abs(d[live] * y[r[live]]).sum(1)
    return dy, dw, mag
