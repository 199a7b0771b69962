"""Plain reference of expert routing (include/nq.h, nq_moe_*) in float64."""
import numpy as np


def numbers(x):
    """Logits or keys, NaN as -inf."""
    x = np.asarray(x, np.float64)
    return np.where(np.isnan(x), -np.inf, x)


def scores(x, kind):
    x = numbers(x)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-x))
        m = x.max(-1, keepdims=True)
        z = np.where(np.isneginf(m), 0.0, np.exp(x - np.where(np.isneginf(m), 0.0, m)))
        s = z.sum(-1, keepdims=True)
        return z / np.where(s == 0, 1.0, s)


def route(x, kind, top_k, bias=None, groups=1, top_groups=1, group_best=1, renormalise=False, scale=1.0):
    """x [tokens, experts] -> ids [tokens, top_k], weights float64."""
    p = scores(x, kind)
    key = numbers(x) if bias is None else p + bias
    summed = numbers(p if bias is None else key)
    ids = np.empty((len(x), top_k), np.int64)
    for t in range(len(x)):
        key_t = np.where(np.isnan(key[t]), -np.inf, key[t])
        allowed = list(range(x.shape[1]))
        if groups > 1:
            size = x.shape[1] // groups
            if group_best == 2:
                score = [np.sort(summed[t, g * size:(g + 1) * size])[-2:].sum() for g in range(groups)]
            else:
                score = [key_t[g * size:(g + 1) * size].max() for g in range(groups)]
            kept = sorted(range(groups), key=lambda g: (-score[g], g))[:top_groups]
            allowed = [e for e in allowed if e // size in kept]
        ids[t] = sorted(allowed, key=lambda e: (-key_t[e], e))[:top_k]
    return ids, weights(x, kind, ids, renormalise, scale)


def weights(x, kind, ids, renormalise, scale):
    w = np.take_along_axis(scores(x, kind), ids, -1)
    if renormalise:
        s = w.sum(-1, keepdims=True)
        w = w / np.where(s == 0, 1.0, s)
    return w * scale


def grad(x, kind, ids, dw, renormalise, scale):
    """d sum(dw * weights) / dx, from the formulas."""
    p = scores(x, kind)
    pk = np.take_along_axis(p, ids, -1)
    d = dw * scale
    if renormalise:
        s = pk.sum(-1, keepdims=True)
        d = (d - (d * pk).sum(-1, keepdims=True) / s) / s
    dp = np.zeros_like(p)
    np.put_along_axis(dp, ids, d, -1)
    if kind == "sigmoid":
        return dp * p * (1 - p)
    return p * (dp - (dp * p).sum(-1, keepdims=True))


def grad_by_differences(x, kind, ids, dw, renormalise, scale, step=1e-5):
    """The same by central differences of the weights, the choice fixed."""
    x = np.asarray(x, np.float64)
    out = np.zeros_like(x)
    for e in range(x.shape[1]):
        hi, lo = x.copy(), x.copy()
        hi[:, e] += step
        lo[:, e] -= step
        f = [(dw * weights(y, kind, ids, renormalise, scale)).sum(-1) for y in (hi, lo)]
        out[:, e] = (f[0] - f[1]) / (2 * step)
    return out
