"""Plain reference of the steps between a decoder layer's products (include/nq.h:
nq_block_norm, nq_rope, nq_moe_sort and its kin) in float64, row by row where
that is the definition."""
import numpy as np


# ---------------------------------------------------------------- norms, gate and residual
def normed(t, eps):
    return t / np.sqrt((t * t).mean(-1, keepdims=True) + eps)


def rows_of_gate(gate, rows):
    """gate [gates, dim] or [dim] -> [rows, dim]."""
    gate = gate if gate.ndim == 2 else gate[None]
    return gate[np.arange(rows) // (rows // len(gate))]


def joined(h, y, post, gate, scale, offset, eps):
    """h_out."""
    if y is None:
        return h
    u = y if post is None else normed(y, eps) * (post + offset)
    if gate is not None:
        u = u * rows_of_gate(gate, len(h))
    return h + scale * u


def block_norm(h, y=None, post=None, gate=None, pre=None, scale=1.0, offset=0.0, eps=1e-6):
    h_out = joined(h, y, post, gate, scale, offset, eps)
    return h_out, None if pre is None else normed(h_out, eps) * (pre + offset)


def norm_back(v, t, eps):
    """The gradient of sum(v * normed(t)) for t."""
    r = 1 / np.sqrt((t * t).mean(-1, keepdims=True) + eps)
    n = t * r
    return r * (v - n * (v * n).mean(-1, keepdims=True))


def block_norm_grad(h_out, y=None, dh_out=None, dz=None, post=None, gate=None, pre=None, scale=1.0, offset=0.0, eps=1e-6):
    """(dh, dy, dpost, dgate, dpre), from the formulas."""
    rows = len(h_out)
    d = np.zeros_like(h_out) if dh_out is None else dh_out.copy()
    dpre = dpost = dgate = dy = None
    if dz is not None:
        dpre = (dz * normed(h_out, eps)).sum(0)
        d = d + norm_back(dz * (pre + offset), h_out, eps)
    if y is not None:
        g = 1.0 if gate is None else rows_of_gate(gate, rows)
        n = normed(y, eps)
        u = y if post is None else n * (post + offset)
        du = scale * g * d
        if post is None:
            dy = du * np.ones_like(y)
        else:
            dpost = (du * n).sum(0)
            dy = norm_back(du * (post + offset), y, eps)
        if gate is not None:
            gates = len(gate) if gate.ndim == 2 else 1
            dgate = (scale * d * u).reshape(gates, rows // gates, -1).sum(1).reshape(gate.shape)
    return d, dy, dpost, dgate, dpre


# ---------------------------------------------------------------- rotary positions
def rope(x, positions, freq, axis=None, layout="halves", scale=1.0, back=False):
    """x [rows, heads, dim], positions [axes, rows]; one pair at a time, as a complex number."""
    out = np.array(x, np.float64)
    half = len(freq)
    for i in range(half):
        a, b = (i, i + half) if layout == "halves" else (2 * i, 2 * i + 1)
        ax = 0 if axis is None else int(axis[i])
        p = positions[ax].astype(np.float64) if 0 <= ax < len(positions) else np.zeros(len(x))
        turn = scale * np.exp((-1j if back else 1j) * p * freq[i])[:, None]
        z = (x[..., a] + 1j * x[..., b]) * turn
        out[..., a], out[..., b] = z.real, z.imag
    return out


# ---------------------------------------------------------------- tokens sorted by expert
def moe_sort(ids, experts):
    """ids [tokens, top_k] uint32 -> starts, place, row_token, row_expert (int64)."""
    tokens, k = ids.shape
    flat = [int(i) for i in ids.reshape(-1)]
    buckets = [[] for _ in range(experts + 1)]
    for p, e in enumerate(flat):
        buckets[min(e, experts)].append(p)
    order = [p for b in buckets for p in b]
    place = np.empty(tokens * k, np.int64)
    place[order] = np.arange(tokens * k)
    starts = np.concatenate([[0], np.cumsum([len(b) for b in buckets[:experts]])])
    return starts.astype(np.int64), place.reshape(tokens, k), np.array([p // k for p in order], np.int64), \
        np.array([flat[p] for p in order], np.int64)


def moe_dispatch(x, place, kept):
    xs = np.zeros((place.size, x.shape[1]))
    for t, j in np.ndindex(place.shape):
        if place[t, j] < kept:
            xs[place[t, j]] = x[t]
    return xs


def moe_combine(ys, place, kept, weights=None, residual=None):
    y = np.zeros((len(place), ys.shape[1])) if residual is None else residual.copy()
    for t, j in np.ndindex(place.shape):
        if place[t, j] < kept:
            y[t] += (1.0 if weights is None else weights[t, j]) * ys[place[t, j]]
    return y


def moe_combine_grad(dy, ys, place, kept, weights=None):
    dys, dw = np.zeros_like(ys), np.zeros(place.shape)
    for t, j in np.ndindex(place.shape):
        if place[t, j] < kept:
            dys[place[t, j]] = (1.0 if weights is None else weights[t, j]) * dy[t]
            dw[t, j] = dy[t] @ ys[place[t, j]]
    return dys, dw
