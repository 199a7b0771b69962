"""Plain reference of the 8-bit key/value cache (include/nq.h, nq_kv_*):
loops over sequences, blocks and heads, products and sums in float64.

The steps that the contract states in fp32 (scales, reciprocals, the value
that is rounded to a code) are taken in numpy float32, whose division and
product are correctly rounded."""
import numpy as np

QMAX = {"int8": 127.0, "fp8": 448.0}
MIN_SCALE = np.float32(2.0 ** -100)
F = np.float32


def e4m3_table():
    v = np.empty(256, np.float64)
    for byte in range(256):
        e, m = byte >> 3 & 15, byte & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            x = np.nan
        v[byte] = -x if byte >> 7 else x
    return v


E4M3 = e4m3_table()
_POSITIVE = E4M3[:127]      # 0 .. 448, rising with the byte


def values(codes, fmt):
    """uint8 codes -> float64 values in units of the scale."""
    return codes.astype(np.float64) - 128.0 if fmt == "int8" else E4M3[codes]


def encode(x, fmt):
    """float32 values in units of the scale -> uint8 codes, ties to even."""
    x = np.asarray(x, np.float64)
    if fmt == "int8":
        return (np.clip(np.rint(x), -127, 127) + 128).astype(np.uint8)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POSITIVE, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _POSITIVE[hi] - a, a - _POSITIVE[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


class Cache:
    """k_codes [blocks, heads, block, dim], v_codes [blocks, heads, dim,
    block], scales [blocks, heads]."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, fmt):
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.fmt = fmt
        self.blocks, self.heads, self.block, self.dim = k_codes.shape

    def slab(self, part, i, h):
        """The codes of one block and head as [block, dim] (a view)."""
        return self.k_codes[i, h] if part == "k" else self.v_codes[i, h].T

    def scales(self, part):
        return self.k_scales if part == "k" else self.v_scales


def block_id(cache, table, b, j):
    if j < 0 or j >= table.shape[1]:
        return -1
    i = int(table[b, j])
    return i if 0 <= i < cache.blocks else -1


def _write_block(cache, part, i, h, lo, x):
    """Rows x [n, dim] (float32) into slots lo .. of block i, head h."""
    qmax = F(QMAX[cache.fmt])
    scales = cache.scales(part)
    a = F(np.abs(x).max())
    codes = cache.slab(part, i, h)
    if not np.isfinite(a):      # from here on the block holds no numbers; codes do not matter
        scales[i, h] = np.nan
        codes[lo:lo + len(x)] = encode(np.zeros_like(x), cache.fmt)
        return
    fresh = max(F(a / qmax), MIN_SCALE) if a > 0 else F(0)
    s = fresh
    if lo > 0:
        s = scales[i, h]
        reach = F(s * qmax)
        if a > reach:
            with np.errstate(divide="ignore", over="ignore"):
                ratio = F(a / reach)
            if s == 0 or ratio > 2.0 ** 20:
                s, shrink = fresh, F(0)
            else:
                j = 0
                while F(2.0 ** j) < ratio:
                    j += 1
                s, shrink = F(s * F(2.0 ** j)), F(2.0 ** -j)
            codes[:lo] = encode(F(values(codes[:lo], cache.fmt)) * shrink, cache.fmt)
    scales[i, h] = s
    inv = F(F(1) / s) if s > 0 else F(0)
    codes[lo:lo + len(x)] = encode((x * inv).astype(F), cache.fmt)


def append(cache, row_start, lengths, table, k, v):
    """k, v [rows, heads, dim] float32."""
    for b in range(len(lengths)):
        r0, r1 = int(row_start[b]), int(row_start[b + 1])
        first = int(lengths[b]) - (r1 - r0)
        for j in range(first // cache.block, -(-int(lengths[b]) // cache.block)) if r1 > r0 else ():
            i = block_id(cache, table, b, j)
            lo, hi = max(first, j * cache.block), min(int(lengths[b]), (j + 1) * cache.block)
            if i < 0 or lo >= hi:
                continue
            for part, x in (("k", k), ("v", v)):
                for h in range(cache.heads):
                    _write_block(cache, part, i, h, lo - j * cache.block, x[r0 + lo - first:r0 + hi - first, h])


def tokens(cache, part, b, t0, t1, table):
    """Tokens t0 .. t1 of sequence b -> (float32 values [t, heads, dim] as
    nq_kv_read gives them before the last rounding, exists [t])."""
    out = np.zeros((t1 - t0, cache.heads, cache.dim), F)
    there = np.zeros(t1 - t0, bool)
    for j in range(t0 // cache.block, -(-t1 // cache.block)):
        i = block_id(cache, table, b, j)
        if i < 0:
            continue
        lo, hi = max(t0, j * cache.block), min(t1, (j + 1) * cache.block)
        there[lo - t0:hi - t0] = True
        for h in range(cache.heads):
            c = values(cache.slab(part, i, h)[lo - j * cache.block:hi - j * cache.block], cache.fmt)
            out[lo - t0:hi - t0, h] = F(c) * cache.scales(part)[i, h]
    return out, there


def read(cache, row_start, lengths, table):
    out = {"k": [], "v": []}
    for b in range(len(lengths)):
        n = int(row_start[b + 1]) - int(row_start[b])
        for part in out:
            out[part].append(tokens(cache, part, b, int(lengths[b]) - n, int(lengths[b]), table)[0])
    return np.concatenate(out["k"]), np.concatenate(out["v"])


def attention(cache, row_start, lengths, table, q, scale, causal=True, window=0):
    """q [rows, q_heads, dim] float64 -> a dict of out and lse, and an error
    bound's ingredients: spread (sum of w |v|), reach (largest scale * sum
    |q||k| over the visible tokens), largest (the largest of w times what its
    token's value scale can hold) and seen (visible tokens), all float64."""
    rows, heads, dim = q.shape
    group = heads // cache.heads
    out, spread = np.zeros((2, rows, heads, dim))
    lse, reach, seen = np.full((rows, heads), -np.inf), np.zeros((rows, heads)), np.zeros(rows, np.int64)
    largest = np.zeros((rows, heads))
    for b in range(len(lengths)):
        r0, r1, length = int(row_start[b]), int(row_start[b + 1]), max(0, int(lengths[b]))
        if r1 <= r0:
            continue
        k, there = tokens(cache, "k", b, 0, length, table)
        v, _ = tokens(cache, "v", b, 0, length, table)
        k, v = k.astype(np.float64), v.astype(np.float64)
        t = np.arange(length)
        holds = np.zeros((length, cache.heads))
        for i in np.flatnonzero(there):
            holds[i] = QMAX[cache.fmt] * cache.v_scales[table[b, i // cache.block]]
        for r in range(r0, r1):
            p = length - r1 + r
            see = there.copy()
            if causal:
                see &= t <= p
            if window:
                see &= t > p - window
            seen[r] = see.sum()
            if not see.any():
                continue
            for h in range(heads):
                z = scale * (k[see, h // group] @ q[r, h])
                m = z.max()
                w = np.exp(z - m)
                out[r, h] = w @ v[see, h // group] / w.sum()
                spread[r, h] = w @ np.abs(v[see, h // group]) / w.sum()
                largest[r, h] = (w * holds[see, h // group]).max() / w.sum()
                lse[r, h] = m + np.log(w.sum())
                reach[r, h] = scale * (np.abs(k[see, h // group]) @ np.abs(q[r, h])).max()
    return {"out": out, "lse": lse, "spread": spread, "reach": reach, "largest": largest, "seen": seen}


def attention_shared(cache, prefix_start, prefix_lengths, prefix_table, row_start, lengths, table, q, scale, causal=True):
    """As attention(), rows prefix_start[p] .. prefix_start[p + 1] seeing all of prefix p's tokens first."""
    rows, heads, dim = q.shape
    group = heads // cache.heads
    out, spread = np.zeros((2, rows, heads, dim))
    lse, reach, seen = np.full((rows, heads), -np.inf), np.zeros((rows, heads)), np.zeros(rows, np.int64)
    largest = np.zeros((rows, heads))

    def whole(b, length, table):
        """Keys, values, what a value's scale can hold, and whether the token is there."""
        k, there = tokens(cache, "k", b, 0, length, table)
        v, _ = tokens(cache, "v", b, 0, length, table)
        holds = np.zeros((length, cache.heads))
        for i in np.flatnonzero(there):
            holds[i] = QMAX[cache.fmt] * cache.v_scales[table[b, i // cache.block]]
        return k.astype(np.float64), v.astype(np.float64), holds, there

    before = [whole(p, max(0, int(n)), prefix_table) for p, n in enumerate(prefix_lengths)]
    for b in range(len(lengths)):
        r0, r1, length = int(row_start[b]), int(row_start[b + 1]), max(0, int(lengths[b]))
        if r1 <= r0:
            continue
        own = whole(b, length, table)
        for r in range(r0, r1):
            see = own[3].copy()
            if causal:
                see &= np.arange(length) <= length - r1 + r
            parts = [[a[see] for a in own[:3]]]
            for p in range(len(prefix_lengths)):
                if prefix_start[p] <= r < prefix_start[p + 1]:
                    parts.insert(0, [a[before[p][3]] for a in before[p][:3]])
            k, v, holds = (np.concatenate(a) for a in zip(*parts))
            seen[r] = len(k)
            if not len(k):
                continue
            for h in range(heads):
                j = h // group
                z = scale * (k[:, j] @ q[r, h])
                m = z.max()
                w = np.exp(z - m)
                out[r, h] = w @ v[:, j] / w.sum()
                spread[r, h] = w @ np.abs(v[:, j]) / w.sum()
                largest[r, h] = (w * holds[:, j]).max() / w.sum()
                lse[r, h] = m + np.log(w.sum())
                reach[r, h] = scale * (np.abs(k[:, j]) @ np.abs(q[r, h])).max()
    return {"out": out, "lse": lse, "spread": spread, "reach": reach, "largest": largest, "seen": seen}
