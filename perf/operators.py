"""What is measured of the 8-bit key/value cache and of the expert router.

Four operators: a cache of keys and values is written in 8 bits (op "write":
the new tokens are quantised into their blocks, then the touched blocks are
read back), whole sequences are read back (op "read"), attention runs over
such a cache (op "attend"), and tokens are routed to experts, with the
gradient where a case trains (op "route").

`own` false computes them with elementary torch operations in 32 bits; true
makes the package's calls.  Both work on the same tensors:

- A cache holds blocks of `block` tokens.  k_codes [blocks, kv_heads, block,
  head_dim] and v_codes [blocks, kv_heads, head_dim, block] are bytes,
  k_scales and v_scales [blocks, kv_heads] float32: a value is its block's
  scale times what its byte stands for, byte - 128 ("int8") or the E4M3
  number ("fp8").
- Sequence b's rows of this call are row_start[b] .. row_start[b + 1]; they
  are the last tokens of its lengths[b]; token t lies in slot t % block of
  block table[b, t // block].
- Writing: a block whose first token is written in this call takes the scale
  a / qmax (a the largest magnitude, qmax 127 or 448, at least 2^-100, zero
  for zeros); a block that holds older tokens keeps its scale, or, when the new
  tokens pass it, takes it times the smallest power of two that holds them, and
  the older codes are rounded to it (to zero past 2^20).  A code is x times the
  reciprocal of the scale, rounded to even.
"""
import math

import torch

own = False

QMAX = {"int8": 127.0, "fp8": 448.0}
MIN_SCALE = 2.0 ** -100
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    """Head layouts are those of this repository's projections: 4096 = 32
    heads of 128 columns, 1024 = 8 key/value heads of 128."""
    return [
        # a serving step of a small batch: every sequence adds one token, some to a fresh block
        _write("write_step", seqs=16, new=1, new_lo=1, length=700, kv=8, dim=128, block=16, fmt="int8", dt="bf16"),
        # prompts of uneven lengths go into the cache, one of them behind a shared prefix that ends inside a block
        _write("write_prompts", seqs=5, new=4096, new_lo=700, length=4199, kv=8, dim=128, block=64, fmt="fp8", dt="bf16"),
        # a short conversation is taken out of the cache in full precision
        _read("read_short", seqs=3, length=411, length_lo=1, kv=2, dim=64, block=32, fmt="fp8", dt="f32"),
        # a batch's caches are read back, to be moved or reused
        _read("read_batch", seqs=32, length=6000, length_lo=500, kv=8, dim=128, block=64, fmt="int8", dt="bf16"),
        # one user's next token: the shortest call, latency counts
        _attend("attend_one", seqs=1, new=1, new_lo=1, length=333, length_lo=333, heads=32, kv=8, dim=128, block=16,
                fmt="int8", dt="bf16"),
        # a serving batch's next tokens, contexts of uneven lengths
        _attend("attend_batch", seqs=64, new=1, new_lo=1, length=8192, length_lo=1024, heads=32, kv=8, dim=128,
                block=64, fmt="int8", dt="bf16"),
        # two very long documents, four draft tokens each to be verified at once
        _attend("attend_long", seqs=2, new=4, new_lo=4, length=131077, length_lo=120001, heads=32, kv=4, dim=128,
                block=128, fmt="fp8", dt="bf16"),
        # prompts are attended to themselves right after they were written
        _attend("attend_prompts", seqs=3, new=4096, new_lo=2047, length=4096, length_lo=2047, heads=32, kv=8, dim=128,
                block=64, fmt="int8", dt="bf16"),
        # a chunk of a long prompt in full precision, within a sliding window
        _attend("attend_window", seqs=3, new=257, new_lo=96, length=9001, length_lo=500, heads=16, kv=2, dim=64,
                block=32, fmt="fp8", dt="f32", window=2048),
        # a serving step's tokens among this repository's 32 experts
        _route("route_step", tokens=16, experts=32, top_k=4, score="softmax", dt="bf16", renorm=True),
        # a prompt's tokens, sigmoid scores with a balance bias, the best groups first
        _route("route_groups", tokens=16384, experts=256, top_k=8, score="sigmoid", dt="f32", renorm=True, bias=True,
               groups=8, top_groups=4, best=2, scale=2.5),
        # a training step: the weights, and the gradient of the logits
        _route("route_train", tokens=32768, experts=64, top_k=6, score="softmax", dt="bf16", renorm=False, train=True),
    ]


def _write(name, **c):
    return {"name": name, "op": "write", "heads": 0, **c}


def _read(name, **c):
    return {"name": name, "op": "read", **c}


def _attend(name, **c):
    return {"name": name, "op": "attend", "causal": True, "window": 0, **c}


def _route(name, **c):
    return {"name": name, "op": "route", "bias": False, "groups": 1, "top_groups": 1, "best": 1, "scale": 1.0,
            "train": False, **c}


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))

    layout = {"kv": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128, 128, 192, 256]),
              "block": rng.choice([16, 32, 64, 128]), "fmt": rng.choice(["int8", "fp8"])}
    dt = rng.choice(["bf16", "bf16", "f32"])
    op = rng.choice(["write", "read", "attend", "attend", "attend", "route"])
    width = layout["kv"] * layout["dim"]
    if op == "write":
        seqs = spread(1, 64)
        new = max(1, min(spread(1, 4096), 9_000_000 // (width * seqs)))
        c = _write("", seqs=seqs, new=new, new_lo=rng.randint(0, new), length=new + spread(1, 2000), dt=dt, **layout)
    elif op == "read":
        seqs = spread(1, 32)
        length = max(1, min(spread(1, 20000), 60_000_000 // (width * seqs)))
        c = _read("", seqs=seqs, length=length, length_lo=rng.randint(1, length), dt=dt, **layout)
    elif op == "attend":
        heads = layout["kv"] * rng.choice([1, 2, 3, 4, 7, 8, 16])
        if rng.random() < 0.6:      # next tokens, one or a few
            seqs, new = spread(1, 96), rng.choice([1, 1, 1, 2, 5])
            length = min(spread(8, 131072), 250_000_000 // (seqs * width))
        else:                       # prompts and their chunks
            seqs, new = spread(1, 4), spread(17, 3000)
            length = new + rng.choice([0, 0, spread(1, 20000)])
            # no more products than the listed prompts have
            pairs = 64_000_000_000 // (seqs * heads * layout["dim"])
            new = min(new, math.isqrt(pairs))
            length = max(new, min(length, pairs // new))
        new = min(new, length)
        c = _attend("", seqs=seqs, new=new, new_lo=rng.randint(1, new), length=length,
                    length_lo=rng.randint(new, length), heads=heads, dt=dt, **layout)
        c["causal"] = rng.random() < 0.85
        if c["causal"] and rng.random() < 0.25:
            c["window"] = spread(64, 4096)
    else:
        score = rng.choice(["softmax", "sigmoid"])
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * rng.choice([8, 16, 20, 32, 48])
        tokens = max(1, min(spread(1, 32768), 2_600_000 // experts))
        top_groups = rng.randint(1, groups)
        c = _route("", tokens=tokens, experts=experts, top_k=rng.randint(1, 8), score=score, dt=dt,
                   renorm=rng.random() < 0.6, bias=rng.random() < 0.5, train=rng.random() < 0.5, groups=groups,
                   top_groups=top_groups, best=rng.choice([1, 2]), scale=rng.choice([1.0, 2.5]))
    del c["name"]
    return c


# ---------------------------------------------------------------- geometry
def _uneven(lo, hi, count):
    """`count` sizes spread unevenly over lo .. hi, the last one hi."""
    return [hi if i == count - 1 else lo + int((hi - lo) * math.modf((i + 1) * 0.6180339887498949)[0])
            for i in range(count)]


def _sizes(c):
    """Rows of this call and lengths after it, for each sequence."""
    n = c["seqs"]
    if c["op"] == "read":
        lengths = _uneven(c["length_lo"], c["length"], n)
        return lengths, lengths
    new = _uneven(c["new_lo"], c["new"], n)
    if c["op"] == "write":      # every third sequence is new, the others have a context before these tokens
        before = [0 if i % 3 == 1 else (c["length"] - c["new"]) - 5 * i % max(1, c["length"] - c["new"])
                  for i in range(n)]
        return new, [a + b for a, b in zip(new, before)]
    return new, [max(a, b) for a, b in zip(new, _uneven(c["length_lo"], c["length"], n))]


def _starts(sizes):
    at = [0]
    for s in sizes:
        at.append(at[-1] + s)
    return at


def work(c):
    wide = 2 if c["dt"] == "bf16" else 4
    if c["op"] == "route":
        out = c["tokens"] * c["top_k"] * 8
        moved = c["tokens"] * c["experts"] * wide + out + (4 * c["experts"] if c["bias"] else 0)
        flops = 6.0 * c["tokens"] * c["experts"]
        if c["train"]:      # the logits again, the chosen ids, the weights' gradient in, the logits' out
            moved += 2 * c["tokens"] * c["experts"] * wide + out
            flops *= 2
        return {"bytes": float(moved), "flops": flops}
    new, lengths = _sizes(c)
    width = c["kv"] * c["dim"]
    if c["op"] == "write":      # rows in, their codes out; the touched blocks' codes in, their values out
        back = sum(_back(n, l, c["block"]) for n, l in zip(new, lengths))
        return {"bytes": 2.0 * width * (sum(new) * (wide + 1) + back * (1 + wide)), "flops": 8.0 * width * sum(new)}
    if c["op"] == "read":
        return {"bytes": 2.0 * width * sum(new) * (1 + wide), "flops": 2.0 * width * sum(new)}
    pairs, seen = 0, 0
    for n, l in zip(new, lengths):
        first = l - n
        for i in range(n):
            hi = first + i + 1 if c["causal"] else l
            pairs += min(hi, c["window"]) if c["window"] else hi
        seen += min(l, c["window"] + n - 1) if c["window"] else l
    return {"bytes": 2.0 * width * seen + 2.0 * sum(new) * c["heads"] * c["dim"] * wide,
            "flops": 4.0 * pairs * c["heads"] * c["dim"]}


def _back(n, length, block):
    """Tokens from the start of the first block that n new tokens touch."""
    return length - (length - n) // block * block if n else 0


# ---------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _cache(c, seed, g):
    """A pool of blocks full of other sequences' leftovers, and a table that takes blocks in any order."""
    new, lengths = _sizes(c)
    need = [(l + c["block"] - 1) // c["block"] for l in lengths]
    wide = max(1, max(need))
    blocks = sum(need) + 3
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((c["seqs"], wide), dtype=torch.int32, device="cuda")
    for b, at in enumerate(_starts(need)[:-1]):
        table[b, : need[b]] = order[at: at + need[b]]
    out = {"new": new, "lengths_host": lengths, "table": table, "spare": order[-1],
           "row_start": torch.tensor(_starts(new), dtype=torch.int32).cuda(),
           "lengths": torch.tensor(lengths, dtype=torch.int32).cuda()}
    for part, shape in (("k", (blocks, c["kv"], c["block"], c["dim"])), ("v", (blocks, c["kv"], c["dim"], c["block"]))):
        codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (c["kv"] * c["block"] * c["dim"]))
        for i in range(0, blocks, step):    # normal values whose largest lie about four deviations out
            x = torch.randn((min(step, blocks - i),) + shape[1:], generator=g, device="cuda") * (QMAX[c["fmt"]] / 4)
            codes[i: i + step] = _encode(x, c["fmt"])
        out[part + "_codes"] = codes
        jitter = torch.rand((blocks, c["kv"]), generator=g, device="cuda") * 0.5 + 0.75
        out[part + "_scales"] = (4 / QMAX[c["fmt"]]) * jitter
    return out


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = {"case": c}
    if c["op"] == "route":
        s.update(_route_inputs(c, g))
        if own:
            import group_wise_affine_quantize_amd as nq
            s["nq"] = nq
            s["router"] = nq.MoERouter(c["experts"], c["top_k"], score=c["score"], groups=c["groups"],
                                       top_groups=c["top_groups"], group_best=c["best"], renormalise=c["renorm"],
                                       scale=c["scale"])
        return s
    s.update(_cache(c, seed, g))
    rows, dt = sum(s["new"]), DTYPES[c["dt"]]
    if c["op"] in ("write", "attend"):
        # queries, keys and values are column ranges of one fused projection's output
        heads = c["heads"] + 2 * c["kv"]
        fused = torch.randn((rows, heads, c["dim"]), generator=g, device="cuda")
        if c["op"] == "write":
            fused *= torch.rand((rows, heads, 1), generator=g, device="cuda") + 0.5
        else:
            fused *= 1.5
        s["fused"] = fused.to(dt)
        s["q"], s["k"], s["v"] = s["fused"].split([c["heads"], c["kv"], c["kv"]], dim=1)
    if c["op"] == "write":
        s["back"] = [_back(n, l, c["block"]) for n, l in zip(s["new"], s["lengths_host"])]
        s["back_start"] = torch.tensor(_starts(s["back"]), dtype=torch.int32).cuda()
    if own:
        import group_wise_affine_quantize_amd as nq
        s["nq"] = nq
        s["cache"] = nq.KVCache.wrap(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], c["fmt"])
        s["seqs"] = nq.KVSequences(s["row_start"], s["lengths"], s["table"], rows)
        if c["op"] == "write":
            s["back_seqs"] = nq.KVSequences(s["back_start"], s["lengths"], s["table"], sum(s["back"]))
    return s


def _route_inputs(c, g):
    """Logits of a gate, a bias as steps of 0.001 make it.  Tokens whose choice
    would hang on the last bits of 32 are drawn again: what is chosen follows
    from the formulas."""
    dt = DTYPES[c["dt"]]
    t, e = c["tokens"], c["experts"]
    bias = None
    if c["bias"]:
        bias = torch.randint(-60, 61, (e,), generator=g, device="cuda").float() * 0.001
    logits = (torch.randn((t, e), generator=g, device="cuda") * 1.5).to(dt)
    for _ in range(12):
        x = logits.double()
        p = torch.softmax(x, -1) if c["score"] == "softmax" else torch.sigmoid(x)
        key = p if bias is None else p + bias.double()
        close = _close(key, min(e, 2 * c["top_k"] + 1))
        if c["groups"] > 1:
            per = torch.sort(key.view(t, c["groups"], -1), -1, descending=True).values
            score = per[..., : c["best"]].sum(-1)
            close |= _close(score, c["groups"])
            order = torch.sort(score, dim=-1, descending=True, stable=True).indices[:, : c["top_groups"]]
            kept = torch.zeros_like(score, dtype=torch.bool).scatter_(1, order, True)
            inside = key.masked_fill(~kept.repeat_interleave(e // c["groups"], 1), -1e30)
            close |= _close(inside, min(e, c["top_k"] + 1))
        fresh = (torch.randn((t, e), generator=g, device="cuda") * 1.5).to(dt)
        logits = torch.where(close[:, None], fresh, logits)
    out = {"logits": logits, "bias": bias}
    if c["train"]:
        out["dweights"] = torch.randn((t, c["top_k"]), generator=g, device="cuda")
    return out


def _close(key, top):
    """Rows whose `top` largest keys hold two that differ by less than 32 bits can tell."""
    s = torch.sort(key, -1, descending=True).values[:, :top]
    gap = s[:, :-1] - s[:, 1:]
    return ((gap > 0) & (gap < 4e-6 * s[:, :1].abs().clamp(min=1e-3))).any(-1)


# ---------------------------------------------------------------- a pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _own_write(s):
    nq = s["nq"]
    nq.nq_kv_append(s["cache"], s["seqs"], s["k"], s["v"])
    k, v = nq.nq_kv_read(s["cache"], s["back_seqs"], out_dtype=s["k"].dtype)
    return {"k": k, "v": v}


def _own_read(s):
    k, v = s["nq"].nq_kv_read(s["cache"], s["seqs"], out_dtype=DTYPES[s["case"]["dt"]])
    return {"k": k, "v": v}


def _own_attend(s):
    c = s["case"]
    return s["nq"].nq_kv_attention(s["cache"], s["seqs"], s["q"], causal=c["causal"], window=c["window"])


def _own_route(s):
    nq = s["nq"]
    ids, weights = nq.nq_moe_route(s["router"], s["logits"], bias=s["bias"])
    out = {"ids": ids, "weights": weights}
    if s["case"]["train"]:
        out["dlogits"] = nq.nq_moe_route_grad(s["router"], s["logits"], ids, s["dweights"])
    return out


_OWN = {"write": _own_write, "read": _own_read, "attend": _own_attend, "route": _own_route}


# ---------------------------------------------------------------- the plain form
def _encode(x, fmt):
    """float32 values in units of the scale -> bytes."""
    if fmt == "int8":
        return (x.round().clamp(-127, 127) + 128).to(torch.uint8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes, fmt):
    """bytes -> float32 values in units of the scale."""
    if fmt == "int8":
        return codes.float() - 128
    return codes.view(torch.float8_e4m3fn).float()


def _sequence(s, b, length):
    """Keys and values of sequence b's first `length` tokens, [kv_heads, length, head_dim] float32."""
    c = s["case"]
    ids = s["table"][b, : (length + c["block"] - 1) // c["block"]].long()
    k = _decode(s["k_codes"][ids], c["fmt"]) * s["k_scales"][ids][:, :, None, None]
    v = _decode(s["v_codes"][ids], c["fmt"]) * s["v_scales"][ids][:, :, None, None]
    k = k.transpose(0, 1).reshape(c["kv"], -1, c["dim"])
    v = v.permute(1, 0, 3, 2).reshape(c["kv"], -1, c["dim"])
    return k[:, :length], v[:, :length]


def _read_rows(s, counts, dt):
    ks, vs = [], []
    for b, (n, length) in enumerate(zip(counts, s["lengths_host"])):
        if n:
            k, v = _sequence(s, b, length)
            ks.append(k[:, length - n:].transpose(0, 1).to(dt))
            vs.append(v[:, length - n:].transpose(0, 1).to(dt))
    return {"k": torch.cat(ks), "v": torch.cat(vs)}


def _plain_write(s):
    c = s["case"]
    block, fmt, qmax = c["block"], c["fmt"], QMAX[c["fmt"]]
    rows = s["k"].shape[0]
    at = torch.arange(rows, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["row_start"][1:].contiguous(), at, right=True)
    pos = s["lengths"][seq] - s["row_start"][seq + 1] + at
    ids = s["table"][seq, (pos // block).long()].long()
    slot = (pos % block).long()
    # each sequence's first touched block may hold older tokens; the others point at a spare block
    counts = s["row_start"][1:] - s["row_start"][:-1]
    first = s["lengths"] - counts
    old = torch.where(counts > 0, first % block, 0)
    at_first = (first // block).long().clamp(max=s["table"].shape[1] - 1)
    old_ids = torch.where(old > 0, s["table"].gather(1, at_first[:, None])[:, 0], s["spare"]).long()
    held = torch.zeros(s["k_scales"].shape[0], dtype=torch.bool, device="cuda")
    held[old_ids] = True
    touched = torch.zeros_like(held)
    touched[ids] = True
    for part in ("k", "v"):
        x = s[part].float()
        codes, scales = s[part + "_codes"], s[part + "_scales"]
        a = torch.zeros_like(scales).scatter_reduce_(0, ids[:, None].expand(-1, c["kv"]), x.abs().amax(-1), "amax")
        fresh = torch.where(a > 0, (a / torch.full_like(a, qmax)).clamp(min=MIN_SCALE), 0.0)
        reach = scales * qmax
        ratio = a / reach
        mant, expo = torch.frexp(ratio)
        expo = torch.where(mant == 0.5, expo - 1, expo)
        lost = ratio > 2.0 ** 20
        grow = a > reach
        grown = torch.where(lost | (scales == 0), fresh, torch.ldexp(scales, expo))
        scale = torch.where(held[:, None], torch.where(grow, grown, scales), fresh)
        # the older codes of blocks that grew are rounded to the new scale
        o = old_ids
        have = codes[o] if part == "k" else codes[o].transpose(2, 3)
        shrink = torch.where(lost | (scales == 0), 0.0, torch.ldexp(torch.ones_like(scales), -expo))[o]
        again = _encode(_decode(have, fmt) * shrink[:, :, None, None], fmt)
        change = (torch.arange(block, device="cuda") < old[:, None])[:, None, :] & grow[o][:, :, None]
        have = torch.where(change[..., None], again, have)
        codes[o] = have if part == "k" else have.transpose(2, 3)
        scales.copy_(torch.where(touched[:, None], scale, scales))
        inv = torch.where(scales > 0, 1.0 / scales, 0.0)
        y = _encode(x * inv[ids][..., None], fmt)
        if part == "k":
            codes[ids, :, slot] = y
        else:
            codes[ids, :, :, slot] = y
    return _read_rows(s, s["back"], s["k"].dtype)


def _plain_read(s):
    return _read_rows(s, s["new"], DTYPES[s["case"]["dt"]])


def _plain_attend(s):
    c = s["case"]
    out, group, at = [], c["heads"] // c["kv"], 0
    for b, (n, length) in enumerate(zip(s["new"], s["lengths_host"])):
        k, v = _sequence(s, b, length)
        q = s["q"][at: at + n].float().view(n, c["kv"], group, c["dim"])
        q = q.permute(1, 0, 2, 3).reshape(c["kv"], n * group, c["dim"])
        at += n
        x = torch.matmul(q, k.transpose(1, 2).contiguous()) * c["dim"] ** -0.5
        if c["causal"]:
            pos = (torch.arange(n, device="cuda") + (length - n)).repeat_interleave(group)[:, None]
            key = torch.arange(length, device="cuda")[None]
            hide = key > pos
            if c["window"]:
                hide |= key <= pos - c["window"]
            x.masked_fill_(hide, float("-inf"))
        x -= x.amax(-1, keepdim=True)
        x.exp_()
        total = x.sum(-1, keepdim=True)
        y = torch.matmul(x, v.contiguous()) / total
        y = y.view(c["kv"], n, group, c["dim"]).permute(1, 0, 2, 3).reshape(n, c["heads"], c["dim"])
        out.append(y.to(s["q"].dtype))
    return torch.cat(out)


def _plain_scores(x, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    z = torch.exp(x - x.amax(-1, keepdim=True))
    return z / z.sum(-1, keepdim=True)


def _plain_route(s):
    c = s["case"]
    x = s["logits"].float()
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    p = _plain_scores(x, c["score"])
    key = p if s["bias"] is None else p + s["bias"]
    # without a bias the scores have the logits' order
    order = x if s["bias"] is None else key
    if c["groups"] > 1:
        per = (key if c["best"] > 1 else order).view(t, c["groups"], -1)
        best = torch.sort(per, -1, descending=True).values[..., : c["best"]].sum(-1)
        chosen = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, : c["top_groups"]]
        kept = torch.zeros_like(best, dtype=torch.bool).scatter_(1, chosen, True)
        order = order.masked_fill(~kept.repeat_interleave(e // c["groups"], 1), float("-inf"))
    ids = torch.sort(order, dim=-1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    total = w.sum(-1, keepdim=True)
    share = w / total if c["renorm"] else w
    out = {"ids": ids.to(torch.int32), "weights": share * c["scale"]}
    if c["train"]:
        d = s["dweights"] * c["scale"]
        if c["renorm"]:
            d = (d - (d * share).sum(-1, keepdim=True)) / total
        if c["score"] == "sigmoid":
            got = d * w * (1 - w)
            dx = torch.zeros_like(x).scatter_(1, ids, got)
        else:
            dp = torch.zeros_like(x).scatter_(1, ids, d)
            dx = p * (dp - (d * w).sum(-1, keepdim=True))
        out["dlogits"] = dx.to(s["logits"].dtype)
    return out


_PLAIN = {"write": _plain_write, "read": _plain_read, "attend": _plain_attend, "route": _plain_route}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"write": _exact_write, "read": _exact_read, "attend": _exact_attend, "route": _exact_route}[case["op"]](s)


def _e4m3_values():
    """The value of each E4M3 byte, from the format: sign, 4 bits of exponent (bias 7), 3 of fraction."""
    v = []
    for byte in range(256):
        sign, e, m = byte >> 7, byte >> 3 & 15, byte & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(math.nan if e == 15 and m == 7 else -x if sign else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _exact_values(codes, fmt):
    return codes.double() - 128 if fmt == "int8" else _e4m3_values()[codes.long()]


def _exact_round(x, fmt):
    """The nearest values of the format, ties to even; x in float64."""
    if fmt == "int8":
        return torch.round(x).clamp(-127, 127)
    x = x.clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _token_values(s, part, b, first, last):
    """Tokens first .. last of sequence b, [tokens, kv_heads, head_dim] float64, one block at a time."""
    c, out = s["case"], []
    for j in range(first // c["block"], (last - 1) // c["block"] + 1):
        i = int(s["table"][b, j])
        x = _exact_values(s[part + "_codes"][i], c["fmt"]) * s[part + "_scales"][i].double()[:, None, None]
        if part == "v":
            x = x.transpose(1, 2)
        lo, hi = max(first - j * c["block"], 0), min(last - j * c["block"], c["block"])
        out.append(x[:, lo:hi].transpose(0, 1))
    return torch.cat(out)


def _exact_read(s):
    out = {}
    for part in ("k", "v"):
        out[part] = torch.cat([_token_values(s, part, b, 0, n) for b, n in enumerate(s["lengths_host"])])
    return out


def _f32(x):
    return x.float().double()


def _exact_write(s):
    c = s["case"]
    block, fmt, qmax = c["block"], c["fmt"], QMAX[c["fmt"]]
    out = {}
    for part in ("k", "v"):
        rows = []
        for b, (n, length, at) in enumerate(zip(s["new"], s["lengths_host"], _starts(s["new"]))):
            first = length - n
            for j in range(first // block, (length - 1) // block + 1) if n else ():
                lo, hi = max(first, j * block), min(length, (j + 1) * block)
                x = s[part][at + lo - first: at + hi - first].double()
                a = x.abs().amax((0, 2))
                scale = torch.where(a > 0, _f32(a / qmax).clamp(min=MIN_SCALE), 0.0)
                older = x[:0]
                if lo > j * block:
                    i = int(s["table"][b, j])
                    codes = _exact_values(s[part + "_codes"][i], fmt)
                    codes = (codes if part == "k" else codes.transpose(1, 2))[:, : lo - j * block].transpose(0, 1)
                    had = s[part + "_scales"][i].double()
                    reach = _f32(had * qmax)
                    ratio = _f32(a / reach)
                    power = torch.exp2(torch.ceil(torch.log2(ratio.clamp(1.0, 2.0 ** 20))))
                    gone = (ratio > 2.0 ** 20) | (had == 0)
                    scale = torch.where(a > reach, torch.where(gone, scale, had * power), had)
                    moved = torch.where((a > reach) & gone, 0.0, 1 / torch.where(a > reach, power, 1.0))
                    older = _exact_round(codes * moved[:, None], fmt) * scale[:, None]
                inverse = torch.where(scale > 0, _f32(1 / scale), 0.0)
                rows += [older, _exact_round(_f32(x * inverse[:, None]), fmt) * scale[:, None]]
        out[part] = torch.cat(rows)
    return out


def _exact_attend(s):
    c = s["case"]
    out, group, at = [], c["heads"] // c["kv"], 0
    for b, (n, length) in enumerate(zip(s["new"], s["lengths_host"])):
        ids = s["table"][b, : (length + c["block"] - 1) // c["block"]].long()
        y = torch.empty((n, c["heads"], c["dim"]), dtype=torch.float64, device="cuda")
        pos = torch.arange(length - n, length, device="cuda")
        for h in range(c["kv"]):
            k = _exact_values(s["k_codes"][ids, h], c["fmt"]) * s["k_scales"][ids, h].double()[:, None, None]
            v = _exact_values(s["v_codes"][ids, h], c["fmt"]) * s["v_scales"][ids, h].double()[:, None, None]
            k = k.reshape(-1, c["dim"])[:length]
            v = v.transpose(1, 2).reshape(-1, c["dim"])[:length]
            for j in range(h * group, (h + 1) * group):
                z = s["q"][at: at + n, j].double() @ k.t() / math.sqrt(c["dim"])
                if c["causal"]:
                    gap = pos[:, None] - torch.arange(length, device="cuda")
                    seen = gap >= 0 if not c["window"] else (gap >= 0) & (gap < c["window"])
                    z = torch.where(seen, z, -math.inf)
                y[:, j] = torch.exp(z - torch.logsumexp(z, -1, keepdim=True)) @ v
        at += n
        out.append(y)
    return torch.cat(out)


def _exact_route(s):
    c = s["case"]
    x = s["logits"].double().requires_grad_(c["train"])
    t, e = x.shape
    p = torch.softmax(x, -1) if c["score"] == "softmax" else torch.sigmoid(x)
    key = (p if s["bias"] is None else p + s["bias"].double()).detach()
    if c["groups"] > 1:
        score = torch.topk(key.view(t, c["groups"], -1), c["best"], -1).values.sum(-1)
        worse = (score[:, None, :] > score[:, :, None]).sum(-1)
        tied = (score[:, None, :] == score[:, :, None]).tril(-1).sum(-1)
        dropped = (worse + tied >= c["top_groups"]).repeat_interleave(e // c["groups"], 1)
        key = key.masked_fill(dropped, -math.inf)
    ids = torch.argsort(key, dim=-1, descending=True, stable=True)[:, : c["top_k"]]
    w = torch.gather(p, 1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    w = w * c["scale"]
    out = {"ids": ids.to(torch.int32), "weights": w.detach()}
    if c["train"]:
        (w * s["dweights"].double()).sum().backward()
        out["dlogits"] = x.grad
    return out
