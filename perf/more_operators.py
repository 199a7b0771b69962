"""What is measured of the steps between a decoder layer's products.

Four operators: norms before and after a block with its gate and residual
scale (op "norm"), rotary positions with one or several axes (op "rope"),
tokens sorted by expert and back (op "moe"), and attention of a batch whose
sequences share prefixes in the 8-bit key/value cache (op "shared").  The first
three with their gradients where a case trains.

`own` false computes them with elementary torch operations in 32 bits (angles
in 64); true makes the package's calls.  Both work on the same tensors:

- norm: h (the residual stream) and y (a block's output) are [rows, dim];
  u = y / sqrt(mean y^2 + eps) * (post + offset), or y without `post`;
  h_out = h + scale * gate * u; z = h_out / sqrt(mean h_out^2 + eps) * (pre +
  offset), from h_out before it is rounded.  gate [gates, dim] serves rows /
  gates neighbouring rows each.  The gradient takes the h_out that the step's
  forward pass stored (`stored`).
- rope: pair i of a head's first rotary_dim columns, which are (i, i +
  rotary_dim / 2) or (2 i, 2 i + 1), is turned by freq[i] times the row's
  position on axis[i]; the columns behind are copied.
- moe: pairs (token, choice) in the stable order of their experts; experts
  outside 0 .. experts - 1 come last and are dropped: their rows are zeros.
- shared: the cache is the one of perf/operators.py (blocks of `block` tokens,
  k_codes [blocks, kv_heads, block, head_dim], v_codes transposed, a scale for
  each block and head).  Rows prefix_start[p] .. prefix_start[p + 1] see all
  prefix_lengths[p] tokens of prefix p, then their own sequence's tokens, of
  which they are the last.
"""
import math

import torch

own = False

QMAX = {"int8": 127.0, "fp8": 448.0}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    """Widths are this repository's (hidden sizes 4096 and 2048; 32, 16, 8 and 4 heads of
    128 and 64; 32 experts, 4 of them for a token) or generic."""
    return [
        # a serving step: the block's output is normed, gated and added, the next block's input normed
        _norm("norm_step", rows=16, dim=4096, dt="bf16", pdt="bf16", gate="channel", scale=0.5),
        # a prompt's tokens through the same, without a gate
        _norm("norm_prompt", rows=8191, dim=4096, dt="bf16", pdt="bf16", offset=1.0),
        # a training step, a gate for each of four sequences, parameters kept in 32 bits
        _norm("norm_train", rows=8192, dim=2048, dt="bf16", pdt="f32", gate="batch", gates=4, train=True),
        # training in full precision at an odd width, a gate for every row
        _norm("norm_train_odd", rows=1501, dim=1407, dt="f32", pdt="f32", gate="rows", scale=0.25, offset=1.0,
              train=True),
        # a serving step far into long contexts: queries and keys of a fused projection
        _rope("rope_step", rows=16, heads=40, behind=8, dim=128, rotary=128, layout="halves", axes=1, far=131072,
              dt="bf16"),
        # training on images and video: time, height and width by turns, in full precision
        _rope("rope_train", rows=9001, heads=18, behind=2, dim=64, rotary=48, layout="pairs", axes=3, far=6000,
              dt="f32", train=True),
        # a serving step's tokens to their experts and back
        _moe("moe_step", tokens=16, top_k=4, experts=32, hidden=2048, dt="bf16", residual=True),
        # a prompt's tokens, an eighth of the experts on this device
        _moe("moe_prompt", tokens=8192, top_k=8, experts=256, hidden=4096, dt="bf16", residual=True, dropped=0.3),
        # a training step
        _moe("moe_train", tokens=8192, top_k=6, experts=64, hidden=2048, dt="bf16", train=True),
        # four users behind one system prompt
        _shared("shared_few", prefixes=1, prefix=700, prefix_lo=700, seqs=4, new=1, length=90, length_lo=17, heads=32,
                kv=8, dim=128, block=16, fmt="int8", dt="bf16"),
        # a serving batch behind a long document
        _shared("shared_batch", prefixes=1, prefix=16384, prefix_lo=16384, seqs=64, new=1, length=700, length_lo=33,
                heads=32, kv=8, dim=128, block=64, fmt="int8", dt="bf16"),
        # drafts of three tokens behind documents of uneven lengths, some sequences behind none
        _shared("shared_groups", prefixes=3, prefix=30011, prefix_lo=9000, seqs=40, new=3, length=1500, length_lo=3,
                heads=16, kv=4, dim=128, block=32, fmt="fp8", dt="bf16", loose=4),
    ]


def _norm(name, **c):
    return {"name": name, "op": "norm", "post": True, "pre": True, "gate": "none", "gates": 1, "scale": 1.0,
            "offset": 0.0, "train": False, **c}


def _rope(name, **c):
    return {"name": name, "op": "rope", "scale": 1.0, "train": False, **c}


def _moe(name, **c):
    return {"name": name, "op": "moe", "residual": False, "dropped": 0.0, "train": False, **c}


def _shared(name, **c):
    return {"name": name, "op": "shared", "loose": 0, **c}


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))

    op = rng.choice(["norm", "norm", "rope", "moe", "moe", "shared", "shared"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    train = rng.random() < 0.5
    if op == "norm":
        dim = spread(64, 8192)
        dim -= rng.choice([0, dim % 8, dim % 8, dim % 64])
        rows = max(1, min(spread(1, 8192), (8_000_000 if train else 16_000_000) // dim))
        gate = rng.choice(["none", "channel", "batch", "rows"])
        gates = {"channel": 1, "rows": rows}.get(gate, 1)
        if gate == "batch":
            gates = rng.randint(2, 5)
            rows = max(1, rows // gates) * gates
        c = _norm("", rows=rows, dim=dim, dt=dt, pdt=rng.choice([dt, "f32"]), gate=gate, gates=gates,
                  scale=rng.choice([1.0, 0.5]), offset=rng.choice([0.0, 1.0]), post=rng.random() < 0.7, train=train)
    elif op == "rope":
        dim = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
        rotary = rng.choice([dim, dim, dim // 2, dim // 4 * 3])
        heads = rng.randint(1, 48)
        c = _rope("", rows=max(1, min(spread(1, 16384), 10_000_000 // (heads * dim))), heads=heads,
                  behind=rng.choice([0, 1, 8]), dim=dim, rotary=rotary, layout=rng.choice(["halves", "pairs"]),
                  axes=rng.choice([1, 2, 3]), far=spread(100, 1_000_000), dt=dt, scale=rng.choice([1.0, 1.0, 1.1]),
                  train=train)
    elif op == "moe":
        top_k, hidden = rng.randint(1, 8), spread(64, 8192)
        hidden -= rng.choice([0, hidden % 8, hidden % 8, hidden % 64])
        tokens = max(1, min(spread(1, 32768), 16_000_000 // (hidden * top_k)))
        c = _moe("", tokens=tokens, top_k=top_k, experts=rng.choice([8, 20, 32, 64, 160, 256]), hidden=hidden, dt=dt,
                 residual=rng.random() < 0.5, dropped=rng.choice([0.0, 0.0, 0.1, 0.8]), train=train)
    else:
        kv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 192, 256])
        seqs, new = spread(1, 80), rng.choice([1, 1, 1, 2, 5])
        heads = kv * rng.choice([1, 2, 4, 4, 8])
        prefixes = rng.choice([1, 1, 2, 4])
        loose = rng.choice([0, 0, 0, 1])
        seqs = max(seqs, prefixes + loose)
        # no more than the largest listed case moves and multiplies
        prefix = min(spread(20, 40000), 8_000_000_000 // (seqs * new * heads * dim * 4) + 20,
                     40_000_000 // (prefixes * kv * dim))
        length = max(new, min(spread(1, 3000), 20_000_000 // (seqs * kv * dim)))
        c = _shared("", prefixes=prefixes, prefix=prefix, prefix_lo=rng.randint(1, prefix), seqs=seqs, new=new,
                    length=length, length_lo=rng.randint(new, length), heads=heads, kv=kv, dim=dim,
                    block=rng.choice([16, 32, 64, 128]), fmt=rng.choice(["int8", "fp8"]), dt=dt, loose=loose)
    del c["name"]
    return c


# ---------------------------------------------------------------- geometry
def _uneven(lo, hi, count):
    """`count` sizes spread unevenly over lo .. hi, the last one hi."""
    return [hi if i == count - 1 else lo + int((hi - lo) * math.modf((i + 1) * 0.6180339887498949)[0])
            for i in range(count)]


def _starts(sizes):
    at = [0]
    for s in sizes:
        at.append(at[-1] + s)
    return at


def _layout(c):
    """Shared prefixes: lengths of the sequences' own tokens, lengths of the
    prefixes, and the prefix of each sequence (-1: none); each prefix takes a
    run of neighbouring sequences."""
    behind = c["seqs"] - c["loose"]
    return (_uneven(c["length_lo"], c["length"], c["seqs"]), _uneven(c["prefix_lo"], c["prefix"], c["prefixes"]),
            [i * c["prefixes"] // behind if i < behind else -1 for i in range(c["seqs"])])


def work(c):
    if c["op"] == "shared":
        lengths, prefixes, of = _layout(c)
        new, wide = c["new"], 2 if c["dt"] == "bf16" else 4
        pairs = sum(new * (l + (prefixes[p] if p >= 0 else 0)) - new * (new - 1) // 2 for l, p in zip(lengths, of))
        rows = c["seqs"] * new
        read = sum(lengths) + sum(prefixes[p] for p in set(of) if p >= 0)
        return {"bytes": 2.0 * c["kv"] * c["dim"] * read + 2.0 * rows * c["heads"] * c["dim"] * wide
                + 4.0 * rows * c["heads"], "flops": 4.0 * pairs * c["heads"] * c["dim"]}
    wide = 2 if c["dt"] == "bf16" else 4
    if c["op"] == "norm":
        size = c["rows"] * c["dim"]
        p = 2 if c["pdt"] == "bf16" else 4
        params = ((c["dim"] if c["post"] else 0) + c["dim"] + (c["gates"] * c["dim"] if c["gate"] != "none" else 0)) * p
        moved, flops = 4.0 * size * wide + params, 10.0 * size
        if c["train"]:      # h_out, y and the two gradients in, two out; parameters in, their gradients out
            moved += 6.0 * size * wide + 2 * params
            flops += 30.0 * size
        return {"bytes": moved, "flops": flops}
    if c["op"] == "rope":
        size = c["rows"] * c["heads"] * c["dim"]
        passes = 2 if c["train"] else 1
        return {"bytes": passes * (2.0 * size * wide + 4.0 * c["axes"] * c["rows"]), "flops": passes * 3.0 * size}
    pairs = c["tokens"] * c["top_k"]
    row = c["hidden"] * wide
    kept = pairs * (1 - c["dropped"])
    moved = 4.0 * pairs * 5 + 4.0 * c["experts"]                # ids, weights; places, tokens, experts
    moved += (c["tokens"] + pairs) * row                        # dispatch
    moved += (kept + c["tokens"] * (2 if c["residual"] else 1)) * row
    flops = 2.0 * kept * c["hidden"]
    if c["train"]:
        moved += (kept + c["tokens"]) * row + (kept + pairs + c["tokens"]) * row + 4.0 * pairs
        flops *= 3.5
    return {"bytes": moved, "flops": flops}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case, **_PREPARE[case["op"]](case, g)}
    if own:
        import group_wise_affine_quantize_amd as nq
        s["nq"] = nq
        c = case
        if c["op"] == "rope":
            s["rope"] = nq.Rope(c["rotary"], freq=s["freq"], axis=s["axis"].tolist(), layout=c["layout"],
                                scale=c["scale"])
        elif c["op"] == "shared":
            s["cache"] = nq.KVCache.wrap(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], c["fmt"])
            rows = c["seqs"] * c["new"]
            s["seqs"] = nq.KVSequences(s["row_start"], s["lengths"], s["table"], rows)
            s["prefix"] = nq.KVSequences(s["prefix_start"], s["prefix_lengths"], s["prefix_table"], rows)
    return s


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _prepare_norm(c, g):
    dt, pdt = DTYPES[c["dt"]], DTYPES[c["pdt"]]
    rows, dim = c["rows"], c["dim"]
    # a residual stream that has grown over the layers, rows of unlike sizes
    s = {"h": (_normal(g, rows, dim) * (1 + 3 * torch.rand((rows, 1), generator=g, device="cuda"))).to(dt),
         "y": (_normal(g, rows, dim) * 0.7).to(dt), "post": None, "gate": None}
    near = lambda *shape: (1 - c["offset"] + 0.2 * _normal(g, *shape)).to(pdt)
    s["pre"] = near(dim)
    if c["post"]:
        s["post"] = near(dim)
    if c["gate"] != "none":
        s["gate"] = (0.5 * _normal(g, c["gates"], dim)).to(pdt)
    if c["train"]:
        s["dh_out"] = (_normal(g, rows, dim) * 0.1).to(dt)
        s["dz"] = (_normal(g, rows, dim) * 0.1).to(dt)
        s["stored"] = _plain_norm({"case": {**c, "train": False}, **s})["h_out"]
    return s


def _prepare_rope(c, g):
    rows, pairs = c["rows"], c["rotary"] // 2
    fused = _normal(g, rows, c["heads"] + c["behind"], c["dim"]).to(DTYPES[c["dt"]])
    s = {"x": fused[:, : c["heads"]], "fused": fused}
    # the axes take pairs by turns; each has frequencies from 1 down to 1 / 10000
    i = torch.arange(pairs, device="cuda", dtype=torch.float64)
    s["axis"] = torch.arange(pairs, device="cuda") % c["axes"]
    s["freq"] = 10000.0 ** (-i / pairs)
    # the first axis counts up from anywhere, the others walk over a picture
    first = torch.randint(0, c["far"], (1,), generator=g, device="cuda")
    at = torch.arange(rows, device="cuda") + first
    s["positions"] = torch.stack([at] + [at % (37 + 24 * a) for a in range(1, c["axes"])]).to(torch.int32)
    if c["train"]:
        s["dout"] = _normal(g, rows, c["heads"], c["dim"]).to(DTYPES[c["dt"]])
    return s


def _prepare_moe(c, g):
    dt = DTYPES[c["dt"]]
    tokens, k, e, hidden = c["tokens"], c["top_k"], c["experts"], c["hidden"]
    # distinct experts of a token, some experts more popular than others
    popular = _normal(g, e)
    ids = torch.topk(_normal(g, tokens, e) + popular, k, dim=-1).indices.to(torch.int32)
    if c["dropped"]:
        gone = torch.rand((tokens, k), generator=g, device="cuda") < c["dropped"]
        ids = torch.where(gone, ids + e, ids).to(torch.int32)
    s = {"ids": ids, "x": _normal(g, tokens, hidden).to(dt), "residual": None}
    w = torch.rand((tokens, k), generator=g, device="cuda") + 0.05
    s["weights"] = w / w.sum(-1, keepdim=True)
    s["ys"] = _normal(g, tokens * k, hidden).to(dt)
    if c["residual"]:
        s["residual"] = _normal(g, tokens, hidden).to(dt)
    if c["train"]:
        s["dy"] = _normal(g, tokens, hidden).to(dt)
        s["dxs"] = _normal(g, tokens * k, hidden).to(dt)
    return s


def _prepare_shared(c, g):
    lengths, prefixes, of = _layout(c)
    block, new = c["block"], c["new"]
    need = [-(-n // block) for n in lengths + prefixes]
    blocks = sum(need) + 3
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(need), max(need)), dtype=torch.int32, device="cuda")
    for b, at in enumerate(_starts(need)[:-1]):
        table[b, : need[b]] = order[at: at + need[b]]
    rows = c["seqs"] * new
    per = [new * sum(1 for o in of if o == p) for p in range(c["prefixes"])]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
    s = {"own_host": lengths, "prefix_host": prefixes, "of": of,
         "table": table[: c["seqs"], : max(need[: c["seqs"]])].contiguous(),
         "prefix_table": table[c["seqs"]:].contiguous(), "row_start": i32([new * i for i in range(c["seqs"] + 1)]),
         "lengths": i32(lengths), "prefix_lengths": i32(prefixes), "prefix_start": i32(_starts(per))}
    for part, shape in (("k", (blocks, c["kv"], block, c["dim"])), ("v", (blocks, c["kv"], c["dim"], block))):
        x = _normal(g, *shape) * (QMAX[c["fmt"]] / 4)
        if c["fmt"] == "int8":
            s[part + "_codes"] = (x.round().clamp(-127, 127) + 128).to(torch.uint8)
        else:
            s[part + "_codes"] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        jitter = torch.rand((blocks, c["kv"]), generator=g, device="cuda") * 0.5 + 0.75
        s[part + "_scales"] = (4 / QMAX[c["fmt"]]) * jitter
    fused = (_normal(g, rows, c["heads"] + 2 * c["kv"], c["dim"]) * 1.5).to(DTYPES[c["dt"]])
    s["fused"] = fused
    s["q"] = fused[:, : c["heads"]]
    s["lse"] = torch.empty((rows, c["heads"]), dtype=torch.float32, device="cuda")
    return s


_PREPARE = {"norm": _prepare_norm, "rope": _prepare_rope, "moe": _prepare_moe, "shared": _prepare_shared}


# ---------------------------------------------------------------- a pass
def run(s):
    op = s["case"]["op"]
    return (_OWN if own else _PLAIN)[op](s)


def _own_norm(s):
    c, nq = s["case"], s["nq"]
    options = {"post": s["post"], "gate": s["gate"], "pre": s["pre"], "scale": c["scale"], "offset": c["offset"],
               "eps": EPS}
    h_out, z = nq.nq_block_norm(s["h"], s["y"], **options)
    out = {"h_out": h_out, "z": z}
    if c["train"]:
        dh, dy, dpost, dgate, dpre = nq.nq_block_norm_grad(s["stored"], s["y"], s["dh_out"], s["dz"], **options)
        out.update(dh=dh, dy=dy, dpre=dpre)
        if s["post"] is not None:
            out["dpost"] = dpost
        if s["gate"] is not None:
            out["dgate"] = dgate
    return out


def _own_rope(s):
    nq = s["nq"]
    out = {"out": nq.nq_rope(s["rope"], s["x"], s["positions"])}
    if s["case"]["train"]:
        out["dx"] = nq.nq_rope_grad(s["rope"], s["dout"], s["positions"])
    return out


def _own_moe(s):
    c, nq = s["case"], s["nq"]
    order = nq.nq_moe_sort(s["ids"], c["experts"])
    out = {"starts": order.starts, "place": order.place, "row_token": order.row_token, "row_expert": order.row_expert,
           "xs": nq.nq_moe_dispatch(order, s["x"]),
           "y": nq.nq_moe_combine(order, s["ys"], s["weights"], residual=s["residual"])}
    if c["train"]:
        out["dx"] = nq.nq_moe_dispatch_grad(order, s["dxs"])
        out["dys"], out["dweights"] = nq.nq_moe_combine_grad(order, s["dy"], s["ys"], s["weights"])
    return out


def _own_shared(s):
    out = s["nq"].nq_kv_attention_shared(s["cache"], s["prefix"], s["seqs"], s["q"], lse=s["lse"])
    return {"out": out, "lse": s["lse"]}


_OWN = {"norm": _own_norm, "rope": _own_rope, "moe": _own_moe, "shared": _own_shared}


# ---------------------------------------------------------------- the plain form
def _spread(c, gate):
    """The gate of each row, float32 (1 where there is none)."""
    if gate is None:
        return 1.0
    return gate.float().repeat_interleave(c["rows"] // c["gates"], 0) if c["gates"] > 1 else gate.float()


def _plain_norm(s):
    c = s["case"]
    dt, o = s["h"].dtype, c["offset"]
    y = s["y"].float()
    ry = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS)
    u = y * ry * (s["post"].float() + o) if c["post"] else y
    gate = _spread(c, s["gate"])
    h = s["h"].float() + c["scale"] * gate * u
    rh = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    z = h * rh * (s["pre"].float() + o)
    out = {"h_out": h.to(dt), "z": z.to(dt)}
    if c["train"]:
        x = s["stored"].float()
        r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        x = x * r
        dz = s["dz"].float()
        v = dz * (s["pre"].float() + o)
        d = s["dh_out"].float() + r * (v - x * (v * x).mean(-1, keepdim=True))
        out["dh"] = d.to(dt)
        du = c["scale"] * gate * d
        if c["post"]:
            yh = y * ry
            v = du * (s["post"].float() + o)
            out["dy"] = (ry * (v - yh * (v * yh).mean(-1, keepdim=True))).to(dt)
        else:
            out["dy"] = du.to(dt)
        out["dpre"] = (dz * x).sum(0).to(s["pre"].dtype)
        if c["post"]:
            out["dpost"] = (du * yh).sum(0).to(s["post"].dtype)
        if s["gate"] is not None:
            t = c["scale"] * (d * u)
            if c["gates"] < c["rows"]:
                t = t.view(c["gates"], -1, c["dim"]).sum(1)
            out["dgate"] = t.to(s["gate"].dtype)
    return out


def _plain_turn(s, x, sign):
    c = s["case"]
    angle = s["positions"].double()[s["axis"]].t() * s["freq"]      # [rows, pairs]
    cos = (torch.cos(angle).float() * c["scale"])[:, None]
    sin = (torch.sin(angle).float() * (sign * c["scale"]))[:, None]
    f = x[..., : c["rotary"]].float()
    if c["layout"] == "halves":
        a, b = f[..., : c["rotary"] // 2], f[..., c["rotary"] // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = f[..., 0::2], f[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned.to(x.dtype), x[..., c["rotary"]:]], -1)


def _plain_rope(s):
    out = {"out": _plain_turn(s, s["x"], 1.0)}
    if s["case"]["train"]:
        out["dx"] = _plain_turn(s, s["dout"], -1.0)
    return out


def _plain_moe(s):
    c = s["case"]
    tokens, k, e, hidden = c["tokens"], c["top_k"], c["experts"], c["hidden"]
    dt = s["x"].dtype
    flat = s["ids"].reshape(-1)
    gone = (flat < 0) | (flat >= e)
    key = torch.where(gone, e, flat.long())
    pair = torch.sort(key, stable=True).indices
    place = torch.empty_like(pair)
    place[pair] = torch.arange(tokens * k, device="cuda")
    counts = torch.zeros(e + 1, dtype=torch.int64, device="cuda").scatter_add_(0, key, torch.ones_like(key))
    starts = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    starts[1:] = counts[:e].cumsum(0)
    kept = ~gone[pair]
    out = {"starts": starts.to(torch.int32), "place": place.view(tokens, k).to(torch.int32),
           "row_token": (pair // k).to(torch.int32), "row_expert": flat[pair]}
    xs = s["x"][pair // k]
    if c["dropped"]:
        xs = torch.where(kept[:, None], xs, torch.zeros((), dtype=dt, device="cuda"))
    out["xs"] = xs
    here = ~gone.view(tokens, k)
    w = torch.where(here, s["weights"], 0.0)

    def back(rows, weights):
        total = torch.zeros((tokens, hidden), device="cuda")
        for j in range(k):
            total += rows[place[j::k]].float() * weights[:, j, None]
        return total

    y = back(s["ys"], w)
    if c["residual"]:
        y = y + s["residual"].float()
    out["y"] = y.to(dt)
    if c["train"]:
        out["dx"] = back(s["dxs"], here.float()).to(dt)
        dy = s["dy"].float()
        dys, dw = torch.empty_like(s["ys"]), torch.empty((tokens, k), device="cuda")
        for j in range(k):
            at = place[j::k]
            dys[at] = (dy * w[:, j, None]).to(dt)
            dw[:, j] = torch.where(here[:, j], (dy * s["ys"][at].float()).sum(-1), 0.0)
        out["dys"], out["dweights"] = dys, dw
    return out


def _tokens(s, table, length):
    """Keys and values of the first `length` tokens, [kv_heads, length, head_dim] float32."""
    c = s["case"]
    ids = table[: -(-length // c["block"])].long()

    def values(codes):
        return codes.float() - 128 if c["fmt"] == "int8" else codes.view(torch.float8_e4m3fn).float()

    k = values(s["k_codes"][ids]) * s["k_scales"][ids][:, :, None, None]
    v = values(s["v_codes"][ids]) * s["v_scales"][ids][:, :, None, None]
    k = k.transpose(0, 1).reshape(c["kv"], -1, c["dim"])
    v = v.permute(1, 0, 3, 2).reshape(c["kv"], -1, c["dim"])
    return k[:, :length], v[:, :length]


def _plain_shared(s):
    c = s["case"]
    n, kv, group, dim = c["new"], c["kv"], c["heads"] // c["kv"], c["dim"]
    before = [_tokens(s, s["prefix_table"][p], length) for p, length in enumerate(s["prefix_host"])]
    out, lse = [], []
    for b, (length, p) in enumerate(zip(s["own_host"], s["of"])):
        k, v = _tokens(s, s["table"][b], length)
        first = 0
        if p >= 0:
            first = s["prefix_host"][p]
            k, v = torch.cat([before[p][0], k], 1), torch.cat([before[p][1], v], 1)
        q = s["q"][b * n: (b + 1) * n].float().view(n, kv, group, dim).permute(1, 0, 2, 3).reshape(kv, n * group, dim)
        x = torch.matmul(q, k.transpose(1, 2).contiguous()) * dim ** -0.5
        last = first + length - n + torch.arange(n, device="cuda").repeat_interleave(group)[:, None]
        x.masked_fill_(torch.arange(first + length, device="cuda")[None] > last, float("-inf"))
        top = x.amax(-1, keepdim=True)
        x = (x - top).exp_()
        total = x.sum(-1, keepdim=True)
        y = torch.matmul(x, v.contiguous()) / total
        out.append(y.view(kv, n, group, dim).permute(1, 0, 2, 3).reshape(n, c["heads"], dim).to(s["q"].dtype))
        lse.append((top + torch.log(total)).view(kv, n, group).permute(1, 0, 2).reshape(n, c["heads"]))
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


_PLAIN = {"norm": _plain_norm, "rope": _plain_rope, "moe": _plain_moe, "shared": _plain_shared}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return _EXACT[case["op"]](s)


def _exact_norm(s):
    """Forward by the definition, gradients by differentiating it."""
    c = s["case"]
    wide = lambda t: None if t is None else t.double()

    def normed(t, weight):
        return t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * (weight + c["offset"])

    def added(y, post, gate):
        u = y if post is None else normed(y, post)
        if gate is not None:
            rows = torch.arange(c["rows"], device="cuda") // (c["rows"] // c["gates"])
            u = u * gate[rows]
        return c["scale"] * u

    h, y, post, gate, pre = (wide(s[n]) for n in ("h", "y", "post", "gate", "pre"))
    h_out = h + added(y, post, gate)
    out = {"h_out": h_out, "z": normed(h_out, pre)}
    if c["train"]:
        leaves = {"y": y, "pre": pre, "post": post, "gate": gate}
        for t in leaves.values():
            if t is not None:
                t.requires_grad_()
        at = s["stored"].double().requires_grad_()
        dh, out["dpre"] = torch.autograd.grad(normed(at, pre), [at, pre], s["dz"].double())
        out["dh"] = dh + s["dh_out"].double()
        names = [n for n in ("y", "post", "gate") if leaves[n] is not None]
        grads = torch.autograd.grad(added(y, post, gate), [leaves[n] for n in names], out["dh"])
        out.update({"d" + n: t for n, t in zip(names, grads)})
    return {n: t.detach() for n, t in out.items()}


def _exact_rope(s):
    c = s["case"]
    half = c["rotary"] // 2

    def turned(x, direction):
        out = x.double().clone()
        for i in range(half):
            a, b = (i, i + half) if c["layout"] == "halves" else (2 * i, 2 * i + 1)
            angle = s["positions"][int(s["axis"][i])].double() * s["freq"][i]
            z = torch.polar(torch.full_like(angle, c["scale"]), direction * angle)[:, None]
            w = torch.complex(x[..., a].double(), x[..., b].double()) * z
            out[..., a], out[..., b] = w.real, w.imag
        return out

    out = {"out": turned(s["x"], 1)}
    if c["train"]:
        out["dx"] = turned(s["dout"], -1)
    return out


def _exact_moe(s):
    c = s["case"]
    tokens, k, e, hidden = c["tokens"], c["top_k"], c["experts"], c["hidden"]
    ids = s["ids"].reshape(-1).cpu().tolist()
    order = sorted(range(len(ids)), key=lambda p: ids[p] if 0 <= ids[p] < e else e)     # sorted() is stable
    place = [0] * len(ids)
    starts = [0] * (e + 1)
    for i, p in enumerate(order):
        place[p] = i
        if 0 <= ids[p] < e:
            starts[ids[p] + 1] += 1
    for i in range(e):
        starts[i + 1] += starts[i]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    out = {"starts": i32(starts), "place": i32(place).view(tokens, k), "row_token": i32([p // k for p in order]),
           "row_expert": i32([ids[p] for p in order])}
    at = torch.tensor(place, device="cuda").view(tokens, k)
    keep = (at < starts[e]).double()
    source = torch.tensor([p // k for p in order], device="cuda")
    out["xs"] = s["x"].double()[source]
    out["xs"][starts[e]:] = 0
    y = torch.zeros((tokens, hidden), dtype=torch.float64, device="cuda")
    for j in range(k):
        y.addcmul_((s["weights"][:, j].double() * keep[:, j])[:, None], s["ys"][at[:, j]].double())
    out["y"] = y if s["residual"] is None else y + s["residual"].double()
    if c["train"]:
        dx, dy = torch.zeros_like(y), s["dy"].double()
        dys = torch.zeros((tokens * k, hidden), dtype=torch.float64, device="cuda")
        dw = torch.zeros((tokens, k), dtype=torch.float64, device="cuda")
        for j in range(k):
            dx.addcmul_(keep[:, j, None], s["dxs"][at[:, j]].double())
            dys[at[:, j]] = (s["weights"][:, j].double() * keep[:, j])[:, None] * dy
            dw[:, j] = keep[:, j] * (dy * s["ys"][at[:, j]].double()).sum(-1)
        out.update(dx=dx, dys=dys, dweights=dw)
    return out


def _e4m3_values():
    """The value of each E4M3 byte, from the format: sign, 4 bits of exponent (bias 7), 3 of fraction."""
    v = []
    for byte in range(256):
        sign, e, m = byte >> 7, byte >> 3 & 15, byte & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(math.nan if e == 15 and m == 7 else -x if sign else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _exact_shared(s):
    c = s["case"]
    if c["fmt"] == "int8":
        byte = torch.arange(256, dtype=torch.float64, device="cuda") - 128
    else:
        byte = _e4m3_values()
    n, group = c["new"], c["heads"] // c["kv"]
    rows = c["seqs"] * n
    out = torch.zeros((rows, c["heads"], c["dim"]), dtype=torch.float64, device="cuda")
    lse = torch.zeros((rows, c["heads"]), dtype=torch.float64, device="cuda")

    def head(part, h, table, length):
        ids = table[: -(-length // c["block"])].long()
        x = byte[s[part + "_codes"][ids, h].long()] * s[part + "_scales"][ids, h].double()[:, None, None]
        return (x if part == "k" else x.transpose(1, 2)).reshape(-1, c["dim"])[:length]

    for h in range(c["kv"]):
        for p in range(-1, c["prefixes"]):
            members = [b for b in range(c["seqs"]) if s["of"][b] == p]
            if not members:
                continue
            kp, vp = (head(part, h, s["prefix_table"][p], s["prefix_host"][p]) if p >= 0 else
                      torch.zeros((0, c["dim"]), dtype=torch.float64, device="cuda") for part in ("k", "v"))
            for b in members:
                k = torch.cat([kp, head("k", h, s["table"][b], s["own_host"][b])])
                v = torch.cat([vp, head("v", h, s["table"][b], s["own_host"][b])])
                q = s["q"][b * n: (b + 1) * n, h * group: (h + 1) * group].double().reshape(n * group, -1)
                z = q @ k.t() / math.sqrt(c["dim"])
                for i in range(n - 1):      # drafts do not see those behind them
                    z[i * group: (i + 1) * group, len(k) - n + i + 1:] = -math.inf
                l = torch.logsumexp(z, -1)
                y = torch.exp(z - l[:, None]) @ v
                out[b * n: (b + 1) * n, h * group: (h + 1) * group] = y.view(n, group, -1)
                lse[b * n: (b + 1) * n, h * group: (h + 1) * group] = l.view(n, group)
    return {"out": out, "lse": lse}


_EXACT = {"norm": _exact_norm, "rope": _exact_rope, "moe": _exact_moe, "shared": _exact_shared}
