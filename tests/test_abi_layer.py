"""Host-side checks of the entry points for norms, rotary positions and tokens
sorted by expert that need no GPU: every argument error is reported before
anything is enqueued (the pointers are made up and never dereferenced)."""
import ctypes

import pytest

from group_wise_affine_quantize_amd import _binding as B

OK, NULL, DTYPE, SHAPE, ALIGN, ALIAS, WORKSPACE = 0, 1, 2, 4, 5, 6, 7
P = 1 << 40         # made-up addresses, 2^32 apart
NAMES = ["h", "y", "post", "gate", "pre", "h_out", "z", "dh_out", "dz", "dh", "dy", "dpost", "dgate", "dpre", "ws", "x",
         "out", "positions", "freq", "axis", "ids", "starts", "place", "row_token", "row_expert", "xs", "weights",
         "residual", "dweights"]
AT = {n: P + (i << 32) for i, n in enumerate(NAMES)}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return B.load_library()


def norm_args(grad, **c):
    a = dict(rows=8, dim=64, gates=4, eps=1e-6, offset=0.0, scale=1.0, h=AT["h"], ldh=64, y=AT["y"], ldy=64, x_dt=1,
             post=AT["post"], gate=AT["gate"], ldg=64, pre=AT["pre"], p_dt=1)
    if grad:
        a.update(dh_out=AT["dh_out"], ldd=64, dz=AT["dz"], ldz=64, dh=AT["dh"], dy=AT["dy"], dpost=AT["dpost"],
                 dgate=AT["dgate"], dpre=AT["dpre"], ws=AT["ws"], ws_bytes=1 << 31)
    else:
        a.update(h_out=AT["h_out"], z=AT["z"])
    assert set(c) <= set(a), set(c) - set(a)
    a.update(c)
    shape = B._BlockNormStruct(*(a[f] for f, _ in B._BlockNormStruct._fields_))
    return a, shape


def norm(lib, shape=True, **c):
    a, s = norm_args(False, **c)
    return lib.nq_block_norm(shape and ctypes.byref(s) or None, a["h"], a["ldh"], a["y"], a["ldy"], a["x_dt"], a["post"], a["gate"],
                             a["ldg"], a["pre"], a["p_dt"], a["h_out"], a["z"], None)


def norm_grad(lib, shape=True, **c):
    a, s = norm_args(True, **c)
    return lib.nq_block_norm_grad(shape and ctypes.byref(s) or None, a["h"], a["ldh"], a["y"], a["ldy"], a["dh_out"], a["ldd"],
                                  a["dz"], a["ldz"], a["x_dt"], a["post"], a["gate"], a["ldg"], a["pre"], a["p_dt"],
                                  a["dh"], a["dy"], a["dpost"], a["dgate"], a["dpre"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("call", [norm, norm_grad])
def test_norm_shapes_and_inputs(lib, call):
    assert call(lib, shape=False) == NULL
    for bad in (dict(dim=0), dict(dim=16385), dict(rows=-1), dict(rows=1 << 31), dict(gates=0), dict(gates=3), dict(gates=-1),
                dict(gates=1 << 31, rows=0), dict(eps=1e-38),
                dict(eps=0.0), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(offset=INF), dict(scale=NAN),
                dict(ldh=63), dict(ldy=10), dict(ldg=63), dict(ldh=1 << 31)):
        assert call(lib, **bad) == SHAPE, bad
        assert b"nq_block_norm" in lib.nq_last_error()
    assert call(lib, x_dt=2) == DTYPE and call(lib, p_dt=-1) == DTYPE
    for bad in (dict(h=0), dict(y=0), dict(y=0, post=0)):
        assert call(lib, **bad) == NULL, bad
    for name, by in (("h", 1), ("y", 1), ("post", 1), ("gate", 1), ("pre", 1)):
        assert call(lib, **{name: AT[name] + by}) == ALIGN, name
    assert call(lib, p_dt=0, pre=AT["pre"] + 2) == ALIGN and call(lib, x_dt=0, h=AT["h"] + 2) == ALIGN


def test_norm_outputs(lib):
    for bad in (dict(z=0), dict(pre=0), dict(h_out=0), dict(y=0, post=0, gate=0), dict(y=0, post=0, gate=0, h_out=0, pre=0, z=0)):
        assert norm(lib, **bad) == NULL, bad
    for bad in (dict(h_out=AT["h"]), dict(z=AT["h"] + 2), dict(z=AT["h_out"]), dict(z=AT["y"]), dict(h_out=AT["gate"] + 16),
                dict(z=AT["pre"]), dict(h_out=AT["post"])):
        assert norm(lib, **bad) == ALIAS, bad
    assert norm(lib, z=AT["z"] + 1) == ALIGN
    # nothing to do: no pointer is needed
    assert norm(lib, rows=0, h=0, y=0, post=0, gate=0, pre=0, h_out=0, z=0) == OK


def test_norm_grad_outputs(lib):
    for bad in (dict(dh_out=0, dz=0), dict(pre=0), dict(dh=0), dict(dy=0), dict(y=0, post=0, gate=0),
                dict(post=0), dict(gate=0), dict(dz=0)):
        assert norm_grad(lib, **bad) == NULL, bad
    for bad in (dict(ldd=63), dict(ldz=63)):
        assert norm_grad(lib, **bad) == SHAPE, bad
    for bad in (dict(dh=AT["h"]), dict(dh=AT["dh_out"]), dict(dy=AT["y"]), dict(dy=AT["dz"]), dict(dh=AT["dy"]),
                dict(dpost=AT["post"]), dict(dgate=AT["dpre"]), dict(dpre=AT["pre"]), dict(rows=80, ws=AT["h"]), dict(rows=80, ws=AT["dh"])):
        assert norm_grad(lib, **bad) == ALIAS, bad
    for name in ("dh", "dy", "dpost", "dgate", "dpre"):
        assert norm_grad(lib, **{name: AT[name] + 1}) == ALIGN, name
    need = B.nq_block_norm_grad_workspace_bytes(80, 64, 4)
    assert need > 0
    assert norm_grad(lib, rows=80, ws=0) == WORKSPACE and norm_grad(lib, rows=80, ws_bytes=need - 1) == WORKSPACE
    assert norm_grad(lib, rows=80, ws=AT["ws"] + 8) == ALIGN
    assert B.nq_block_norm_grad_workspace_bytes(0, 64) == 0 and B.nq_block_norm_grad_workspace_bytes(8, 0) == 0


def rope(lib, plan=True, grad=False, **c):
    a = dict(freq=AT["freq"], axis=AT["axis"], rotary_dim=64, axes=3, layout=1, scale=1.0, x=AT["x"], x_dt=1, rows=8, ldx=640,
             heads=5, head_dim=128, positions=AT["positions"], ldp=8, out=AT["out"], ldo=640)
    assert set(c) <= set(a)
    a.update(c)
    s = B._RopeStruct(*(a[f] for f, _ in B._RopeStruct._fields_))
    return (lib.nq_rope_grad if grad else lib.nq_rope)(plan and ctypes.byref(s) or None, a["x"], a["x_dt"], a["rows"], a["ldx"],
                                                       a["heads"], a["head_dim"], a["positions"], a["ldp"], a["out"], a["ldo"], None)


@pytest.mark.parametrize("grad", [False, True])
def test_rope_arguments(lib, grad):
    assert rope(lib, plan=False, grad=grad) == NULL
    for bad in (dict(layout=0), dict(layout=3), dict(rotary_dim=0), dict(rotary_dim=63), dict(rotary_dim=130), dict(rotary_dim=-2),
                dict(head_dim=1025, ldx=1 << 20, ldo=1 << 20), dict(axes=0), dict(axes=17), dict(scale=0.0), dict(scale=NAN),
                dict(heads=0), dict(heads=65536), dict(rows=-1), dict(rows=1 << 31), dict(ldp=7), dict(ldp=-1), dict(ldx=639), dict(ldo=639),
                dict(ldp=1 << 62)):
        assert rope(lib, grad=grad, **bad) == SHAPE, bad
        assert (b"nq_rope_grad" if grad else b"nq_rope:") in lib.nq_last_error()
    assert rope(lib, grad=grad, x_dt=3) == DTYPE
    for name in ("freq", "positions", "x", "out"):
        assert rope(lib, grad=grad, **{name: 0}) == NULL, name
    for bad in (dict(freq=AT["freq"] + 4), dict(axis=AT["axis"] + 2), dict(positions=AT["positions"] + 1), dict(x=AT["x"] + 1),
                dict(out=AT["out"] + 1)):
        assert rope(lib, grad=grad, **bad) == ALIGN, bad
    # in place is the very same rows, or nothing
    for bad in (dict(out=AT["x"] + 2), dict(out=AT["x"], ldo=1280), dict(out=AT["positions"]), dict(out=AT["freq"]),
                dict(out=AT["axis"])):
        assert rope(lib, grad=grad, **bad) == ALIAS, bad
    assert rope(lib, grad=grad, rows=0, freq=0, axis=0, x=0, positions=0, out=0) == OK


def sort(lib, **c):
    a = dict(ids=AT["ids"], tokens=9000, top_k=4, experts=64, starts=AT["starts"], place=AT["place"], row_token=AT["row_token"],
             row_expert=AT["row_expert"], ws=AT["ws"], ws_bytes=1 << 31)
    assert set(c) <= set(a)
    a.update(c)
    return lib.nq_moe_sort(*a.values(), None)


def test_sort_arguments(lib):
    for bad in (dict(tokens=-1), dict(tokens=1 << 29), dict(tokens=1 << 62), dict(top_k=0), dict(top_k=33), dict(experts=0),
                dict(experts=1025)):
        assert sort(lib, **bad) == SHAPE, bad
    for name in ("ids", "starts", "place", "row_token", "row_expert"):
        assert sort(lib, **{name: 0}) == NULL, name
        assert sort(lib, **{name: AT[name] + 2}) == ALIGN, name
    for bad in (dict(place=AT["ids"]), dict(starts=AT["place"] + 4), dict(row_token=AT["row_expert"]), dict(ws=AT["ids"]),
                dict(ws=AT["starts"])):
        assert sort(lib, **bad) == ALIAS, bad
    need = B.nq_moe_sort_workspace_bytes(9000, 4, 64)
    assert need > 0 and B.nq_moe_sort_workspace_bytes(16, 4, 64) == 0
    assert sort(lib, ws=0) == WORKSPACE and sort(lib, ws_bytes=need - 1) == WORKSPACE and sort(lib, ws=AT["ws"] + 4) == ALIGN
    assert B.nq_moe_sort_workspace_bytes(-1, 4, 64) == 0 and B.nq_moe_sort_workspace_bytes(9000, 0, 64) == 0


def order(**c):
    a = dict(starts=AT["starts"], place=AT["place"], tokens=8, top_k=4, experts=64)
    a.update(c)
    return B._MoEOrderStruct(*(a[f] for f, _ in B._MoEOrderStruct._fields_))


def dispatch(lib, o, x=AT["x"], dt=1, ld=64, hidden=64, out=AT["xs"]):
    return lib.nq_moe_dispatch(o and ctypes.byref(o), x, dt, ld, hidden, out, None)


def dispatch_grad(lib, o, x=AT["x"], dt=1, hidden=64, out=AT["xs"]):
    return lib.nq_moe_dispatch_grad(o and ctypes.byref(o), x, dt, hidden, out, None)


def combine(lib, o, x=AT["x"], dt=1, hidden=64, weights=AT["weights"], residual=AT["residual"], ld=64, out=AT["xs"]):
    return lib.nq_moe_combine(o and ctypes.byref(o), x, dt, hidden, weights, residual, ld, out, None)


def combine_grad(lib, o, x=AT["x"], dt=1, ld=64, hidden=64, ys=AT["y"], weights=AT["weights"], out=AT["xs"], dw=AT["dweights"]):
    return lib.nq_moe_combine_grad(o and ctypes.byref(o), x, dt, ld, hidden, ys, weights, out, dw, None)


@pytest.mark.parametrize("call", [dispatch, dispatch_grad, combine, combine_grad])
def test_moving_arguments(lib, call):
    assert call(lib, None) == NULL
    for bad in (dict(tokens=-1), dict(tokens=1 << 31), dict(top_k=0), dict(experts=0)):
        assert call(lib, order(**bad)) == SHAPE, bad
        assert call.__name__.encode() in lib.nq_last_error()
    assert call(lib, order(starts=0)) == NULL and call(lib, order(place=0)) == NULL and call(lib, order(place=AT["place"] + 2)) == ALIGN
    for hidden in (0, -1, 1 << 31):
        assert call(lib, order(), hidden=hidden) == SHAPE
    assert call(lib, order(tokens=1 << 24), hidden=1 << 20) == SHAPE
    assert call(lib, order(), dt=5) == DTYPE
    assert call(lib, order(), x=0) == NULL and call(lib, order(), out=0) == NULL
    assert call(lib, order(), x=AT["x"] + 1) == ALIGN and call(lib, order(), out=AT["xs"] + 1) == ALIGN
    for out in (AT["x"], AT["starts"], AT["place"] + 4):
        assert call(lib, order(), out=out) == ALIAS
    assert call(lib, order(tokens=0, starts=0, place=0), x=0, out=0) == OK


def test_combine_arguments(lib):
    o = order()
    assert dispatch(lib, o, ld=63) == SHAPE and combine(lib, o, ld=63) == SHAPE and combine_grad(lib, o, ld=63) == SHAPE
    assert combine(lib, o, weights=AT["weights"] + 2) == ALIGN and combine(lib, o, residual=AT["residual"] + 1) == ALIGN
    assert combine(lib, o, weights=AT["xs"]) == ALIAS and combine(lib, o, residual=AT["xs"]) == ALIAS
    assert combine_grad(lib, o, ys=0) == NULL and combine_grad(lib, o, dw=AT["dweights"] + 2) == ALIGN
    for bad in (dict(ys=AT["xs"]), dict(weights=AT["xs"]), dict(dw=AT["xs"]), dict(dw=AT["x"]), dict(dw=AT["y"]),
                dict(dw=AT["weights"]), dict(dw=AT["place"])):
        assert combine_grad(lib, o, **bad) == ALIAS, bad


def test_shared_attention_arguments(lib):
    from test_abi_kv import AT as KV
    from test_abi_kv import BAD_CACHES, BAD_SEQS, QUANT, cache, seqs  # noqa: F401
    far = {n: a + (1 << 50) for n, a in KV.items()}

    def prefix(**s):
        return seqs(**{**dict(row_start=far["row_start"], lengths=far["lengths"], block_table=far["table"], batch=2), **s})

    def attend(c=cache(), p=prefix(), s=seqs(), q=KV["q"], dt=1, ldq=1024, heads=8, scale=0.1, causal=1, out=KV["out"], lse=None,
               ws=KV["ws"], ws_bytes=1 << 31):
        r = lambda x: x and ctypes.byref(x)
        return lib.nq_kv_attention_shared(r(c), r(p), r(s), q, dt, ldq, heads, scale, causal, out, lse, ws, ws_bytes, None)

    assert attend(c=None) == NULL and attend(p=None) == NULL and attend(s=None) == NULL
    for bad, status in BAD_CACHES:
        assert attend(c=cache(**bad)) == status, bad
        assert b"nq_kv_attention_shared" in lib.nq_last_error()
    for bad, status in BAD_SEQS:
        assert attend(s=seqs(**bad)) == status, bad
        assert attend(p=prefix(**bad)) == status, bad
    assert attend(p=prefix(rows=8)) == SHAPE and attend(s=seqs(rows=6)) == SHAPE
    assert attend(dt=9) == DTYPE and attend(heads=7) == SHAPE and attend(scale=0.0) == SHAPE and attend(ldq=1025) == ALIGN
    assert attend(q=None) == NULL and attend(out=0) == NULL and attend(lse=KV["lse"] + 2) == ALIGN
    for bad in (dict(out=KV["q"]), dict(out=far["table"]), dict(lse=far["lengths"]), dict(lse=KV["out"]), dict(out=KV["k_codes"]),
                dict(ws=far["row_start"]), dict(ws=KV["out"])):
        assert attend(**bad) == ALIAS, bad
    need = lib.nq_kv_attention_shared_workspace_bytes(ctypes.byref(cache()), ctypes.byref(prefix()), ctypes.byref(seqs()), 8, 1)
    # the prefix's states: O and three sums for every row and head
    assert need >= 7 * 8 * (128 + 4) * 4
    assert attend(ws=None) == WORKSPACE and attend(ws_bytes=need - 1) == WORKSPACE and attend(ws=KV["ws"] + 8) == ALIGN
    assert lib.nq_kv_attention_shared_workspace_bytes(ctypes.byref(cache()), ctypes.byref(prefix(rows=9)), ctypes.byref(seqs()), 8, 1) == 0
    assert lib.nq_kv_attention_shared_workspace_bytes(ctypes.byref(cache()), None, ctypes.byref(seqs()), 8, 1) == 0
    empty = dict(row_start=0, lengths=0, block_table=0, rows=0)
    assert attend(p=prefix(**empty), s=seqs(**empty), q=None, out=None) == OK
