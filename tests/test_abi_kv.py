"""Host-side checks of the key/value cache and routing entry points that need
no GPU: every argument error is reported before anything is enqueued (the
pointers are made up and never dereferenced)."""
import ctypes

import pytest

from group_wise_affine_quantize_amd import _binding as B

OK, NULL, DTYPE, QUANT, SHAPE, ALIGN, ALIAS, WORKSPACE = 0, 1, 2, 3, 4, 5, 6, 7
P = 1 << 40         # made-up addresses, 2^32 apart
AT = {n: P + (i << 32) for i, n in enumerate(
    ["k_codes", "v_codes", "k_scales", "v_scales", "row_start", "lengths", "table", "k", "v", "q", "out", "lse", "ws",
     "logits", "bias", "ids", "weights", "dweights", "dlogits"])}


@pytest.fixture(scope="module")
def lib():
    return B.load_library()


def cache(**c):
    a = dict(k_codes=AT["k_codes"], v_codes=AT["v_codes"], k_scales=AT["k_scales"], v_scales=AT["v_scales"], blocks=10,
             kv_heads=2, head_dim=128, block_tokens=32, format=1)
    a.update(c)
    return B._KVCacheStruct(*(a[f] for f, _ in B._KVCacheStruct._fields_))


def seqs(**s):
    a = dict(row_start=AT["row_start"], lengths=AT["lengths"], block_table=AT["table"], batch=3, max_blocks=4,
             table_stride=4, rows=7)
    a.update(s)
    return B._KVSeqsStruct(*(a[f] for f, _ in B._KVSeqsStruct._fields_))


def router(**r):
    a = dict(experts=64, score=1, groups=8, top_groups=4, group_best=2, top_k=6, renormalise=1, scale=1.0)
    a.update(r)
    return B._MoERouterStruct(*(a[f] for f, _ in B._MoERouterStruct._fields_))


def append(lib, c=None, s=None, k=AT["k"], ldk=256, v=AT["v"], ldv=256, dt=1):
    return lib.nq_kv_append(c and ctypes.byref(c), s and ctypes.byref(s), k, ldk, v, ldv, dt, None)


def read(lib, c=None, s=None, k=AT["k"], v=AT["v"], dt=1):
    return lib.nq_kv_read(c and ctypes.byref(c), s and ctypes.byref(s), k, v, dt, None)


def attend(lib, c=None, s=None, q=AT["q"], dt=1, ldq=1024, heads=8, scale=0.1, causal=1, window=0, out=AT["out"],
           lse=None, ws=AT["ws"], ws_bytes=1 << 31):
    return lib.nq_kv_attention(c and ctypes.byref(c), s and ctypes.byref(s), q, dt, ldq, heads, scale, causal, window,
                               out, lse, ws, ws_bytes, None)


BAD_CACHES = [(dict(format=0), QUANT), (dict(format=3), QUANT), (dict(block_tokens=8), QUANT),
              (dict(block_tokens=48), QUANT), (dict(head_dim=0), SHAPE), (dict(head_dim=96), SHAPE),
              (dict(head_dim=512), SHAPE), (dict(kv_heads=0), SHAPE), (dict(kv_heads=65536), SHAPE),
              (dict(blocks=0), SHAPE), (dict(blocks=-1), SHAPE), (dict(blocks=1 << 31), SHAPE),
              (dict(blocks=1 << 30, kv_heads=60000), SHAPE), (dict(k_codes=0), NULL), (dict(v_scales=0), NULL),
              (dict(v_codes=AT["v_codes"] + 8), ALIGN), (dict(k_scales=AT["k_scales"] + 2), ALIGN)]
BAD_SEQS = [(dict(batch=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(max_blocks=-1), SHAPE), (dict(rows=1 << 31), SHAPE),
            (dict(table_stride=3), SHAPE), (dict(batch=1 << 25), SHAPE), (dict(row_start=0), NULL),
            (dict(lengths=0), NULL), (dict(block_table=0), NULL), (dict(lengths=AT["lengths"] + 1), ALIGN)]


@pytest.mark.parametrize("call", [append, read, attend])
def test_bad_caches_and_sequences(lib, call):
    assert call(lib, None, seqs()) == NULL and call(lib, cache(), None) == NULL
    for bad, status in BAD_CACHES:
        assert call(lib, cache(**bad), seqs()) == status, bad
        assert b"nq_kv_" in lib.nq_last_error()
    for bad, status in BAD_SEQS:
        assert call(lib, cache(), seqs(**bad)) == status, bad
    assert call(lib, cache(), seqs(), dt=7) == DTYPE
    # nothing to do: no pointer is needed
    empty = dict(row_start=0, lengths=0, block_table=0)
    assert call(lib, cache(k_codes=0, v_codes=0, k_scales=0, v_scales=0), seqs(rows=0, **empty)) == OK
    assert call(lib, cache(k_codes=0), seqs(batch=0, **empty)) == OK


def test_append_arguments(lib):
    c, s = cache(), seqs()
    assert append(lib, c, s, k=None) == NULL and append(lib, c, s, v=0) == NULL
    assert append(lib, c, s, k=AT["k"] + 4) == ALIGN
    assert append(lib, c, s, ldk=255) == SHAPE and append(lib, c, s, ldv=257) == ALIGN
    assert append(lib, c, s, k=AT["k_codes"]) == ALIAS and append(lib, c, s, v=AT["v_scales"]) == ALIAS
    assert append(lib, cache(v_codes=AT["k_codes"] + 16), s) == ALIAS
    assert append(lib, c, seqs(lengths=AT["k_codes"])) == ALIAS


def test_read_arguments(lib):
    c, s = cache(), seqs()
    assert read(lib, c, s, k=None) == NULL
    assert read(lib, c, s, v=AT["v"] + 8) == ALIGN
    assert read(lib, c, s, v=AT["k"] + 16) == ALIAS
    assert read(lib, c, s, k=AT["v_codes"]) == ALIAS and read(lib, c, s, k=AT["table"]) == ALIAS


def test_attention_arguments(lib):
    c, s = cache(), seqs()
    for heads in (0, -2, 7, 65536):
        assert attend(lib, c, s, heads=heads, ldq=1 << 23) == SHAPE
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert attend(lib, c, s, scale=scale) == SHAPE
    assert attend(lib, c, s, window=-1) == SHAPE and attend(lib, c, s, window=5, causal=0) == SHAPE
    assert attend(lib, c, s, q=None) == NULL and attend(lib, c, s, out=None) == NULL
    assert attend(lib, c, s, ldq=1020) == SHAPE and attend(lib, c, s, ldq=1025) == ALIGN
    assert attend(lib, c, s, lse=AT["lse"] + 2) == ALIGN
    assert attend(lib, c, s, out=AT["q"]) == ALIAS and attend(lib, c, s, lse=AT["out"]) == ALIAS
    assert attend(lib, c, s, out=AT["k_codes"]) == ALIAS
    # contexts of up to 16 tiles of 64 tokens are not split: no workspace
    assert lib.nq_kv_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(s), 8, 1) == 0
    s = seqs(max_blocks=100, table_stride=100)
    need = lib.nq_kv_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(s), 8, 1)
    assert need > 0
    assert attend(lib, c, s, ws=None) == WORKSPACE and attend(lib, c, s, ws_bytes=need - 1) == WORKSPACE
    assert attend(lib, c, s, ws=AT["ws"] + 8) == ALIGN and attend(lib, c, s, ws=AT["out"]) == ALIAS
    assert lib.nq_kv_attention_workspace_bytes(ctypes.byref(cache(head_dim=5)), ctypes.byref(s), 8, 1) == 0


BAD_ROUTERS = [(dict(score=0), QUANT), (dict(score=3), QUANT), (dict(experts=0), SHAPE), (dict(experts=1025), SHAPE),
               (dict(groups=0), SHAPE), (dict(groups=7), SHAPE), (dict(experts=130, groups=65), SHAPE),
               (dict(top_groups=0), SHAPE), (dict(top_groups=9), SHAPE), (dict(group_best=0), SHAPE),
               (dict(group_best=3), SHAPE), (dict(groups=64, top_groups=64), SHAPE), (dict(top_k=0), SHAPE),
               (dict(top_k=33), SHAPE), (dict(top_groups=1, top_k=9), SHAPE), (dict(scale=float("nan")), SHAPE)]


def test_routing_arguments(lib):
    def route(r=router(), logits=AT["logits"], dt=0, tokens=5, ld=64, bias=None, ids=AT["ids"], w=AT["weights"]):
        return lib.nq_moe_route(r and ctypes.byref(r), logits, dt, tokens, ld, bias, ids, w, None)

    def grad(r=router(), logits=AT["logits"], dt=0, tokens=5, ld=64, ids=AT["ids"], dw=AT["dweights"],
             dx=AT["dlogits"]):
        return lib.nq_moe_route_grad(r and ctypes.byref(r), logits, dt, tokens, ld, ids, dw, dx, None)

    for call in (route, grad):
        assert call(r=None) == NULL
        for bad, status in BAD_ROUTERS:
            assert call(r=router(**bad)) == status, bad
        assert call(dt=2) == DTYPE and call(tokens=-1) == SHAPE and call(ld=63) == SHAPE
        assert call(tokens=0, logits=None, ids=None) == OK
        assert call(logits=None) == NULL and call(ids=None) == NULL
        assert call(logits=AT["logits"] + 2) == ALIGN and call(ids=AT["ids"] + 1) == ALIGN
    assert route(w=None) == NULL and route(w=AT["ids"]) == ALIAS and route(ids=AT["logits"]) == ALIAS
    assert route(bias=AT["bias"] + 2) == ALIGN and route(bias=AT["weights"]) == ALIAS
    assert grad(dw=None) == NULL and grad(dx=AT["logits"]) == ALIAS and grad(dx=AT["dweights"]) == ALIAS


def test_binding_refuses_cpu_tensors():
    import torch
    with pytest.raises(ValueError):
        B.KVCache(2, 1, 16, 64, device="cpu")
    with pytest.raises(ValueError):
        B.nq_moe_route(B.MoERouter(8, 2), torch.zeros(3, 8))
    with pytest.raises(ValueError):
        B.MoERouter(8, 2, score="tanh")


def test_attention_of_more_sequences_than_rows_returns():
    """The bound of the list of work counts sequences that can have rows: with 2^24 sequences of 128 heads the search
    for its unit size ends (no GPU is visible here, so the call then fails at the launch)."""
    import os
    import subprocess
    import sys
    program = """
import ctypes, sys
sys.path[:0] = sys.argv[1:]
import test_abi_kv as t
lib = t.B.load_library()
c = t.cache(kv_heads=128, head_dim=64, block_tokens=128)
s = t.seqs(batch=1 << 24, rows=4, max_blocks=8, table_stride=8)
print(t.attend(lib, c, s, ldq=128 * 64, heads=128), flush=True)
"""
    here = os.path.dirname(os.path.abspath(__file__))
    env = {**os.environ, "HIP_VISIBLE_DEVICES": "-1", "ROCR_VISIBLE_DEVICES": ""}
    done = subprocess.run([sys.executable, "-c", program, here, os.path.dirname(here)], env=env, capture_output=True,
                          text=True, timeout=60)
    assert done.stdout.split() == ["8"], done.stderr[-500:]


def test_a_router_that_calls_go_by_does_not_change():
    router = B.MoERouter(32, 4, renormalise=True)
    for name in ("top_k", "experts", "scale", "score", "groups", "_struct"):
        with pytest.raises(AttributeError):
            setattr(router, name, 8)
    assert router.top_k == router._struct.top_k == 4
