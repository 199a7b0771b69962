"""Attention behind shared prefixes on the GPU against the plain reference
(oracle/kv.py), within the bounds of its roundings.  Ways to make a cache are
test_gpu_kv.py's."""
import numpy as np
import pytest
import torch

from gpu_helpers import bits_equal
from group_wise_affine_quantize_amd import _binding as B
from oracle import kv as K
from test_gpu_kv import Pair, filled, gpu, i32, rows, tables  # noqa: F401  (gpu: the fixture)

pytestmark = pytest.mark.gpu


def attend(p, prefix, own, q, fill=None, **how):
    """prefix and own: (row_start, lengths, table).  out and lse, both holding `fill` before the call."""
    seqs = [B.KVSequences(i32(s), i32(n), i32(t), q.shape[0]) for s, n, t in (prefix, own)]
    out, lse = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    if fill is not None:
        out.fill_(fill), lse.fill_(fill)
    B.nq_kv_attention_shared(p.dev, *seqs, q, out=out, lse=lse, **how)
    return out, lse


def limits(p, prefix, own, q, scale=None, causal=True):
    """out and lse in 64 bits, and how far they may be off.  The roundings, relative: the scores' sums (dim terms) and exponents (24 bits of log2 e * |z|, twice), value scales
    of up to 2^120 in the exponent, the weights (2^-12 as fp16, 2^-22 as two of them), sums over the tokens, and three
    more where the two parts join; for fp32 the query's 22 bits.  Weights times value scales end at 2^-37 of the largest."""
    dim, wide = p.host.dim, q.dtype == torch.float32
    scale = dim ** -0.5 if scale is None else scale
    want = K.attention_shared(p.host, *prefix, *own, q.float().cpu().double().numpy(), scale, causal)
    z = (want["reach"] + 20)[..., None]
    weight = 2 * ((dim + 8) * 2.0 ** -24 + 2.0 ** -22) * z + (2.0 ** -21 if wide else 2.0 ** -11) + 4 * 120 * 2.0 ** -24
    rest = (want["seen"][:, None, None] + 3) * 2.0 ** -24
    bound = (weight + rest) * want["spread"] + np.abs(want["out"]) * (2.0 ** -22 if wide else 2.0 ** -8) + 1e-37
    bound += (want["seen"][:, None] * want["largest"])[..., None] * 2.0 ** -37
    lse = weight[..., 0] + rest[..., 0] + 2.0 ** -22 * np.abs(np.where(np.isneginf(want["lse"]), 0, want["lse"])) + 2.0 ** -20
    return want, bound, lse


def check(p, prefix, own, q, out, lse, rows_of=None, scale=None, causal=True):
    want, bound, lim = limits(p, prefix, own, q, scale, causal)
    at = slice(None) if rows_of is None else rows_of
    err = np.abs(out.double().cpu().numpy() - want["out"])[at]
    assert np.all(np.isfinite(err)) and np.all(err <= bound[at]), float((err / bound[at]).max())
    g, w = lse.double().cpu().numpy()[at], want["lse"][at]
    none = np.isneginf(w)
    assert np.array_equal(np.isneginf(g), none)
    assert np.all(np.abs(g[~none] - w[~none]) <= lim[at][~none])


def starts(counts, first=0):
    return (first + np.concatenate([[0], np.cumsum(counts)])).astype(int)


CASES = [
    # prefix lengths, sequences of each prefix, sequences behind none, rows per sequence, own lengths, q heads, kv heads,
    # dim, block, format, dtype, options
    ([1], [1], 0, [1], [1], 1, 1, 64, 16, "int8", "bf16", {}),
    ([64], [3], 0, [1, 1, 1], [1, 17, 64], 4, 1, 128, 16, "int8", "bf16", {}),
    ([200], [4], 0, [1, 1, 1, 1], [90, 1, 33, 5], 8, 2, 128, 64, "fp8", "bf16", {}),
    ([1500], [5], 0, [1] * 5, [10, 20, 3, 70, 1], 6, 1, 64, 32, "int8", "f32", {}),                 # a split prefix
    ([333], [20], 0, [1] * 20, [(7 * i) % 90 + 1 for i in range(20)], 8, 2, 128, 64, "int8", "bf16", {}),    # tiles
    ([2100], [24], 0, [2] * 24, [(11 * i) % 60 + 2 for i in range(24)], 8, 1, 128, 16, "fp8", "bf16", {}),   # split tiles
    ([777, 0, 40], [3, 2, 30], 3, [1] * 38, [(5 * i) % 50 + 1 for i in range(38)], 4, 1, 64, 32, "int8", "bf16", {}),
    ([100, 300], [2, 1], 1, [40, 3, 70, 1], [40, 50, 80, 9], 4, 2, 128, 64, "int8", "bf16", {}),    # prompts behind prefixes
    ([100, 300], [2, 1], 1, [40, 3, 70, 1], [40, 50, 80, 9], 4, 2, 192, 32, "fp8", "f32", {}),
    ([130], [2], 0, [90, 90], [90, 1400], 4, 4, 64, 16, "int8", "f32", {}),                         # both parts split
    ([50], [3], 1, [1, 0, 2, 1], [0, 9, 1, 0], 4, 2, 128, 16, "fp8", "bf16", {}),                   # rows before the first token
    ([90], [2], 1, [3, 20, 7], [30, 20, 7], 6, 2, 256, 32, "int8", "bf16", {"causal": False}),
    ([90], [2], 1, [33, 20, 7], [33, 20, 7], 6, 1, 256, 128, "fp8", "f32", {"causal": False, "scale": 0.2}),
    ([0, 0], [1, 1], 1, [1, 2, 1], [5, 5, 5], 2, 1, 64, 16, "int8", "bf16", {}),
    ([8000], [2], 0, [1, 1], [40, 7000], 3, 1, 64, 64, "int8", "bf16", {}),                         # over 64 parts of both
    ([8100], [9], 0, [2] * 9, [(31 * i) % 40 + 2 for i in range(9)], 4, 1, 64, 128, "fp8", "f32", {}),   # the same, of tiles
    # more segments than one launch takes for both passes: prefixes by tiles, one of them and three, and streamed
    ([2100], [200], 0, [1] * 200, [(11 * i) % 130 + 1 for i in range(200)], 32, 8, 64, 64, "int8", "bf16", {}),
    ([900, 0, 3000], [70, 60, 90], 5, [1] * 225, [(13 * i) % 1200 + 1 for i in range(225)], 32, 8, 64, 128, "fp8", "f32", {}),
    ([(97 * i) % 400 for i in range(40)], [6] * 40, 10, [1] * 250, [(17 * i) % 200 for i in range(250)], 16, 8, 64, 16, "int8", "f32", {}),
    ([1300, 70, 2], [90, 1, 90], 0, [1] * 181, [(29 * i) % 900 + 1 for i in range(181)], 32, 8, 128, 32, "int8", "bf16", {}),
]


@pytest.mark.parametrize("prefixes,behind,loose,n,lengths,heads,kv,dim,block,fmt,dtype,how", CASES)
def test_shared_attention_matches_the_reference(prefixes, behind, loose, n, lengths, heads, kv, dim, block, fmt, dtype, how):
    p, table = filled(20, fmt, block, dim, kv, lengths + prefixes)
    own_table, prefix_table = table[:len(lengths)], table[len(lengths):]
    start = starts(n)
    assert sum(behind) + loose == len(n)
    prefix_start = start[starts(behind)]
    q = rows(30, sum(n), heads, dim, dtype, 2.0, fused=2)
    prefix, own = (prefix_start, prefixes, prefix_table), (start, lengths, own_table)
    out, lse = attend(p, prefix, own, q, fill=7.0, **how)
    check(p, prefix, own, q, out, lse, **how)
    again = attend(p, prefix, own, q.contiguous(), fill=3.0, **how)
    assert bits_equal(out, again[0]) and bits_equal(lse, again[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_no_sequence_or_no_prefix_has(dtype):
    """Spare rows before, between and behind stay as they were; sequences outside the prefixes see their own tokens."""
    p, table = filled(40, "int8", 32, 64, 2, [90, 40, 200])
    q = rows(41, 60, 8, 64, dtype, 2.0)
    own = ([5, 6, 30], [90, 40], table[:2])
    for first, last in ((0, 60), (5, 6), (6, 30), (10, 20), (31, 60), (7, 7)):
        prefix = ([first, last], [200], table[2:])
        out, lse = attend(p, prefix, own, q, fill=7.0)
        mine = np.zeros(60, bool)
        mine[5:30] = True
        check(p, prefix, own, q, out, lse, mine)
        assert (out[:5] == 7).all() and (out[30:] == 7).all() and (lse[30:] == 7).all()


def test_many_prefixes_and_sequences():
    """More of both than a wave has lanes; prefixes with no rows among them."""
    rng = np.random.default_rng(5)
    lengths = rng.integers(1, 60, 150).tolist()
    prefixes = rng.integers(0, 90, 80).tolist()
    behind = rng.integers(0, 4, 80)
    behind[-1] += 140 - min(140, behind.sum())
    p, table = filled(21, "fp8", 16, 64, 1, lengths + prefixes)
    start = starts([1] * 150)
    prefix_start = np.minimum(starts(behind, 4), 150)
    q = rows(31, 150, 2, 64, "bf16")
    prefix, own = (prefix_start, prefixes, table[150:]), (start, lengths, table[:150])
    check(p, prefix, own, q, *attend(p, prefix, own, q))


@pytest.mark.parametrize("count", [3, 40])
def test_equal_to_tables_that_repeat_the_prefix(count):
    """The same attention with the prefix's blocks at the head of every table: within two roundings of each other."""
    block, long = 32, 96
    p, table = filled(50, "int8", block, 128, 2, [30] * count + [long])
    q = rows(51, count, 8, 128, "f32", 2.0)
    own = (starts([1] * count), [30] * count, table[:count])
    out, lse = attend(p, ([0, count], [long], table[count:]), own, q)
    repeat = np.concatenate([np.repeat(table[count:, :3], count, 0), table[:count, :1]], 1)
    want_lse = torch.empty_like(lse)
    want = B.nq_kv_attention(p.dev, B.KVSequences(i32(own[0]), i32([30 + long] * count), i32(repeat), count), q, lse=want_lse)
    assert (out - want).abs().max() <= 2.0 ** -17 * want.abs().max() and (lse - want_lse).abs().max() <= 2.0 ** -17 * want_lse.abs().max()


@pytest.mark.parametrize("seqs", [3, 30])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("prefix_e,own_e", [([0, 40, None, -90], [0, 1]), ([0, 1], [None, -100]), ([None], [None]),
                                            ([100, -20], [None, 0]), ([-100, -100], [60, 0])])
def test_value_scales_of_unlike_parts(prefix_e, own_e, dtype, seqs):
    """Blocks of values about 2^e (None: zeros), so that one part's sum of weights has a reference of its own and the
    other's has not."""
    block, dim = 32, 64
    blocks = len(prefix_e) + seqs * len(own_e)
    p = Pair(60, blocks, 1, block, dim, "int8")
    table = np.random.default_rng(61).permutation(blocks).astype(np.int32)
    all_e = list(prefix_e) + list(own_e) * seqs
    k = rows(62, block * blocks, 1, dim, "f32")
    v = rows(63, block * blocks, 1, dim, "f32")
    for j, e in enumerate(all_e):
        v[block * j:block * (j + 1)] *= 0.0 if e is None else 2.0 ** e
    p.append([0, block * blocks], [block * blocks], table[None], k, v)
    n = len(prefix_e)
    prefix = ([0, seqs], [block * n], table[None, :n])
    own = (starts([1] * seqs), [block * len(own_e) - 5] * seqs, table[n:].reshape(seqs, len(own_e)))
    q = rows(64, seqs, 4, dim, dtype, 2.0)
    check(p, prefix, own, q, *attend(p, prefix, own, q))


@pytest.mark.parametrize("seqs", [4, 40])
def test_numbers_that_are_none(seqs):
    """A block of NaN in a prefix reaches the rows behind it, one in a sequence that sequence, a query of NaN its own head."""
    p, table = filled(70, "fp8", 16, 64, 1, [20] * seqs + [50, 60])
    own = (starts([1] * seqs), [20] * seqs, table[:seqs])
    half = seqs // 2
    prefix = ([0, half, seqs], [50, 60], table[seqs:])
    q = rows(71, seqs, 4, 64, "bf16")
    clean, clean_lse = attend(p, prefix, own, q)
    q[1, 2, 5] = float("nan")
    p.dev.v_scales[int(table[seqs + 1, 3])] = float("nan")     # the second prefix's tokens 48 on
    p.dev.k_scales[int(table[0, 1])] = float("nan")            # the first sequence's tokens 16 on
    out, lse = attend(p, prefix, own, q)
    lost = torch.zeros((seqs, 4), dtype=torch.bool, device="cuda")
    lost[half:] = True
    lost[0] = True
    lost[1, 2] = True
    assert out[lost].isnan().all() and lse[lost].isnan().all()
    assert bits_equal(out[~lost], clean[~lost]) and bits_equal(lse[~lost], clean_lse[~lost])


def test_arrays_of_any_content_touch_nothing_else():
    p, table = filled(80, "int8", 16, 64, 1, [40, 40, 40])
    p.dev.k_scales.nan_to_num_(1.0), p.dev.v_scales.nan_to_num_(1.0)
    q = rows(81, 50, 4, 64, "f32")
    wild = np.array([[3, -1, 99], [0, 2 ** 31 - 1, -2 ** 31], [1, 2, 3]], np.int32)
    before = [t.clone() for t in (p.dev.k_codes, p.dev.v_codes, p.dev.k_scales, p.dev.v_scales)]
    for prefix_start in ([-5, 12, 3, 2 ** 31 - 1], [50, 40, 30, 20], [0, 50, 50, 50], [-2 ** 31, -1, 60, 70]):
        for lengths in ([40, 48, -7], [2 ** 31 - 1, 3, 0]):
            out, lse = torch.full((70, 4, 64), 7.0, device="cuda"), torch.full((70, 4), 7.0, device="cuda")
            prefix = B.KVSequences(i32(prefix_start), i32(lengths), i32(wild), 50)
            own = B.KVSequences(i32([0, 10, 30, 50]), i32([40, 20, 25]), i32(wild), 50)
            B.nq_kv_attention_shared(p.dev, prefix, own, q, out=out[10:60], lse=lse[10:60])
            assert (out[:10] == 7).all() and (out[60:] == 7).all() and (lse[:10] == 7).all() and (lse[60:] == 7).all()
    assert all(torch.equal(a, b) for a, b in zip(before, (p.dev.k_codes, p.dev.v_codes, p.dev.k_scales, p.dev.v_scales)))


def test_serving_steps_replay_from_a_graph():
    """Lengths grow on the device; replays between eager calls give the eager results, on any stream."""
    seqs, heads = 20, 8
    p, table = filled(90, "int8", 32, 128, 2, [64] * seqs + [1200])
    lengths = i32([20] * seqs)
    prefix = B.KVSequences(i32([0, seqs]), i32([1200]), i32(table[seqs:]), seqs)
    own = B.KVSequences(i32(starts([1] * seqs)), lengths, i32(table[:seqs]), seqs)
    q = rows(91, seqs, heads, 128, "bf16")
    lse = torch.empty((seqs, heads), device="cuda")
    B.nq_kv_attention_shared(p.dev, prefix, own, q, lse=lse)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        out = B.nq_kv_attention_shared(p.dev, prefix, own, q, lse=lse)
    for step in range(4):
        lengths += 7
        q.copy_(rows(100 + step, seqs, heads, 128, "bf16"))
        graph.replay()
        got, got_lse = out.clone(), lse.clone()
        want_lse = torch.empty_like(lse)
        want = B.nq_kv_attention_shared(p.dev, prefix, own, q, lse=want_lse)
        torch.cuda.synchronize()
        assert bits_equal(got, want) and bits_equal(got_lse, want_lse)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        other = B.nq_kv_attention_shared(p.dev, prefix, own, q, stream=s)
        s.synchronize()
        assert bits_equal(other, want)
        check(p, ([0, seqs], [1200], table[seqs:]), (starts([1] * seqs), lengths.tolist(), table[:seqs]), q, want, want_lse)


def test_more_rows_than_one_launch_has_threads_for():
    """2^26 rows and heads and some: at 64 threads to each in the join, their threads pass 32 bits."""
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of memory")
    n, heads, period = (1 << 20) + 8, 64, 7
    p, table = filled(97, "int8", 16, 64, 1, [70, 1])
    some = rows(98, period, heads, 64, "bf16")
    q = some[torch.arange(n, device="cuda") % period]
    prefix, own = ([0, n], [70], table[:1]), ([0, n], [0], table[1:])
    out, lse = attend(p, prefix, own, q, fill=7.0)
    want, bound, lim = limits(p, ([0, period], *prefix[1:]), ([0, period], *own[1:]), some)
    want, bound, want_lse, lim = (torch.tensor(t, device="cuda") for t in (want["out"], bound, want["lse"], lim))
    for at in torch.arange(n, device="cuda").split(1 << 17):
        which = at % period
        assert ((out[at] - want[which]).abs() <= bound[which]).all() and ((lse[at] - want_lse[which]).abs() <= lim[which]).all()


def test_empty_calls_and_refusals():
    p, table = filled(95, "int8", 16, 64, 1, [20, 20])
    q = rows(96, 2, 2, 64, "bf16")
    own = B.KVSequences(i32([0, 1, 2]), i32([20, 20]), i32(table), 2)
    # no prefix at all: attention of the sequences
    none = B.KVSequences(i32([0]), i32([]), torch.empty((0, 1), dtype=torch.int32, device="cuda"), 2)
    assert bits_equal(B.nq_kv_attention_shared(p.dev, none, own, q), B.nq_kv_attention(p.dev, own, q))
    prefix = B.KVSequences(i32([0, 2]), i32([20]), i32(table[:1]), 2)
    zero = [B.KVSequences(i32([0, 0]), i32([20]), i32(table[:1]), 0) for _ in range(2)]
    assert B.nq_kv_attention_shared(p.dev, *zero, q[:0]).shape == (0, 2, 64)
    three = B.KVSequences(i32([0, 2]), i32([20]), i32(table[:1]), 3)
    for call in (lambda: B.nq_kv_attention_shared(p.dev, three, own, q), lambda: B.nq_kv_attention_shared(p.dev, prefix, own, q[:1]),
                 lambda: B.nq_kv_attention_shared(p.dev, prefix, own, q, out=q), lambda: B.nq_kv_attention_shared(p.dev, prefix, own, q.half()),
                 lambda: B.nq_kv_attention_shared(p.dev, prefix, own, q, lse=torch.empty(2, 2)),
                 lambda: B.nq_kv_attention_shared(p.dev, prefix, own, q, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
                 lambda: B.nq_kv_attention_shared(p.dev, prefix, own, q, scale=-1.0)):
        with pytest.raises((ValueError, TypeError, B.NQError)):
            call()
