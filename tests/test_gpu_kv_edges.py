"""The 8-bit key/value cache on the GPU where its kernels can go wrong: spare
rows, value scales from one end of their range to the other, numbers that are
none.  References and the ways to make a cache are test_gpu_kv.py's."""
import numpy as np
import pytest
import torch

from gpu_helpers import bits_equal
from group_wise_affine_quantize_amd import _binding as B
from oracle import kv as K
from test_gpu_kv import Pair, filled, gpu, i32, rows, tables  # noqa: F401  (gpu: the fixture)

pytestmark = pytest.mark.gpu


def attend(p, start, lengths, table, q, fill=None, **how):
    """out and lse, both holding `fill` before the call."""
    seqs = B.KVSequences(i32(start), i32(lengths), i32(table), q.shape[0])
    out, lse = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    if fill is not None:
        out.fill_(fill), lse.fill_(fill)
    B.nq_kv_attention(p.dev, seqs, q, out=out, lse=lse, **how)
    return out, lse


def check(p, start, lengths, table, q, out, lse, own=None, scale=None, **how):
    """Rows `own` (default: all) against the reference.  The roundings, relative: the scores' sums (dim terms) and
    exponents (24 bits of log2 e * |z|, twice), the weights (2^-12 as fp16, 2^-22 as two of them) and sums over the
    tokens; for fp32 the query's 22 bits.  Weights times value scales end at 2^-37 of a row's largest."""
    dim, wide = p.host.dim, q.dtype == torch.float32
    scale = dim ** -0.5 if scale is None else scale
    want = K.attention(p.host, start, lengths, table, q.float().cpu().double().numpy(), scale, **how)
    z = (want["reach"] + 20)[..., None]
    weight = 2 * ((dim + 8) * 2.0 ** -24 + 2.0 ** -22) * z + (2.0 ** -21 if wide else 2.0 ** -11)
    # value scales are powers of two up to 2^120: their logarithm takes part in the exponent, 24 bits of it
    weight = weight + 4 * 120 * 2.0 ** -24
    rest = want["seen"][:, None, None] * 2.0 ** -24
    bound = (weight + rest) * want["spread"] + np.abs(want["out"]) * (2.0 ** -22 if wide else 2.0 ** -8) + 1e-37
    bound += (want["seen"][:, None] * want["largest"])[..., None] * 2.0 ** -37
    own = slice(None) if own is None else own
    err = np.abs(out.double().cpu().numpy() - want["out"])[own]
    assert np.all(np.isfinite(err)) and np.all(err <= bound[own]), float((err / bound[own]).max())
    g, w = lse.double().cpu().numpy()[own], want["lse"][own]
    none = np.isneginf(w)
    assert np.array_equal(np.isneginf(g), none)
    lim = (weight[..., 0] + rest[..., 0])[own] + 2.0 ** -22 * np.abs(np.where(none, 0, w)) + 2.0 ** -20
    assert np.all(np.abs(g[~none] - w[~none]) <= lim[~none])


@pytest.mark.parametrize("total,first,used", [(17, 0, 1), (17, 5, 4), (32, 0, 4), (32, 9, 16), (100, 3, 10), (100, 99, 1),
                                              (100, 0, 16), (100, 40, 17), (100, 7, 0)])
def test_one_sequence_among_spare_rows(total, first, used):
    """A buffer of fixed size, of which the sequence has some rows: those are answered, the others stay."""
    p, table = filled(40, "int8", 32, 64, 2, [90])
    q = rows(41, total, 8, 64, "bf16", 2.0)
    start = [first, first + used]
    out, lse = attend(p, start, [90], table, q, fill=7.0)
    own = np.zeros(total, bool)
    own[first:first + used] = True
    check(p, start, [90], table, q, out, lse, own)
    spare = torch.from_numpy(~own)
    assert (out.cpu()[spare] == 7).all() and (lse.cpu()[spare] == 7).all()


# What the kernels see: few query columns of a head go through the streaming kernel, more through the tile kernel; a
# table of more than 16 tiles of 64 tokens lets the first split its tokens, few workgroups the second.
SHAPES = {"stream": (2, 4), "stream, two groups": (5, 4), "tile": (20, 4)}


def blocks_of(seed, exponents, block, dim, fmt, wide=None):
    """One sequence; the values of its block j lie about 2^exponents[j] (None: all zero)."""
    n = len(exponents) * block - 3
    wide = wide or len(exponents)
    p = Pair(seed, wide + 2, 1, block, dim, fmt)
    table = tables(seed + 1, 1, wide, wide + 2)
    k, v = rows(seed + 2, n, 1, dim, "f32"), rows(seed + 3, n, 1, dim, "f32").clamp(-4, 4)
    for j, e in enumerate(exponents):
        v[block * j:block * (j + 1)] *= 0.0 if e is None else 2.0 ** e
    p.append([0, n], [n], table, k, v)
    return p, table, n


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("e", [0, 60, 75, 118, -95, None])
def test_blocks_of_zeros_count_beside_values_of_any_size(e, dtype, split, shape):
    """Half of the tokens are zeros: they have their share of the sum of weights, whatever the others' values."""
    n, heads = SHAPES[shape]
    exponents = [None, e] * (34 if split else 4)
    p, table, length = blocks_of(50, exponents, 32, 64, "int8")
    for q in (torch.zeros((n, heads, 64), device="cuda"), rows(51, n, heads, 64, "f32", 2.0)):
        q = q.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
        out, lse = attend(p, [0, n], [length], table, q)
        check(p, [0, n], [length], table, q, out, lse)


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_value_scales_over_their_whole_range(fmt, split, shape):
    """Scales from 2^-100 to 2^118 and zeros side by side, with scores in both directions."""
    n, heads = SHAPES[shape]
    some = [-98, 3, None, -60, 110, 0, -20, 70, -75, 30, None, 100]
    for exponents in (some, some[::-1], [0, 0, -98, -98], [-98, None, -98, -90], [None, -98, 0, 5]):
        exponents = exponents * (-(-70 // len(exponents)) if split else 1)
        p, table, length = blocks_of(60, exponents, 16, 64, fmt, wide=80 if split else None)
        for dtype, sigma in (("bf16", 1.0), ("f32", 12.0)):
            q = rows(61, n, heads, 64, dtype, sigma)
            out, lse = attend(p, [0, n], [length], table, q)
            check(p, [0, n], [length], table, q, out, lse)


@pytest.mark.parametrize("shape", list(SHAPES))
def test_long_contexts_of_tiny_values(shape):
    """30000 equal keys whose values have the smallest scale: the sum of weights over it passes fp32, the answer does
    not, and the log of the sum does not depend on the values."""
    n, heads = SHAPES[shape]
    length, block, dim = 30000, 128, 64
    wide = -(-length // block)
    p = Pair(70, wide + 2, 1, block, dim, "int8")
    table = tables(71, 1, wide, wide + 2)
    k = rows(72, 1, 1, dim, "f32").expand(length, 1, dim).contiguous()
    v = rows(73, length, 1, dim, "f32") * 1e-30
    p.append([0, length], [length], table, k, v)
    for dtype in ("bf16", "f32"):
        q = rows(74, n, heads, dim, dtype)
        out, lse = attend(p, [0, n], [length], table, q)
        check(p, [0, n], [length], table, q, out, lse)


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_sharp_scores_and_uneven_scales_in_every_kernel(fmt, shape):
    """Scores of several hundred, value scales over 2^60, zero keys and zero values."""
    n, heads = SHAPES[shape]
    p = Pair(80, 12, 1, 16, 64, fmt)
    table = tables(81, 1, 10, 12)
    k, v = rows(82, 150, 1, 64, "f32", 20.0), rows(83, 150, 1, 64, "f32")
    for j, e in enumerate((0, -40, 20, 3, -7, 0, 1, -30, 12, 0)):
        v[16 * j:16 * j + 16] *= 2.0 ** e
    v[48:64] = 0
    k[96:112] = 0
    p.append([0, 150], [150], table, k, v)
    for dtype in ("bf16", "f32"):
        q = rows(84, n, heads, 64, dtype, 6.0)
        out, lse = attend(p, [0, n], [150], table, q)
        check(p, [0, n], [150], table, q, out, lse)


# ---- numbers that are none
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("length", [150, 2500])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_query_that_is_no_number_gives_nan_in_both_outputs(bad, dtype, length, shape):
    n, heads = SHAPES[shape]
    p, table = filled(90, "fp8", 16, 64, 1, [length])
    q = rows(91, n, heads, 64, dtype)
    want, want_lse = attend(p, [0, n], [length], table, q)
    q[1, 2, 13] = bad
    got, lse = attend(p, [0, n], [length], table, q)
    keep = torch.ones((n, heads), dtype=torch.bool)
    keep[1, 2] = False
    assert bits_equal(got.cpu()[keep], want.cpu()[keep]) and bits_equal(lse.cpu()[keep], want_lse.cpu()[keep])
    assert got[1, 2].isnan().all() and lse[1, 2].isnan()
    # a row that sees nothing has no answer to spoil
    out, lse = attend(p, [0, n], [0], table, q)
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("fp8", "f32")])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_number_that_is_none_makes_its_block_nan(bad, fmt, dtype):
    """The head's block reads as NaN from then on, also for tokens written before and after, until its first token is
    written again; other blocks, heads and the other part are as they would be."""
    block, dim, heads = 16, 64, 2
    p, clean = Pair(95, 6, heads, block, dim, fmt), Pair(95, 6, heads, block, dim, fmt)
    table = tables(96, 1, 4, 6)
    calls = [(20, 20), (5, 25), (1, 26), (30, 56)]      # rows, length after them
    for i, (n, length) in enumerate(calls):
        k, v = rows(97 + i, n, heads, dim, dtype), rows(107 + i, n, heads, dim, dtype)
        clean.append([0, n], [length], table, k, v)
        if i == 1:
            k[2, 1, 7] = bad        # token 22, block 1
        if i == 3:
            v[20, 0, 63] = bad      # token 46, block 2
        p.append([0, n], [length], table, k, v)
    for name, block_no, head in (("k", 1, 1), ("v", 2, 0)):
        got, want = getattr(p.dev, name + "_scales").cpu(), getattr(clean.dev, name + "_scales").cpu().clone()
        assert got[table[0, block_no], head].isnan()
        want[table[0, block_no], head] = float("nan")
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())
    seqs = B.KVSequences(i32([0, 56]), i32([56]), i32(table), 56)
    for out in (torch.float32, torch.bfloat16):
        got, want = B.nq_kv_read(p.dev, seqs, out_dtype=out), B.nq_kv_read(clean.dev, seqs, out_dtype=out)
        for g, w, lo, hi, head in ((got[0], want[0], 16, 32, 1), (got[1], want[1], 32, 48, 0)):
            assert g[lo:hi, head].isnan().all()
            g[lo:hi, head] = w[lo:hi, head]
            assert bits_equal(g, w)
    host = K.read(p.host, [0, 56], [56], table)
    got = B.nq_kv_read(p.dev, seqs, out_dtype=torch.float32)
    assert all(np.array_equal(g.cpu().numpy(), w, equal_nan=True) for g, w in zip(got, host))
    # written anew from its first token, a block is whole again: tokens 32 on, of block 2
    k, v = rows(120, 24, heads, dim, dtype), rows(121, 24, heads, dim, dtype)
    p.append([0, 24], [56], table, k, v)
    assert torch.isfinite(p.dev.v_scales.cpu()[table[0]]).all()


@pytest.mark.parametrize("part", ["k", "v"])
@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("fp8", "f32")])
@pytest.mark.parametrize("n,length", [(3, 150), (150, 150), (5, 1500), (90, 1500)])
def test_a_block_of_nan_reaches_the_rows_that_see_it_and_no_other(n, length, fmt, dtype, part):
    """Masked rows and the other head keep their bits; rows that see a token of the block get NaN."""
    block, dim, kv, heads = 16, 64, 2, 4
    p, table = filled(130, fmt, block, dim, kv, [length])
    q = rows(131, n, heads, dim, dtype)
    want, want_lse = attend(p, [0, n], [length], table, q)
    near = attend(p, [0, n], [length], table, q, window=9)
    hurt = (length - n // 2) // block       # the block of a token that some of the rows may not see
    getattr(p.dev, part + "_scales")[int(table[0, hurt]), 1] = float("nan")
    got, lse = attend(p, [0, n], [length], table, q)
    pos = np.arange(length - n, length)
    sees = torch.from_numpy(pos >= hurt * block)
    for r in range(n):
        assert bits_equal(got[r, :2], want[r, :2]) and bits_equal(lse[r, :2], want_lse[r, :2])
        if sees[r]:
            assert got[r, 2:].isnan().all() and lse[r, 2:].isnan().all()
        else:
            assert bits_equal(got[r, 2:], want[r, 2:]) and bits_equal(lse[r, 2:], want_lse[r, 2:])
    got, lse = attend(p, [0, n], [length], table, q, window=9)
    sees = torch.from_numpy((pos >= hurt * block) & (pos - 8 < (hurt + 1) * block)).cuda()
    assert torch.equal(got[:, 2:].isnan().all(-1).all(-1), sees) and torch.equal(lse[:, 2:].isnan().all(-1), sees)
    assert bits_equal(got[~sees], near[0][~sees]) and bits_equal(got[:, :2], near[0][:, :2])


def test_descriptions_that_calls_go_by_do_not_change():
    """Shapes are checked against a description's attributes, kernels go by its struct: were the two apart, rows past
    a tensor's end would be read and written."""
    cache = B.KVCache(4, 1, 16, 64, "int8")
    seqs = B.KVSequences(i32([0, 2]), i32([2]), i32([[1, 2]]), 2)
    for one, names in ((cache, ("k_codes", "v_scales", "blocks", "kv_heads", "format", "block_tokens")),
                       (seqs, ("rows", "lengths", "row_start", "block_table", "batch"))):
        for name in names:
            with pytest.raises(AttributeError):
                setattr(one, name, getattr(one, name))
    seqs.lengths.add_(1)    # in place: the same tensor
    assert seqs.lengths.item() == 3


def test_more_blocks_than_one_launch_has_threads_for():
    """Two sequences of 2^27 rows and some in blocks of 16, nearly all of which do not exist: the last ones are written
    and read as those of a short sequence are, the others read as zeros."""
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of memory")
    half, block, dim, tail = 1 << 27, 16, 64, 55
    n = 2 * half + 23
    wide = -(-(half + 23) // block)
    table = torch.full((2, wide), -1, dtype=torch.int32, device="cuda")
    table[1, -4:] = torch.tensor([3, 0, 2, 1], dtype=torch.int32)
    k = torch.empty((n, 1, dim), dtype=torch.bfloat16, device="cuda")
    first = n - tail        # the first token of the table's last four blocks
    assert first - half == (wide - 4) * block
    k[first:] = rows(140, tail, 1, dim, "bf16")
    cache, small = B.KVCache(4, 1, block, dim, "int8"), B.KVCache(4, 1, block, dim, "int8")
    for c in (cache, small):
        for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
            t.zero_()
    seqs = B.KVSequences(i32([0, half, n]), i32([half, half + 23]), table, n)
    B.nq_kv_append(cache, seqs, k, k)
    short = B.KVSequences(i32([0, tail]), i32([tail]), i32([[3, 0, 2, 1]]), tail)
    x = k[first:].contiguous()
    B.nq_kv_append(small, short, x, x)
    for a, b in ((cache.k_codes, small.k_codes), (cache.v_codes, small.v_codes), (cache.k_scales, small.k_scales),
                 (cache.v_scales, small.v_scales)):
        assert torch.equal(a, b)
    k.fill_(3.0)
    v = torch.full_like(k, 3.0)
    B.nq_kv_read(cache, seqs, k=k, v=v)
    want = B.nq_kv_read(small, short)
    for got, w in zip((k, v), want):
        assert torch.equal(got[first:], w) and not got[:first].any()
    del k, v
    torch.cuda.empty_cache()
