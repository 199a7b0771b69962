"""The 8-bit key/value cache on the GPU against the plain reference
(oracle/kv.py): writes and reads bit for bit, attention within bounds derived
from its roundings."""
import numpy as np
import pytest
import torch

from gpu_helpers import bits_equal
from group_wise_affine_quantize_amd import _binding as B
from group_wise_affine_quantize_amd import synthetic
from oracle import kv as K

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    B.load_library()


def f32_of(t):
    return t.float().cpu().numpy()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


class Pair:
    """A cache on the GPU and its plain twin.  Memory starts as noise: codes of
    every kind (E4M3 NaNs among them) and scales NaN, so that anything read
    without having been written shows."""

    def __init__(self, seed, blocks, heads, block, dim, fmt):
        rng = np.random.default_rng(seed)
        kc = rng.integers(0, 256, (blocks, heads, block, dim), dtype=np.uint8)
        vc = rng.integers(0, 256, (blocks, heads, dim, block), dtype=np.uint8)
        s = np.full((blocks, heads), np.nan, np.float32)
        self.host = K.Cache(kc, s.copy(), vc, s.copy(), fmt)
        self.dev = B.KVCache.wrap(*(torch.from_numpy(a.copy()).cuda() for a in (kc, s, vc, s)), fmt)

    def append(self, row_start, lengths, table, k, v):
        seqs = B.KVSequences(i32(row_start), i32(lengths), i32(table), k.shape[0])
        B.nq_kv_append(self.dev, seqs, k, v)
        K.append(self.host, row_start, lengths, table, f32_of(k), f32_of(v))

    def check_equal(self):
        for name in ("k_scales", "v_scales", "k_codes", "v_codes"):
            got, want = getattr(self.dev, name).cpu().numpy(), getattr(self.host, name)
            assert np.array_equal(got.view(np.uint8), want.view(np.uint8)), name


def rows(seed, n, heads, dim, dtype, sigma=1.0, fused=0):
    """n rows of `heads` heads; fused: column ranges of wider rows."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, heads + fused, dim), dtype=np.float32) * np.float32(sigma)
    return torch.from_numpy(x).cuda().to(DT[dtype])[:, fused:]


def tables(seed, batch, wide, blocks):
    """Every sequence has blocks of its own, in any order."""
    return np.random.default_rng(seed).permutation(blocks)[:batch * wide].reshape(batch, wide).astype(np.int32)


# (row counts, lengths after the call) of a batch, in calls that follow each other
STEPS = {
    "one token": [([1], [1])],
    "token by token": [([1], [i + 1]) for i in range(35)],
    "prompt then tokens": [([37, 0, 5], [37, 0, 5]), ([1, 16, 1], [38, 16, 6]), ([1, 1, 90], [39, 17, 96])],
    "more rows than tokens": [([9, 4], [3, 4]), ([2, 40], [5, 20])],
}


@pytest.mark.parametrize("steps", list(STEPS))
@pytest.mark.parametrize("fmt,dtype,block,dim,heads", [("int8", "bf16", 16, 128, 2), ("fp8", "bf16", 32, 64, 3),
                                                       ("int8", "f32", 64, 192, 1), ("fp8", "f32", 128, 256, 2)])
def test_append_and_read_match_the_reference(steps, fmt, dtype, block, dim, heads):
    calls = STEPS[steps]
    batch = len(calls[0][0])
    p = Pair(1, 8 * batch + 2, heads, block, dim, fmt)
    table = tables(2, batch, 8, 8 * batch + 2)
    for i, (n, lengths) in enumerate(calls):
        start = np.concatenate([[0], np.cumsum(n)])
        # magnitudes that rise and fall from call to call: some scales grow, some do not
        k = rows(10 + i, sum(n), heads, dim, dtype, 2.0 ** ((i * 7) % 5), fused=1)
        v = rows(50 + i, sum(n), heads, dim, dtype, 1.3 ** i)
        p.append(start, lengths, table, k, v)
    p.check_equal()
    whole = np.minimum(calls[-1][1], 8 * block)
    start = np.concatenate([[0], np.cumsum(whole)])
    seqs = B.KVSequences(i32(start), i32(calls[-1][1]), i32(table), int(start[-1]))
    want = K.read(p.host, start, calls[-1][1], table)
    for out in ("f32", "bf16"):
        got = B.nq_kv_read(p.dev, seqs, out_dtype=DT[out])
        for g, w in zip(got, want):
            assert bits_equal(g.cpu(), torch.from_numpy(w).to(DT[out]))


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_scales_that_grow_vanish_and_overflow(fmt):
    """A held block's scale: zero, kept, grown by exact and inexact powers,
    grown past what old codes can hold, and values too small for any scale."""
    dim, block = 64, 32
    qmax = K.QMAX[fmt]
    p = Pair(3, 3, 1, block, dim, fmt)
    table = np.array([[1]], np.int32)
    sizes = [0.0, 0.0, qmax, qmax * 0.5, qmax, qmax * 2, qmax * 2.0000002, qmax * 64, 1.0, 2.0 ** 31, 3e38, 1e-35]
    for t, top in enumerate(sizes):
        x = np.random.default_rng(t).uniform(-1, 1, (1, 1, dim)).astype(np.float32)
        x[0, 0, t] = 1.0
        x = torch.from_numpy(x * np.float32(top)).cuda()
        p.append([0, 1], [t + 1], table, x, -x)
        p.check_equal()
    p = Pair(4, 3, 1, block, dim, fmt)
    x = torch.full((3, 1, dim), 1e-37, device="cuda")
    p.append([0, 3], [3], table, x, x)
    p.check_equal()
    assert p.host.k_scales[1, 0] == np.float32(2.0 ** -100)


def test_halfway_values_round_to_even():
    dim = 64
    for fmt, step in (("int8", 1.0), ("fp8", 32.0)):
        p = Pair(5, 2, 1, 16, dim, fmt)
        qmax = K.QMAX[fmt]
        x = np.zeros((2, 1, dim), np.float32)
        x[0, 0, 0] = qmax                           # scale 1
        x[0, 0, 1:41] = (np.arange(40) + 0.5) * step
        x[1, 0, :40] = -(np.arange(40) + 0.5) * 2.0 ** -9     # between E4M3's smallest numbers
        x = torch.from_numpy(np.clip(x, -qmax, qmax)).cuda()
        p.append([0, 2], [2], np.array([[0]], np.int32), x, x)
        p.check_equal()


def test_ids_lengths_and_row_starts_out_of_range_touch_nothing_else():
    """Every kind of bad content: the cache's other blocks and the rows that no
    sequence has stay as they were; absent tokens read as zeros."""
    heads, dim, block = 2, 64, 16
    p = Pair(6, 6, heads, block, dim, "int8")
    table = np.array([[3, -1, 99], [0, 6, 2], [5, 2 ** 31 - 1, -2 ** 31]], np.int32)
    k, v = rows(1, 90, heads, dim, "bf16"), rows(2, 90, heads, dim, "bf16")
    start, lengths = [0, 40, 80, 90], [40, 48, -7]
    p.append([0, 0, 8, 8], [0, 8, 0], table, k[80:88], v[80:88])     # the second sequence's first tokens
    p.append(start, lengths, table, k, v)
    p.check_equal()
    q = rows(3, 90, 4, dim, "f32")
    seqs = B.KVSequences(i32(start), i32(lengths), i32(table), 90)
    want = K.read(p.host, start, lengths, table)
    got = B.nq_kv_read(p.dev, seqs, out_dtype=torch.float32)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    check_attention(p, start, lengths, table, q, dict(causal=True))
    # row_start that falls, is negative or passes the rows: clamped
    k0 = p.dev.k_codes.clone()
    for scales in (p.dev.k_scales, p.dev.v_scales):     # these sequences also see tokens that nobody wrote
        scales.nan_to_num_(1.0)
    out = torch.full((20, 4, dim), 7.0, device="cuda")
    wild = B.KVSequences(i32([-5, 12, 3, 2 ** 31 - 1]), i32([12, 20, 5]), i32(table), 20)
    B.nq_kv_attention(p.dev, wild, q[:20].contiguous(), out=out)
    got = B.nq_kv_read(p.dev, wild)
    B.nq_kv_append(p.dev, wild, k[:20], v[:20])
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and got[0].shape == (20, heads, dim)
    same = [i for i in range(6) if i not in (3, 0, 5, 2)]
    assert torch.equal(p.dev.k_codes[same], k0[same])


# ---------------------------------------------------------------- attention
def check_attention(p, start, lengths, table, q, how, scale=None, lse=True):
    dim, heads = p.host.dim, q.shape[1]
    scale = dim ** -0.5 if scale is None else scale
    seqs = B.KVSequences(i32(start), i32(lengths), i32(table), q.shape[0])
    got_lse = torch.full((q.shape[0], heads), 5.0, device="cuda")
    out = B.nq_kv_attention(p.dev, seqs, q, scale=scale, lse=got_lse if lse else None, **how)
    assert out.dtype == q.dtype and out.shape == q.shape
    want = K.attention(p.host, start, lengths, table, q.float().cpu().double().numpy(), scale, **how)
    # roundings, relative: the scores' sums (dim terms) and exponents (24 bits
    # of log2 e * |z|, twice), the weights (2^-12 as fp16, 2^-22 as two of
    # them) and sums over the tokens; for fp32 the query's 22 bits.  And, as the
    # kernels state, weights times value scales end about 2^-39 below the largest
    wide = q.dtype == torch.float32
    z = (want["reach"] + 20)[..., None]
    weight = 2 * ((dim + 8) * 2.0 ** -24 + 2.0 ** -22) * z + (2.0 ** -21 if wide else 2.0 ** -11)
    rest = want["seen"][:, None, None] * 2.0 ** -24
    bound = (weight + rest) * want["spread"] + np.abs(want["out"]) * (2.0 ** -22 if wide else 2.0 ** -8) + 1e-37
    bound += (want["seen"][:, None] * want["largest"])[..., None] * 2.0 ** -39
    err = np.abs(out.double().cpu().numpy() - want["out"])
    assert np.all(np.isfinite(err)) and np.all(err <= bound), (float((err / bound).max()), how)
    if lse:
        g = got_lse.double().cpu().numpy()
        none = np.isneginf(want["lse"])
        assert np.array_equal(np.isneginf(g), none)
        both = ~none
        lim = (weight[..., 0] + rest[..., 0]) + 2.0 ** -22 * np.abs(want["lse"], where=both, out=np.zeros_like(g)) + 2.0 ** -20
        assert np.all(np.abs(g[both] - want["lse"][both]) <= lim[both])
    return out


def filled(seed, fmt, block, dim, heads, lengths, wide=None, spare=3, sigma=1.0):
    """A cache that holds random tokens of every sequence."""
    need = [max(1, -(-max(0, n) // block)) for n in lengths]
    wide = wide or max(need)
    blocks = len(lengths) * wide + spare
    p = Pair(seed, blocks, heads, block, dim, fmt)
    table = tables(seed + 1, len(lengths), wide, blocks)
    start = np.concatenate([[0], np.cumsum(lengths)])
    k = rows(seed + 2, int(start[-1]), heads, dim, "bf16", sigma)
    v = rows(seed + 3, int(start[-1]), heads, dim, "bf16")
    p.append(start, lengths, table, k, v)
    return p, table


CASES = [
    # rows per sequence, lengths, q heads, kv heads, dim, block, format, dtype, options
    ([1], [1], 1, 1, 64, 16, "int8", "bf16", {}),
    ([1], [63], 4, 1, 128, 16, "int8", "bf16", {}),
    ([1], [64], 8, 2, 128, 64, "fp8", "bf16", {}),
    ([1], [65], 7, 1, 128, 128, "int8", "f32", {}),
    ([1, 1, 1], [17, 200, 1], 6, 2, 192, 32, "fp8", "bf16", {}),
    ([1, 1, 1, 1], [129, 16, 500, 333], 16, 1, 256, 16, "int8", "bf16", {}),
    ([1, 1], [2500, 40], 40, 2, 64, 64, "fp8", "f32", {}),               # more than 16 queries of a head
    ([3, 0, 1, 5], [100, 50, 0, 5], 4, 2, 128, 32, "int8", "bf16", {}),   # a sequence without rows, one without tokens
    ([5, 2], [3, 90], 2, 1, 64, 16, "fp8", "bf16", {}),                  # rows before the first token
    ([1, 1], [700, 300], 8, 4, 128, 64, "int8", "bf16", {"window": 100}),
    ([40, 7], [40, 600], 4, 4, 64, 16, "int8", "f32", {"window": 33}),
    ([33], [33], 3, 1, 128, 32, "fp8", "bf16", {"causal": False}),
    ([19, 1], [400, 90], 12, 4, 192, 128, "int8", "f32", {"causal": False}),
    ([77], [177], 8, 2, 128, 64, "int8", "bf16", {}),
    ([130, 64, 1], [130, 200, 150], 6, 2, 128, 64, "fp8", "bf16", {}),
    ([150], [333], 5, 1, 64, 32, "int8", "f32", {}),
    ([65, 66], [65, 300], 2, 2, 256, 16, "fp8", "bf16", {}),
    ([90], [290], 4, 2, 256, 64, "int8", "f32", {"window": 70}),
    ([300, 5], [300, 129], 4, 1, 192, 64, "fp8", "bf16", {"window": 128}),
    ([257], [257], 16, 1, 128, 16, "int8", "bf16", {}),
]


@pytest.mark.parametrize("n,lengths,heads,kv,dim,block,fmt,dtype,how", CASES)
def test_attention_matches_the_reference(n, lengths, heads, kv, dim, block, fmt, dtype, how):
    p, table = filled(20, fmt, block, dim, kv, lengths)
    start = np.concatenate([[0], np.cumsum(n)])
    q = rows(30, sum(n), heads, dim, dtype, 2.0, fused=2)
    check_attention(p, start, lengths, table, q, how)
    check_attention(p, start, lengths, table, q.contiguous(), how, scale=0.3, lse=False)


def test_attention_of_prompts_among_single_tokens():
    """Sequences for the tile kernel and for the streaming one in one batch,
    long contexts split between workgroups, more of them than a wave has lanes."""
    rng = np.random.default_rng(3)
    lengths = [int(rng.integers(1, 40)) for _ in range(70)] + [1500, 700, 90]
    n = [1] * 40 + [0] * 20 + [3] * 10 + [1, 200, 90]
    lengths = [max(a, b) for a, b in zip(n, lengths)]
    p, table = filled(26, "int8", 32, 64, 1, lengths)
    start = np.concatenate([[0], np.cumsum(n)])
    for dtype in ("bf16", "f32"):
        check_attention(p, start, lengths, table, rows(8, sum(n), 2, 64, dtype), {})
    check_attention(p, start, lengths, table, rows(8, sum(n), 2, 64, "bf16"), {"window": 300})


def test_attention_over_many_sequences():
    """More sequences than a wave has lanes, uneven, with gaps."""
    rng = np.random.default_rng(7)
    lengths = rng.integers(0, 90, 150).tolist()
    n = [int(rng.integers(0, 3)) for _ in lengths]
    p, table = filled(21, "int8", 16, 64, 1, lengths)
    start = np.concatenate([[0], np.cumsum(n)])
    check_attention(p, start, lengths, table, rows(31, sum(n), 2, 64, "bf16"), {})
    # writing and reading find their sequences the same way
    want = K.read(p.host, np.concatenate([[0], np.cumsum(lengths)]), lengths, table)
    seqs = B.KVSequences(i32(np.concatenate([[0], np.cumsum(lengths)])), i32(lengths), i32(table), sum(lengths))
    got = B.nq_kv_read(p.dev, seqs, out_dtype=torch.float32)
    assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_attention_with_sharp_scores_and_uneven_scales(fmt):
    """Scores of several hundred, value scales over 2^60, zero blocks."""
    block, dim = 16, 64
    lengths = [150]
    p = Pair(8, 12, 1, block, dim, fmt)
    table = tables(9, 1, 10, 12)
    k, v = rows(1, 150, 1, dim, "f32", 20.0), rows(2, 150, 1, dim, "f32")
    for j, e in enumerate((0, -40, 20, 3, -7, 0, 1, -30, 12, 0)):
        v[16 * j:16 * j + 16] *= 2.0 ** e
    v[48:64] = 0
    k[96:112] = 0
    p.append([0, 150], lengths, table, k, v)
    for dtype in ("bf16", "f32"):
        q = rows(3, 20, 4, dim, dtype, 6.0)
        check_attention(p, [0, 20], lengths, table, q, {})
    # all values zero
    v[:] = 0
    p.append([0, 150], lengths, table, k, v)
    out = check_attention(p, [0, 20], lengths, table, rows(3, 20, 4, dim, "bf16"), {})
    assert not out.any()


@pytest.mark.parametrize("scale_of_q", [1e-30, 1e-6, 1e4, 3e37])
def test_attention_over_the_range_of_queries(scale_of_q):
    p, table = filled(22, "int8", 32, 128, 1, [70])
    q = rows(5, 2, 3, 128, "f32", 1.0) * scale_of_q
    check_attention(p, [0, 2], [70], table, q, {}, scale=min(0.1, 0.3 / scale_of_q))
    q[:, 1] = 0
    check_attention(p, [0, 2], [70], table, q, {}, scale=min(0.1, 0.3 / scale_of_q))


def test_a_row_of_nan_spoils_no_other():
    p, table = filled(23, "int8", 16, 64, 1, [50])
    q = rows(5, 6, 2, 64, "bf16")
    seqs = B.KVSequences(i32([0, 6]), i32([50]), i32(table), 6)
    want = B.nq_kv_attention(p.dev, seqs, q)
    q[2, 1] = float("nan")
    got = B.nq_kv_attention(p.dev, seqs, q)
    keep = torch.ones(6, 2, dtype=torch.bool)
    keep[2, 1] = False
    assert bits_equal(got.cpu()[keep], want.cpu()[keep])


def test_offsets_past_32_bits():
    """Blocks at the end of a cache of 2.5e9 bytes of keys and as many values."""
    heads, block, dim = 8, 128, 128
    blocks = 19100
    cache = B.KVCache(blocks, heads, block, dim, "int8")
    ids = [blocks - 1, 17, blocks - 2]
    table = np.array([ids], np.int32)
    n = 2 * block + 9
    k, v = rows(1, n, heads, dim, "bf16"), rows(2, n, heads, dim, "bf16")
    seqs = B.KVSequences(i32([0, n]), i32([n]), i32(table), n)
    B.nq_kv_append(cache, seqs, k, v)
    small = Pair(1, 3, heads, block, dim, "int8")
    local = np.array([[0, 1, 2]], np.int32)
    small.append([0, n], [n], local, k, v)
    for part in ("k", "v"):
        got = getattr(cache, part + "_scales")[ids].cpu().numpy()
        assert np.array_equal(got, getattr(small.host, part + "_scales"))
    back = B.nq_kv_read(cache, seqs, out_dtype=torch.float32)
    want = K.read(small.host, [0, n], [n], local)
    assert np.array_equal(back[0].cpu().numpy(), want[0]) and np.array_equal(back[1].cpu().numpy(), want[1])
    q = rows(3, 140, 16, dim, "bf16")
    a = B.nq_kv_attention(cache, B.KVSequences(i32([0, 140]), i32([n]), i32(table), 140), q)
    b = B.nq_kv_attention(small.dev, B.KVSequences(i32([0, 140]), i32([n]), i32(local), 140), q)
    assert bits_equal(a, b)


def test_streams_and_repeats_give_the_same_bits():
    """On a stream of its own, with tensors of that stream, and again: split
    contexts are joined in a fixed order."""
    lengths = [3000, 700]
    p, table = filled(24, "int8", 64, 128, 2, lengths)
    q = rows(5, 2, 8, 128, "bf16")
    seqs = B.KVSequences(i32([0, 1, 2]), i32(lengths), i32(table), 2)
    want = B.nq_kv_attention(p.dev, seqs, q)
    k, v = B.nq_kv_read(p.dev, seqs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = B.nq_kv_attention(p.dev, seqs, q, stream=s)
        k2, v2 = B.nq_kv_read(p.dev, seqs, stream=s)
        s.synchronize()
        assert bits_equal(got, want) and bits_equal(k, k2) and bits_equal(v, v2)


def test_serving_steps_replay_from_a_graph():
    """A step (lengths grow on the device, append, attention) captured once and
    replayed, against the same steps called one by one."""
    heads, kv, dim, block, batch, steps = 8, 2, 128, 32, 3, 5
    lengths = [40, 3, 95]
    outs = []
    for captured in (False, True):
        p, table = filled(25, "int8", block, dim, kv, lengths, wide=5)
        new = rows(6, steps * batch, heads + 2 * kv, dim, "bf16").view(steps, batch, heads + 2 * kv, dim)
        have = i32(lengths)
        seqs = B.KVSequences(i32([0, 1, 2, 3]), have, i32(table), batch)
        x = new[0].clone()
        q, k, v = x.split([heads, kv, kv], dim=1)
        out = torch.empty((batch, heads, dim), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(B.nq_kv_attention_workspace_bytes(p.dev, seqs, heads, torch.bfloat16), dtype=torch.uint8,
                         device="cuda")

        def step():
            have.add_(1)
            B.nq_kv_append(p.dev, seqs, k, v)
            B.nq_kv_attention(p.dev, seqs, q, out=out, workspace=ws)

        got = []
        if captured:
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                B.nq_kv_attention(p.dev, seqs, q, out=out, workspace=ws)     # loads the kernels
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
        for i in range(steps):
            x.copy_(new[i])
            if captured:
                g.replay()
            else:
                step()
            torch.cuda.synchronize()
            got.append(out.clone())
        outs.append(torch.stack(got))
    assert bits_equal(outs[0], outs[1])


def test_empty_calls_do_nothing():
    cache = B.KVCache(2, 1, 16, 64, "fp8")
    none = B.KVSequences(i32([0]), torch.zeros(0, dtype=torch.int32, device="cuda"),
                         torch.zeros((0, 1), dtype=torch.int32, device="cuda"), 0)
    x = torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    B.nq_kv_append(cache, none, x, x)
    k, v = B.nq_kv_read(cache, none)
    out = B.nq_kv_attention(cache, none, x)
    torch.cuda.synchronize()
    assert k.shape == (0, 1, 64) and out.shape == (0, 1, 64)
    # rows that no sequence has are left alone
    out = torch.full((4, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    seqs = B.KVSequences(i32([1, 1]), i32([0]), i32([[0]]), 4)
    B.nq_kv_attention(cache, seqs, torch.zeros_like(out), out=out)
    assert (out == 3).all()
