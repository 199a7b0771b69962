"""Attention behind shared prefixes on the GPU in batches as servers have them:
block tables that are wider than the contexts in them, a prompt's chunk among
single tokens, one prompt behind a prefix.  References, bounds and ways to make a cache are
test_gpu_kv_shared.py's and test_gpu_kv.py's."""
import numpy as np
import pytest
import torch

from gpu_helpers import bits_equal
from group_wise_affine_quantize_amd import _binding as B
from test_gpu_kv import filled, gpu, i32, rows  # noqa: F401  (gpu: the fixture)
from test_gpu_kv_shared import attend, check, starts

pytestmark = pytest.mark.gpu


def widened(table, by):
    """The same table with `by` times the columns, of which the rest name no block."""
    return np.concatenate([table, np.full((len(table), table.shape[1] * (by - 1)), -1, np.int32)], 1)


# prefix lengths, sequences of each, own lengths, rows of each sequence, q heads, kv heads, dim, block, format, dtype:
# prefixes by tiles and streamed, one and several, own tokens cut up and whole, both passes in one launch
WIDE = [
    ([16400], [40], [(37 * i) % 300 + 1030 for i in range(40)], 1, 16, 2, 128, 64, "int8", "bf16"),
    ([6000, 9100], [20, 22], [(37 * i) % 300 + 1030 for i in range(42)], 3, 8, 2, 128, 32, "fp8", "bf16"),
    ([9000], [40], [(53 * i) % 300 + 1030 for i in range(40)], 2, 16, 2, 128, 128, "int8", "f32"),
    ([1100, 1300], [2, 1], [1300, 4000, 1100], 1, 4, 4, 64, 16, "int8", "bf16"),
]


@pytest.mark.parametrize("prefixes,behind,lengths,new,heads,kv,dim,block,fmt,dtype", WIDE)
def test_tables_wider_than_their_contexts(prefixes, behind, lengths, new, heads, kv, dim, block, fmt, dtype):
    """Work is dealt by lengths: 32 times the columns change no bit of the results (nor does what the workspace held)."""
    p, table = filled(150, fmt, block, dim, kv, lengths + prefixes)
    n = len(lengths)
    start = starts([new] * n)
    q = rows(151, new * n, heads, dim, dtype, 2.0)
    own, prefix = (start, lengths, table[:n]), (start[starts(behind)], prefixes, table[n:])
    out, lse = attend(p, prefix, own, q)
    check(p, prefix, own, q, out, lse)
    for by in (4, 32):
        wide = [(s, l, widened(t, by)) for s, l, t in (prefix, own)]
        seqs = [B.KVSequences(i32(s), i32(l), i32(t), q.shape[0]) for s, l, t in wide]
        need = B.nq_kv_attention_shared_workspace_bytes(p.dev, *seqs, heads, q.dtype)
        got = attend(p, *wide, q, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
        assert bits_equal(out, got[0]) and bits_equal(lse, got[1])


@pytest.mark.parametrize("chunk,singles,heads,kv,dim,block,fmt,dtype", [(300, 120, 16, 1, 64, 32, "int8", "bf16"),
                                                                      (520, 130, 8, 1, 128, 64, "fp8", "f32")])
@pytest.mark.parametrize("at", [0, 60])
def test_a_long_chunk_among_single_tokens(chunk, singles, heads, kv, dim, block, fmt, dtype, at):
    """Long and short sequences take a kernel each, wherever in the batch the long one is; some rows without a prefix."""
    n, lengths = [1] * singles, [(7 * i) % 90 + 1 for i in range(singles)]
    n.insert(at, chunk), lengths.insert(at, chunk + 45)
    p, table = filled(160, fmt, block, dim, kv, lengths + [500])
    start = starts(n)
    q = rows(161, sum(n), heads, dim, dtype, 2.0)
    prefix, own = ([0, start[singles - 10]], [500], table[-1:]), (start, lengths, table[:-1])
    out, lse = attend(p, prefix, own, q, fill=7.0)
    check(p, prefix, own, q, out, lse)


@pytest.mark.parametrize("n,length,prefix", [(150, 150, 300), (150, 2000, 1000), (40, 900, 65), (65, 10, 64)])
@pytest.mark.parametrize("heads,kv,dim,fmt,dtype", [(8, 2, 128, "int8", "bf16"), (2, 1, 64, "fp8", "f32"), (4, 2, 256, "int8", "bf16")])
def test_one_prompt_behind_a_prefix(n, length, prefix, heads, kv, dim, fmt, dtype):
    """Rows see their own tokens up to themselves, cut up between workgroups where there are many, and all of the prefix."""
    p, table = filled(170, fmt, 32, dim, kv, [length, prefix])
    q = rows(171, n, heads, dim, dtype, 2.0, fused=1)
    before, own = ([0, n], [prefix], table[1:]), ([0, n], [length], table[:1])
    out, lse = attend(p, before, own, q, fill=7.0)
    check(p, before, own, q, out, lse)
