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
