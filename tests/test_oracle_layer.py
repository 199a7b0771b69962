"""The plain references of oracle/layer.py, pinned by hand-worked values, by
identities and by differences."""
import numpy as np
import pytest

from oracle import layer as L


def test_norm_by_hand():
    h, y = np.array([[1.0, 2.0, 2.0, 4.0]]), np.array([[3.0, -3.0, 3.0, 3.0]])
    post, gate, pre = np.array([1.0, 2.0, 3.0, 4.0]), np.array([1.0, 0.0, -1.0, 2.0]), np.array([1.0, 1.0, 1.0, 0.5])
    # the norm of y is (1, -1, 1, 1); u = (2, -3, 4, 5) with offset 1; h + 2 * gate * u
    h_out, z = L.block_norm(h, y, post, gate, pre, scale=2.0, offset=1.0, eps=0.0)
    assert np.allclose(h_out, [[5.0, 2.0, -6.0, 24.0]], rtol=1e-15)
    r = np.sqrt((25 + 4 + 36 + 576) / 4)
    assert np.allclose(z, np.array([[10.0, 4.0, -12.0, 36.0]]) / r, rtol=1e-15)
    # without a block, z is the norm of h; eps below the mean square
    _, z = L.block_norm(h, pre=np.ones(4), eps=2.75)
    assert np.allclose(z, h / 3.0, rtol=1e-15)


@pytest.mark.parametrize("post,gates,pre,dh,dz", [(1, 0, 1, 1, 1), (1, 1, 1, 1, 1), (1, 3, 1, 0, 1), (0, 6, 1, 1, 1),
                                                  (1, 6, 0, 1, 0), (0, 0, 1, 1, 1)])
def test_norm_gradient_by_differences(post, gates, pre, dh, dz):
    rng = np.random.default_rng(post + 10 * gates)
    rows, dim, o = 6, 5, dict(scale=0.7, offset=0.25, eps=1e-3)
    p = {"h": rng.standard_normal((rows, dim)), "y": rng.standard_normal((rows, dim)),
         "post": rng.standard_normal(dim) if post else None,
         "gate": rng.standard_normal((gates, dim) if gates != 1 else dim) if gates else None,
         "pre": rng.standard_normal(dim) if pre else None}
    a, b = rng.standard_normal((2, rows, dim))

    def loss(q):
        h_out, z = L.block_norm(**q, **o)
        return (a * h_out).sum() * dh + ((b * z).sum() if pre and dz else 0.0)

    h_out, _ = L.block_norm(**p, **o)
    got = L.block_norm_grad(h_out, p["y"], a if dh else None, b if dz else None, p["post"], p["gate"], p["pre"], **o)
    for name, g in zip(("h", "y", "post", "gate", "pre"), got):
        if p[name] is None or (name == "pre" and not dz):
            assert g is None
            continue
        assert g.shape == p[name].shape
        for i in np.ndindex(g.shape):
            q = [{**p, name: p[name].copy()} for _ in range(2)]
            q[0][name][i] += 1e-5
            q[1][name][i] -= 1e-5
            assert abs((loss(q[0]) - loss(q[1])) / 2e-5 - g[i]) < 1e-8 * (1 + abs(g[i]))


def test_rope_by_hand():
    x = np.array([[[1.0, 0.0, 0.0, 2.0, 9.0]]])
    quarter = np.pi / 2
    # halves: pairs (0, 2) and (1, 3); a quarter turn and a half turn
    out = L.rope(x, np.array([[1], [1]]), [quarter, 2 * quarter], [0, 1])
    assert np.allclose(out, [[[0.0, 0.0, 1.0, -2.0, 9.0]]], atol=1e-15)
    # neighbours: (1, 0) by a quarter turn, (0, 2) by three
    out = L.rope(x, np.array([[1], [3]]), [quarter, quarter], [0, 1], layout="pairs", scale=2.0)
    assert np.allclose(out, [[[0.0, 2.0, 4.0, 0.0, 9.0]]], atol=1e-15)


@pytest.mark.parametrize("layout", ["halves", "pairs"])
def test_rope_gradient_is_the_adjoint(layout):
    rng = np.random.default_rng(1)
    x, d = rng.standard_normal((2, 7, 3, 10))
    p, freq, axis = rng.integers(-50, 50, (3, 7)), rng.random(4), [0, 2, 1, 2]
    fwd = L.rope(x, p, freq, axis, layout, 1.3)
    back = L.rope(d, p, freq, axis, layout, 1.3, back=True)
    assert abs((fwd * d)[..., :8].sum() - (x * back)[..., :8].sum()) < 1e-12
    assert np.array_equal(fwd[..., 8:], x[..., 8:])
    # lengths are kept, and turning by a relative angle depends on the distance alone
    assert np.allclose((fwd[..., :8] ** 2).sum(-1), 1.69 * (x[..., :8] ** 2).sum(-1))


def test_sort_by_hand():
    ids = np.array([[2, 0], [7, 2], [0, 2]], np.uint32)
    starts, place, token, expert = L.moe_sort(ids, 4)
    assert starts.tolist() == [0, 2, 2, 5, 5]
    assert place.tolist() == [[2, 0], [5, 3], [1, 4]]
    assert token.tolist() == [0, 2, 0, 1, 2, 1] and expert.tolist() == [0, 0, 2, 2, 2, 7]


def test_moving_is_linear_and_its_gradient_the_adjoint():
    rng = np.random.default_rng(2)
    ids = rng.integers(0, 6, (9, 3)).astype(np.uint32)      # 5 is dropped
    starts, place, _, _ = L.moe_sort(ids, 5)
    kept = starts[-1]
    x, dy = rng.standard_normal((2, 9, 4))
    ys, dxs, w = rng.standard_normal((27, 4)), rng.standard_normal((27, 4)), rng.standard_normal((9, 3))
    xs = L.moe_dispatch(x, place, kept)
    assert np.all(xs[kept:] == 0)
    assert abs((xs * dxs).sum() - (x * L.moe_combine(dxs, place, kept)).sum()) < 1e-12
    dys, dw = L.moe_combine_grad(dy, ys, place, kept, w)
    y = L.moe_combine(ys, place, kept, w)
    # linear in ys and in the weights
    assert abs((y * dy).sum() - (dys * ys).sum()) < 1e-12 and abs((y * dy).sum() - (dw * w).sum()) < 1e-12
    assert np.all(dys[kept:] == 0) and np.all(dw[ids >= 5] == 0)


def test_shared_attention_is_attention_over_the_joined_tokens():
    """A prefix of whole blocks can also be had by repeating its blocks in every sequence's table."""
    from oracle import kv as K
    rng = np.random.default_rng(4)
    cache = K.Cache(rng.integers(0, 256, (9, 2, 4, 8), dtype=np.uint8), rng.random((9, 2)).astype(np.float32),
                    rng.integers(0, 256, (9, 2, 8, 4), dtype=np.uint8), rng.random((9, 2)).astype(np.float32), "int8")
    q = rng.standard_normal((5, 4, 8))
    start, lengths, table = [0, 1, 3, 5], [3, 6, 2], np.array([[2, 0], [3, 4], [5, 0]])
    # rows 1 .. 4 (the second and third sequence) behind blocks 7 and 8
    for causal in (True, False):
        got = K.attention_shared(cache, [1, 5], [8], np.array([[7, 8]]), start, lengths, table, q, 0.01, causal)
        want = K.attention(cache, start, [3, 14, 10], np.array([[2, 0, 0, 0], [7, 8, 3, 4], [7, 8, 5, 0]]), q, 0.01, causal)
        for name in want:
            assert np.allclose(got[name], want[name], rtol=1e-13), name
