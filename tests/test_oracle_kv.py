"""Pins of the plain references of the key/value cache and of routing: the
properties that their contracts state, checked without the library."""
import numpy as np
import pytest

from oracle import kv as K
from oracle import moe as M


def test_e4m3_codes_round_trip_and_round_to_even():
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    again = K.encode(K.values(codes, "fp8").astype(np.float32), "fp8")
    assert np.array_equal(again, codes)
    pos = K.values(np.arange(127, dtype=np.uint8), "fp8")
    mid = (pos[1:] + pos[:-1]) / 2      # exact in float32
    even = np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(1, 127))
    assert np.array_equal(K.encode(mid.astype(np.float32), "fp8"), even.astype(np.uint8))
    assert K.encode(np.float32([1e9, -1e9]), "fp8").tolist() == [126, 254]


def _cache(fmt, blocks=4, heads=1, block=16, dim=64):
    return K.Cache(np.full((blocks, heads, block, dim), 77, np.uint8), np.full((blocks, heads), np.nan, np.float32),
                   np.full((blocks, heads, dim, block), 77, np.uint8), np.full((blocks, heads), np.nan, np.float32), fmt)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_a_block_written_at_once_is_within_half_a_step(fmt):
    rng = np.random.default_rng(0)
    c = _cache(fmt)
    x = rng.standard_normal((20, 1, 64)).astype(np.float32)
    table = np.array([[2, 0]], np.int32)
    K.append(c, [0, 20], [20], table, x, -x)
    k, v = K.read(c, [0, 20], [20], table)
    scale = np.where(np.arange(20) < 16, c.k_scales[2, 0], c.k_scales[0, 0])[:, None, None]
    # half a step: 1/2 for integers; half of 2^-3 of the value (E4M3), 2^-10 below the normal range
    step = 0.5 if fmt == "int8" else np.maximum(np.abs(x) / scale / 16, 2.0 ** -10)
    assert np.all(np.abs(k - x) <= scale * step * (1 + 1e-6))
    assert np.array_equal(v, -k)
    assert np.isnan(c.k_scales[1, 0]) and np.all(c.k_codes[3] == 77)     # untouched


def test_growing_scales_keep_old_values_within_one_step():
    """Largest magnitudes that creep up by 7 % a token: the case in which
    scales that grew to a / qmax each time would let old codes drift."""
    rng = np.random.default_rng(1)
    c = _cache("int8")
    table = np.array([[1]], np.int32)
    x = rng.uniform(-1, 1, (16, 1, 64)).astype(np.float32) * (1.07 ** np.arange(16, dtype=np.float32))[:, None, None]
    for t in range(16):
        K.append(c, [0, 1], [t + 1], table, x[t:t + 1], x[t:t + 1])
    k, _ = K.read(c, [0, 16], [16], table)
    assert np.all(np.abs(k - x) <= c.k_scales[1, 0] * (1 + 1e-6))
    assert c.k_scales[1, 0] < 2 * np.abs(x).max() / 127


def test_attention_of_equal_keys_is_the_mean_of_the_visible_values():
    c = _cache("int8", dim=64)
    c.k_scales[:], c.v_scales[:] = 1, 1
    c.k_codes[:] = 130
    c.v_codes[:] = (128 + np.arange(16)).astype(np.uint8)[None, None, None, :]
    table = np.array([[0, 1]], np.int32)
    got = K.attention(c, [0, 3], [20], table, np.ones((3, 1, 64)), 0.1, window=6)
    for r, p in enumerate((17, 18, 19)):
        assert np.allclose(got["out"][r, 0], np.mean([t % 16 for t in range(p - 5, p + 1)]))
        assert np.isclose(got["lse"][r, 0], 0.1 * 128 + np.log(6))
    none = K.attention(c, [0, 2], [0], table, np.ones((2, 1, 64)), 0.1)
    assert np.all(none["out"] == 0) and np.all(np.isneginf(none["lse"]))


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_routing_gradient_matches_differences(kind, renormalise):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((7, 24))
    ids, _ = M.route(x, kind, 4, groups=3, top_groups=2, group_best=2, renormalise=renormalise, scale=2.5)
    dw = rng.standard_normal((7, 4))
    g = M.grad(x, kind, ids, dw, renormalise, 2.5)
    d = M.grad_by_differences(x, kind, ids, dw, renormalise, 2.5)
    assert np.max(np.abs(g - d)) < 1e-8     # step^2 and rounding / step, both about 1e-10


def test_routing_takes_the_lowest_index_among_equals():
    ids, w = M.route(np.array([[1.0, 2.0, 2.0, 2.0, 0.0, 1.0]]), "softmax", 4)
    assert ids.tolist() == [[1, 2, 3, 0]]
    ids, _ = M.route(np.array([[1.0, 0.0, 1.0, 0.0, 1.0, 5.0]]), "sigmoid", 2, groups=3, top_groups=2, group_best=1)
    assert ids.tolist() == [[5, 0]]
    ids, w = M.route(np.full((1, 4), -np.inf), "softmax", 2, renormalise=True)
    assert ids.tolist() == [[0, 1]] and np.all(w == 0)


@pytest.mark.parametrize("best,first", [(1, 0), (2, 1)])
def test_a_nan_key_adds_nothing_to_its_group(best, first):
    """{0.9, 0.1, NaN, 0.2} has the best single key, but with its second best only 1.1 against 1.3."""
    keys = np.array([0.9, 0.1, np.nan, 0.2, 0.7, 0.6, 0.0, 0.0])
    ids, _ = M.route(np.full((1, 8), -1000.0), "sigmoid", 1, bias=keys, groups=2, top_groups=1, group_best=best)
    assert ids.tolist() == [[4 * first]]


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_number_that_is_none_takes_its_block_along(bad):
    c = _cache("fp8", heads=2)
    table = np.array([[2, 0]], np.int32)
    x = np.random.default_rng(4).standard_normal((20, 2, 64)).astype(np.float32)
    K.append(c, [0, 5], [5], table, x[:5], x[:5])
    y = x[5:9].copy()
    y[1, 1, 3] = bad
    K.append(c, [0, 4], [9], table, x[5:9], y)
    K.append(c, [0, 11], [20], table, x[9:], x[9:])
    k, v = K.read(c, [0, 20], [20], table)
    assert np.isfinite(k).all() and np.isnan(v[:16, 1]).all() and np.isfinite(v[:16, 0]).all() and np.isfinite(v[16:]).all()
    K.append(c, [0, 20], [20], table, x, x)
    assert np.isfinite(K.read(c, [0, 20], [20], table)[1]).all()
