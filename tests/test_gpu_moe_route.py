"""Expert routing on the GPU against the plain reference (oracle/moe.py)."""
import numpy as np
import pytest
import torch

from gpu_helpers import bits_equal
from group_wise_affine_quantize_amd import _binding as B
from oracle import moe as M

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    B.load_library()


def logits_of(seed, tokens, experts, dtype, sigma=1.5):
    x = np.random.default_rng(seed).standard_normal((tokens, experts)).astype(np.float32) * sigma
    return torch.from_numpy(x).cuda().to(DT[dtype])


def f64(t):
    return t.double().cpu().numpy()


# tokens, experts, top_k, score, dtype, router options, bias
CASES = [
    (1, 1, 1, "softmax", "f32", {}, False),
    (1, 8, 2, "softmax", "bf16", {"renormalise": True}, False),
    (5, 32, 4, "sigmoid", "bf16", {"scale": 2.5}, True),
    (17, 64, 6, "softmax", "f32", {}, True),
    (33, 65, 7, "softmax", "f32", {"renormalise": True}, False),
    (16, 60, 5, "sigmoid", "f32", {"groups": 4, "top_groups": 2, "group_best": 2, "renormalise": True}, False),
    (9, 128, 32, "sigmoid", "bf16", {"renormalise": True}, False),
    (40, 256, 8, "sigmoid", "f32", {"groups": 8, "top_groups": 4, "group_best": 2, "renormalise": True, "scale": 2.5},
     True),
    (21, 160, 6, "softmax", "f32", {"groups": 8, "top_groups": 3, "group_best": 1, "scale": 16.0}, False),
    (3, 257, 3, "softmax", "bf16", {}, False),
    (6, 512, 10, "sigmoid", "f32", {"groups": 16, "top_groups": 1, "group_best": 1}, True),
    (2, 1000, 32, "softmax", "f32", {"renormalise": True}, False),
    (4, 1024, 8, "sigmoid", "f32", {"groups": 64, "top_groups": 8, "group_best": 2}, True),
    (3, 48, 12, "softmax", "f32", {"groups": 48, "top_groups": 12}, False),     # groups of one expert
]


@pytest.mark.parametrize("tokens,experts,top_k,score,dtype,options,biased", CASES)
def test_route_and_gradient_match_the_reference(tokens, experts, top_k, score, dtype, options, biased):
    options = {"groups": 1, "top_groups": 1, "group_best": 1, "renormalise": False, "scale": 1.0, **options}
    router = B.MoERouter(experts, top_k, score=score, **options)
    x = logits_of(experts + tokens, tokens, experts, dtype)
    bias = torch.from_numpy(np.random.default_rng(5).integers(-50, 50, experts).astype(np.float32) / 64).cuda() \
        if biased else None
    ids, w = B.nq_moe_route(router, x, bias=bias)
    want_ids, want_w = M.route(f64(x), score, top_k, None if bias is None else f64(bias), **options)
    # the order may only differ where keys are equal to 32-bit accuracy; these seeds have no such pair
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    # p: an exponential, a quotient and a sum over the experts; renormalised, a sum and a quotient more
    tol = (experts + top_k + 16) * 2.0 ** -24
    assert np.all(np.abs(f64(w) - want_w) <= tol * np.abs(want_w))

    dw = torch.from_numpy(np.random.default_rng(6).standard_normal((tokens, top_k)).astype(np.float32)).cuda()
    dx = B.nq_moe_route_grad(router, x, ids, dw)
    want = M.grad(f64(x), score, want_ids, f64(dw), options["renormalise"], options["scale"])
    differences = M.grad_by_differences(f64(x), score, want_ids, f64(dw), options["renormalise"], options["scale"])
    # p's tolerance on each of the formula's terms (the largest stands for all), and the output's rounding
    p = M.scores(f64(x), score)
    pk = np.take_along_axis(p, want_ids, -1)
    total = pk.sum(-1, keepdims=True) if options["renormalise"] else 1.0
    terms = np.abs(f64(dw)).sum(-1, keepdims=True) * abs(options["scale"]) / total
    spread = p if score == "softmax" and not options["renormalise"] else np.where(want != 0, p, 0)
    bound = 4 * tol * terms * spread + np.abs(want) * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -22)
    assert np.all(np.abs(f64(dx) - want) <= bound)
    assert np.all(np.abs(f64(dx) - differences) <= bound + 1e-8 * max(1.0, abs(options["scale"])))
    assert dx.dtype == x.dtype and dx.shape == x.shape


def test_equal_keys_take_the_lowest_index():
    x = torch.from_numpy(np.random.default_rng(1).integers(0, 3, (50, 96)).astype(np.float32)).cuda()
    x[0] = 0.0
    x[1, ::2] = -0.0
    for options in ({}, {"groups": 6, "top_groups": 2, "group_best": 1}, {"groups": 6, "top_groups": 3, "group_best": 2}):
        for bias in (None, torch.zeros(96, device="cuda")):
            router = B.MoERouter(96, 9, score="sigmoid", **options)
            ids, _ = B.nq_moe_route(router, x, bias=bias)
            o = {"top_groups": 1, **options}
            want, _ = M.route(f64(x), "sigmoid", 9, None if bias is None else f64(bias), **o)
            assert np.array_equal(ids.cpu().numpy(), want)


def test_order_without_a_bias_is_the_logits():
    """Logits whose scores are equal in 32 bits are still told apart."""
    x = torch.arange(30, 62, device="cuda").float()[None]
    ids, w = B.nq_moe_route(B.MoERouter(32, 3, score="sigmoid"), x)
    assert ids.tolist() == [[31, 30, 29]] and w.tolist() == [[1.0, 1.0, 1.0]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_masked_and_nan_logits(score, renormalise):
    low = float(torch.finfo(torch.bfloat16).min)
    x = torch.full((4, 20), float("-inf"), device="cuda", dtype=torch.bfloat16)
    x[1, 7], x[1, 3] = 1.0, 2.0
    x[2] = low
    x[2, 19] = 0.5
    x[3, ::2] = float("nan")
    x[3, 1] = 0.0
    router = B.MoERouter(20, 3, score=score, renormalise=renormalise)
    ids, w = B.nq_moe_route(router, x)
    assert ids.tolist()[:3] == [[0, 1, 2], [3, 7, 0], [19, 0, 1]]
    assert ids.tolist()[3][0] == 1 and len(set(ids.tolist()[3])) == 3
    assert w[0].tolist() == [0.0, 0.0, 0.0]
    clean = f64(x[1:3])
    want = M.weights(clean, score, ids[1:3].cpu().numpy().astype(np.int64), renormalise, 1.0)
    assert np.allclose(f64(w[1:3]), want, rtol=1e-5, atol=0)
    dx = B.nq_moe_route_grad(router, x[:3], ids[:3], torch.ones((3, 3), device="cuda"))
    assert torch.isfinite(dx).all() and not dx[0].any()


def test_row_strides_streams_and_replays():
    wide = logits_of(9, 37, 200, "f32")
    router = B.MoERouter(64, 4, renormalise=True)
    dw = torch.randn(37, 4, device="cuda")
    for first in (0, 3, 64):        # aligned to 16 bytes and not
        x = wide[:, first:first + 64]
        ids, w = B.nq_moe_route(router, x)
        dx = B.nq_moe_route_grad(router, x, ids, dw)
        ids2, w2 = B.nq_moe_route(router, x.contiguous())
        assert torch.equal(ids, ids2) and bits_equal(w, w2)
        assert bits_equal(dx, B.nq_moe_route_grad(router, x.contiguous(), ids, dw))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ids3, w3 = B.nq_moe_route(router, x, stream=s)
    s.synchronize()
    assert torch.equal(ids, ids3) and bits_equal(w, w3)
    g = torch.cuda.CUDAGraph()
    x = x.clone()
    with torch.cuda.graph(g):
        ids4, w4 = B.nq_moe_route(router, x)
        dx4 = B.nq_moe_route_grad(router, x, ids4, dw)
    for i in range(4):
        x.copy_(logits_of(40 + i, 37, 64, "f32"))
        g.replay()
        torch.cuda.synchronize()
        ids5, w5 = B.nq_moe_route(router, x)
        assert torch.equal(ids4, ids5) and bits_equal(w4, w5)
        assert bits_equal(dx4, B.nq_moe_route_grad(router, x, ids5, dw))


def test_gradient_skips_ids_past_the_experts():
    x = logits_of(3, 6, 24, "f32")
    router = B.MoERouter(24, 3, score="sigmoid")
    ids, _ = B.nq_moe_route(router, x)
    dw = torch.ones((6, 3), device="cuda")
    bad = ids.clone()
    bad[:, 1] = -1
    bad[0, 2] = 24
    got = B.nq_moe_route_grad(router, x, bad, dw)
    dw[:, 1] = 0
    dw[0, 2] = 0
    assert bits_equal(got, B.nq_moe_route_grad(router, x, ids, dw))


@pytest.mark.parametrize("experts,top_k,options", [(20, 3, {}), (200, 8, {}), (200, 9, {}),
                                                   (256, 8, {"groups": 8, "top_groups": 2, "group_best": 2})])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_logits_and_biases_count_as_minus_infinity(experts, top_k, options, score):
    """Also where keys are scores plus a bias."""
    x = logits_of(7, 12, experts, "f32")
    x[:, ::3] = float("nan")
    x[3, 1::3] = float("-inf")
    bias = torch.arange(experts, device="cuda").float() % 7 / 64
    options = {"groups": 1, "top_groups": 1, "group_best": 1, **options}
    router = B.MoERouter(experts, top_k, score=score, **options)
    for b in (None, bias):
        ids, w = B.nq_moe_route(router, x, bias=b)
        want, ww = M.route(x.double().cpu().numpy(), score, top_k, None if b is None else f64(b), **options)
        assert np.array_equal(ids.cpu().numpy(), want)
        assert np.all(np.abs(f64(w) - ww) <= (experts + top_k + 16) * 2.0 ** -24 * np.abs(ww))
    bias[5] = float("nan")
    ids, _ = B.nq_moe_route(router, torch.zeros_like(x), bias=bias)
    assert not (ids == 5).any()


# group sizes that a power of two of lanes holds, and others; more than 256 experts
@pytest.mark.parametrize("experts,groups,top_k", [(32, 4, 3), (60, 4, 3), (120, 8, 9), (256, 8, 8), (480, 16, 5), (1024, 64, 8)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_biases_add_nothing_to_a_group(experts, groups, top_k, best, score):
    """A NaN key counts as -infinity in its group's score too: it is not the second best, and does not stand in for it."""
    options = {"groups": groups, "top_groups": 2, "group_best": best}
    x = logits_of(experts, 25, experts, "f32")
    size = experts // groups
    bias = torch.arange(experts, device="cuda").float() % 7 / 64
    bias[1::3] = float("nan")
    bias[:size] = float("nan")                      # a group without any key,
    bias[size:2 * size - 1] = float("nan")          # and one with a single one
    bias[-size:-1:2] = float("-inf")
    router = B.MoERouter(experts, top_k, score=score, **options)
    ids, w = B.nq_moe_route(router, x, bias=bias)
    want, ww = M.route(f64(x), score, top_k, f64(bias), **options)
    assert np.array_equal(ids.cpu().numpy(), want)
    assert np.all(np.abs(f64(w) - ww) <= (experts + top_k + 16) * 2.0 ** -24 * np.abs(ww))


def test_the_second_best_of_a_group_is_a_number():
    """{0.9, 0.1, NaN, 0.2} has 1.1, not 1.8, and {0.7, 0.6, 0, 0} is the better one."""
    keys = torch.tensor([0.9, 0.1, float("nan"), 0.2, 0.7, 0.6, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0], device="cuda")
    x = torch.full((1, 12), -100.0, device="cuda")      # sigmoids of zero: the keys are the bias
    ids, _ = B.nq_moe_route(B.MoERouter(12, 2, score="sigmoid", groups=3, top_groups=1, group_best=2), x, bias=keys)
    assert ids.tolist() == [[4, 5]]
    # the same among 480 experts, whose groups of 30 no power of two of lanes holds
    x = torch.full((1, 480), -100.0, device="cuda")
    bias = torch.zeros(480, device="cuda")
    bias[:4], bias[30:34] = keys[:4], keys[4:8]
    ids, _ = B.nq_moe_route(B.MoERouter(480, 2, score="sigmoid", groups=16, top_groups=1, group_best=2), x, bias=bias)
    assert ids.tolist() == [[30, 31]]


def test_more_tokens_than_one_launch_has_threads_for():
    """2^28 tokens and some: at 16 lanes to a token their threads pass 32 bits."""
    tokens = (1 << 28) + 40
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB of memory")
    x = (torch.arange(tokens, device="cuda") % 7).to(torch.bfloat16)[:, None]
    router = B.MoERouter(1, 1, score="sigmoid")
    ids = torch.full((tokens, 1), 9, dtype=torch.int32, device="cuda")
    w = torch.full((tokens, 1), 9.0, device="cuda")
    B.nq_moe_route(router, x, ids=ids, weights=w)
    assert not ids.any()
    want, at = B.nq_moe_route(router, x[:7])[1], torch.arange(tokens, device="cuda") % 7
    assert torch.equal(w[:, 0], want[:, 0][at])
    dx = torch.full((tokens, 1), 9.0, dtype=torch.bfloat16, device="cuda")
    B.nq_moe_route_grad(router, x, ids, w, dlogits=dx)
    want = B.nq_moe_route_grad(router, x[:7], ids[:7], w[:7])
    assert torch.equal(dx[:, 0], want[:, 0][at])
