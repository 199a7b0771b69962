"""The example decoder layer (cache, attention, routing and products together)
against the same layer in plain float32 on dequantized weights and on the
cache's own values."""
import pytest
import torch

from group_wise_affine_quantize_amd import _binding as B
from group_wise_affine_quantize_amd.decoder_layer import DecoderLayer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    B.load_library()


def plain(layer, x, positions, cache, table, start, lengths, ids):
    """The layer with the experts `ids`, keys and values as the cache holds them."""
    f = lambda w, bits=4: B.nq_dequantize(*w, layer.GROUP, bits, out_dtype=torch.float32)
    norm = lambda t: DecoderLayer._norm(t.to(torch.bfloat16)).float()
    h, kv, d = layer.heads, layer.kv_heads, layer.head_dim
    fused = (norm(x) @ f(layer.qkv).t()).view(len(x), h + 2 * kv, d)
    q = layer._rotate(fused[:, :h], positions)
    out = torch.empty(len(x), h, d, device="cuda")
    for b, n in enumerate(lengths):
        one = B.KVSequences(torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                            torch.tensor([n], dtype=torch.int32, device="cuda"), table[b:b + 1], n)
        k, v = B.nq_kv_read(cache, one, out_dtype=torch.float32)
        for r in range(start[b], start[b + 1]):
            p = n - start[b + 1] + r
            kk, vv = (t[:p + 1].repeat_interleave(h // kv, 1) for t in (k, v))
            w = torch.softmax((q[r][None] * kk).sum(-1) * d ** -0.5, 0)
            out[r] = (w[..., None] * vv).sum(0)
    x = x.float() + out.reshape(len(x), -1) @ f(layer.out).t()
    z = norm(x)
    p = torch.softmax(z @ f(layer.gate, 8).t(), -1).gather(1, ids.long())
    p = p / p.sum(-1, keepdim=True)
    up, down = f(layer.up), f(layer.down)
    for r in range(len(x)):
        for j, e in enumerate(ids[r].tolist()):
            a, b = (up[e] @ z[r]).chunk(2)
            x[r] += p[r, j] * (down[e] @ (torch.nn.functional.silu(a) * b))
    return x


@pytest.mark.parametrize("format", ["int8", "fp8"])
def test_prompts_then_steps(format):
    layer = DecoderLayer(hidden=256, heads=4, kv_heads=2, head_dim=64, experts=8, expert_hidden=128, top_k=2)
    prompts, wide = [19, 5, 40], 4
    cache = layer.new_cache(12, 16, format)
    table = torch.randperm(12, generator=torch.Generator().manual_seed(1))[:12].view(3, wide).to(torch.int32).cuda()
    lengths = torch.tensor(prompts, dtype=torch.int32).cuda()
    start = [0, 19, 24, 64]
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn(64, 256, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.cat([torch.arange(n) for n in prompts]).cuda()
    seqs = B.KVSequences(torch.tensor(start, dtype=torch.int32).cuda(), lengths, table, 64)
    y, ids = layer.forward(x, pos, cache, seqs)
    want = plain(layer, x, pos, cache, table, start, prompts, ids)
    # bf16 activations at half a dozen places, each 2^-9 of values up to the largest
    assert (y.float() - want).abs().max() <= 2.0 ** -5 * want.abs().max()

    step = B.KVSequences(torch.arange(4, dtype=torch.int32, device="cuda"), lengths, table, 3)
    x = y[[18, 23, 63]]
    for i in range(3):
        lengths += 1
        y, ids = layer.forward(x, lengths - 1, cache, step)
        want = plain(layer, x, lengths - 1, cache, table, [0, 1, 2, 3], lengths.tolist(), ids)
        assert (y.float() - want).abs().max() <= 2.0 ** -5 * want.abs().max()
        x = DecoderLayer._norm(y)
