"""The example decoder layer behind a shared prefix against the same layer with
the prefix's blocks repeated at the head of every sequence's table: the same
keys and values, so the same output up to the order of the attention's sums."""
import pytest
import torch

from group_wise_affine_quantize_amd import _binding as B
from group_wise_affine_quantize_amd import decoder_layer
from group_wise_affine_quantize_amd.decoder_layer import DecoderLayer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    B.load_library()


def i32(a):
    return torch.tensor(a, dtype=torch.int32).cuda()


@pytest.mark.parametrize("format", ["int8", "fp8"])
def test_prompts_and_steps_behind_a_shared_prefix(format):
    layer = DecoderLayer(hidden=256, heads=4, kv_heads=2, head_dim=64, experts=8, expert_hidden=128, top_k=2)
    block, system, prompts = 16, 48, [19, 5, 40]
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x0 = torch.randn(system, 256, generator=g, device="cuda").to(torch.bfloat16)
    x1 = torch.randn(sum(prompts), 256, generator=g, device="cuda").to(torch.bfloat16)
    steps = torch.randn(3, 3, 256, generator=g, device="cuda").to(torch.bfloat16)
    start = [0, 19, 24, 64]
    positions = torch.cat([torch.arange(n) for n in prompts]).cuda() + system
    out = []
    for shared in (True, False):
        cache = layer.new_cache(3 + 12, block, format)
        head, own = i32([[14, 0, 7]]), i32([[1, 2, 3, 4], [5, 6, 8, 9], [10, 11, 12, 13]])
        layer.forward(x0, torch.arange(system, device="cuda"), cache, B.KVSequences(i32([0, system]), i32([system]), head, system))
        extra = 0 if shared else system
        table = own if shared else torch.cat([head.expand(3, 3), own], 1).contiguous()
        lengths = i32(prompts) + extra
        before = lambda rows: B.KVSequences(i32([0, rows]), i32([system]), head, rows) if shared else None
        got = [layer.forward(x1, positions, cache, B.KVSequences(i32(start), lengths, table, 64), before(64))]
        one = B.KVSequences(i32([0, 1, 2, 3]), lengths, table, 3)
        for x in steps:
            lengths += 1
            got.append(layer.forward(x, lengths - extra + system - 1, cache, one, before(3)))
        out.append((torch.cat([y for y, _ in got]).float(), torch.cat([ids for _, ids in got])))
    (a, ids_a), (b, ids_b) = out
    same = (ids_a == ids_b).all(-1)
    assert same.float().mean() >= 0.9       # scores a rounding apart may choose differently
    # bf16 activations at half a dozen places, each 2^-9 of values up to the largest
    assert (a - b)[same].abs().max() <= 2.0 ** -5 * b.abs().max()


def test_the_example_runs(capsys):
    decoder_layer.main()
    assert "us a step" in capsys.readouterr().out
