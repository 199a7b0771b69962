"""Example: one quantized mixture-of-experts decoder layer, served from an
8-bit key/value cache.

    python -m group_wise_affine_quantize_amd.decoder_layer

Every product, the cache, the attention and the routing are libnq calls;
norms, the position rotation and the activation between the experts' products
are plain torch.  The demonstration fills the cache with a few prompts of
uneven lengths, then serves tokens step by step, as a server would: lengths
grow on the device, and the same tensors describe every step.
"""
import torch

from . import _binding as B


class DecoderLayer:
    """x -> x + attention(norm(x)) -> x + experts(norm(x)), weights in 4 bits
    (groups of 64), the router's in 8, activations bf16."""

    GROUP, BITS, ROUTER_BITS = 64, 4, 8

    def __init__(self, hidden=2048, heads=16, kv_heads=4, head_dim=128, experts=32, expert_hidden=1408, top_k=4,
                 seed=0, device="cuda"):
        self.hidden, self.heads, self.kv_heads, self.head_dim = hidden, heads, kv_heads, head_dim
        self.router = B.MoERouter(experts, top_k, score="softmax", renormalise=True)
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def quantized(*shape, bits=self.BITS):
            w = torch.randn(shape, generator=g, device=device) * shape[-1] ** -0.5
            return B.nq_quantize(w.to(torch.bfloat16), self.GROUP, bits)

        self.qkv = quantized((heads + 2 * kv_heads) * head_dim, hidden)
        self.out = quantized(hidden, heads * head_dim)
        self.gate = quantized(experts, hidden, bits=self.ROUTER_BITS)
        self.up = quantized(experts, 2 * expert_hidden, hidden)
        self.down = quantized(experts, hidden, expert_hidden)

    def new_cache(self, blocks, block_tokens=64, format="int8"):
        return B.KVCache(blocks, self.kv_heads, block_tokens, self.head_dim, format)

    @staticmethod
    def _norm(x):
        f = x.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def _rotate(self, x, positions):
        half = self.head_dim // 2
        freq = 10000.0 ** (-torch.arange(half, device=x.device) / half)
        angle = positions[:, None, None] * freq
        a, b = x.float().split(half, -1)
        return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1).to(x.dtype)

    def forward(self, x, positions, cache, seqs):
        """x [rows, hidden] bf16, positions [rows] (of each row in its
        sequence); seqs' lengths already count these rows.  Returns the
        layer's output and the experts chosen."""
        rows, h, kv, d = x.shape[0], self.heads, self.kv_heads, self.head_dim
        fused = B.nq_qmm(self._norm(x), *self.qkv, self.GROUP, self.BITS).view(rows, h + 2 * kv, d)
        fused[:, : h + kv] = self._rotate(fused[:, : h + kv], positions)
        q, k, v = fused.split([h, kv, kv], dim=1)       # column ranges: no copies
        B.nq_kv_append(cache, seqs, k, v)
        y = B.nq_kv_attention(cache, seqs, q)
        x = x + B.nq_qmm(y.view(rows, h * d), *self.out, self.GROUP, self.BITS)

        z = self._norm(x)
        logits = B.nq_qmm(z, *self.gate, self.GROUP, self.ROUTER_BITS)
        ids, weights = B.nq_moe_route(self.router, logits)
        chosen, top_k = ids.view(-1), ids.shape[1]
        token = torch.arange(rows, device=x.device, dtype=torch.int32).repeat_interleave(top_k)
        up = B.nq_gather_qmm_lhs(z.view(rows, 1, -1), *self.up, self.GROUP, self.BITS, token, chosen)
        a, b = up.chunk(2, -1)
        mid = (torch.nn.functional.silu(a.float()) * b.float()).to(x.dtype).contiguous()
        down = B.nq_gather_qmm(mid, *self.down, self.GROUP, self.BITS, chosen).view(rows, top_k, -1)
        return x + (down.float() * weights[..., None]).sum(1).to(x.dtype), ids


def main():
    import time
    layer = DecoderLayer()
    prompts, steps, block = [700, 33, 1, 410], 32, 64
    batch, wide = len(prompts), -(-(max(prompts) + steps) // block)
    cache = layer.new_cache(batch * wide, block)
    table = torch.randperm(batch * wide, device="cuda").to(torch.int32).view(batch, wide)
    lengths = torch.tensor(prompts, dtype=torch.int32).cuda()

    rows = sum(prompts)
    start = torch.tensor([0] + prompts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    positions = torch.cat([torch.arange(n) for n in prompts]).cuda()
    x = torch.randn(rows, layer.hidden, device="cuda").to(torch.bfloat16)
    y, _ = layer.forward(x, positions, cache, B.KVSequences(start, lengths, table, rows))
    print(f"{batch} prompts of {prompts} tokens: output {tuple(y.shape)}")

    seqs = B.KVSequences(torch.arange(batch + 1, dtype=torch.int32, device="cuda"), lengths, table, batch)
    x = y[(start[1:] - 1).long()]       # each sequence's last row
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(steps):
        lengths += 1
        x, ids = layer.forward(x, lengths - 1, cache, seqs)
        x = DecoderLayer._norm(x)       # in the place of the layers and the sampling between
    torch.cuda.synchronize()
    each = (time.perf_counter() - began) / steps
    print(f"{steps} steps of {batch} tokens: {each * 1e6:.0f} us a step; lengths {lengths.tolist()}, "
          f"last experts of the first sequence {ids[0].tolist()}")


if __name__ == "__main__":
    main()
