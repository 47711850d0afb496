"""One decoder block on the library's operators: packed prompts, then one new
token per sequence at a time.

    x1 = x + W_o attention(rotate(W_qkv x)),   y = x1 + moe_layer(x1)

The projections are plain matrix products; everything between them is the
library's: kv_append rotates the queries and keys and stores keys and values
in the paged cache, attn_prefill attends within the prompts, attn_decode over
the cache, and the routed-MoE layer follows.  Norms and weights of a real
model are left out: weights are random.

    python examples/decoder_block.py            (an MI355X and the built library)
"""

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_fp4_sqrtsoftplus_amd as moe  # noqa: E402


class Pages:
    """A free list of cache pages and the block table of a fixed batch."""

    def __init__(self, pages, page_size, batch, width, device="cuda"):
        self.page_size, self.free = page_size, list(range(pages))
        self.table = torch.full((batch, width), -1, dtype=torch.int32)
        self.lens = [0] * batch
        self.device = device

    def grow(self, counts):
        """Adds counts[b] tokens to every sequence b: their slots and positions, packed, and the table and lengths
        on the device."""
        slots, positions = [], []
        for b, n in enumerate(counts):
            for pos in range(self.lens[b], self.lens[b] + n):
                if pos % self.page_size == 0:
                    if not self.free:
                        raise RuntimeError("the cache has no free page")
                    self.table[b, pos // self.page_size] = self.free.pop()
                slots.append(int(self.table[b, pos // self.page_size]) * self.page_size + pos % self.page_size)
                positions.append(pos)
            self.lens[b] += n
        d = self.device
        return (torch.tensor(slots, dtype=torch.int64, device=d), torch.tensor(positions, dtype=torch.int32, device=d),
                self.table.to(d), torch.tensor(self.lens, dtype=torch.int32, device=d))


class DecoderBlock:
    def __init__(self, hidden=1024, heads=16, kv_heads=4, head_dim=128, inter=512, experts=16, top_k=4, pages=64,
                 page_size=16, batch=3, kv_format=moe.KV_BF16, max_positions=4096, window=0, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(rows, cols):
            return (torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5).bfloat16()

        self.hidden, self.heads, self.kv_heads, self.dim, self.window = hidden, heads, kv_heads, head_dim, window
        self.w_qkv, self.w_o = w((heads + 2 * kv_heads) * head_dim, hidden), w(hidden, heads * head_dim)
        self.w_gate = w(experts, hidden)
        u8 = dict(dtype=torch.uint8, device="cuda", generator=g)

        def expert(n, k):   # E2M1 nibbles with scales of 2^-7 .. 2^-5 per 32
            return (torch.randint(0, 256, (experts, n, k // 2), **u8),
                    torch.randint(120, 123, (experts, n, k // 32), **u8))

        self.experts = dict(zip(("w1", "w1_scale", "w3", "w3_scale", "w2", "w2_scale"),
                                (*expert(inter, hidden), *expert(inter, hidden), *expert(hidden, inter))))
        self.moe_sizes = dict(hidden=hidden, inter=inter, n_experts=experts, top_k=top_k)
        self.rope = moe.Rope.of(max_positions, head_dim)
        self.cache = moe.KVCache.empty(pages, page_size, kv_heads, head_dim, kv_format)
        self.pages = Pages(pages, page_size, batch, pages)
        self.decode_attention = moe.DecodeAttention(self.cache, batch, heads, window=window)

    def _qkv(self, x):
        qkv = torch.nn.functional.linear(x, self.w_qkv).view(len(x), -1, self.dim)
        return qkv[:, :self.heads], qkv[:, self.heads:-self.kv_heads], qkv[:, -self.kv_heads:]

    def _rest(self, x, attended):
        x1 = x + torch.nn.functional.linear(attended.flatten(1), self.w_o)
        return x1 + moe.layer(moe.Config(tokens=len(x), **self.moe_sizes), x1, self.experts, w_gate=self.w_gate)

    def attend_prompts(self, x, lengths):
        """Attention of packed prompts x [sum(lengths), hidden]; their keys and values enter the cache."""
        slots, positions, _, _ = self.pages.grow(lengths)
        q, k, v = self._qkv(x)
        moe.kv_append(self.cache, k, v, slots, positions, self.rope, q, q_out=q, k_out=k)   # q, k rotated in place
        cu = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")
        return moe.attn_prefill(q, k, v, cu, window=self.window)

    def attend_tokens(self, x):
        """Attention of one new token per sequence, x [batch, hidden], over the cache."""
        slots, positions, table, lens = self.pages.grow([1] * len(x))
        q, k, v = self._qkv(x)
        q = moe.kv_append(self.cache, k, v, slots, positions, self.rope, q)
        return self.decode_attention(q, table, lens)

    def prompts(self, x, lengths):
        return self._rest(x, self.attend_prompts(x, lengths))

    def tokens(self, x):
        return self._rest(x, self.attend_tokens(x))


def main():
    torch.manual_seed(0)
    for name, fmt in (("bf16", moe.KV_BF16), ("fp8", moe.KV_FP8)):
        block = DecoderBlock(hidden=4096, heads=32, kv_heads=8, head_dim=128, inter=2048, experts=64, top_k=6,
                             pages=512, page_size=64, batch=4, kv_format=fmt)
        lengths = [1500, 37, 800, 2048]
        x = torch.randn(sum(lengths), 4096, device="cuda").bfloat16()
        y = block.prompts(x, lengths)
        last = y[torch.tensor(lengths, device="cuda").cumsum(0) - 1]
        torch.cuda.synchronize()
        start, steps = time.perf_counter(), 32
        for _ in range(steps):
            last = block.tokens(torch.nn.functional.rms_norm(last.float(), (4096,)).bfloat16())
        torch.cuda.synchronize()
        ms = (time.perf_counter() - start) / steps * 1e3
        print(f"{name} cache: {sum(lengths)} prompt tokens, {steps} steps of {len(lengths)} sequences, "
              f"{ms:.3f} ms a step, output rms {last.float().square().mean().sqrt().item():.3f}")
        assert torch.isfinite(last.float()).all()


if __name__ == "__main__":
    main()
