"""A few serving steps of one window-attention layer, from request lengths to attention output.

Each step: block tables and slot maps from the requests' lengths, the residual addition and norm with 8-bit rows,
a projection of those rows (plain torch here), the K/V cache write and attention over the paged cache with a sliding
window and a few first tokens that stay visible.  The indexer's key cache shares the block tables, as the cache of a
sparse layer would.

    python examples/serve_step.py        (needs a GB300 and the built library)
"""

import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))
from dsa_sparse_attention_fp8_gb300 import binding  # noqa: E402

PAGE = binding.PAGE_TOKENS


class WindowLayer:
    """A layer's weights, caches and step buffers."""

    def __init__(self, *, width=1024, heads=16, kv_heads=4, dim=128, window=256, sinks=4, pages=256, requests=8,
                 max_blocks=64, fp8_cache=True, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.window, self.sinks = heads, kv_heads, dim, window, sinks
        self.norm = torch.ones(width, dtype=torch.bfloat16, device="cuda")
        n = (heads + 2 * kv_heads) * dim + binding.HEAD_DIM
        self.weight = torch.randn(width, n, generator=g, device="cuda") * width ** -0.5
        kind = torch.uint8 if fp8_cache else torch.bfloat16
        self.k_cache, self.v_cache = (torch.zeros(pages, PAGE, kv_heads, dim, dtype=kind, device="cuda") for _ in "kv")
        self.k_scale = self.v_scale = None
        if fp8_cache:
            self.k_scale, self.v_scale = (torch.ones(pages, kv_heads, PAGE, device="cuda") for _ in "kv")
        self.index_cache = torch.zeros(pages, binding.PAGE_BYTES, dtype=torch.uint8, device="cuda")
        self.table = torch.full((requests, max_blocks), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.workspace = binding.alloc_attention_workspace()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(self, x, residual, query_lens, seq_lens):
        """One step's rows x, residual [T, width] (BF16) -> attention output [T, heads, dim]; residual is updated."""
        T, R = x.shape[0], query_lens.shape[0]
        start = torch.empty(R + 1, dtype=torch.int32, device="cuda")
        positions = torch.empty(T, dtype=torch.int32, device="cuda")
        slots = torch.empty(T, dtype=torch.int64, device="cuda")
        used = torch.empty(1, dtype=torch.int32, device="cuda")
        binding.build_block_tables(query_lens, seq_lens, self.free, self.table, start, positions, slots, used,
                                   status=self.status)
        codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
        scales = torch.empty(T, -(-x.shape[1] // binding.NORM_GROUP), device="cuda")
        binding.add_rms_norm(x, residual, self.norm, 1e-6, residual_out=residual, codes=codes, scales=scales)
        rows = codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(binding.NORM_GROUP, 1)[:, : x.shape[1]]
        y = rows @ self.weight
        h, k = self.heads, self.kv_heads
        index_key = y[:, -binding.HEAD_DIM:].contiguous()
        qkv = y[:, : -binding.HEAD_DIM].to(torch.bfloat16).view(T, h + 2 * k, self.dim)
        binding.write_k(index_key, start, seq_lens, self.table, self.index_cache, status=self.status)
        binding.kv_write(qkv[:, h:h + k], qkv[:, h + k:], slots, self.k_cache, self.v_cache, self.k_scale, self.v_scale,
                         status=self.status)
        out, _ = binding.paged_attention(qkv[:, :h], self.k_cache, self.v_cache, start, seq_lens, self.table,
                                         self.dim ** -0.5, self.workspace, window=self.window, num_sinks=self.sinks,
                                         k_scale=self.k_scale, v_scale=self.v_scale, status=self.status)
        self.free = self.free[int(used):].contiguous()     # the host's free list drops the pages taken
        return out, qkv, positions


def main(steps=4, requests=8, prompt=200, **kw):
    layer = WindowLayer(requests=requests, **kw)
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
    for i in range(steps):
        # prompts of several lengths first, then a token each
        new = torch.tensor([prompt + 13 * r if i == 0 else 1 for r in range(requests)], dtype=torch.int32, device="cuda")
        lens += new
        T = int(new.sum())
        x, residual = (torch.randn(T, layer.norm.shape[0], generator=g, device="cuda").bfloat16() for _ in "xr")
        out, _, positions = layer.step(x, residual, new, lens)
        print(f"step {i}: {T} rows, positions to {int(positions.max())}, |out| {out.float().abs().mean():.4f}, "
              f"free pages {layer.free.numel()}, status {int(layer.status)}")
    return layer


if __name__ == "__main__":
    main()
