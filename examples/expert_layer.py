"""A few serving steps of one layer's experts, from the residual stream and back to it.

Each step: the residual addition and norm with 8-bit rows, the router's logits (plain torch here), each token's experts and
the groups that they make, the two expert products (the first gathers its rows, gates them and writes 8-bit rows), the
shared expert's two products, and the weighted sum.  The step's launches are captured once, for a batch padded to a fixed
size, and replayed with each step's number of tokens.

    python examples/expert_layer.py        (needs a GB300 and the built library)
"""

import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))
from dsa_sparse_attention_fp8_gb300 import binding  # noqa: E402

GROUP = binding.NORM_GROUP


def quantised_weights(w):
    """E4M3 codes of weights [..., N, K] and one scale for each 128 x 128 block."""
    n, k = w.shape[-2:]
    blocks = torch.nn.functional.pad(w, (0, -k % GROUP, 0, -n % GROUP)).unflatten(-1, (-1, GROUP)).unflatten(-3, (-1, GROUP))
    amax = blocks.abs().amax((-3, -1))
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / 448.0)
    codes = (blocks / scale[..., :, None, :, None]).to(torch.float8_e4m3fn)
    codes = codes.flatten(-4, -3).flatten(-2, -1)[..., :n, :k].contiguous()
    return codes.view(torch.uint8), scale.contiguous()


class ExpertLayer:
    """A layer's weights and step buffers for up to `tokens` rows."""

    def __init__(self, *, width=1024, inner=512, experts=32, top_k=4, runs=4, top_runs=2, tokens=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5  # noqa: E731
        empty = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.top_k, self.runs, self.top_runs = top_k, runs, top_runs
        self.norm = torch.ones(width, dtype=torch.bfloat16, device="cuda")
        self.router, self.bias = rand(experts, width), torch.zeros(experts, device="cuda")
        self.up, self.down = quantised_weights(rand(experts, 2 * inner, width)), quantised_weights(rand(experts, width, inner))
        self.shared_up, self.shared_down = quantised_weights(rand(2 * inner, width)), quantised_weights(rand(width, inner))
        u8, i32, bf = torch.uint8, torch.int32, torch.bfloat16
        pairs, scales = tokens * top_k, -(-width // GROUP)
        self.x, self.residual, self.y = (torch.zeros(tokens, width, dtype=bf, device="cuda") for _ in "xry")
        self.codes, self.scales = empty(tokens, width, dtype=u8), empty(tokens, scales)
        self.ids, self.places, self.weights = empty(tokens, top_k, dtype=i32), empty(tokens, top_k, dtype=i32), empty(tokens, top_k)
        self.starts, self.rows = empty(experts + 1, dtype=i32), torch.zeros(pairs, dtype=i32, device="cuda")
        self.hidden = empty(pairs, inner, dtype=u8), empty(pairs, -(-inner // GROUP))
        self.shared = empty(tokens, inner, dtype=u8), empty(tokens, -(-inner // GROUP))
        self.expert_out, self.out = empty(pairs, width, dtype=bf), empty(tokens, width, dtype=bf)
        self.num, self.status = torch.zeros(1, dtype=i32, device="cuda"), torch.zeros(1, dtype=i32, device="cuda")
        self.graph = None

    def launch(self):
        b, status = binding, self.status
        b.add_rms_norm(self.x, self.residual, self.norm, 1e-6, residual_out=self.residual, out=self.y, codes=self.codes,
                       scales=self.scales)
        logits = self.y.float() @ self.router.T
        b.route_experts(logits, self.top_k, self.ids, self.weights, self.starts, self.rows, self.places, bias=self.bias,
                        num_groups=self.runs, top_groups=self.top_runs, num_tokens=self.num)
        b.grouped_matmul(self.codes, self.up[0], self.starts, self.scales, self.up[1], rows=self.rows, gated=True,
                         out_codes=self.hidden[0], out_scales=self.hidden[1], status=status)
        b.grouped_matmul(self.hidden[0], self.down[0], self.starts, self.hidden[1], self.down[1], out=self.expert_out, status=status)
        b.fp8_matmul(self.codes, self.scales, *self.shared_up, gated=True, out_codes=self.shared[0], out_scales=self.shared[1],
                     status=status)
        b.fp8_matmul(*self.shared, *self.shared_down, out=self.out, status=status)
        b.combine_experts(self.expert_out, self.places, self.weights, add=self.out, out=self.out, status=status)

    def step(self, x):
        """One step's rows x [n, width] (BF16), n up to the layer's tokens -> the layer's output for them."""
        self.x[: len(x)].copy_(x)
        self.num.fill_(len(x))
        if self.graph is None:
            self.launch()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.launch()
        else:
            self.graph.replay()
        return self.out[: len(x)]


def main(steps=4, tokens=64, **kw):
    layer = ExpertLayer(tokens=tokens, **kw)
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(steps):
        n = max(1, tokens - 7 * i)
        out = layer.step(torch.randn(n, layer.x.shape[1], generator=g, device="cuda").bfloat16())
        counts = layer.starts.diff()
        print(f"step {i}: {n} rows, {int((counts > 0).sum())} experts used, most rows to one {int(counts.max())}, "
              f"|out| {out.float().abs().mean():.4f}, status {int(layer.status)}")
    return layer


if __name__ == "__main__":
    main()
