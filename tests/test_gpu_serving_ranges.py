"""Attention and norm at the ends of their types' ranges, and in place (GPU)."""

import math

import pytest
import torch

from test_gpu_serving import BF, HF, B, ints, ws  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, HF, torch.float32])
@pytest.mark.parametrize("T,N", [(3, 32768), (2, 16392), (1300, 4096), (5, 7161)])
def test_norm_over_its_inputs(B, T, N, dtype):  # noqa: F811
    """The sum written over x, or over the residual: the same sums, rows and codes as into memory of its own."""
    g = torch.Generator(device="cuda").manual_seed(N)
    x, res = (torch.randn(T, N, generator=g, device="cuda").to(dtype) for _ in "xr")
    w = (1 + 0.3 * torch.randn(N, generator=g, device="cuda")).to(dtype)

    def run(x, res, total):
        out, codes = torch.empty_like(x), torch.empty(T, N, dtype=torch.uint8, device="cuda")
        scales = torch.empty(T, -(-N // 128), device="cuda")
        B.add_rms_norm(x, res, w, 1e-6, residual_out=total, out=out, codes=codes, scales=scales)
        return total, out, codes, scales
    want = run(x, res, torch.empty_like(x))
    assert torch.equal(want[0], (x.float() + res.float()).to(dtype))
    over_x, over_res = x.clone(), res.clone()
    for got in (run(over_x, res, over_x), run(x, over_res, over_res)):
        for a, b in zip(got, want):
            assert torch.equal(a, b)
