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


@pytest.mark.parametrize("at", [0, 31, 5000, 59999])
@pytest.mark.parametrize("gap", [10.0, 14.0, 17.0])
def test_many_small_probabilities_in_fp16(B, ws, at, gap):  # noqa: F811
    """One key of a long context far above the others, which weigh little each and something together (requests enough
    that few are split: a part without that key has a maximum of its own).

    A row's probabilities are rounded over a maximum that leaves its largest one at 2^6 at least, so each is off by
    half a step of itself (2^-11) or by 2^-25 of 2^6 where it falls below FP16's normal numbers: 2^-31 of the row's
    sum for each key.  The output is rounded once; sums of 60,000 terms in FP32."""
    n, d, heads, requests = 60000, 64, 4, 304
    pages = -(-n // 64)
    kc, vc = torch.zeros(pages, 64, 1, d, dtype=HF, device="cuda"), torch.ones(pages, 64, 1, d, dtype=HF, device="cuda")
    kc[at // 64, at % 64, 0, 0], vc[at // 64, at % 64] = gap, 0
    q = torch.zeros(requests, heads, d, dtype=HF, device="cuda")
    q[..., 0] = 1
    table = torch.arange(pages, device="cuda").int().repeat(requests, 1)       # all read the same pages
    out, lse = B.paged_attention(q, kc, vc, torch.arange(requests + 1, device="cuda").int(), ints([n] * requests), table,
                                 1.0, ws)
    torch.cuda.synchronize()
    rest = (n - 1) * math.exp(-gap)
    want = rest / (1 + rest)
    bar = (2 * 2.0 ** -11 + 2.0 ** -18 + n * 2.0 ** -23) * want + 2.0 ** -31 * n + 2.0 ** -25
    assert ((out.double() - want).abs() <= bar).all(), f"{want} became {out.min().item()} to {out.max().item()}"
    assert ((lse.double() - (gap + math.log1p(rest))).abs() <= n * 2.0 ** -23 + 2.0 ** -18 + 2.0 ** -22 * gap).all()


def test_norm_of_the_smallest_numbers(B):  # noqa: F811
    """A group whose scale would underflow is a group of zeros: finite codes and scales."""
    x = torch.ones(2, 256, device="cuda")
    x[:, ::2] = 0
    w = torch.full((256,), 1e-43, device="cuda")
    w[128:] = 1.0
    codes, scales = torch.empty(2, 256, dtype=torch.uint8, device="cuda"), torch.empty(2, 2, device="cuda")
    B.add_rms_norm(x, None, w, 1e-6, codes=codes, scales=scales)
    torch.cuda.synchronize()
    value = codes.view(torch.float8_e4m3fn).double().cpu() * scales.double().cpu().repeat_interleave(128, 1)
    want = x.double().cpu() * math.sqrt(2) * w.double().cpu()
    assert (scales > 0).all() and torch.isfinite(scales).all()
    # half a code's step of the group's largest (2^-4), or an FP32 number below the normal ones
    assert ((value - want).abs() <= want.abs() * (2.0 ** -4 + 2.0 ** -18) + 3e-43).all()
