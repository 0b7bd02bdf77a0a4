"""Outputs that a call allocates belong to the stream that writes them (GPU)."""

import pytest
import torch

from test_gpu_serving import B, Batch, Case, ws  # noqa: F401

pytestmark = pytest.mark.gpu


def test_attention_outputs_come_from_the_launch_stream(B, ws):  # noqa: F811
    """Memory that the current stream's queued work may still use is not handed to a launch on another stream."""
    b = Batch(Case([1, 3], [70, 200], heads=32, kv=4))
    want = b.run(B, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    freed = [torch.empty(b.T, 32, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(b.T, 32, device="cuda")]
    at = [t.data_ptr() for t in freed]
    del freed                                # as after a step whose work is still queued
    out, lse = B.paged_attention(b.q, b.kc, b.vc, b.start, b.seq, b.table, b.scale, ws, stream=side)
    side.synchronize()
    assert out.data_ptr() not in at and lse.data_ptr() not in at
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_codes_come_from_the_launch_stream(B):  # noqa: F811
    x = torch.randn(4096, 128, device="cuda")
    want = B.quantize_fp8_blocks(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    freed = [torch.empty(4096, 128, dtype=torch.uint8, device="cuda"), torch.empty(4096, device="cuda")]
    at = [t.data_ptr() for t in freed]
    del freed
    got = B.quantize_fp8_blocks(x, stream=side)
    side.synchronize()
    assert got[0].data_ptr() not in at and got[1].data_ptr() not in at
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
