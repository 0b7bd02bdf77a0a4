"""The attention kernel's bounded waits give up cleanly (GPU).

DSA_WAIT_LIMIT=0 makes the kernel's loading warp give up at once, so that every other role waits for what does not come
until it sees that.
The kernel has to say so (DSA_STATUS_TIMEOUT) and leave, its own copies and products drained and tensor memory freed, so
that the next call, over a workspace that is zeroed again, gives what it gave before.  Nothing here faults or hangs
the GPU: the failure is a wait that stops early.
"""

import pytest
import torch

from test_gpu_serving import B, HF, Batch, Case  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = {
    "one": Case([1], [300]),
    "many units": Case([1, 130, 2, 77] * 60, [700, 300, 65, 500] * 60, heads=16),
    "window, fp16": Case([70, 1] * 40, [900, 640] * 40, heads=9, kv=3, d=96, dtype=HF, window=77, sinks=130),
    "dim 64": Case([150, 1], [3000, 20000], d=64),
    "fp8 one": Case([1], [300], fp8=True),
    "fp8 many units": Case([1, 130, 2, 77] * 60, [700, 300, 65, 500] * 60, heads=16, fp8=True),
    "fp8 long": Case([1, 1], [30001, 64], heads=4, kv=1, fp8=True),
}


@pytest.mark.parametrize("name", CASES)
def test_waits_time_out_then_the_next_call_is_correct(B, monkeypatch, name):  # noqa: F811
    b = Batch(CASES[name])
    ws = B.alloc_attention_workspace()
    want = b.run(B, ws)
    assert want[2] == 0
    monkeypatch.setenv("DSA_WAIT_LIMIT", "0")
    _, _, status = b.run(B, ws)
    assert status == B.STATUS_TIMEOUT
    monkeypatch.delenv("DSA_WAIT_LIMIT")
    ws.zero_()
    for _ in range(2):
        out, lse, status = b.run(B, ws)
        assert status == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    b.check(out, lse)
