"""The product kernels' bounded waits give up cleanly (GPU).

DSA_WAIT_LIMIT=0 makes the loading warp give up at once, so that every other role, in every CTA that shares a tile, waits
for what does not come until it sees that.  The kernel has to say so (DSA_STATUS_TIMEOUT) and leave, its own copies and
products drained and tensor memory freed, so that the next call gives what it gave before.  Nothing here faults or hangs
the GPU: the failure is a wait that stops early.
"""

import pytest
import torch

from test_gpu_experts import BF, F32, U8, B, Product, ints  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = {
    "one row, shared K": ([1], 200, 4096),
    "gated rows, shared K": ([60], 512, 4096, U8, False, True),
    "one CTA a tile": ([100], 4000, 128),
    "16 bits": ([70, 3], 300, 640, BF),
    "gathered": ([5, 0, 9], 300, 1024, U8, True),
    "many groups": ([3] * 80, 1024, 256),
    "many groups, gated, gathered": ([3] * 80, 1024, 256, U8, True, True),
    "many rows": ([3000], 1500, 512),
    "many rows, gathered": ([1500, 1, 900, 700], 1500, 512, U8, True),
    "many rows, 16 bits, gated": ([1500, 1, 900, 700], 1500, 512, BF, False, True),
}


@pytest.mark.parametrize("name", CASES)
def test_waits_time_out_then_the_next_call_is_correct(B, monkeypatch, name):  # noqa: F811
    p = Product(*CASES[name])
    want = p.call(B, out_dtype=F32)
    status = ints([0])
    monkeypatch.setenv("DSA_WAIT_LIMIT", "0")
    p.call(B, out_dtype=F32, status=status)
    assert status.item() == B.STATUS_TIMEOUT
    monkeypatch.delenv("DSA_WAIT_LIMIT")
    status.zero_()
    for _ in range(2):
        got = p.call(B, out_dtype=F32, status=status)
        assert status.item() == 0 and torch.equal(got, want)
    p.check(B, F32)
