"""The product kernels give up in the midst of a call and leave cleanly (GPU).

DSA_LOAD_STAGES=n makes every loading warp stop after n stages (those of CTAs of odd rank in a cluster one later or earlier),
with copies, gathered rows and products under way, so that every other role waits for what does not come.  The kernel has to
say so (DSA_STATUS_TIMEOUT), end what is under way, free its tensor memory and leave; the next calls give what they gave
before.  Nothing here faults or hangs the GPU: the failure is a role that stops early.

A wait that ran to its own limit would take seconds; a role sees within some milliseconds that another has left.  So a call
that ends within a second has had no wait run out, those for its last copies and products among them.
"""

import time

import pytest
import torch

from test_gpu_experts import BF, F32, U8, B, Product, ints  # noqa: F401

pytestmark = pytest.mark.gpu

# (each CTA's part has more than 21 stages)
CASES = {
    "one row, shared K": ([1], 200, 24576),
    "gated rows, shared K": ([60], 512, 24576, U8, False, True),
    "gathered rows, shared K": ([5, 0, 9], 300, 24576, U8, True),
    "16 bits": ([70, 3], 300, 12288, BF),
    "one CTA a tile": ([100], 12000, 4096),
    "many groups": ([3] * 80, 1024, 2048),
    "many groups, gated, gathered": ([3] * 80, 1024, 2048, U8, True, True),
    "many rows": ([3000], 1500, 4096),
    "many rows, gathered": ([1500, 1, 900, 700], 1500, 4096, U8, True),
    "many rows, 16 bits, gated": ([1500, 1, 900, 700], 1500, 4096, BF, False, True),
    "many rows, second CTAs without any": ([100, 300, 20, 90, 256, 1, 5, 128] * 4, 2048, 4096),
}


@pytest.mark.parametrize("stages", [1, 2, 4, 7, 8, 9, 21])
@pytest.mark.parametrize("name", CASES)
def test_a_call_that_gives_up_midway_ends_what_is_under_way(B, monkeypatch, name, stages):  # noqa: F811
    p = Product(*CASES[name])
    want = p.call(B, out_dtype=F32)
    status = ints([0])
    torch.cuda.synchronize()
    monkeypatch.setenv("DSA_LOAD_STAGES", str(stages))
    start = time.monotonic()
    p.call(B, out_dtype=F32, status=status)
    torch.cuda.synchronize()
    took = time.monotonic() - start
    monkeypatch.delenv("DSA_LOAD_STAGES")
    assert status.item() == B.STATUS_TIMEOUT and took < 1.0
    status.zero_()
    for _ in range(2):
        got = p.call(B, out_dtype=F32, status=status)
        assert status.item() == 0 and torch.equal(got, want)
