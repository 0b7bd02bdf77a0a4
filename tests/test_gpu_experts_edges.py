"""The products, the router and the experts' sum where their CTAs depend on one another, and at calls that the other tests do
not make (GPU), against the same 64-bit formulas and bars."""

import pytest
import torch

from test_gpu_experts import F32, B, Product, check_route  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k", [(17, 8, 2), (100, 256, 8), (113, 512, 16), (127, 64, 4), (129, 256, 8), (130, 16, 1)])
def test_route_where_some_ctas_have_no_tokens(B, T, E, k):  # noqa: F811
    """A CTA that has nothing to choose is ready to tell the others its counts at once."""
    torch.manual_seed(T)
    logits, bias = torch.randn(T, E, device="cuda"), 0.05 * torch.randn(E, device="cuda")
    check_route(B, logits, k, bias=bias)
    outs = []
    for _ in range(50):
        ids, places, rows = (torch.full(s, -9, dtype=torch.int32, device="cuda") for s in ((T, k), (T, k), (T * k,)))
        weights, starts = torch.full((T, k), -9.0, device="cuda"), torch.full((E + 1,), -9, dtype=torch.int32, device="cuda")
        outs.append((ids, weights, starts, rows, places))
    for o in outs:
        B.route_experts(logits, k, *o, bias=bias)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs[1:] for a, b in zip(o, outs[0]))


@pytest.mark.parametrize("counts,N,K,gather,gated,calls", [
    ([1500, 1, 900, 700], 1536, 1024, True, True, 12),       # pairs, of which the second CTA gathers too
    ([700, 0, 1030, 3, 513], 1101, 400, True, False, 12),
    ([60], 4096, 2176, False, True, 30),                      # a tile joined in one round
    ([200], 2112, 2048, False, False, 30),                    # and in several
    ([128, 40], 640, 2176, True, True, 30),
    ([3] * 40, 256, 1024, True, False, 30),
])
def test_what_ctas_hand_to_one_another(B, counts, N, K, gather, gated, calls):  # noqa: F811
    """Rows that one CTA of a pair gathers and the other multiplies, and sums that a cluster's CTAs read from one another,
    round by round: right, and the same each time."""
    p = Product(counts, N, K, gather=gather, gated=gated)
    p.check(B, F32)
    want = p.call(B, out_dtype=F32)
    got = [p.call(B, out_dtype=F32) for _ in range(calls)]
    assert all(torch.equal(g, want) for g in got)
