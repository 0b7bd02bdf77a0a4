"""What the kernels' results rest on and no run shows, because it goes well by luck of timing (no GPU): the order of
barriers and accesses as the source has them."""

import re

import pytest

from kernel_source import kernels

# another CTA's shared memory, or tensor memory that a pair of CTAs asks for together
PEER = r"\b(?:st_cluster_u32|ld_cluster_v4|mbar_arrive_cluster\w*|mbar_arrive_remote|tmem_alloc_pair)\s*\("
MET = r"\b(?:cluster_sync|cluster_wait)\s*\("


@pytest.mark.parametrize("file", ["matmul.cuh", "route.cuh"])
def test_a_cta_touches_another_only_after_they_have_met(file):
    """CTAs of a cluster are placed together, but one may store to another before that one has started: a cluster barrier
    has to come first."""
    seen = 0
    for name, body in kernels(file).items():
        touch, met = re.search(PEER, body), re.search(MET, body)
        if touch:
            seen += 1
            assert met and met.start() < touch.start(), f"{name}: {touch.group(0)} before any cluster barrier"
    assert seen == 2
