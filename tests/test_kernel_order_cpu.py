"""What the kernels' results rest on and no run shows, because it goes well by luck of timing (no GPU): the order of
barriers and accesses as the source has them."""

import re

import pytest

from kernel_source import CSRC, kernels

# another CTA's shared memory, or tensor memory that a pair of CTAs asks for together
PEER = r"\b(?:st_cluster_u32|ld_cluster_v4|mbar_arrive_cluster\w*|mbar_arrive_shared|mbar_arrive_remote|tmem_alloc_pair)\s*\("
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


def test_arrivals_at_another_cta_have_the_clusters_scope():
    """An arrival without a scope orders memory within its own CTA alone.  Relaxed ones are for accumulators, whose reads the
    tensor core's own fences order, or stand behind a fence for shared memory."""
    arrivals = re.findall(r"(mbarrier\.arrive[^ ]*shared::cluster[^ ]*) _", (CSRC / "ptx_matmul.cuh").read_text())
    assert len(arrivals) == 3 and all(re.match(r"mbarrier\.arrive\.(release|relaxed)\.cluster\.", a) for a in arrivals), arrivals
    text = (CSRC / "ptx_matmul.cuh").read_text()
    assert "fence.release.sync_restrict::shared::cta.cluster;\\n\\tmbarrier.arrive.relaxed.cluster" in text
    assert "@p fence.acquire.sync_restrict::shared::cluster.cluster" in text
    many = kernels("matmul.cuh")["many_rows_kernel"]
    assert set(re.findall(r"mbar_arrive_cluster_relaxed\(map_to\((\w+)", many)) == {"acc_empty"}


def test_rows_that_the_second_cta_gathered_are_waited_for_with_the_clusters_scope():
    """The second CTA arrives at the first one's barrier of a stage, and the first multiplies what the second has written."""
    many = kernels("matmul.cuh")["many_rows_kernel"]
    product = many[many.index("warp == 9 && rank == 0"):many.index("umma_f8_k128_pair")]
    assert re.search(r"p\.rows\)? .*mbar_wait_cluster<true>\(landed\(s\)", product)
    told = many[many.index("warp == 9 && p.rows"):many.index("warp >= 10 && p.rows")]
    assert re.search(r"fence_proxy_async_smem\(\);\s*mbar_arrive_shared\(map_to\(landed\(s\), 0\)\)", told)


@pytest.mark.parametrize("file", ["matmul.cuh", "ptx_matmul.cuh", "route.cuh", "combine.cuh"])
def test_what_the_kernel_before_writes_is_read_by_ordinary_loads(file):
    """A kernel launched programmatically lives while the one before it writes: read-only loads (__ldg, .nc, and ptx.cuh's
    ld_ahead, which is one) would promise that nobody does."""
    text = re.sub(r"//[^\n]*", "", (CSRC / file).read_text())
    assert not re.search(r"__ldg\b|ld\.global\.nc|\bld_ahead\w*\(|__restrict__", text)
