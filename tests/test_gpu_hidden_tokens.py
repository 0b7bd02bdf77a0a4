"""Attention over caches whose hidden tokens hold anything (GPU).

A token that no row of its request sees may share a page with tokens that are seen: those before the window's first
position, those after the first `sinks` tokens.  Neither its key, its value nor (E4M3 caches) its scales may reach a
result.  Bars as in test_gpu_serving.py.
"""

import math

import pytest
import torch

from test_gpu_serving import B, BF, HF, NAN_CODE, Batch, Case, ws  # noqa: F401

pytestmark = pytest.mark.gpu

WINDOWS = {
    "decode": Case([1] * 5, [1000, 130, 257, 700, 64], window=100, sinks=5),
    "prompt": Case([200, 1, 3], [700, 1000, 130], heads=16, window=100, sinks=5),
    "window 1": Case([70, 1], [300, 200], window=1),
    "sinks end inside a page": Case([64, 1], [512, 640], window=128, sinks=3),
    "sinks past a tile": Case([111, 1], [640, 641], heads=9, kv=3, d=96, window=77, sinks=130),
    "one tile": Case([1, 2, 20], [120, 125, 90], window=30, sinks=5),
    "dim 64": Case([150, 1], [300, 200], d=64, window=50, sinks=3),
    "group of 128": Case([3, 1], [500, 300], heads=128, kv=1, window=90, sinks=70),
    "split": Case([1, 2], [20000, 9000], heads=8, kv=1, window=7001, sinks=200),
}


def spoil(b, put):
    """Calls put(page, places) for the tokens of each seen page that no row of their request sees."""
    c, n = b.c, 0
    for r, (a, s) in enumerate(zip(c.q, c.seq)):
        far = max(0, s - a - c.window + 1)
        for block, page in enumerate(b.table[r].tolist()):
            if page >= 0:
                p = torch.arange(64 * block, min(64 * block + 64, s))
                at = (p[(p < far) & (p >= c.sinks)] % 64).cuda()
                n += len(at)
                put(page, at)
    assert n > 0


def case(name, **kw):
    return Case(**{**WINDOWS[name].__dict__, **kw})


def check(B, ws, b):  # noqa: F811
    out, lse, status = b.run(B, ws)
    assert status == 0
    b.check(out, lse)


@pytest.mark.parametrize("name", WINDOWS)
@pytest.mark.parametrize("dtype,value", [(BF, math.nan), (BF, math.inf), (HF, math.nan), (HF, -math.inf)])
def test_hidden_keys_and_values(B, ws, name, dtype, value):  # noqa: F811
    b = Batch(case(name, dtype=dtype))

    def put(page, at):
        b.kc[page, at] = value
        b.vc[page, at] = value
    spoil(b, put)
    check(B, ws, b)


@pytest.mark.parametrize("name", WINDOWS)
def test_hidden_codes(B, ws, name):  # noqa: F811
    b = Batch(case(name, fp8=True))

    def put(page, at):
        b.kc[page, at] = NAN_CODE
        b.vc[page, at] = NAN_CODE
    spoil(b, put)
    check(B, ws, b)


# ------------------------------------------------------------------ scales of keys
@pytest.mark.parametrize("name", WINDOWS)
@pytest.mark.parametrize("value", [0.0, math.nan, -1.0, math.inf, -math.inf])
def test_hidden_scales_of_keys(B, ws, name, value):  # noqa: F811
    b = Batch(case(name, fp8=True))
    spoil(b, lambda page, at: b.ks[page].index_fill_(1, at, value))
    check(B, ws, b)


def rescale(b, factors):
    """Multiplies the scales of the keys of request r at position p by factors(p), and the exact keys alike."""
    for r, s in enumerate(b.c.seq):
        p = torch.arange(s)
        f = factors(p)
        for block in range(-(-s // 64)):
            i = p[64 * block:64 * block + 64]
            b.ks[int(b.table[r, block]), :, : len(i)] *= f[i].cuda()
        b.kv[r][0] *= f.double()[:, None, None]


CHUNKS = [Case([130, 1, 77], [400, 300, 77], heads=16, fp8=True), Case([300], [900], heads=8, kv=1, d=64, fp8=True),
          Case([200, 1], [700, 300], window=100, sinks=5, fp8=True)]


@pytest.mark.parametrize("c", CHUNKS)
def test_scales_of_keys_of_zero_and_below(B, ws, c):  # noqa: F811
    """Finite scales of tokens that some rows see and others do not: a key of scale 0 is a key of zeros."""
    b = Batch(Case(**{**c.__dict__, "window": 0, "sinks": 0}))
    b.c = c
    rescale(b, lambda p: torch.where(p % 7 == 3, 0.0, torch.where(p % 7 == 5, -1.0, 1.0)))
    check(B, ws, b)


@pytest.mark.parametrize("c", CHUNKS)
@pytest.mark.parametrize("small", [1.0, 2.0 ** -30])
def test_query_rows_of_zeros(B, ws, c, small):  # noqa: F811
    """Rows of zeros, and rows of the smallest numbers, weigh all the tokens they see alike, whatever the scales."""
    b = Batch(Case(**{**c.__dict__, "window": 0, "sinks": 0}))
    b.c = c
    b.q[::3] = 0
    b.q[1::3] = 2.0 ** -133
    rescale(b, lambda p: torch.full(p.shape, small))
    check(B, ws, b)


# ------------------------------------------------------------------ scales of values
@pytest.mark.parametrize("name", WINDOWS)
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_hidden_scales_of_values(B, ws, name, value):  # noqa: F811
    b = Batch(case(name, fp8=True))

    def put(page, at):
        b.ks[page].index_fill_(1, at, value)
        b.vs[page].index_fill_(1, at, value)
    spoil(b, put)
    check(B, ws, b)


@pytest.mark.parametrize("window,sinks", [(100, 5), (0, 0)])
def test_scales_of_pages_that_are_not_loaded(B, ws, window, sinks):  # noqa: F811
    """A prompt's first rows see one page of a tile only, and bad pages are skipped: neither page brings scales.  What an
    earlier tile of another request left in their place (hidden tokens' NaN) decides nothing."""
    n = 60
    b = Batch(Case([1, 300] * n, [1000, 300] * n, heads=16, window=100, sinks=5, fp8=True))

    def put(page, at):
        b.ks[page].index_fill_(1, at, math.nan)
        b.vs[page].index_fill_(1, at, math.nan)
    spoil(b, put)
    hidden = []
    if not window:                # bad pages instead: blocks inside the prompts' windows
        for r in range(1, 2 * n, 4):
            b.table[r, 3] = -1
            hidden.append((r, 3))
    out, lse, status = b.run(B, ws)
    assert status == (1 if hidden else 0)
    b.check(out, lse, hidden_pages=hidden)
