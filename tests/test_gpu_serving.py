"""Block tables and slot maps, the K/V cache write, attention over the paged K/V cache and the residual + RMS norm
(GPU), against plain implementations in 64 bits.

Whole numbers, copied rows and quantised rows are exact.  Attention's bar is worst-case, per (row, head, dimension),
from the roundings the kernel makes, evaluated on the 64-bit values (w_s the exact softmax weights, A = sum_s w_s
|v_s|, u = eps/2 of the 16-bit type: bf16 2^-8, fp16 2^-11):
  * each probability is rounded once to 16 bits before it multiplies v (its sum is not): <= u A;
  * the output is rounded once: <= u |o|;
  * a score is a sum of D products in FP32, scaled: |dz| <= scale (D + 4) 2^-23 sum_j |q_j k_j|, which moves weights
    by at most 2 |dz| each (numerator and sum); exp2 and the scaling add a few 2^-22 of the score's size:
    <= A (2 max dz + 2^-18);
  * FP32 sums over S keys, even truncating: <= S 2^-23 A.
lse has no 16-bit rounding: |d| <= max dz + S 2^-23 + 2^-18 + 2^-22 |lse|.
"""

import dataclasses
import math

import pytest
import torch

from conftest import gpu_available

pytestmark = pytest.mark.gpu
LN2 = math.log(2.0)
NAN_CODE = 0x7F


@pytest.fixture(scope="module")
def B(lib):
    if not gpu_available():
        pytest.skip("no CUDA device")
    from dsa_sparse_attention_fp8_gb300 import binding
    return binding


@pytest.fixture(scope="module")
def ws(B):
    return B.alloc_attention_workspace()


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


# ------------------------------------------------------------------ tables
def plain_tables(q, seq, free, table, T):
    """The definition, request by request; bad requests hold rows only."""
    table = [list(r) for r in table]
    start, pos, slot, used, status = [0], [0] * T, [-1] * T, 0, 0
    for r, (a, c) in enumerate(zip(q, seq)):
        ok = 0 <= a <= T and a <= c <= 64 * len(table[r])
        if not 0 <= a <= T:
            a = 0
        t0 = start[-1]
        start.append(t0 + a)
        if not ok:
            status |= 2
            continue
        have, need = -(-(c - a) // 64), -(-c // 64)
        for b in range(have, need):
            table[r][b] = free[used] if used < len(free) else -1
            status |= 0 if used < len(free) else 8
            used += 1
        for i in range(a):
            p = c - a + i
            if t0 + i < T:
                pg = table[r][p // 64]
                if p // 64 < have and pg < 0:
                    status |= 1
                pos[t0 + i], slot[t0 + i] = p, pg * 64 + p % 64 if pg >= 0 else -1
    if start[-1] > T:
        status |= 2
    return table, start, pos, slot, used, status


def run_tables(B, q, seq, free, table, T):
    d = dict(start=torch.full((len(q) + 1,), -9, dtype=torch.int32, device="cuda"),
             pos=torch.full((T,), -9, dtype=torch.int32, device="cuda"),
             slot=torch.full((T,), -9, dtype=torch.int64, device="cuda"),
             used=ints([-9]), status=ints([0]), table=ints(table))
    B.build_block_tables(ints(q), ints(seq), ints(free), d["table"], d["start"], d["pos"], d["slot"], d["used"],
                         status=d["status"])
    torch.cuda.synchronize()
    return (d["table"].tolist(), d["start"].tolist(), d["pos"].tolist(), d["slot"].tolist(), d["used"].item(),
            d["status"].item())


def tables_case(q, seq, width=None, spare=3, seed=0):
    g = torch.Generator().manual_seed(seed)
    width = width or max(1, max(-(-c // 64) for c in seq))
    have = [max(0, -(-(c - a) // 64)) for a, c in zip(q, seq)]
    need = sum(max(0, -(-c // 64) - h) for c, h in zip(seq, have))
    pages = torch.randperm(sum(have) + need + spare, generator=g).tolist()
    at, table = 0, []
    for h in have:
        table.append((pages[at:at + h] + [-7] * width)[:width])
        at += h
    return pages[at:], table


@pytest.mark.parametrize("q,seq", [
    ([1], [1]), ([0], [0]), ([64], [64]), ([65], [65]), ([1], [64]), ([1], [65]), ([3, 0, 1, 200, 0], [3, 70, 129, 264, 0]),
    ([1] * 700, [1 + 13 * i % 517 for i in range(700)]),
    ([i % 67 for i in range(1500)], [i % 67 + 31 * i % 400 for i in range(1500)]),
])
def test_tables(B, q, seq):
    free, table = tables_case(q, seq)
    T = sum(q)
    assert run_tables(B, q, seq, free, table, T) == plain_tables(q, seq, free, table, T)
    # a batch padded to more rows
    assert run_tables(B, q, seq, free, table, T + 77) == plain_tables(q, seq, free, table, T + 77)


def test_tables_most_requests(B):
    n = 16384
    q, seq = [1] * n, [1 + i % 130 for i in range(n)]
    free, table = tables_case(q, seq)
    assert run_tables(B, q, seq, free, table, n) == plain_tables(q, seq, free, table, n)


def test_tables_faults(B):
    q, seq = [5, -1, 4, 9, 2, 1], [5, 10, 3, 1000, 70, 129]      # q < 0, seq < q, seq past the row
    free, table = tables_case([5, 2, 1], [5, 70, 129], width=4)
    table = [table[0], [1, 2, 3, 4], [5, 6, 7, 8], [9, 10, 11, 12], table[1], table[2]]
    want = plain_tables(q, seq, free, table, 21)
    assert want[-1] == 2
    assert run_tables(B, q, seq, free, table, 21) == want
    # too few free pages
    q, seq = [100, 100, 1], [100, 300, 1]
    free, table = tables_case(q, seq)
    want = plain_tables(q, seq, free[:3], table, 201)
    assert want[-1] == 8
    assert run_tables(B, q, seq, free[:3], table, 201) == want
    # a hole under an old block, and more tokens than rows
    table[1][3] = -1
    want = plain_tables(q, seq, free, table, 150)
    assert want[-1] == 3
    assert run_tables(B, q, seq, free, table, 150) == want


# ------------------------------------------------------------------ K/V write
def quantised(x):
    """E4M3 codes and scales by the library's rule, in IEEE FP32 steps (exact; on the CPU, where a division by a
    number is a division)."""
    on, x = x.device, x.float().cpu()
    amax = x.abs().amax(-1)
    s = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, 448.0))
    return (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).to(on), s.to(on)


def pool(pages, h, d, dtype, layout, fill):
    """An empty cache in one of three layouts, as [pages, 64, h, d] views."""
    if layout == "tokens":
        return torch.full((pages, 64, h, d), fill, dtype=dtype, device="cuda"), \
            torch.full((pages, 64, h, d), fill, dtype=dtype, device="cuda")
    if layout == "heads":
        return torch.full((pages, h, 64, d), fill, dtype=dtype, device="cuda").transpose(1, 2), \
            torch.full((pages, h, 64, d), fill, dtype=dtype, device="cuda").transpose(1, 2)
    both = torch.full((pages, 2, 64, h, d + 16), fill, dtype=dtype, device="cuda")   # interleaved, padded heads
    return both[:, 0, :, :, :d], both[:, 1, :, :, :d]


@pytest.mark.parametrize("layout", ["tokens", "heads", "interleaved"])
@pytest.mark.parametrize("T,h,d,dtype,fp8", [
    (1, 1, 16, torch.bfloat16, False), (7, 3, 48, torch.float16, False), (130, 8, 128, torch.bfloat16, False),
    (1, 1, 16, torch.bfloat16, True), (7, 3, 80, torch.float16, True), (333, 8, 128, torch.bfloat16, True),
])
def test_kv_write(B, T, h, d, dtype, fp8, layout):
    torch.manual_seed(T + d)
    pages = T // 64 + 3
    kc, vc = pool(pages, h, d, torch.uint8 if fp8 else dtype, layout, 7)
    rows = torch.randn(T, 2 * h + 1, d, device="cuda").to(dtype)
    rows[T // 2, 0] = 0                                    # an all-zero head
    k, v = rows[:, :h], rows[:, h:2 * h]
    slots = torch.randperm(pages * 64, device="cuda")[:T].contiguous()
    if T > 3:
        slots[2], slots[3] = -1, pages * 64 + 5             # padding, and past the pool
    ks, vs = (torch.full((pages, h, 64), 3.0, device="cuda") for _ in "kv") if fp8 else (None, None)
    want = [x.clone() for x in (kc, vc)] + [x.clone() for x in (ks, vs) if x is not None]
    for t in range(T):
        s = slots[t].item()
        if 0 <= s < pages * 64:
            for i, x in enumerate((k[t], v[t])):
                if fp8:
                    c, sc = quantised(x)
                    want[i][s // 64, s % 64], want[2 + i][s // 64, :, s % 64] = c, sc
                else:
                    want[i][s // 64, s % 64] = x
    status = ints([0])
    B.kv_write(k, v, slots, kc, vc, ks, vs, status=status)
    torch.cuda.synchronize()
    assert status.item() == (1 if T > 3 else 0)
    for got, w in zip([kc, vc] + ([ks, vs] if fp8 else []), want):
        assert torch.equal(got, w)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_kv_write_codes_near_borders(B, dtype):
    """Codes are those of the IEEE quotient, ties and subnormal codes included: rows over every exponent below their
    maximum, with maxima that make the quotients exact, and with ones that do not."""
    torch.manual_seed(5)
    T, h, d = 600, 2, 128
    x = torch.randint(0, 1 << 15, (T, 2 * h, d)).short()
    top = 0x4000 + torch.randint(0, 200, (T, 2 * h)).short()
    top[::2] = torch.tensor(448.0, dtype=dtype).view(torch.int16)      # s = 1: many quotients are ties
    x = torch.minimum(x, top[..., None])                               # (positive bit patterns order like their values)
    # near the maximum too, where codes are coarse
    x[:, :, ::3] = torch.maximum(top[..., None] - x[:, :, ::3] % 2000, torch.tensor(0, dtype=torch.int16))
    x[:, :, 0] = top
    x = x.contiguous().view(dtype) * (1 - 2 * torch.randint(0, 2, (T, 2 * h, d))).to(dtype)
    x = x.cuda()
    pages = T // 64 + 1
    kc, vc = (torch.zeros(pages, 64, h, d, dtype=torch.uint8, device="cuda") for _ in "kv")
    ks, vs = (torch.zeros(pages, h, 64, device="cuda") for _ in "kv")
    status = ints([0])
    B.kv_write(x[:, :h], x[:, h:], torch.arange(T, device="cuda"), kc, vc, ks, vs, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for cache, scale, rows in ((kc, ks, x[:, :h]), (vc, vs, x[:, h:])):
        codes, want = quantised(rows)
        assert torch.equal(scale.transpose(1, 2).reshape(-1, h)[:T], want)
        assert torch.equal(cache.view(-1, h, d)[:T], codes)


# ------------------------------------------------------------------ attention
@dataclasses.dataclass
class Case:
    q: list
    seq: list
    heads: int = 8
    kv: int = 2
    d: int = 128
    dtype: torch.dtype = torch.bfloat16
    fp8: bool = False
    window: int = 0
    sinks: int = 0
    layout: str = "tokens"
    pad: int = 0           # rows past the last request
    spread: float = 2.0    # standard deviation of the scores
    scale: float = 0.0     # softmax scale (0: 1 / sqrt(d))


class Batch:
    """Inputs of a case.  Every place that no row sees holds NaN: free pages, the ends of last pages, pages and
    tokens outside the windows (whose table entries are -1)."""

    def __init__(self, c: Case, seed=0):
        self.c = c
        g = torch.Generator().manual_seed(seed)
        self.T = sum(c.q) + c.pad
        blocks = [-(-s // 64) for s in c.seq]
        n_pages = sum(blocks) + 3
        perm = torch.randperm(n_pages, generator=g).tolist()
        self.scale = c.scale or c.d ** -0.5
        self.q = (c.spread * torch.randn(self.T, c.heads + 1, c.d, generator=g)).to(c.dtype).cuda()[:, :c.heads]
        kc, vc = pool(n_pages, c.kv, c.d, torch.uint8 if c.fp8 else c.dtype, c.layout, NAN_CODE if c.fp8 else math.nan)
        ks, vs = (torch.full((n_pages, c.kv, 64), math.nan, device="cuda") for _ in "kv") if c.fp8 else (None, None)
        self.table = torch.full((len(c.q), max(1, max(blocks))), -1, dtype=torch.int32)
        self.kv = []       # per request: exact keys and values in 64 bits [seq, kv, d]
        at = 0
        for r, (a, s) in enumerate(zip(c.q, c.seq)):
            pages = perm[at:at + blocks[r]]
            at += blocks[r]
            far = max(0, s - a - c.window + 1) if c.window else 0
            rows = []
            for cache, scale in ((kc, ks), (vc, vs)):
                x = torch.randn(s, c.kv, c.d, generator=g).to(c.dtype)
                if c.fp8:
                    codes, sc = quantised(x)
                    rows.append(codes.view(torch.float8_e4m3fn).double() * sc.double()[..., None])
                else:
                    codes, sc = x, None
                    rows.append(x.double())
                for b, page in enumerate(pages):
                    p = torch.arange(64 * b, min(s, 64 * b + 64))
                    if c.window:
                        held = bool(((p >= far) | (p < c.sinks)).any())
                    else:
                        held = True
                    if not held or len(p) == 0 or a == 0:
                        continue
                    self.table[r, b] = page
                    cache[page, : len(p)] = codes[p].cuda()
                    if c.fp8:
                        scale[page, :, : len(p)] = sc[p].T.cuda()
            self.kv.append(rows)
        self.kc, self.vc, self.ks, self.vs = kc, vc, ks, vs
        self.start = torch.tensor([0] + c.q).cumsum(0).to(torch.int32).cuda()
        self.seq = ints(c.seq)
        self.table = self.table.cuda()

    def run(self, B, ws, **kw):
        c = self.c
        status = ints([0])
        out = torch.full((self.T, c.heads + 2, c.d), 5.0, dtype=c.dtype, device="cuda")
        lse = torch.full((self.T, c.heads), 5.0, device="cuda")
        args = dict(window=c.window, num_sinks=c.sinks, k_scale=self.ks, v_scale=self.vs, out=out[:, 1:-1], lse=lse,
                    status=status)
        args.update(kw)
        B.paged_attention(self.q, self.kc, self.vc, self.start, self.seq, self.table, self.scale, ws, **args)
        torch.cuda.synchronize()
        assert (out[:, 0] == 5).all() and (out[:, -1] == 5).all(), "wrote outside its heads"
        return out[:, 1:-1], lse, status.item()

    def reference(self, hidden_pages=()):
        """(out, out's bar, lse, lse's bar) in 64 bits; hidden_pages: (request, block) pairs that are skipped."""
        c = self.c
        u = torch.finfo(c.dtype).eps / 2
        o, ob = torch.zeros(self.T, c.heads, c.d).double(), torch.zeros(self.T, c.heads, c.d).double()
        l = torch.full((self.T, c.heads), -math.inf).double()
        lb = torch.zeros(self.T, c.heads).double()
        group, t0 = c.heads // c.kv, 0
        q = self.q.double().cpu()
        for r, (a, s) in enumerate(zip(c.q, c.seq)):
            key, pos = torch.arange(s), torch.arange(s - a, s)[:, None]
            seen = key <= pos
            if c.window:
                seen &= (key > pos - c.window) | (key < c.sinks)
            for hr, b in hidden_pages:
                if hr == r:
                    seen[:, 64 * b:64 * b + 64] = False
            some = seen.any(1)
            for h in range(c.heads if a else 0):
                k, v = (x[:, h // group] for x in self.kv[r])
                qq = q[t0:t0 + a, h]
                z = torch.where(seen, self.scale * (qq @ k.T), -math.inf)
                size = torch.where(seen, self.scale * (qq.abs() @ k.abs().T), 0.0).amax(1, keepdim=True)
                dz = (c.d + 4) * 2.0 ** -23 * size
                lse = torch.logsumexp(z, 1, keepdim=True)
                w = torch.where(some[:, None], (z - lse).exp(), 0.0)
                A = w @ v.abs()
                o[t0:t0 + a, h] = w @ v
                small = 2 * dz + 2.0 ** -18 + s * 2.0 ** -23
                ob[t0:t0 + a, h] = u * A * (1 + u) + u * (w @ v).abs() + small * A
                if c.dtype == torch.float16:          # steps below the smallest normal number: probabilities and outputs
                    ob[t0:t0 + a, h] += 2.0 ** -25 * (1 + (w > 0).double() @ v.abs())
                l[t0:t0 + a, h] = lse[:, 0]
                lb[t0:t0 + a, h] = (dz + s * 2.0 ** -23 + 2.0 ** -18 + 2.0 ** -22 * lse.abs())[:, 0]
            t0 += a
        return o, ob, l, lb

    def check(self, out, lse, hidden_pages=()):
        o, ob, l, lb = self.reference(hidden_pages)
        out, lse = out.double().cpu(), lse.double().cpu()
        assert torch.isfinite(out).all(), "NaN or infinity came through"
        empty = torch.isinf(l)
        assert (out[empty] == 0).all() and (lse[empty] == -math.inf).all()
        assert torch.isfinite(lse[~empty]).all()
        worst = ((out - o).abs() - ob).max().item()
        assert worst <= 0, f"out is {worst:.3g} past its bar"
        worst = ((lse - l).abs() - lb)[~empty].max().item() if (~empty).any() else 0
        assert worst <= 0, f"lse is {worst:.3g} past its bar"


BF, HF = torch.bfloat16, torch.float16
CASES = {
    "one token": Case([1], [1]),
    "one token, long": Case([1], [2500], heads=16),
    "page borders": Case([1] * 9, [63, 64, 65, 127, 128, 129, 191, 192, 193]),
    "empty requests": Case([0, 1, 0, 0, 5, 0], [0, 70, 64, 0, 5, 9], pad=3),
    "prompt": Case([300], [300]),
    "prompt after prefix": Case([257], [900], heads=4, kv=1),
    "two tiles": Case([33, 32, 16, 17], [33, 500, 161, 17], heads=16),
    "mixed": Case([1, 130, 1, 1, 77, 2], [700, 1000, 1, 65, 77, 2000]),
    "one head each": Case([40, 1], [200, 333], heads=3, kv=3),
    "odd groups": Case([50, 1, 9], [90, 257, 140], heads=15, kv=3, dtype=HF),
    "group of 7": Case([61, 1], [130, 129], heads=14, kv=2, d=112),
    "group of 128": Case([3, 1], [200, 300], heads=128, kv=1, d=64),
    "group of 100": Case([3, 1], [200, 300], heads=100, kv=1, d=64),
    "dim 16": Case([20, 1], [100, 200], d=16, dtype=HF),
    "dim 64": Case([150, 1], [300, 200], d=64),
    "dim 80": Case([150, 1], [300, 200], d=80, dtype=HF),
    "dim 96, heads first": Case([70, 1], [300, 200], d=96, layout="heads"),
    "interleaved": Case([70, 1], [300, 200], layout="interleaved", dtype=HF),
    "fp16": Case([130, 1, 1], [260, 1000, 64], dtype=HF),
    "peaked": Case([65, 1], [500, 900], spread=30.0),
    "flat": Case([65, 1], [500, 900], spread=0.01),
    "small scale": Case([65, 1], [500, 900], spread=2e4, scale=1e-5),
    "fp8 one": Case([1], [1], fp8=True),
    "fp8 mixed": Case([1, 130, 1, 1, 77, 2], [700, 1000, 1, 65, 77, 2000], fp8=True, heads=16),
    "fp8 dim 64": Case([70, 1], [300, 200], fp8=True, d=64),
    "fp8 dim 48, interleaved": Case([70, 1], [300, 200], fp8=True, d=48, layout="interleaved"),
    "fp8 heads first": Case([70, 1], [300, 200], fp8=True, layout="heads"),
    "window 1": Case([70, 1], [300, 200], window=1),
    "window 1, sinks": Case([70, 1], [300, 200], window=1, sinks=4),
    "window 100": Case([200, 1, 1], [700, 1000, 50], window=100),
    "window, sinks": Case([200, 1, 1, 3], [700, 1000, 50, 130], window=100, sinks=5),
    "window, many sinks": Case([200, 1, 1], [900, 1000, 50], window=128, sinks=200),
    "window on borders": Case([64, 128, 1, 1], [512, 640, 256, 257], window=128, sinks=64),
    "window past all": Case([64, 1], [300, 400], window=100000, sinks=3),
    "sinks past all": Case([64, 1], [300, 400], window=10, sinks=100000),
    "fp8 window": Case([200, 1, 1, 3], [700, 1000, 50, 130], window=100, sinks=5, fp8=True),
    "fp16 window, odd": Case([111, 1], [640, 641], heads=9, kv=3, d=96, dtype=HF, window=77, sinks=130),
    "long, split": Case([1, 2], [20000, 9000], heads=8, kv=1),
    "long chunk, split": Case([300], [6000], heads=8, kv=1),
    "fp8 long": Case([1, 1], [20001, 64], heads=4, kv=1, fp8=True),
}


@pytest.mark.parametrize("name", CASES)
def test_attention(B, ws, name):
    b = Batch(CASES[name])
    out, lse, status = b.run(B, ws)
    assert status == 0
    b.check(out, lse)


def test_attention_many_requests(B, ws):
    n = 900
    b = Batch(Case([1 + (i % 5 == 0) for i in range(n)], [2 + 7 * i % 200 for i in range(n)], heads=4, kv=1, d=64))
    out, lse, status = b.run(B, ws)
    assert status == 0
    b.check(out, lse)


def test_attention_repeats_bit_for_bit(B, ws):
    b = Batch(CASES["long, split"])
    first = b.run(B, ws)
    other = Batch(CASES["mixed"], seed=3)
    other.run(B, ws)                       # another batch through the same workspace
    again = b.run(B, ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_bad_pages_are_skipped(B, ws, fp8):
    b = Batch(Case([1, 70, 1], [300, 400, 64], fp8=fp8))
    b.table[0, 2], b.table[1, 0], b.table[1, 3], b.table[2, 0] = -5, 1 << 30, b.kc.shape[0], -1
    out, lse, status = b.run(B, ws)
    assert status == 1
    b.check(out, lse, hidden_pages=[(0, 2), (1, 0), (1, 3), (2, 0)])


def test_attention_bad_metadata(B, ws):
    b = Batch(Case([2, 3, 1], [100, 70, 64]))
    good = b.run(B, ws)
    b.seq = ints([100, 2, 64])             # fewer tokens than rows
    out, lse, status = b.run(B, ws)
    assert status == 2
    assert (out[2:5] == 0).all() and (lse[2:5] == -math.inf).all()
    assert torch.equal(out[:2], good[0][:2]) and torch.equal(out[5:], good[0][5:])
    b.seq = ints([100, 70, 64 * b.table.shape[1] + 1])   # longer than its table row
    out, lse, status = b.run(B, ws)
    assert status == 2
    assert (out[5] == 0).all() and torch.equal(out[:5], good[0][:5])
    b.seq = ints([100, 70, 64])
    b.start = ints([0, 2, 1, 1 << 20])     # decreasing, then past the rows
    out, lse, status = b.run(B, ws)
    assert status == 2 and torch.equal(out[:2], good[0][:2])
    assert (out[2:] == 0).all() and (lse[2:] == -math.inf).all()


def test_attention_without_optional_outputs_and_on_a_stream(B, ws):
    b = Batch(CASES["mixed"])
    want = b.run(B, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse = B.paged_attention(b.q, b.kc, b.vc, b.start, b.seq, b.table, b.scale, ws)
    s.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,d,q,seq", [(4, 128, [1, 2], [30011, 20500]), (128, 64, [1, 0, 1], [16001, 9, 33000]),
                                           (48, 128, [5], [25003])])
def test_units_split_over_many_ctas(B, ws, heads, d, q, seq, fp8):
    """One key head and few requests: each unit is most of the grid's work, its parts joined in groups; again and again
    the same bits, so every call leaves the counts of arrivals at zero."""
    b = Batch(Case(q, seq, heads=heads, kv=1, d=d, fp8=fp8))
    out, lse, status = b.run(B, ws)
    assert status == 0
    b.check(out, lse)
    for _ in range(3):
        again = b.run(B, ws)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", [3, 5, 7])
def test_results_do_not_depend_on_what_ran_before(B, ws, group, fp8):
    """Head groups that leave rows of a query tile over: the bits are the same whatever other calls left there."""
    b = Batch(Case([40, 1, 3, 100], [300, 200, 77, 500], heads=4 * group, kv=4, fp8=fp8))
    other = Batch(Case([256, 1], [900, 700], heads=32, kv=4, spread=30.0, fp8=fp8), seed=1)
    out, lse, status = b.run(B, ws)
    assert status == 0
    b.check(out, lse)
    for scale in (1.0, 30.0, 300.0):
        other.scale = scale
        other.run(B, ws)
        again = b.run(B, ws)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_attention_in_a_graph_reads_new_lengths(B, ws):
    c = Case([1, 1, 1], [500, 64, 1000])
    b = Batch(c)
    out, lse = torch.empty_like(b.q, memory_format=torch.contiguous_format), torch.empty(3, c.heads, device="cuda")
    call = lambda: B.paged_attention(b.q, b.kc, b.vc, b.start, b.seq, b.table, b.scale, ws, out=out, lse=lse)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seq in ([500, 64, 1000], [129, 3, 999]):
        b.seq.copy_(ints(seq))
        b.c = dataclasses.replace(c, seq=seq)
        g.replay()
        torch.cuda.synchronize()
        short = Batch.__new__(Batch)
        short.__dict__ = dict(b.__dict__, kv=[[x[:n] for x in rows] for rows, n in zip(b.kv, seq)])
        short.check(out, lse)


@pytest.mark.parametrize("fp8", [False, True])
def test_dimensions_of_one_with_odd_strides(B, ws, fp8):
    """One key head, one page, one row, one query head, each with a stride that would be refused over more."""
    torch.manual_seed(8)
    d, n = 64, 40

    def odd(t, dim):  # the same view with an odd stride at a dimension of one element
        assert t.shape[dim] == 1
        return t.as_strided(t.shape, [3 if i == dim else s for i, s in enumerate(t.stride())])
    k, v = torch.randn(n, 1, d, device="cuda").to(BF), torch.randn(n, 1, d, device="cuda").to(BF)
    kc, vc = (odd(odd(torch.zeros(1, 64, 1, d, dtype=torch.uint8 if fp8 else BF, device="cuda"), 0), 2) for _ in "kv")
    ks, vs = (odd(torch.zeros(1, 64, 1, device="cuda").transpose(1, 2), 1) for _ in "kv") if fp8 else (None, None)
    status = ints([0])
    B.kv_write(odd(k, 1), odd(v, 1), torch.arange(n, device="cuda"), kc, vc, ks, vs, status=status)
    q = odd(odd(torch.randn(1, 1, d, device="cuda").to(BF), 0), 1)
    out, lse = B.paged_attention(q, kc, vc, ints([0, 1]), ints([n]), ints([[0]]), d ** -0.5, ws, k_scale=ks, v_scale=vs,
                                 status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    b = Batch.__new__(Batch)
    b.c, b.T, b.q, b.scale = Case([1], [n], heads=1, kv=1, d=d, fp8=fp8), 1, q.contiguous(), d ** -0.5
    b.kv = [[]]
    for x in (k, v):
        if fp8:
            c, s = quantised(x)
            x = c.view(torch.float8_e4m3fn).double() * s.double()[..., None]
        b.kv[0].append(x.double().cpu())
    b.check(out, lse)


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("dtype", [BF, HF, torch.float32])
@pytest.mark.parametrize("T,N", [(1, 1), (3, 7), (2, 128), (5, 129), (2, 1000), (3, 2048), (2, 2560), (4, 7168),
                                 (2, 7169), (3, 32768), (700, 256)])
def test_norm(B, T, N, dtype):
    torch.manual_seed(N)
    wide = torch.randn(T, 2 * N + 3).to(dtype)
    x, res = wide[:, :N], (3 * wide[:, N:2 * N]).contiguous()
    w = (1 + 0.3 * torch.randn(N)).to(dtype)
    if T > 2:
        x, res = x.clone(), res.clone()
        x[1], res[1] = 0, 0                                     # a row of zeros
    xd, rd, wd = wide.cuda()[:, :N], res.cuda(), w.cuda()
    if T > 2:
        xd[1] = 0
    g = -(-N // 128)
    h, y = torch.empty(T, N, dtype=dtype, device="cuda"), torch.empty(T, N + 5, dtype=dtype, device="cuda")[:, :N]
    codes, scales = torch.empty(T, N, dtype=torch.uint8, device="cuda"), torch.empty(T, g, device="cuda")
    B.add_rms_norm(xd, rd, wd, 1e-6, residual_out=h, out=y, codes=codes, scales=scales)
    torch.cuda.synchronize()
    hw = (x.float() + res.float()).to(dtype)
    assert torch.equal(h.cpu(), hw)
    hd = hw.double()
    yw = hd / (hd.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double()
    # FP32: N terms summed (each half a step off), root, division, two products
    near = (N / 2 + 8) * 2.0 ** -24
    u = torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0
    tiny = 2.0 ** -25 if dtype == HF else 0.0
    assert ((y.double().cpu() - yw).abs() <= (near + u * (1 + near)) * yw.abs() + tiny).all()
    pad = torch.nn.functional.pad(yw, (0, g * 128 - N)).view(T, g, 128)
    amax = pad.abs().amax(2)
    sw = torch.where(amax == 0, 1.0, amax / 448)
    assert ((scales.double().cpu() - sw).abs() <= (near + 2.0 ** -23) * sw).all()
    # a code is at most half a step off: 2^-4 of the value, or 2^-10 below the smallest normal number 2^-6
    got = codes.view(torch.float8_e4m3fn).double().cpu()
    t = yw / sw.repeat_interleave(128, 1)[:, :N]
    assert ((got - t).abs() <= torch.maximum(t.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10)) + 4 * (near + 2.0 ** -22) * t.abs()).all()
    # in place, without codes; without a residual
    x2 = xd.contiguous().clone()
    y2 = torch.empty(T, N, dtype=dtype, device="cuda")
    B.add_rms_norm(x2, rd, wd, 1e-6, residual_out=x2, out=y2)
    assert torch.equal(x2, h) and torch.equal(y2, y)
    y3 = torch.empty(T, N, dtype=dtype, device="cuda")
    B.add_rms_norm(h, None, wd, 1e-6, out=y3)
    assert torch.equal(y3, y)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,N", [(1300, 1024), (1217, 1033), (1400, 7168)])
def test_norm_of_many_rows(B, T, N, dtype):
    test_norm(B, T, N, dtype)


def test_tables_write_attention_together(B, ws):
    """Tables built from lengths, rows written at the slot map, attention over what was written: equal to
    attention over keys and values in order."""
    torch.manual_seed(1)
    steps = [([70, 5, 1], [70, 5, 1]), ([1, 60, 3], [71, 65, 4]), ([64, 1, 1], [135, 66, 5])]
    h, heads, d = 2, 8, 64
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(12, device="cuda").to(torch.int32)
    kc, vc = pool(12, h, d, BF, "tokens", math.nan)
    ks = [torch.zeros(0, h, d, dtype=BF, device="cuda") for _ in range(3)]
    vs = [torch.zeros(0, h, d, dtype=BF, device="cuda") for _ in range(3)]
    for q_lens, seq in steps:
        T = sum(q_lens)
        start, pos = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda")
        slots, used, status = torch.empty(T, dtype=torch.int64, device="cuda"), ints([0]), ints([0])
        B.build_block_tables(ints(q_lens), ints(seq), free, table, start, pos, slots, used, status=status)
        k, v = torch.randn(T, h, d, device="cuda").to(BF), torch.randn(T, h, d, device="cuda").to(BF)
        B.kv_write(k, v, slots, kc, vc, status=status)
        q = torch.randn(T, heads, d, device="cuda").to(BF)
        out, lse = B.paged_attention(q, kc, vc, start, ints(seq), table, d ** -0.5, ws, status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        free = free[used.item():].contiguous()
        ks = [torch.cat([a, b]) for a, b in zip(ks, k.split(q_lens))]
        vs = [torch.cat([a, b]) for a, b in zip(vs, v.split(q_lens))]
        b = Batch.__new__(Batch)
        b.c, b.T, b.q, b.scale = Case(q_lens, seq, heads=heads, kv=h, d=d), T, q, d ** -0.5
        b.kv = [[x.double().cpu(), y.double().cpu()] for x, y in zip(ks, vs)]
        b.check(out, lse)


@pytest.mark.parametrize("fp8", [False, True])
def test_the_example_attends_over_what_it_wrote(B, fp8):
    """The example's steps: attention of the last step equals attention over the kept keys and values."""
    import importlib.util

    from conftest import ROOT
    spec = importlib.util.spec_from_file_location("serve_step", ROOT / "examples" / "serve_step.py")
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    layer = ex.WindowLayer(requests=3, width=384, heads=8, kv_heads=2, dim=64, window=100, sinks=3, fp8_cache=fp8)
    torch.manual_seed(2)
    kept, lens = [[[], []] for _ in range(3)], [0, 0, 0]
    for new in ([150, 1, 70], [1, 1, 1], [3, 1, 1]):
        lens = [a + b for a, b in zip(lens, new)]
        T = sum(new)
        out, qkv, positions = layer.step(torch.randn(T, 384, device="cuda").to(BF), torch.randn(T, 384, device="cuda").to(BF),
                                         ints(new), ints(lens))
        assert positions.tolist() == [p for n, c in zip(new, lens) for p in range(c - n, c)]
        for r, rows in enumerate(qkv.split(new)):
            for i, part in enumerate((rows[:, 8:10], rows[:, 10:])):
                if fp8:
                    codes, sc = quantised(part)
                    part = codes.view(torch.float8_e4m3fn).double() * sc.double()[..., None]
                kept[r][i].append(part.double().cpu())
    assert int(layer.status) == 0
    b = Batch.__new__(Batch)
    b.c, b.T, b.q, b.scale = Case([3, 1, 1], lens, heads=8, kv=2, d=64, window=100, sinks=3), T, qkv[:, :8], 64 ** -0.5
    b.kv = [[torch.cat(k), torch.cat(v)] for k, v in kept]
    o, ob, _, _ = b.reference()
    assert ((out.double().cpu() - o).abs() <= ob).all()
