"""The products, the router and the experts' sum where their CTAs depend on one another, and at calls that the other tests do
not make (GPU), against the same 64-bit formulas and bars."""

import pytest
import torch

from test_gpu_experts import BF, E4M3, F32, U8, B, Product, check_route, ints  # noqa: F401

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


def e4m3(*shape):
    return (100 * torch.randn(*shape, device="cuda")).clamp(-448, 448).to(E4M3).view(U8)


def test_a_call_right_behind_another_sees_its_scales(B):  # noqa: F811
    """A chain of products in which each reads the codes and the scales that the one before has just written, of inputs that
    change from chain to chain in the same buffers: as with a wait after each call."""
    torch.manual_seed(4)
    n, sizes = 512, [700, 700, 300, 64, 1]
    w, ws = e4m3(2 * n, n), torch.full((8, 4), 1.6 * n ** -0.5 / 100, device="cuda")
    codes, scales = [torch.empty(700, n, dtype=U8, device="cuda") for _ in sizes], [torch.empty(700, 4, device="cuda") for _ in sizes]
    inputs = [(e4m3(700, n), (0.5 + torch.rand(700, 4, device="cuda")) / 100) for _ in range(10)]

    def chains(wait):
        got = []
        for c, s in inputs:
            codes[0].copy_(c), scales[0].copy_(s)
            for i in range(1, len(sizes)):
                t = sizes[i]
                B.fp8_matmul(codes[i - 1][:t], scales[i - 1][:t], w, ws, gated=True, out_codes=codes[i][:t], out_scales=scales[i][:t])
                if wait:
                    torch.cuda.synchronize()
            got.append([x[i][:sizes[i]].clone() for i in range(1, len(sizes)) for x in (codes, scales)])
        torch.cuda.synchronize()
        return got
    want = chains(True)
    assert all(s.isfinite().all() and (s > 0).all() for one in want for s in one[1::2])
    assert len({one[1][0, 0].item() for one in want}) == len(inputs)               # (scales that a stale one would change)
    for _ in range(10):
        assert all(torch.equal(a, b) for x, y in zip(chains(False), want) for a, b in zip(x, y))


@pytest.mark.parametrize("T", [40, 1500])
def test_steps_right_behind_one_another_see_each_others_results(B, T):  # noqa: F811
    """Router, gathered product, product and sum over the same buffers, step after step with nothing between them: groups,
    rows, scales, places and weights are all fresh from the call before."""
    torch.manual_seed(T)
    E, k, n, i32 = 12, 3, 256, torch.int32
    x, xs = e4m3(T, n), (0.5 + torch.rand(T, 2, device="cuda")) / 100
    w1, s1 = e4m3(E, 2 * n, n), torch.full((E, 4, 2), n ** -0.5 / 100, device="cuda")
    w2, s2 = e4m3(E, n, n), torch.full((E, 2, 2), n ** -0.5 / 100, device="cuda")
    ids, places, rows = (torch.empty(s, dtype=i32, device="cuda") for s in ((T, k), (T, k), (T * k,)))
    weights, starts = torch.empty(T, k, device="cuda"), torch.empty(E + 1, dtype=i32, device="cuda")
    h, hs, y = torch.empty(T * k, n, dtype=U8, device="cuda"), torch.empty(T * k, 2, device="cuda"), torch.empty(T * k, n, dtype=BF, device="cuda")
    logits = [torch.randn(T, E, device="cuda") for _ in range(10)]

    def steps(wait):
        outs = [torch.empty(T, n, dtype=BF, device="cuda") for _ in logits]
        for l, out in zip(logits, outs):
            for call in (lambda: B.route_experts(l, k, ids, weights, starts, rows, places),
                         lambda: B.grouped_matmul(x, w1, starts, xs, s1, rows=rows, gated=True, out_codes=h, out_scales=hs),
                         lambda: B.grouped_matmul(h, w2, starts, hs, s2, out=y),
                         lambda: B.combine_experts(y, places, weights, out=out)):
                call()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs
    want = steps(True)
    assert not any(torch.equal(a, want[0]) for a in want[1:])
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(steps(False), want))


@pytest.mark.parametrize("N,K,kind,gated", [(128, 256, U8, False), (4096, 256, U8, False), (2048, 2048, BF, False), (8192, 256, U8, True)])
@pytest.mark.parametrize("starts", [[0, 639, 0, 640], [0, 639, 0, 600, 640], [0, 640] * 8, [0, 300, 100, 640, 639, 0, 640]])
def test_groups_that_overlap_keep_all_their_rows(B, starts, N, K, kind, gated):  # noqa: F811
    """Starts that go back: the group that does is skipped, and each element of the others' rows is the result of a group that
    its row lies in, although together they have more rows than there are.  (A row's columns are written tile by tile, so
    groups that share it may each have some of them.)"""
    M, E = 640, len(starts) - 1
    p = Product([M] + [0] * (E - 1), N, K, kind, gated=gated)
    each = []
    for e in range(E):                                           # every row by every group's weights
        p.starts_list = [0] * (e + 1) + [M] * (E - e)
        each.append(p.want())
    status, out = ints([0]), torch.full((M, N // 2 if gated else N), 7.0, device="cuda")
    p.starts = ints(starts)
    p.call(B, out=out, status=status)
    assert status.item() == 2
    for i in [0, 1, 63, 64, 99, 100, 255, 256, 299, 300, 599, 600, 638, 639]:
        groups = [e for e in range(E) if starts[e] <= i < starts[e + 1]]
        near = [(out[i].double() - each[e][0][i]).abs() <= each[e][1][i] + 2.0 ** -23 * each[e][0][i].abs() for e in groups]
        assert groups and torch.stack(near).any(0).all(), i


@pytest.mark.parametrize("T", [3, 100, 2000])
def test_the_gate_is_exact_to_a_few_units(B, T):  # noqa: F811
    """silu(g) u of products that are exact (one element of K to the gates, one to what they gate, each with a scale of its
    own), over all g: five units in the last place, 5 x 2^-23 of the result.  Below -87.3 exp(g) is subnormal, a number in
    steps of 2^-149 that g multiplies, and silu(g) has such steps too: (|g| + 1) 2^-149 more, times u, and the result's own."""
    torch.manual_seed(T)
    g = torch.cat([torch.linspace(-104, 90, T, device="cuda")[: T - 1], torch.full((1,), -88.5, device="cuda")])
    u = (10.0 ** (8 * torch.rand(T, device="cuda"))) * torch.where(torch.rand(T, device="cuda") < 0.5, -1.0, 1.0)
    x, w = torch.zeros(T, 256, dtype=U8, device="cuda"), torch.zeros(512, 256, dtype=U8, device="cuda")
    x[:, 5], x[:, 200], w[:256, 5], w[256:, 200] = 0x38, 0x38, 0x38, 0x38             # ones
    out = torch.empty(T, 256, device="cuda")
    B.fp8_matmul(x, torch.stack([g, u], 1).contiguous(), w, torch.ones(4, 2, device="cuda"), gated=True, out=out)
    want = g.double() / (1 + torch.exp(-g.double())) * u.double()
    bar = 5 * 2.0 ** -23 * want.abs() + 2.0 ** -149 * (1 + (g.double().abs() + 1) * u.double().abs())
    assert ((out.double() - want[:, None]).abs() <= bar[:, None]).all()


@pytest.mark.parametrize("size", [30.0, 1e3, 1e6])
def test_run_values_whose_large_parts_cancel(B, size):  # noqa: F811
    """A run's value is the sum of its best two: where a bias makes them large and of opposite signs, the sum is small but as
    uncertain in FP32 as they are."""
    torch.manual_seed(2)
    bias = torch.tensor([size, -size] * 3 + [0.3, 0.2] * 3, device="cuda")
    for T in (60, 400):
        logits = torch.randn(T, 12, device="cuda")
        check_route(B, logits, 4, "sigmoid", bias, 6, 3)
        check_route(B, logits, 2, "softmax", bias, 6, 2)
        check_route(B, logits, 2, "softmax", bias[torch.randperm(12)], 3, 1)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_weights_to_a_few_units(B, dtype):  # noqa: F811
    """A sigmoid: its exponential off by one unit in the last place, sum and quotient by half of one each: two.  Divided by a
    sum of 16 such in five additions, 2 + 2 + 2.5, a quotient and the scale half each: 7.5 units, below 2^-20, and half a step
    of a subnormal number.  A softmax's difference is off by 2^-24 |l - max l|, twice (the sum's too), its sum of 16 to a lane
    and five between lanes by 10.5 units: below 2^-19 with the same quotients."""
    torch.manual_seed(8)
    T, E, k, i32 = 300, 64, 16, torch.int32
    logits = torch.cat([torch.randn(T, E - 8, device="cuda") * 3, torch.linspace(-100, 100, 8 * T, device="cuda").view(8, T).T], 1).to(dtype)
    logits[0] = -88.5 + 0.01 * logits[0]
    l = logits.double()
    for scoring, scale in (("sigmoid", 1.0), ("sigmoid", 2.5), ("softmax", 1.0)):
        s = 1 / (1 + torch.exp(-l)) if scoring == "sigmoid" else torch.softmax(l, 1)
        for normalize in (False, True):
            ids, places, rows = (torch.empty(x, dtype=i32, device="cuda") for x in ((T, k), (T, k), (T * k,)))
            weights, starts = torch.empty(T, k, device="cuda"), torch.empty(E + 1, dtype=i32, device="cuda")
            B.route_experts(logits, k, ids, weights, starts, rows, places, scoring=scoring, normalize=normalize, scale=scale)
            want = s.gather(1, ids.long())
            if normalize:
                want = want / want.sum(1, keepdim=True)
            want = want * scale
            rel = 2.0 ** -20 if scoring == "sigmoid" else 2.0 ** -19 + 2.0 ** -23 * (l.amax(1, keepdim=True) - l.gather(1, ids.long()))
            assert ((weights.double() - want).abs() <= rel * want + 2.0 ** -149 * scale).all(), (scoring, scale, normalize)


def test_a_shared_expert_beside_the_others_in_a_graph(B):  # noqa: F811
    """A captured step that forks: the shared expert's products on a stream of their own beside the router and the experts',
    joined before the sum, replayed with other inputs, against the same calls one after the other."""
    torch.manual_seed(9)
    T, E, k, n, i32 = 70, 8, 2, 512, torch.int32
    x, xs, logits = e4m3(T, n), (0.5 + torch.rand(T, 4, device="cuda")) / 100, torch.randn(T, E, device="cuda")
    w1, s1, w2, s2 = e4m3(E + 1, 2 * n, n), torch.full((E + 1, 8, 4), 4e-4, device="cuda"), e4m3(E + 1, n, n), torch.full((E + 1, 4, 4), 4e-4, device="cuda")
    ids, places, rows = (torch.empty(s, dtype=i32, device="cuda") for s in ((T, k), (T, k), (T * k,)))
    weights, starts = torch.empty(T, k, device="cuda"), torch.empty(E + 1, dtype=i32, device="cuda")
    h, hs, y = torch.empty(T * k, n, dtype=U8, device="cuda"), torch.empty(T * k, 4, device="cuda"), torch.empty(T * k, n, dtype=BF, device="cuda")
    g, gs, shared, out = torch.empty(T, n, dtype=U8, device="cuda"), torch.empty(T, 4, device="cuda"), torch.empty(T, n, dtype=BF, device="cuda"), torch.empty(T, n, dtype=BF, device="cuda")

    def experts():
        B.route_experts(logits, k, ids, weights, starts, rows, places)
        B.grouped_matmul(x, w1[:E], starts, xs, s1[:E], rows=rows, gated=True, out_codes=h, out_scales=hs)
        B.grouped_matmul(h, w2[:E], starts, hs, s2[:E], out=y)

    def beside():
        B.fp8_matmul(x, xs, w1[E], s1[E], gated=True, out_codes=g, out_scales=gs)
        B.fp8_matmul(g, gs, w2[E], s2[E], out=shared)

    def plain():
        experts(), beside()
        torch.cuda.synchronize()
        return B.combine_experts(y, places, weights, add=shared).clone()
    plain()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            beside()
        experts()
        main.wait_stream(side)
        B.combine_experts(y, places, weights, add=shared, out=out)
    for _ in range(20):
        x.copy_(e4m3(T, n)), logits.copy_(torch.randn(T, E, device="cuda")), xs.copy_((0.5 + torch.rand(T, 4, device="cuda")) / 100)
        want = plain()
        for t in (ids, places, rows, starts, h, g, y, shared, out, hs, gs, weights):
            t.zero_()
        graph.replay()
        assert torch.equal(out, want)
