"""Cases of the operators behind the norm's 8-bit rows: the matrix product with a scale for each block of 128, the
products grouped by expert, the router that makes the groups, and the weighted sum that brings the experts' rows back
to their tokens.

`run` computes an operator in its plain form (elementary torch operations) or, with `own`, through the library's
binding; `exact` computes it from its definition in 64 bits.
"""

import torch

own = False

GROUP = 128        # elements that share one scale of an 8-bit row; weights have one for 128 x 128
FP8_MAX = 448.0    # largest E4M3 value
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one user's new token through a projection down to a latent: latency
        {"name": "projection one row", "op": "matmul", "tokens": 1, "k": 7168, "n": 2112, "gated": False, "out": "bf16"},
        # a decode batch through the first half of a gated feed-forward layer, 8-bit rows out
        {"name": "gated batch", "op": "matmul", "tokens": 64, "k": 7168, "n": 4096, "gated": True, "out": "fp8"},
        # a chunk of a long prompt through an output projection
        {"name": "projection chunk", "op": "matmul", "tokens": 8192, "k": 7168, "n": 7168, "gated": False, "out": "bf16"},
        # odd sizes: a prompt of 1003 tokens, widths that no tile divides, 32-bit logits out
        {"name": "projection odd", "op": "matmul", "tokens": 1003, "k": 1040, "n": 577, "gated": False, "out": "fp32"},
        # one token's eight experts: latency, eight weights of which each serves one row
        {"name": "experts one token", "op": "grouped", "tokens": 1, "top": 8, "experts": 64, "k": 7168, "n": 4096, "gather": True,
         "type": "fp8", "gated": True, "out": "fp8"},
        # a decode batch's first expert product: few rows to an expert, every expert's weights are read
        {"name": "experts batch", "op": "grouped", "tokens": 64, "top": 8, "experts": 64, "k": 7168, "n": 4096, "gather": True,
         "type": "fp8", "gated": True, "out": "fp8"},
        # a prefill chunk's first expert product
        {"name": "experts chunk", "op": "grouped", "tokens": 8192, "top": 8, "experts": 64, "k": 7168, "n": 4096, "gather": True,
         "type": "fp8", "gated": True, "out": "fp8"},
        # the second product of unquantised experts over sorted rows, ragged, some experts without a row
        {"name": "experts ragged 16-bit", "op": "grouped", "tokens": 1500, "top": 4, "experts": 61, "k": 1408, "n": 2048, "gather": False,
         "type": "bf16", "gated": False, "out": "bf16"},
        # the router of a decode step, experts chosen within the best 4 of 8 groups
        {"name": "route batch", "op": "route", "tokens": 64, "experts": 256, "top": 8, "groups": 8, "top_groups": 4, "scoring": "sigmoid",
         "bias": True, "type": "fp32"},
        # and of a chunk
        {"name": "route chunk", "op": "route", "tokens": 8192, "experts": 256, "top": 8, "groups": 8, "top_groups": 4, "scoring": "sigmoid",
         "bias": True, "type": "fp32"},
        # the experts' rows of a decode batch back to its tokens, beside a shared expert's
        {"name": "combine batch", "op": "combine", "tokens": 64, "top": 8, "n": 7168, "add": True, "type": "bf16"},
        # and of a chunk
        {"name": "combine chunk", "op": "combine", "tokens": 8192, "top": 8, "n": 7168, "add": True, "type": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "matmul", "grouped", "grouped", "grouped", "route", "combine"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        top_groups = rng.randint(1, groups)
        experts = groups * _spread(rng, 2, 256 // groups)
        return {"op": op, "tokens": _spread(rng, 1, 8192), "experts": experts, "top": rng.randint(1, min(8, experts // groups * top_groups)),
                "groups": groups, "top_groups": top_groups, "scoring": rng.choice(["sigmoid", "softmax"]), "bias": rng.random() < 0.5,
                "type": rng.choice(["fp32", "bf16"])}
    if op == "combine":
        return {"op": op, "tokens": _spread(rng, 1, 8192), "top": rng.randint(1, 8), "n": _spread(rng, 16, 7168), "add": rng.random() < 0.5,
                "type": rng.choice(["bf16", "fp16", "fp32"])}
    gated = rng.random() < 0.4
    n = 128 * _spread(rng, 1, 32) if gated else _spread(rng, 16, 4096)
    k = rng.choice([16 * _spread(rng, 1, 448), 128 * _spread(rng, 1, 56)])
    if op == "matmul":
        return {"op": op, "tokens": _spread(rng, 1, 8192), "k": k, "n": n if gated else _spread(rng, 16, 7168), "gated": gated,
                "out": rng.choice(["bf16", "fp8"] if gated else ["bf16", "fp16", "fp32"])}
    kind = rng.choice(["fp8", "fp8", "bf16", "fp16"])
    experts = rng.choice([1, 3, 8, 16, 64])
    return {"op": op, "tokens": _spread(rng, 1, 4096), "top": rng.randint(1, min(8, experts)), "experts": experts, "k": k, "n": n,
            "gather": rng.random() < 0.5, "type": kind, "gated": gated,
            "out": "fp8" if gated and kind == "fp8" else "bf16" if kind == "fp8" else kind}


# ------------------------------------------------------------------------------------------------- the inputs
def _choices(case):
    """Each token's experts [tokens, top], the same for every seed so that the work of a case is a fixed number: some
    experts are chosen four times as often as others, and one in sixteen hardly ever."""
    g = torch.Generator().manual_seed(case["tokens"] * 1009 + case["experts"])
    n = case["experts"]
    lean = 1.4 * torch.arange(n).mul(0.618034).frac() - 9.0 * (torch.arange(n) % 16 == 5)
    noise = -(-torch.rand(case["tokens"], n, generator=g).clamp(1e-6, 1 - 1e-6).log()).log()
    return (noise + lean).topk(case["top"], 1).indices


def _quantised(x):
    """E4M3 codes (uint8) of a matrix's rows and one scale for each 128 elements, by the library's rule."""
    n = x.shape[1]
    y = torch.nn.functional.pad(x.float(), (0, -n % GROUP)).view(x.shape[0], -1, GROUP)
    amax = y.abs().amax(-1)
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / FP8_MAX)
    return (y / scale[..., None]).to(torch.float8_e4m3fn).flatten(1)[:, :n].contiguous().view(torch.uint8), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    empty = lambda *shape, dtype: torch.empty(*shape, device="cuda", dtype=dtype)  # noqa: E731
    s, t = dict(case), case["tokens"]
    if case["op"] == "route":
        e, top = case["experts"], case["top"]
        s["logits"] = (1.5 * rand(t, e)).to(TYPES[case["type"]])
        s["correction"] = 0.05 * rand(e) if case["bias"] else None
        s["ids"], s["places"] = empty(t, top, dtype=torch.int32), empty(t, top, dtype=torch.int32)
        s["weights"] = empty(t, top, dtype=torch.float32)
        s["starts"], s["rows"] = empty(e + 1, dtype=torch.int32), empty(t * top, dtype=torch.int32)
        return s
    if case["op"] == "combine":
        kind, n, top = TYPES[case["type"]], case["n"], case["top"]
        s["y"] = rand(t * top, n).to(kind)
        s["shared"] = rand(t, n).to(kind) if case["add"] else None
        s["places"] = torch.randperm(t * top, generator=g, device="cuda").view(t, top).int()
        weights = torch.rand(t, top, generator=g, device="cuda") + 0.05
        s["weights"] = 2.5 * weights / weights.sum(1, keepdim=True)
        s["result"] = empty(t, n, dtype=kind)
        return s

    k, n, grouped = case["k"], case["n"], case["op"] == "grouped"
    e, blocks = (case["experts"], -(-n // GROUP)) if grouped else (1, -(-n // GROUP))
    m = t * case["top"] if grouped else t
    source = t if not grouped or case["gather"] else m  # rows of x
    if grouped:
        ids = _choices(case).cuda()[torch.randperm(t, generator=g, device="cuda")].flatten()  # the same counts for every seed
        s["starts"] = torch.cat([ids.new_zeros(1), torch.cumsum(torch.bincount(ids, minlength=e), 0)]).int()
        s["rows"] = (torch.argsort(ids, stable=True) // case["top"]).int() if case["gather"] else None
        s["most"] = int(_choices(case).flatten().bincount().max())
    if not grouped or case["type"] == "fp8":
        s["x"], s["x_scale"] = _quantised(rand(source, k))
        # weights with a deviation of K^-1/2, the scale of each block its largest element's
        s["w"] = empty(e, n, k, dtype=torch.uint8)
        for one in s["w"]:
            one.copy_((110 * rand(n, k)).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8))
        s["w_scale"] = k ** -0.5 / 110 * (0.8 + 0.4 * torch.rand(e, blocks, -(-k // GROUP), generator=g, device="cuda"))
        if not grouped:
            s["w"], s["w_scale"] = s["w"][0], s["w_scale"][0]
    else:
        kind = TYPES[case["type"]]
        s["x"] = rand(source, k).to(kind)
        s["w"] = empty(e, n, k, dtype=kind)
        for one in s["w"]:
            one.copy_(k ** -0.5 * rand(n, k))
        s["x_scale"] = s["w_scale"] = None
    width = n // 2 if case["gated"] else n
    if case["out"] == "fp8":
        s["result"] = None
        s["codes"], s["scales"] = empty(m, width, dtype=torch.uint8), empty(m, -(-width // GROUP), dtype=torch.float32)
    else:
        s["result"], s["codes"], s["scales"] = empty(m, width, dtype=TYPES[case["out"]]), None, None
    return s


# ------------------------------------------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    return {"matmul": _matmul, "grouped": _grouped, "route": _route, "combine": _combine}[s["op"]](s)


def _own(s):
    from dsa_sparse_attention_fp8_gb300 import binding as B

    if s["op"] == "route":
        B.route_experts(s["logits"], s["top"], s["ids"], s["weights"], s["starts"], s["rows"], s["places"], scoring=s["scoring"],
                        bias=s["correction"], num_groups=s["groups"], top_groups=s["top_groups"], normalize=True, scale=2.5)
        return s["ids"], s["weights"], s["starts"], s["rows"], s["places"]
    if s["op"] == "combine":
        return B.combine_experts(s["y"], s["places"], s["weights"], add=s["shared"], out=s["result"])
    if s["op"] == "matmul":
        B.fp8_matmul(s["x"], s["x_scale"], s["w"], s["w_scale"], gated=s["gated"], out=s["result"], out_codes=s["codes"], out_scales=s["scales"])
    else:
        B.grouped_matmul(s["x"], s["w"], s["starts"], s["x_scale"], s["w_scale"], rows=s["rows"], gated=s["gated"], out=s["result"],
                         out_codes=s["codes"], out_scales=s["scales"])
    return s["result"] if s["codes"] is None else (s["codes"].view(torch.float8_e4m3fn), s["scales"])


def _values(codes, scales, rows):
    """The FP32 values of E4M3 matrices with a scale for each `rows` x 128 block."""
    wide = scales.repeat_interleave(GROUP, -1)[..., : codes.shape[-1]]
    if rows > 1:
        wide = wide.repeat_interleave(rows, -2)[..., : codes.shape[-2], :]
    return codes.view(torch.float8_e4m3fn).float() * wide


def _finish(s, y):
    """The activation, then the one rounding, of a product's FP32 rows."""
    if s["gated"]:
        gate, up = y.chunk(2, 1)
        y = gate / (1 + torch.exp(-gate)) * up
    if s["codes"] is None:
        return y.to(s["result"].dtype)
    codes, scales = _quantised(y)
    return codes.view(torch.float8_e4m3fn), scales


def _matmul(s):
    return _finish(s, _values(s["x"], s["x_scale"], 1) @ _values(s["w"], s["w_scale"], GROUP).T)


def _grouped(s):
    x, w = s["x"], s["w"]
    x = x.float() if s["x_scale"] is None else _values(x, s["x_scale"], 1)
    w = w.float() if s["w_scale"] is None else _values(w, s["w_scale"], GROUP)
    if s["rows"] is not None:
        x = x[s["rows"].long()]
    starts = s["starts"].long()
    m = x.shape[0]
    at = starts[:-1, None] + torch.arange(s["most"], device="cuda")  # each expert's rows, padded to the most of any
    y = x[at.clamp(max=m - 1)] @ w.transpose(1, 2)
    i = torch.arange(m, device="cuda")
    e = torch.searchsorted(starts, i, right=True) - 1
    return _finish(s, y[e, i - starts[e]])


def _route(s):
    logits, t, n = s["logits"].double(), s["tokens"], s["experts"]
    score = torch.sigmoid(logits) if s["scoring"] == "sigmoid" else torch.softmax(logits, 1)
    value = score if s["correction"] is None else score + s["correction"].double()
    if s["groups"] > 1:
        inside = value.view(t, s["groups"], -1)
        best = inside.sort(dim=2, descending=True).values[:, :, :2].sum(2)
        chosen = best.sort(dim=1, descending=True, stable=True).indices[:, : s["top_groups"]]
        kept = torch.zeros_like(best, dtype=torch.bool).scatter_(1, chosen, True)
        value = inside.masked_fill(~kept[:, :, None], -torch.inf).view(t, n)
    ids = value.sort(dim=1, descending=True, stable=True).indices[:, : s["top"]]
    weights = score.gather(1, ids)
    weights = 2.5 * weights / weights.sum(1, keepdim=True)
    flat = ids.flatten()
    order = flat.argsort(stable=True)
    places = torch.empty_like(order)
    places[order] = torch.arange(order.numel(), device="cuda")
    starts = torch.searchsorted(flat[order], torch.arange(n + 1, device="cuda"))
    return ids.int(), weights.float(), starts.int(), (order // s["top"]).int(), places.view(t, -1).int()


def _combine(s):
    out = (s["y"][s["places"].long()].float() * s["weights"][..., None]).sum(1)
    if s["shared"] is not None:
        out = out + s["shared"].float()
    return out.to(s["result"].dtype)


# ------------------------------------------------------------------------------------------------- work and exact values
def work(case):
    t, top = case["tokens"], case.get("top", 1)
    if case["op"] == "route":
        e = case["experts"]
        return {"bytes": t * e * TYPES[case["type"]].itemsize + 16 * t * top + 4 * (e + 1) + (4 * e if case["bias"] else 0), "flops": 8 * t * e}
    if case["op"] == "combine":
        n, size = case["n"], TYPES[case["type"]].itemsize
        return {"bytes": t * n * size * (top + 1 + case["add"]) + 8 * t * top, "flops": 2 * t * top * n}
    k, n, kind = case["k"], case["n"], case.get("type", "fp8")
    size = 1 if kind == "fp8" else 2
    scales = 4 if kind == "fp8" else 0
    m, used, source, extra = t, 1, t, 0
    if case["op"] == "grouped":
        m, used, source = t * top, _choices(case).unique().numel(), t if case["gather"] else t * top
        extra = 4 * (case["experts"] + 1) + (4 * m if case["gather"] else 0)
    width = n // 2 if case["gated"] else n
    out = width + 4 * -(-width // GROUP) if case["out"] == "fp8" else width * TYPES[case["out"]].itemsize
    weight = n * k * size + scales * -(-n // GROUP) * -(-k // GROUP)
    return {"bytes": used * weight + source * (k * size + scales * -(-k // GROUP)) + m * out + extra, "flops": 2 * m * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "combine":
        out = s["shared"].double() if case["add"] else torch.zeros(case["tokens"], case["n"], dtype=torch.float64, device="cuda")
        for j in range(case["top"]):
            out = torch.addcmul(out, s["weights"][:, j, None].double(), s["y"][s["places"][:, j].long()].double())
        return out
    if case["op"] == "route":
        l = s["logits"].double()
        p = 1 / (1 + torch.exp(-l)) if case["scoring"] == "sigmoid" else torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
        v = p + s["correction"].double() if case["bias"] else p.clone()
        per = case["experts"] // case["groups"]
        if case["groups"] > 1:
            best = torch.stack([c.topk(min(2, per), 1).values.sum(1) for c in v.split(per, 1)], 1)
            rank = (best[:, None, :] > best[:, :, None]).sum(2) + torch.tril(best[:, None, :] == best[:, :, None], -1).sum(2)
            v = v.masked_fill((rank >= case["top_groups"]).repeat_interleave(per, 1), -torch.inf)
        taken = []
        for _ in range(case["top"]):
            best = (v == v.max(1, keepdim=True).values).int().argmax(1, keepdim=True)  # the lowest index of the largest
            taken.append(p.gather(1, best))
            v = v.scatter(1, best, -torch.inf)
        w = torch.cat(taken, 1)
        return None, 2.5 * w / w.sum(1, keepdim=True), None, None, None
    # products, one expert and a slice of rows at a time
    if case["op"] == "matmul":
        bounds, weights, w_scale = [0, case["tokens"]], s["w"][None], s["w_scale"][None]
    else:
        bounds, weights, w_scale = s["starts"].tolist(), s["w"], s["w_scale"]
    x, wide = s["x"], lambda scale, n: scale.double().repeat_interleave(GROUP, 1)[:, :n]  # noqa: E731
    out = []
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if a == b:
            continue
        w = weights[e]
        if w_scale is None:
            w = w.double()
        else:
            w = w.view(torch.float8_e4m3fn).double() * wide(wide(w_scale[e], case["k"]).T, case["n"]).T
        take = torch.arange(a, b, device="cuda") if s.get("rows") is None else s["rows"][a:b].long()
        for part in take.split(2048):
            r = x[part]
            r = r.double() if w_scale is None else r.view(torch.float8_e4m3fn).double() * wide(s["x_scale"][part], case["k"])
            y = r @ w.T
            if case["gated"]:
                h = case["n"] // 2
                y = y[:, :h] * torch.sigmoid(y[:, :h]) * y[:, h:]
            out.append(y)
    y = torch.cat(out)
    if case["out"] != "fp8":
        return y
    scale = torch.stack([g.abs().max(1).values for g in y.split(GROUP, 1)], 1) / FP8_MAX
    scale[scale == 0] = 1
    return y / wide(scale, y.shape[1]), scale
