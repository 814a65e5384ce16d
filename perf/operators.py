"""The routed expert operators as measured cases: routing, grouping rows by expert, 8-bit block
quantisation and 8-bit products.

`run` computes one case with plain torch operations, or, with `own` set, with this package's
kernels (`muon_newton_schulz_momentum_amd.experts`); `exact` gives the same outputs from
the operators' definitions in float64.

    route     x: logits (T, E).  A logit of -inf or NaN takes its expert out for the token; +inf
              counts as the largest finite value.  Scores s: softmax over the token's
              experts, or sigmoid.  Key: s + bias, or x where there is no bias.  With groups, the
              experts of the `top_groups` groups with the largest sums of their two largest
              scores (plus bias) stay.  The top_k largest keys are chosen, ties to the lowest
              index, in falling order; missing ones are -1 with weight 0.  Weights:
              scale * s, or scale * s / (sum of the chosen s) (0 where that sum is 0).
    group     the T * k choices in stable order of their expert, each expert's segment padded to
              a multiple of `align` with -1; then the balance step of the selection bias,
              bias + rate * sign(mean load - load).
    quantize  blocks of 1 x 128 or 128 x 128 values share the scale 2^e, e the least with
              amax <= 448 * 2^e (e4m3; 57344 for e5m2), clamped to [-127, 127]; a code is the value
              * 2^-e rounded once, to nearest even.  Rows are padded to multiples of 128 codes and of
              4 scales (padding is a block of zeros: code 0, scale 2^-127).  The transposed copy's
              blocks run along the other dimension.
    product   sums over k of the values the codes stand for: one matrix by another
              (dense), row segments each by its expert's matrix (rows), or column
              segments of both operands, a result per expert (depth: weight gradients).
"""
import math

import numpy as np
import torch

own = False

E4M3, E5M2, E8M0 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
BLOCK = 128
NUM = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": E4M3, "e5m2": E5M2}
F32_MAX = 3.4028234663852886e38


def up(v, step):
    return -(-v // step) * step


# ---- cases ------------------------------------------------------------------------------

def listed():
    return [
        # one decoding step of 16 sequences through a 512-expert router: latency
        dict(name="route_decode", op="route", tokens=16, experts=512, top_k=7, score="sigmoid", bias=True, groups=1,
             top_groups=1, renormalize=True, scale=1.0, dtype="f32", backward=False, padded=0),
        # a training microbatch, bf16 logits, device-limited groups, both directions, padding tokens
        dict(name="route_train", op="route", tokens=8192, experts=512, top_k=7, score="sigmoid", bias=True, groups=8,
             top_groups=4, renormalize=True, scale=2.5, dtype="bf16", backward=True, padded=37),
        # a long packed batch through a softmax router, float32 logits, whole-row gradient
        dict(name="route_long", op="route", tokens=65537, experts=512, top_k=7, score="softmax", bias=False, groups=1,
             top_groups=1, renormalize=False, scale=1.0, dtype="f32", backward=True, padded=0),
        # the same decoding step's 112 choices, no padding
        dict(name="group_decode", op="group", tokens=16, top_k=7, experts=512, align=1, padded=0),
        # a long packed batch's choices, segments padded for the 128-blocks of the weight gradients
        dict(name="group_long", op="group", tokens=65537, top_k=7, experts=512, align=128, padded=100),
        # the decoding step's rows, gathered into expert order
        dict(name="quantize_decode", op="quantize", batch=1, rows=112, cols=4096, dtype="bf16", block="row",
             format="e4m3", transpose=False, per=7),
        # a training microbatch's tokens gathered into expert order, with the copy for the weight gradients
        dict(name="quantize_tokens", op="quantize", batch=1, rows=57344, cols=4096, dtype="bf16", block="row",
             format="e4m3", transpose=True, per=7),
        # 64 experts' float32 master weights after a step, both orientations
        dict(name="quantize_weights", op="quantize", batch=64, rows=1024, cols=4096, dtype="f32", block="square",
             format="e4m3", transpose=True, per=0),
        # the decoding step's rows through the 512 experts' gate: each touched expert's weights from memory
        dict(name="product_decode", op="product", mode="rows", groups=512, rows=112, n=1024, k=4096, format="e4m3",
             out="bf16"),
        # a training microbatch through the gates of 128 experts, uneven loads
        dict(name="product_experts", op="product", mode="rows", groups=128, rows=57344, n=1024, k=4096, format="e4m3",
             out="bf16"),
        # weight gradients of 64 experts' down projections, e5m2 gradients, float32 for the step
        dict(name="product_weight_grad", op="product", mode="depth", groups=64, rows=28672, n=1024, k=4096,
             format="e5m2", out="f32"),
        # a dense 2048 -> 5632 projection of an odd number of tokens
        dict(name="product_dense", op="product", mode="dense", groups=1, rows=16381, n=5632, k=2048, format="e4m3",
             out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "group", "quantize", "quantize", "product", "product", "product"])
    if op in ("route", "group"):
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 8, 512 // groups)
        top_groups = rng.randint(max(1, groups // 2), groups)
        top_k = rng.randint(1, min(12, experts // groups * top_groups))
        tokens = _log(rng, 1, 60000)
        padded = rng.choice([0, 0, tokens // 16])
        if op == "group":
            return dict(op=op, tokens=tokens, top_k=top_k, experts=experts, align=rng.choice([1, 16, 128]), padded=padded)
        return dict(op=op, tokens=tokens, experts=experts, top_k=top_k, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, renormalize=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]), backward=rng.random() < 0.6,
                    padded=padded)
    if op == "quantize":
        block, cols = rng.choice(["row", "row", "square"]), _log(rng, 128, 8704)
        batch = rng.randint(1, 16) if block == "square" else 1
        rows = _log(rng, 1, max(2, min(50000, (200 << 20) // (cols * batch))))
        return dict(op=op, batch=batch, rows=rows, cols=cols, dtype=rng.choice(["f32", "bf16"]), block=block,
                    format=rng.choice(["e4m3", "e4m3", "e5m2"]), transpose=rng.random() < 0.5,
                    per=rng.choice([0, 1, 7]) if block == "row" else 0)
    mode = rng.choice(["rows", "rows", "depth", "dense"])
    groups = 1 if mode == "dense" else _log(rng, 1, 128)
    n, k = _log(rng, 128, 5632), _log(rng, 128, 5632)
    while groups * n * k > 1 << (28 if mode == "depth" else 29):
        groups = max(1, groups // 2)
        n, k = (n, k) if groups > 1 else (min(n, 4096), min(k, 4096))
    rows = _log(rng, 1, max(2, min(57344, int(2.0e11) // (n * k))))
    return dict(op=op, mode=mode, groups=groups, rows=rows, n=n, k=k, format=rng.choice(["e4m3", "e4m3", "e5m2"]),
                out=rng.choice(["bf16", "f32"]))


def loads(case):
    """Rows of each group: uneven, some empty; fixed by the case, dealt to the experts by the seed."""
    g = np.random.Generator(np.random.PCG64([case["groups"], case["rows"], 17]))
    share = np.exp(g.normal(0.0, 0.5, case["groups"]))
    return g.multinomial(case["rows"], share / share.sum())


# ---- inputs -----------------------------------------------------------------------------

def _codes(gen, shape, fmt, square):
    """Quantised normal values of `shape` in the padded layout, made expert by expert."""
    *lead, rows, cols = shape
    n = lead[0] if lead else 1
    kp, kb = up(cols, BLOCK), -(-cols // BLOCK)
    srows = -(-rows // BLOCK) if square else rows
    codes = torch.empty(n, rows, kp, dtype=NUM[fmt], device="cuda")
    scales = torch.zeros(n, srows, up(kb, 4), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (rows * kp))
    for i in range(0, n, step):
        m = min(step, n - i)
        x = torch.zeros(m, rows, kp, device="cuda")
        x[:, :, :cols] = torch.randn(m, rows, cols, device="cuda", generator=gen)
        x *= torch.exp(0.5 * torch.randn(m, rows, 1, device="cuda", generator=gen))
        c, s = _plain_blocks(x, fmt, square)
        codes[i:i + m] = c
        scales[i:i + m, :, :kb] = s.view(torch.uint8)
    scales = scales.view(E8M0)
    return (codes, scales) if lead else (codes[0], scales[0])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 13)
    st = dict(case=case)
    if case["op"] == "route":
        T, E = case["tokens"], case["experts"]
        x = torch.randn(T, E, device="cuda", generator=gen) * 1.5
        if E >= 16:
            x[:, (seed * 31) % E] = -math.inf                     # an expert that is switched off
        if case["padded"]:
            x[T - case["padded"]:] = -math.inf                    # padding tokens go nowhere
        st["logits"] = x.to(NUM[case["dtype"]])
        st["bias"] = torch.randn(E, device="cuda", generator=gen) * 0.05 if case["bias"] else None
        st["grad"] = torch.randn(T, case["top_k"], device="cuda", generator=gen)
        return st
    if case["op"] == "group":
        T, E = case["tokens"], case["experts"]
        popular = torch.randn(E, device="cuda", generator=gen)
        noise = -torch.log(-torch.log(torch.rand(T, E, device="cuda", generator=gen).clamp(1e-9, 1 - 1e-7)))
        ex = (noise + popular).topk(case["top_k"], dim=-1).indices.to(torch.int32)
        if case["padded"]:
            ex[T - case["padded"]:] = -1
        st["experts"] = ex
        st["bias"] = torch.randn(E, device="cuda", generator=gen) * 0.05
        return st
    if case["op"] == "quantize":
        B, R, K, per = case["batch"], case["rows"], case["cols"], case["per"]
        S = -(-R // per) if per else R
        x = torch.randn(B, S, K, device="cuda", generator=gen)
        x *= torch.exp(torch.randn(B, 1, K, device="cuda", generator=gen))   # some channels are large
        st["src"] = x.to(NUM[case["dtype"]])
        if case["block"] == "row":
            st["src"] = st["src"][0]
        if per:
            # every choice once, in some expert order, then the unused end of the list
            used = R - R // 50
            rows = torch.randperm(S * per, device="cuda", generator=gen)[:R].to(torch.int32)
            rows[torch.randperm(R, device="cuda", generator=gen)[:R // 20]] = -1          # segment padding
            rows[used:] = -1
            st["rows"] = rows
            st["limit"] = torch.tensor([used], dtype=torch.int32, device="cuda")
            kb, rb, f = -(-K // BLOCK), -(-R // BLOCK), NUM[case["format"]]
            zero = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
            # buffers kept from batch to batch: rows behind the limit stay as they are
            st["out"] = [zero(R, kb * BLOCK).view(f), zero(R, up(kb, 4)).view(E8M0)]
            if case["transpose"]:
                st["out"] += [zero(K, rb * BLOCK).view(f), zero(K, up(rb, 4)).view(E8M0)]
        return st
    mode, G, R, n, k = (case[x] for x in ("mode", "groups", "rows", "n", "k"))
    sizes = loads(case)[np.random.Generator(np.random.PCG64(seed)).permutation(G)]
    if mode == "dense":
        st["a"], st["b"] = _codes(gen, (R, k), case["format"], False), _codes(gen, (n, k), "e4m3", True)
        return st
    step = 128 if mode == "depth" else 1
    padded = -(-sizes // step) * step
    ends = np.concatenate([[0], np.cumsum(padded)])
    st["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    if mode == "rows":
        st["a"], st["b"] = _codes(gen, (R, k), case["format"], False), _codes(gen, (G, n, k), "e4m3", True)
    else:
        total = max(int(ends[-1]), 128)
        st["a"], st["b"] = _codes(gen, (n, total), case["format"], False), _codes(gen, (k, total), "e4m3", False)
        pos = np.concatenate([np.arange(e - p + s, e) for s, p, e in zip(sizes, padded, ends[1:])] or [np.zeros(0)])
        pos = torch.tensor(pos.astype(np.int64), device="cuda")
        for codes, _ in (st["a"], st["b"]):
            codes.view(torch.uint8)[:, pos] = 0                   # the columns that pad a segment
    # which experts have rows, and where each of their rows (or columns) lies, padded to the longest
    present = np.nonzero(sizes)[0]
    longest = int(padded.max())
    at = ends[present][:, None] + np.arange(longest)[None, :]
    st["present"] = torch.tensor(present, device="cuda")
    st["inside"] = torch.tensor(at < ends[present + 1][:, None], device="cuda")
    st["at"] = torch.tensor(np.minimum(at, max(int(ends[-1]) - 1, 0)), device="cuda")
    return st


# ---- plain forms ------------------------------------------------------------------------

def _scores(logits, score):
    """Scores in float64: the choice sits on their borders."""
    x = logits.double().clamp(max=F32_MAX)
    there = x > -math.inf
    if score == "sigmoid":
        return x, there, torch.where(there, torch.sigmoid(x), 0.0)
    top = torch.where(there, x, -math.inf).amax(-1, keepdim=True)
    e = torch.where(there, torch.exp(x - top), 0.0)
    z = e.sum(-1, keepdim=True)
    return x, there, torch.where(z > 0, e / z, 0.0)


def _plain_route(st, c):
    x, there, s = _scores(st["logits"], c["score"])
    biased = s if st["bias"] is None else s + st["bias"].double()
    if c["groups"] > 1:
        in_groups = torch.where(there, biased, -math.inf).unflatten(-1, (c["groups"], -1))
        two = in_groups.topk(min(2, in_groups.shape[-1]), dim=-1).values
        worth = torch.where(two > -math.inf, two, 0.0).sum(-1)
        worth = torch.where(two[..., 0] > -math.inf, worth, -math.inf)
        best = worth.sort(dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros_like(worth, dtype=torch.bool).scatter_(1, best, True)
        there = there & kept.repeat_interleave(in_groups.shape[-1], dim=-1)
    key = torch.where(there, x if st["bias"] is None else biased, -math.inf)
    order = key.sort(dim=-1, descending=True, stable=True)
    chosen = order.indices[:, :c["top_k"]]
    taken = order.values[:, :c["top_k"]] > -math.inf
    w = torch.where(taken, s.gather(1, chosen), 0.0)
    total = w.sum(-1, keepdim=True)
    if c["renormalize"]:
        w = torch.where(total > 0, w / total, 0.0)
    out = [torch.where(taken, chosen, -1).to(torch.int32), (w * c["scale"]).float()]
    if c["backward"]:
        g = torch.where(taken, st["grad"].double() * c["scale"], 0.0)
        if c["renormalize"]:
            g = torch.where(total > 0, (g - (g * w).sum(-1, keepdim=True)) / total, 0.0)
        ds = torch.zeros_like(s).scatter_add_(1, chosen, torch.where(taken, g, 0.0))
        if c["score"] == "sigmoid":
            dx = ds * s * (1.0 - s)
        else:
            dx = s * (ds - (ds * s).sum(-1, keepdim=True))
        out.append(dx.to(st["logits"].dtype))
    return out


def _capacity(c):
    n = c["tokens"] * c["top_k"]
    return up(n + min(n, c["experts"]) * (c["align"] - 1), c["align"])


def _plain_group(st, c):
    E, align = c["experts"], c["align"]
    flat = st["experts"].reshape(-1).long()
    n, cap = flat.numel(), _capacity(c)
    key = torch.where(flat < 0, E, flat)
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda").scatter_add_(0, key, torch.ones_like(key))
    starts = counts.cumsum(0) - counts
    padded = (counts[:E] + align - 1) // align * align
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = padded.cumsum(0)
    order = key.sort(stable=True).indices
    sorted_key = key[order]
    place = offsets[sorted_key.clamp(max=E - 1)] + torch.arange(n, device="cuda") - starts[sorted_key]
    place = torch.where(sorted_key < E, place, cap)
    rows = torch.full((cap + 1,), -1, dtype=torch.int32, device="cuda")
    rows[place] = torch.where(sorted_key < E, order, -1).to(torch.int32)
    position = torch.empty(n, dtype=torch.int32, device="cuda")
    position[order] = torch.where(place < cap, place, -1).to(torch.int32)
    counts = counts[:E]
    bias = st["bias"] + 0.001 * torch.sign(counts.sum() - counts * E).float()
    return [counts.to(torch.int32), offsets.to(torch.int32), rows[:cap], position.view_as(st["experts"]), bias]


def _plain_blocks(x, fmt, square):
    """Codes and scales of x (float32, both last sizes' padding included; rows padded here)."""
    rows, kp = x.shape[-2], x.shape[-1]
    if square:
        x = torch.nn.functional.pad(x, (0, 0, 0, up(rows, BLOCK) - rows))
        t = x.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK))           # .., rb, 128, kb, 128
        amax = t.abs().amax((-1, -3), keepdim=True)
    else:
        t = x.unflatten(-1, (-1, BLOCK))
        amax = t.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)
    e = e - (9 if fmt == "e4m3" else 16) + (m > 0.875).to(e.dtype)            # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e, -127).clamp(-127, 127)
    inverse = ((127 - e) << 23).view(torch.float32)                           # 2^-e
    codes = (t * inverse).to(NUM[fmt])
    scales = (e + 127).to(torch.uint8)
    if square:
        return codes.view(torch.uint8).reshape(x.shape)[..., :rows, :].view(NUM[fmt]), scales[..., 0, :, 0].view(E8M0)
    return codes.view(torch.uint8).reshape(x.shape).view(NUM[fmt]), scales[..., 0].view(E8M0)


def _pad_last(t, n):
    return torch.nn.functional.pad(t, (0, n - t.shape[-1]))


def _plain_quantize(st, c):
    x = st["src"].float()
    if c["per"]:
        rows = st["rows"].long()
        live = (rows >= 0) & (torch.arange(c["rows"], device="cuda") < st["limit"])
        x = torch.where(live[:, None], x[rows.clamp(min=0) // c["per"]], 0.0)
    square, fmt = c["block"] == "square", c["format"]

    def one(v):
        codes, scales = _plain_blocks(_pad_last(v, up(v.shape[-1], BLOCK)), fmt, square)
        wide = up(scales.shape[-1], 4)
        return codes, _pad_last(scales.view(torch.uint8), wide).view(E8M0)
    out = list(one(x))
    if c["transpose"]:
        out += one(x.transpose(-1, -2).contiguous())
    if c["per"]:
        for buf, new in zip(st["out"], out):
            buf.copy_(new)
        out = st["out"]
    return out


def _values(pair, square, rows=None):
    """float32 values of codes and scales; of the stack's matrices or of the rows `rows` alone."""
    codes, scales = pair
    if rows is not None:
        codes = codes.view(torch.uint8)[rows].view(codes.dtype)
        scales = scales.view(torch.uint8)[rows].view(E8M0)
    kb = codes.shape[-1] // BLOCK
    s = scales[..., :kb].float()
    if square:
        s = s.repeat_interleave(BLOCK, dim=-2)[..., :codes.shape[-2], :]
    return (codes.float().unflatten(-1, (kb, BLOCK)) * s.unsqueeze(-1)).flatten(-2)


def _plain_product(st, c):
    out_t = NUM[c["out"]]
    if c["mode"] == "dense":
        return (_values(st["a"], False) @ _values(st["b"], True).T).to(out_t)
    at, inside = st["at"], st["inside"]
    if c["mode"] == "rows":
        # every present expert's rows, padded to the longest segment, in one batched product
        x = _values(st["a"], False)[at]
        y = torch.bmm(x, _values(st["b"], True, st["present"]).transpose(1, 2).contiguous())
        out = torch.zeros(c["rows"], c["n"], device="cuda", dtype=out_t)
        out[at[inside]] = y[inside].to(out_t)
        return out
    a = torch.where(inside[:, None, :], _values(st["a"], False)[:, at].transpose(0, 1), 0.0)
    b = _values(st["b"], False)[:, at].transpose(0, 1)
    out = torch.zeros(c["groups"], c["n"], c["k"], device="cuda", dtype=out_t)
    out[st["present"]] = torch.bmm(a.contiguous(), b.transpose(1, 2).contiguous()).to(out_t)
    return out


# ---- one pass ---------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if not own:
        return {"route": _plain_route, "group": _plain_group, "quantize": _plain_quantize,
                "product": _plain_product}[c["op"]](state, c)
    from muon_newton_schulz_momentum_amd import experts
    if c["op"] == "route":
        chosen, weights = experts.route(state["logits"], c["top_k"], bias=state["bias"], score=c["score"],
                                        groups=c["groups"], top_groups=c["top_groups"],
                                        renormalize=c["renormalize"], scale=c["scale"])
        if not c["backward"]:
            return [chosen, weights]
        return [chosen, weights, experts.route_backward(state["logits"], chosen, state["grad"], score=c["score"],
                                                        renormalize=c["renormalize"], scale=c["scale"])]
    if c["op"] == "group":
        g = experts.group_rows(state["experts"], c["experts"], align=c["align"])
        bias = experts.balance_step(state["bias"], g.counts, 0.001)
        return [g.counts, g.offsets, g.rows, g.position, bias]
    if c["op"] == "quantize":
        kept = state.get("out")
        if kept is not None:
            shape = (c["rows"], c["cols"])
            kept = [experts.Fp8(kept[i], kept[i + 1], shape[1 - i // 2], False) for i in range(0, len(kept), 2)]
        got = experts.quantize(state["src"], block=c["block"], format=c["format"], transpose=c["transpose"],
                               rows=state.get("rows"), per=c["per"] or 1, limit=state.get("limit"), out=kept)
        return [t for q in (got if c["transpose"] else [got]) for t in (q.codes, q.scales)]
    cols = c["rows"] if c["mode"] == "depth" else c["k"]
    if c["mode"] == "depth":
        cols = state["a"][0].shape[-1]
    a = experts.Fp8(*state["a"], cols, False)
    b = experts.Fp8(*state["b"], cols, c["mode"] != "depth")
    return experts.product(a, b, offsets=state.get("offsets"), group=None if c["mode"] == "dense" else c["mode"],
                           dtype=NUM[c["out"]])


def work(case):
    """Bytes and operations of one pass that nothing can avoid: every input read and every output written once."""
    c = case
    if c["op"] == "route":
        size = 4 if c["dtype"] == "f32" else 2
        n, sel = c["tokens"] * c["experts"], c["tokens"] * c["top_k"]
        both = c["backward"]
        return {"bytes": n * size * (2 if both else 1) + sel * (12 if both else 8), "flops": n * (12 if both else 8)}
    if c["op"] == "group":
        n = c["tokens"] * c["top_k"]
        return {"bytes": 8 * n + 4 * _capacity(c) + 16 * c["experts"], "flops": n}
    if c["op"] == "quantize":
        size = 4 if c["dtype"] == "f32" else 2
        n, R, K = c["batch"] * c["rows"] * c["cols"], c["rows"], c["cols"]
        src = (-(-R // c["per"]) * K if c["per"] else n) * size
        return {"bytes": src + n * (2 if c["transpose"] else 1) * (1 + 1 / 128), "flops": 3 * n}
    G, R, n, k = c["groups"], c["rows"], c["n"], c["k"]
    out = 4 if c["out"] == "f32" else 2
    if c["mode"] == "depth":
        return {"bytes": R * (n + k) * (1 + 1 / 128) + G * n * k * out, "flops": 2.0 * R * n * k}
    used = 1 if c["mode"] == "dense" else int((loads(c) > 0).sum())
    return {"bytes": R * k * (1 + 1 / 128) + used * n * k + R * n * out, "flops": 2.0 * R * n * k}


# ---- the definitions in 64 bits ---------------------------------------------------------

def _exact_route(st, c):
    x = st["logits"].double().cpu().numpy()
    x = np.minimum(x, F32_MAX)
    T, E = x.shape
    there = x > -np.inf
    with np.errstate(all="ignore"):
        if c["score"] == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-x))
        else:
            s = np.exp(x - np.max(np.where(there, x, -np.inf), axis=1, keepdims=True))
            s = np.where(there, s, 0.0)
            s = s / np.maximum(s.sum(axis=1, keepdims=True), 1e-300)
    s = np.where(there, s, 0.0)
    bias = np.zeros(E) if st["bias"] is None else st["bias"].double().cpu().numpy()
    if c["groups"] > 1:
        v = np.where(there, s + bias, -np.inf).reshape(T, c["groups"], -1)
        v = -np.sort(-v, axis=2)[:, :, :2]
        worth = np.where(np.isfinite(v), v, 0.0).sum(axis=2)
        worth = np.where(np.isfinite(v[:, :, 0]), worth, -np.inf)
        keep = np.zeros_like(worth, dtype=bool)
        for _ in range(c["top_groups"]):
            best = np.argmax(np.where(keep, -np.inf, worth), axis=1)
            free = ~keep[np.arange(T), best]
            keep[np.arange(T)[free], best[free]] = True
        there = there & np.repeat(keep, E // c["groups"], axis=1)
    key = np.where(there, x if st["bias"] is None else s + bias, -np.inf)
    chosen, left = np.full((T, c["top_k"]), -1), key.copy()
    r = np.arange(T)
    for j in range(c["top_k"]):
        best = np.argmax(left, axis=1)
        ok = left[r, best] > -np.inf
        chosen[:, j] = np.where(ok, best, -1)
        left[r, best] = -np.inf
    taken = chosen >= 0
    sel = np.where(taken, s[r[:, None], chosen], 0.0)
    total = sel.sum(axis=1, keepdims=True)
    safe = np.where(total > 0, total, 1.0)
    w = sel / safe if c["renormalize"] else sel
    out = [chosen.astype(np.int32), w * c["scale"]]
    if c["backward"]:
        g = np.where(taken, st["grad"].double().cpu().numpy(), 0.0) * c["scale"]
        if c["renormalize"]:
            g = np.where(total > 0, (g - (g * w).sum(axis=1, keepdims=True)) / safe, 0.0)
        dx = np.zeros((T, E))
        if c["score"] == "sigmoid":
            np.put_along_axis(dx, np.where(taken, chosen, 0), 0.0, axis=1)
            for j in range(c["top_k"]):
                ok = taken[:, j]
                dx[r[ok], chosen[ok, j]] += (g * sel * (1.0 - sel))[ok, j]
        else:
            dx = -s * (g * sel).sum(axis=1, keepdims=True)
            for j in range(c["top_k"]):
                ok = taken[:, j]
                dx[r[ok], chosen[ok, j]] += (g * sel)[ok, j]
        out.append(dx)
    return out


def _exact_group(st, c):
    ex = st["experts"].cpu().numpy()
    flat, E, align = ex.reshape(-1), c["experts"], c["align"]
    counts = np.bincount(flat[flat >= 0], minlength=E)
    offsets = np.concatenate([[0], np.cumsum(-(-counts // align) * align)])
    rows, position = np.full(_capacity(c), -1), np.full(flat.size, -1)
    for e in range(E):
        ids = np.nonzero(flat == e)[0]
        rows[offsets[e]:offsets[e] + ids.size] = ids
        position[ids] = offsets[e] + np.arange(ids.size)
    bias = st["bias"].double().cpu().numpy() + 0.001 * np.sign(counts.sum() - counts * E)
    return [counts.astype(np.int32), offsets.astype(np.int32), rows.astype(np.int32),
            position.reshape(ex.shape).astype(np.int32), bias]


def _exact_blocks(x, fmt, square):
    """The values the codes and scales stand for, by arithmetic in float64."""
    *lead, rows, cols = x.shape
    kp = up(cols, BLOCK)
    height = up(rows, BLOCK) if square else rows
    big = torch.zeros(*lead, height, kp, dtype=torch.float64, device=x.device)
    big[..., :rows, :cols] = x
    tall = BLOCK if square else 1
    t = big.reshape(*lead, height // tall, tall, kp // BLOCK, BLOCK)
    amax = t.abs().amax(dim=(-3, -1), keepdim=True)
    limit, bits, lowest = (448.0, 3, -6) if fmt == "e4m3" else (57344.0, 2, -14)
    e = torch.ceil(torch.log2(torch.clamp(amax, min=1e-300) / limit))
    e = torch.where(amax > limit * torch.exp2(e), e + 1, e)
    e = torch.where(amax <= limit * torch.exp2(e - 1), e - 1, e).clamp(-127, 127)
    y = t * torch.exp2(-e)
    exponent = torch.frexp(y).exponent.sub_(1).clamp_(min=lowest)
    step = torch.exp2((exponent - bits).double())
    y = torch.round(y.div_(step)).mul_(step)
    s = torch.exp2(e).reshape(*lead, height // tall, kp // BLOCK)
    wide = torch.full((*lead, height // tall, up(kp // BLOCK, 4)), 2.0 ** -127, dtype=torch.float64, device=x.device)
    wide[..., :kp // BLOCK] = s
    return y.reshape(*lead, height, kp)[..., :rows, :], wide


def _exact_quantize(st, c):
    x = st["src"].double()
    if c["per"]:
        rows = st["rows"].long().clone()
        used = int(st["limit"])
        rows[used:] = -1
        x = torch.where(rows[:, None] >= 0, x[torch.div(rows.clamp(min=0), c["per"], rounding_mode="floor")], 0.0)
    square = c["block"] == "square"
    out = list(_exact_blocks(x, c["format"], square))
    if c["transpose"]:
        out += _exact_blocks(x.transpose(-1, -2), c["format"], square)
    return out


def _exact_values(codes, scales, square):
    v = codes.double()
    s = scales.double()
    for kb in range(v.shape[-1] // BLOCK):
        col = s[..., kb:kb + 1]
        if square:
            col = col.repeat_interleave(BLOCK, dim=-2)[..., :v.shape[-2], :]
        v[..., kb * BLOCK:(kb + 1) * BLOCK] *= col
    return v


def _exact_product(st, c):
    (ac, asc), (bc, bsc) = st["a"], st["b"]
    if c["mode"] == "dense":
        return _exact_values(ac, asc, False) @ _exact_values(bc, bsc, True).T
    ends = st["offsets"].tolist()
    if c["mode"] == "rows":
        out = torch.zeros(c["rows"], c["n"], dtype=torch.float64, device="cuda")
        for g in range(c["groups"]):
            lo, hi = ends[g], ends[g + 1]
            if hi > lo:
                out[lo:hi] = _exact_values(ac[lo:hi], asc[lo:hi], False) @ _exact_values(bc[g], bsc[g], True).T
        return out
    out = torch.zeros(c["groups"], c["n"], c["k"], dtype=torch.float64, device="cuda")
    for g in range(c["groups"]):
        lo, hi = ends[g], ends[g + 1]
        if hi > lo:
            a = _exact_values(ac[:, lo:hi], asc[:, lo // BLOCK:hi // BLOCK], False)
            out[g] = a @ _exact_values(bc[:, lo:hi], bsc[:, lo // BLOCK:hi // BLOCK], False).T
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"route": _exact_route, "group": _exact_group, "quantize": _exact_quantize,
            "product": _exact_product}[case["op"]](st, case)
