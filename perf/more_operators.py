"""Operators of an expert layer as measured cases: the gated feed-forward block and its gradients, matrix products
in 8-bit integers, and rows gathered to the experts and combined back.

`run` computes one case with plain torch operations, or, with `own` set, with this package's
kernels (`muon_newton_schulz_momentum_amd.experts`); `exact` gives the same outputs from
the operators' definitions in float64.

    gated     h = act(x G^T) * (x U^T) for rows x of k values and matrices G, U of n x k; with `groups`
              experts the rows offsets[e] .. offsets[e + 1] - 1 go by matrices G[e], U[e].  act(v): v / (1 + exp(-v))
              (silu), v * P(N < v) (gelu), max(v, 0) (relu).  The operands are bfloat16, or 8-bit integers
              with a float32 scale for each row of either.  With `save`, x G^T and x U^T come back too.
    backward  from the gradient d of h, and the saved g = x G^T and u = x U^T as bfloat16: dg = d u act'(g),
              du = d act(g), and the gradients of x, dg G + du U, of G, dg^T x and of U, du^T x, the last two
              over each expert's rows (zeros for an expert without rows).
    quantize  a row's scale is s = max |x| / 127 in float32, its codes are x / s to the nearest whole number, ties
              to even (0 where s is 0); rows are padded to multiples of 128 codes with zeros.
    product   (sum over k of a's codes times b's) times a's row's scale times b's row's scale: one
              matrix by another (groups 0), or row segments each by its expert's matrix.
    combine   out[t] = sum over j of weights[t][j] * y[position[t][j]], and backwards dy[r] = weights[c] * d[c / top_k] for
              the choice c in row r (zeros in a row that pads a segment, rows behind the last segment stay as
              they were), dweights[c] = sum of d[c / top_k] * y[r] (0 for a choice without a row).
"""
import math

import numpy as np
import torch

own = False

NUM = {"f32": torch.float32, "bf16": torch.bfloat16}


def up(v, step):
    return -(-v // step) * step


# ---- cases ------------------------------------------------------------------------------

def listed():
    return [
        # one token through a dense 2048 -> 5632 gated projection: the smallest serving call, bound by the weights
        dict(name="gated_token", op="gated", type="bf16", groups=0, rows=1, n=5632, k=2048, act="silu", save=False),
        # one decoding step of 16 sequences through 512 experts, 8-bit integer weights: each touched expert's once
        dict(name="gated_decode", op="gated", type="int8", groups=512, rows=112, n=1024, k=4096, act="silu", save=False),
        # a training microbatch through 128 experts, uneven loads, what the backward pass needs saved
        dict(name="gated_train", op="gated", type="bf16", groups=128, rows=57344, n=1024, k=4096, act="silu", save=True),
        # the gradients of such a layer's 64 experts: of the rows and of both projections
        dict(name="backward_experts", op="backward", groups=64, rows=28672, n=1024, k=4096, act="silu"),
        # the gradients of a dense block for an odd number of tokens
        dict(name="backward_dense", op="backward", groups=0, rows=8191, n=5632, k=2048, act="gelu"),
        # the decoding step's rows, gathered into expert order
        dict(name="quantize_decode", op="quantize", batch=1, rows=112, cols=4096, type="bf16", per=7),
        # a long prompt's activations at the full width
        dict(name="quantize_prompt", op="quantize", batch=1, rows=16381, cols=8704, type="bf16", per=0),
        # one token through a dense down projection
        dict(name="product_token", op="product", groups=0, rows=1, n=2048, k=5632, out="bf16"),
        # the decoding step's rows through the 512 experts' down projections
        dict(name="product_decode", op="product", groups=512, rows=112, n=4096, k=1024, out="bf16"),
        # a long prompt of an odd number of tokens through a dense down projection, float32
        dict(name="product_prompt", op="product", groups=0, rows=16381, n=2048, k=5632, out="f32"),
        # the decoding step's rows back to their 16 tokens
        dict(name="combine_decode", op="combine", tokens=16, top_k=7, groups=512, cols=4096, type="bf16", align=1,
             padded=0, backward=False),
        # a training microbatch's rows back to their tokens, both directions, some tokens without experts
        dict(name="combine_train", op="combine", tokens=8192, top_k=7, groups=512, cols=4096, type="bf16", align=16,
             padded=37, backward=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "backward", "quantize", "product", "product", "combine"])
    if op == "combine":
        groups = _log(rng, 8, 512)
        cols, top_k = _log(rng, 64, 8704), rng.randint(1, min(8, groups))
        tokens = _log(rng, 1, max(2, min(8192, (230 << 20) // (cols * top_k))))
        return dict(op=op, tokens=tokens, top_k=top_k, groups=groups, cols=cols, type=rng.choice(["bf16", "bf16", "f32"]),
                    align=rng.choice([1, 16, 128]), padded=rng.choice([0, 0, tokens // 16]), backward=rng.random() < 0.5)
    if op == "quantize":
        batch, cols = rng.choice([1, 1, 8]), _log(rng, 64, 16000)
        rows = _log(rng, 1, max(2, min(50000, (140 << 20) // (cols * batch))))
        return dict(op=op, batch=batch, rows=rows, cols=cols, type=rng.choice(["f32", "bf16"]),
                    per=rng.choice([0, 1, 7]) if batch == 1 else 0)
    groups = rng.choice([0, _log(rng, 1, 128)])
    n, k = _log(rng, 64, 5632), _log(rng, 64, 5632)
    while groups * n * k > 1 << 29:
        groups //= 2
    most = {"gated": 2.2e11, "backward": 1.1e11, "product": 1.8e11}[op]
    rows = _log(rng, 1, max(2, min(57344, int(most) // (n * k))))
    case = dict(op=op, groups=groups, rows=rows, n=n, k=k)
    if op == "product":
        return dict(case, out=rng.choice(["bf16", "f32"]))
    case["act"] = rng.choice(["silu", "silu", "gelu", "relu"])
    if op == "backward":
        return case
    kind = rng.choice(["bf16", "bf16", "int8"])
    return dict(case, type=kind, save=kind == "bf16" and rng.random() < 0.5)


def loads(case):
    """Rows of each group: uneven, some empty; fixed by the case, dealt to the experts by the seed."""
    g = np.random.Generator(np.random.PCG64([case["groups"], case["rows"], 23]))
    share = np.exp(g.normal(0.0, 0.5, case["groups"]))
    return g.multinomial(case["rows"], share / share.sum())


# ---- inputs -----------------------------------------------------------------------------

def _int8(gen, shape):
    """Codes and scales of normal values in the padded layout, a few rows at a time."""
    *lead, rows, cols = shape
    total = rows * (lead[0] if lead else 1)
    codes = torch.zeros(total, up(cols, 128), dtype=torch.int8, device="cuda")
    scales = torch.empty(total, device="cuda")
    step = max(1, (1 << 28) // cols)
    for i in range(0, total, step):
        x = torch.randn(min(step, total - i), cols, device="cuda", generator=gen)
        s = x.abs().amax(-1, keepdim=True) / 127
        codes[i:i + step, :cols] = (x / s).round().to(torch.int8)
        scales[i:i + step] = s[:, 0] / math.sqrt(cols)
    return codes.view(*lead, rows, -1), scales.view(*lead, rows)


def _bf16(gen, *shape, std=1.0):
    out = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
    for part in out.view(-1).split(1 << 28):
        part.copy_(torch.randn(part.numel(), device="cuda", generator=gen) * std)
    return out


def _segments(st, case, seed):
    """Offsets of the experts' rows, which experts have rows, and where each of their rows lies, padded to the longest."""
    sizes = loads(case)[np.random.Generator(np.random.PCG64(seed)).permutation(case["groups"])]
    ends = np.concatenate([[0], np.cumsum(sizes)])
    present = np.nonzero(sizes)[0]
    at = ends[present][:, None] + np.arange(int(sizes.max()))[None, :]
    st["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    st["present"] = torch.tensor(present, device="cuda")
    st["inside"] = torch.tensor(at < ends[present + 1][:, None], device="cuda")
    st["at"] = torch.tensor(np.minimum(at, case["rows"] - 1), device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 29)
    st = dict(case=case)
    if case["op"] == "quantize":
        B, R, K, per = case["batch"], case["rows"], case["cols"], case["per"]
        S = -(-R // per) if per else R
        x = torch.randn(B, S, K, device="cuda", generator=gen)
        x *= torch.exp(torch.randn(B, 1, K, device="cuda", generator=gen))   # some channels are large
        x = x.to(NUM[case["type"]])
        st["src"] = x if B > 1 else x[0]
        if per:
            # every choice once, in some expert order, then the unused end of the list
            used = R - R // 50
            rows = torch.randperm(S * per, device="cuda", generator=gen)[:R].to(torch.int32)
            rows[torch.randperm(R, device="cuda", generator=gen)[:R // 20]] = -1          # segment padding
            rows[used:] = -1
            st["rows"] = rows
            st["limit"] = torch.tensor([used], dtype=torch.int32, device="cuda")
            # buffers kept from batch to batch: rows behind the limit stay as they are
            st["out"] = [torch.zeros(R, up(K, 128), dtype=torch.int8, device="cuda"), torch.zeros(R, device="cuda")]
        return st
    if case["op"] == "combine":
        T, k, E, d, align = (case[x] for x in ("tokens", "top_k", "groups", "cols", "align"))
        popular = torch.randn(E, device="cuda", generator=gen)
        noise = -torch.log(-torch.log(torch.rand(T, E, device="cuda", generator=gen).clamp(1e-9, 1 - 1e-7)))
        chosen = (noise + popular).topk(k, dim=-1).indices
        w = torch.rand(T, k, device="cuda", generator=gen) + 0.05
        w = w / w.sum(-1, keepdim=True)
        if case["padded"]:
            chosen[T - case["padded"]:] = E
            w[T - case["padded"]:] = 0.0
        flat = chosen.reshape(-1)
        n = T * k
        counts = torch.bincount(flat, minlength=E + 1)
        order = flat.sort(stable=True).indices
        padded = (counts[:E] + align - 1) // align * align
        offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), padded.cumsum(0)])
        place = offsets[flat[order].clamp(max=E - 1)] + torch.arange(n, device="cuda") - (counts.cumsum(0) - counts)[flat[order]]
        placed = flat[order] < E
        capacity = up(n + min(n, E) * (align - 1), align)
        rows = torch.full((capacity,), -1, dtype=torch.int32, device="cuda")
        rows[place[placed]] = order[placed].to(torch.int32)
        position = torch.full((n,), -1, dtype=torch.int32, device="cuda")
        position[order[placed]] = place[placed].to(torch.int32)
        st.update(weights=w, rows=rows, position=position.view(T, k), limit=offsets[-1:].to(torch.int32))
        st["y"] = torch.randn(capacity, d, device="cuda", generator=gen).to(NUM[case["type"]])
        if case["backward"]:
            st["grad"] = torch.randn(T, d, device="cuda", generator=gen).to(NUM[case["type"]])
            # kept from batch to batch: rows behind the last segment stay as they are
            st["grad_y"] = torch.zeros(capacity, d, device="cuda", dtype=NUM[case["type"]])
        return st
    G, R, n, k = (case[x] for x in ("groups", "rows", "n", "k"))
    lead = (G,) if G else ()
    if case["op"] == "product":
        st["a"], st["b"] = _int8(gen, (R, k)), _int8(gen, (*lead, n, k))
    elif case["op"] == "gated" and case["type"] == "int8":
        st["x"], st["gate"], st["up"] = _int8(gen, (R, k)), _int8(gen, (*lead, n, k)), _int8(gen, (*lead, n, k))
        st["x"][1].mul_(math.sqrt(k))
    else:
        st["x"] = _bf16(gen, R, k)
        st["gate"], st["up"] = (_bf16(gen, *lead, n, k, std=1 / math.sqrt(k)) for _ in range(2))
        if case["op"] == "backward":
            st["grad"], st["pre_gate"], st["pre_up"] = _bf16(gen, R, n, std=0.1), _bf16(gen, R, n), _bf16(gen, R, n)
    if G:
        _segments(st, case, seed)
    return st


# ---- plain forms ------------------------------------------------------------------------

def _plain_act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return g * 0.5 * torch.erfc(g * -math.sqrt(0.5)) if act == "gelu" else torch.where(g > 0, g, 0.0)


def _plain_act_grad(g, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    if act == "gelu":
        return 0.5 * torch.erfc(g * -math.sqrt(0.5)) + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    return torch.where(g > 0, 1.0, 0.0)


def _plain_values(t, k, rows=None):
    """float32 values of bfloat16 numbers, or the whole numbers of codes beside their rows' scales."""
    if isinstance(t, tuple):
        codes, scales = t if rows is None else (t[0][rows], t[1][rows])
        return codes[..., :k].float(), scales
    return (t if rows is None else t[rows]).float(), None


def _plain_product(st, c, a, b):
    """Rows of a times the transpose of b, each row's by its expert's matrix; both scaled."""
    if not c["groups"]:
        (x, sx), (w, sw) = _plain_values(a, c["k"]), _plain_values(b, c["k"])
        y = x @ w.T
        return y if sx is None else y * sx[:, None] * sw
    at, inside = st["at"], st["inside"]
    (x, sx), (w, sw) = _plain_values(a, c["k"], at), _plain_values(b, c["k"], st["present"])
    y = torch.bmm(x, w.transpose(1, 2).contiguous())           # every present expert's rows, padded to the longest segment
    if sx is not None:
        y = y * sx[:, :, None] * sw[:, None, :]
    out = torch.zeros(c["rows"], c["n"], device="cuda")
    out[at[inside]] = y[inside]
    return out


def _plain_gated(st, c):
    g, u = _plain_product(st, c, st["x"], st["gate"]), _plain_product(st, c, st["x"], st["up"])
    h = (_plain_act(g, c["act"]) * u).bfloat16()
    return [h, g.bfloat16(), u.bfloat16()] if c["save"] else [h]


def _plain_backward(st, c):
    g, u, d, x = (st[v].float() for v in ("pre_gate", "pre_up", "grad", "x"))
    dg, du = d * u * _plain_act_grad(g, c["act"]), d * _plain_act(g, c["act"])
    if not c["groups"]:
        return [v.bfloat16() for v in (dg @ st["gate"].float() + du @ st["up"].float(), dg.T @ x, du.T @ x)]
    at, inside, present = st["at"], st["inside"], st["present"]
    dg, du, x = (torch.where(inside[..., None], v[at], 0.0) for v in (dg, du, x))
    y = torch.bmm(dg, st["gate"][present].float()) + torch.bmm(du, st["up"][present].float())
    dx = torch.zeros(c["rows"], c["k"], device="cuda", dtype=torch.bfloat16)
    dx[at[inside]] = y[inside].bfloat16()
    out = torch.zeros(2, c["groups"], c["n"], c["k"], device="cuda", dtype=torch.bfloat16)
    out[0, present] = torch.bmm(dg.transpose(1, 2).contiguous(), x).bfloat16()
    out[1, present] = torch.bmm(du.transpose(1, 2).contiguous(), x).bfloat16()
    return [dx, out[0], out[1]]


def _plain_quantize(st, c):
    x = st["src"].float()
    if c["per"]:
        rows = st["rows"].long()
        live = (rows >= 0) & (torch.arange(c["rows"], device="cuda") < st["limit"])
        x = torch.where(live[:, None], x[rows.clamp(min=0) // c["per"]], 0.0)
    s = (x.abs().amax(-1, keepdim=True).double() / 127).float()
    q = x.double() / s                                         # 64 bits: some quotients lie next to a border
    codes = torch.where(s > 0, q, 0.0).round().clamp(-127, 127).to(torch.int8)
    out = [torch.nn.functional.pad(codes, (0, up(c["cols"], 128) - c["cols"])), s[..., 0]]
    if c["per"]:
        kept = torch.arange(c["rows"], device="cuda") >= st["limit"]
        st["out"][0].copy_(torch.where(kept[:, None], st["out"][0], out[0]))
        st["out"][1].copy_(torch.where(kept, st["out"][1], out[1]))
        out = st["out"]
    return out


def _plain_combine(st, c):
    y, position, w = st["y"], st["position"].long(), st["weights"]
    there = position >= 0
    rows_y = y[position.clamp(min=0)].float()
    out = [torch.where(there[..., None], w[..., None] * rows_y, 0.0).sum(1).to(y.dtype)]
    if c["backward"]:
        d = st["grad"].float()
        choice = st["rows"].long()
        at = choice.clamp(min=0)
        dy = torch.where(choice[:, None] >= 0, w.reshape(-1)[at][:, None] * d[at // c["top_k"]], 0.0).to(y.dtype)
        kept = torch.arange(choice.numel(), device="cuda") >= st["limit"]
        st["grad_y"].copy_(torch.where(kept[:, None], st["grad_y"], dy))
        dw = torch.where(there, (d[:, None] * rows_y).sum(-1), 0.0)
        out += [st["grad_y"], dw]
    return out


# ---- one pass ---------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if not own:
        if c["op"] == "product":
            return _plain_product(state, c, state["a"], state["b"]).to(NUM[c["out"]])
        return {"gated": _plain_gated, "backward": _plain_backward, "quantize": _plain_quantize,
                "combine": _plain_combine}[c["op"]](state, c)
    from muon_newton_schulz_momentum_amd import experts
    if c["op"] == "quantize":
        kept = None if "out" not in state else experts.Int8(*state["out"], c["cols"])
        q = experts.quantize_int8(state["src"], rows=state.get("rows"), per=c["per"] or 1, limit=state.get("limit"), out=kept)
        return [q.codes, q.scales]
    if c["op"] == "combine":
        out = [experts.combine_rows(state["y"], state["position"], state["weights"])]
        if c["backward"]:
            out += experts.combine_rows_backward(state["grad"], state["y"], state["rows"], state["position"], state["weights"],
                                                 limit=state["limit"], out=state["grad_y"])
        return out
    if c["op"] == "product":
        a, b = (experts.Int8(*state[v], c["k"]) for v in "ab")
        return experts.product_int8(a, b, offsets=state.get("offsets"), dtype=NUM[c["out"]])
    if c["op"] == "backward":
        return list(experts.gated_backward(state["grad"], state["x"], state["gate"], state["up"], state["pre_gate"],
                                           state["pre_up"], activation=c["act"], offsets=state.get("offsets")))
    x, gate, up_ = (experts.Int8(*state[v], c["k"]) if c["type"] == "int8" else state[v] for v in ("x", "gate", "up"))
    out = experts.gated(x, gate, up_, activation=c["act"], offsets=state.get("offsets"), save=c["save"])
    return list(out) if c["save"] else [out]


def work(case):
    """Bytes and operations of one pass that nothing can avoid: every input read and every output written once."""
    c = case
    if c["op"] == "quantize":
        size = 4 if c["type"] == "f32" else 2
        n, R, K = c["batch"] * c["rows"] * c["cols"], c["rows"], c["cols"]
        return {"bytes": (-(-R // c["per"]) * K if c["per"] else n) * size + n, "flops": 3 * n}
    if c["op"] == "combine":
        size = 4 if c["type"] == "f32" else 2
        n, d = (c["tokens"] - c["padded"]) * c["top_k"], c["cols"]
        both = c["backward"]
        return {"bytes": (n * (2 if both else 1) + c["tokens"] * (2 if both else 1)) * d * size + n * (16 if both else 8),
                "flops": (5 if both else 2) * n * d}
    G, R, n, k = c["groups"], c["rows"], c["n"], c["k"]
    used = int((loads(c) > 0).sum()) if G else 1
    if c["op"] == "product":
        return {"bytes": R * k + used * n * k + R * n * (4 if c["out"] == "f32" else 2), "flops": 2.0 * R * n * k}
    if c["op"] == "gated":
        size = 1 if c["type"] == "int8" else 2
        return {"bytes": (R * k + 2 * used * n * k) * size + R * n * (6 if c["save"] else 2), "flops": 4.0 * R * n * k}
    return {"bytes": 2 * (3 * R * n + 2 * R * k + 2 * used * n * k + 2 * max(G, 1) * n * k), "flops": 8.0 * R * n * k}


# ---- the definitions in 64 bits ---------------------------------------------------------

def _exact_matrix(t, k):
    if isinstance(t, tuple):
        return t[0][..., :k].double() * t[1][..., None].double()
    return t.double()


def _exact_spans(st, c):
    if not c["groups"]:
        return [(None, 0, c["rows"])]
    ends = st["offsets"].tolist()
    return [(g, ends[g], ends[g + 1]) for g in range(c["groups"]) if ends[g + 1] > ends[g]]


def _exact_part(t, g):
    if g is None:
        return t
    return (t[0][g], t[1][g]) if isinstance(t, tuple) else t[g]


def _exact_rows(t, lo, hi):
    return (t[0][lo:hi], t[1][lo:hi]) if isinstance(t, tuple) else t[lo:hi]


def _exact_product(st, c, a, b):
    out = torch.zeros(c["rows"], c["n"], dtype=torch.float64, device="cuda")
    for g, lo, hi in _exact_spans(st, c):
        out[lo:hi] = _exact_matrix(_exact_rows(a, lo, hi), c["k"]) @ _exact_matrix(_exact_part(b, g), c["k"]).T
    return out


def _exact_gated(st, c):
    g, u = _exact_product(st, c, st["x"], st["gate"]), _exact_product(st, c, st["x"], st["up"])
    a = {"silu": lambda v: v * torch.sigmoid(v), "gelu": lambda v: v * torch.special.ndtr(v),
         "relu": lambda v: v.clamp(min=0)}[c["act"]](g)
    return [a * u, g, u] if c["save"] else [a * u]


def _exact_backward(st, c):
    g, u, d, x = (st[v].double() for v in ("pre_gate", "pre_up", "grad", "x"))
    if c["act"] == "silu":
        p = torch.sigmoid(g)
        act, slope = g * p, p + g * p * torch.sigmoid(-g)
    elif c["act"] == "gelu":
        p = torch.special.ndtr(g)
        act, slope = g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    else:
        slope = (g > 0).double()
        act = g * slope
    dg, du = d * u * slope, d * act
    dx = torch.zeros(c["rows"], c["k"], dtype=torch.float64, device="cuda")
    out = torch.zeros(2, max(c["groups"], 1), c["n"], c["k"], dtype=torch.float64, device="cuda")
    for g_, lo, hi in _exact_spans(st, c):
        G, U = _exact_part(st["gate"], g_).double(), _exact_part(st["up"], g_).double()
        dx[lo:hi] = dg[lo:hi] @ G + du[lo:hi] @ U
        out[0, g_ or 0], out[1, g_ or 0] = dg[lo:hi].T @ x[lo:hi], du[lo:hi].T @ x[lo:hi]
    if not c["groups"]:
        out = out[:, 0]
    return [dx, out[0], out[1]]


def _exact_quantize(st, c):
    x = st["src"].double()
    if c["per"]:
        rows = st["rows"].long().clone()
        rows[int(st["limit"]):] = -1
        x = torch.where(rows[:, None] >= 0, x[torch.div(rows.clamp(min=0), c["per"], rounding_mode="floor")], 0.0)
    # codes are defined by the scale as it is kept, in float32
    s = (x.abs().amax(-1) / 127).float()
    x = x / torch.where(s > 0, s, 1.0).double()[..., None]
    low = torch.floor(x)
    part = x - low
    codes = low + ((part > 0.5) | ((part == 0.5) & (low % 2 != 0))).double()
    wide = torch.zeros(*codes.shape[:-1], up(c["cols"], 128), dtype=torch.int8, device="cuda")
    wide[..., :c["cols"]] = codes.clamp(-127, 127).to(torch.int8)
    return [wide, s.double()]


def _exact_combine(st, c):
    y, w = st["y"].double(), st["weights"].double()
    position = st["position"].long()
    T, k, d = c["tokens"], c["top_k"], c["cols"]
    out = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    grad_y = torch.zeros_like(y)
    grad_w = torch.zeros_like(w)
    for j in range(k):
        t = torch.nonzero(position[:, j] >= 0)[:, 0]
        p = position[t, j]
        out[t] += w[t, j, None] * y[p]
        if c["backward"]:
            g = st["grad"][t].double()
            grad_y[p] = w[t, j, None] * g
            grad_w[t, j] = (g * y[p]).sum(-1)
    return [out, grad_y, grad_w] if c["backward"] else [out]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "product":
        return _exact_product(st, case, st["a"], st["b"])
    return {"gated": _exact_gated, "backward": _exact_backward, "quantize": _exact_quantize,
            "combine": _exact_combine}[case["op"]](st, case)
