"""The expert layers' operators on the GPU against their float64 definitions (oracle/layers_oracle.py).

Tolerances.  u = 2^-24 is float32's half step, h = 2^-8 bfloat16's.
  * a sum of k bfloat16 products: the products are exact in float32; instructions add 16 of them at a time into a float32
    sum, and a tile may add up to 8 partial sums: (ceil(k / 16) + 16 + 8) roundings of at most 2 u (a sum that cuts
    off rather than rounds) of the sum of magnitudes S: sum_tol(k) S;
  * the activations' slopes are at most 1.13 (gelu; silu 1.1), so a pre-activation's error e moves the value by
    1.13 e and what lies beyond it in second order; 1.2 covers both here, where e is far below 1;
    the exponential's argument is off by 1.5 u (silu) or 2.5 u (gelu) of itself, v or v^2 / 2: 75 u at |v| < 7.7 (inputs here
    are normal with 1.5 or less), the fitted tail by 8 u, what is left is some 20 roundings and hardware steps of 2 u: 160 u;
  * 8-bit integer sums are exact: conversion to float32 and two products, 3 u;
  * every result: its own rounding, u or h, and 2^-126 where it is below the normal numbers;
  * codes and scales are compared for equality.
Gradients of x and of the weights are compared with the definition's of the pre-activations' gradients that the call
formed and rounded (with reuse they are left where the saved values were), and these with theirs.
"""
import itertools
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from oracle import layers_oracle as orc  # noqa: E402

U, H, TINY = 2.0 ** -24, 2.0 ** -8, 2.0 ** -126
HALF = {torch.float32: U, torch.bfloat16: H}
ACTS = ("silu", "gelu", "relu")


def X():
    from muon_newton_schulz_momentum_amd import experts
    return experts


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _np(t):
    return t.detach().double().cpu().numpy()


def sum_tol(k):
    return (-(-k // 16) + 24) * 2 * U


def _close(got, want, tol, what=""):
    got, off = _np(got), np.abs(_np(got) - want)
    worst = np.unravel_index(np.argmax(off - tol), off.shape) if off.size else ()
    assert (off <= tol).all(), f"{what} at {worst}: {got[worst]} is not {want[worst]} within {np.broadcast_to(tol, off.shape)[worst]}"


def _matrix(seed, *shape, std=1.0, dtype=torch.bfloat16, gap=0):
    """Normal values; with a gap between the rows, which holds NaN."""
    *lead, rows, cols = shape
    t = torch.full((*lead, rows, cols + gap), float("nan"), dtype=dtype, device="cuda")
    t[..., :cols] = (torch.randn(*shape, device="cuda", generator=_gen(seed)) * std).to(dtype)
    return t[..., :cols]


def _offsets(ends):
    return None if ends is None else torch.tensor(ends, dtype=torch.int32, device="cuda")


# rows, n, k, offsets, gap
SHAPES = [
    (1, 1, 1, None, 0),
    (1, 64, 64, None, 0),
    (2, 40, 96, None, 8),
    (3, 7, 31, None, 0),
    (5, 130, 8, None, 1),
    (17, 65, 257, None, 3),
    (33, 256, 128, None, 0),
    (64, 129, 200, None, 0),
    (129, 128, 64, None, 8),
    (255, 300, 192, None, 0),
    (257, 384, 320, None, 0),
    (300, 127, 999, None, 0),
    (513, 520, 130, None, 2),
    (1, 24, 40, [0, 1], 0),
    (1, 24, 40, [0, 0, 1, 1], 0),
    (7, 33, 72, [0, 0, 3, 3, 7], 0),
    (60, 64, 128, [5, 20, 20, 41], 0),                     # rows before the first and behind the last segment
    (60, 70, 65, [-3, 10, 30, 900], 5),                    # bounds outside the rows
    (300, 136, 264, [0, 1, 2, 130, 130, 299, 300], 0),
    (700, 257, 136, [0, 256, 300, 300, 699, 700], 8),
    (900, 128, 192, [0, 10, 520, 890], 0),
    (40, 96, 80, [20] * 9, 0),                             # no segment has a row
    (2000, 40, 24, list(range(0, 2001, 10)), 0),           # many short segments
    (1500, 512, 640, [0, 700, 1500], 0),
    (1100, 1024, 512, None, 0),
    (48, 2048, 1024, None, 0),
    (16900, 512, 128, None, 0),                            # tiles for little more than all compute units: rows in two launches
    (16900, 1024, 128, None, 0),
    (16900, 64, 1030, None, 8),
    (96, 5003, 2000, None, 3),
    # full tiles and ends of all lengths, more tiles than compute units, segments without rows, without full tiles, without ends
    (24000, 1030, 136, [3, 3, 259, 300, 812, 1000, 1700, 1700, 1701, 3000, 7096, 7100, 9990, 12289, 12350, 15000, 20120, 20120, 23990], 0),
    (20000, 520, 200, [0] + [17 * i * i // 10 for i in range(4, 108)] + [30000], 8),
    (9, 1000, 2056, [0, 2, 2, 9], 0),
]


def _rows_kept(t, hit, sentinel):
    return bool((t[~torch.from_numpy(hit).cuda()] == sentinel).all())


@pytest.mark.parametrize("m,n,k,ends,gap", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_gated(m, n, k, ends, gap, act):
    lead = () if ends is None else (len(ends) - 1,)
    x, w = _matrix(1, m, k, gap=gap), [_matrix(2 + i, *lead, n, k, std=1.5 / math.sqrt(k), gap=gap) for i in range(2)]
    out = torch.full((m, n + gap), 7.0, dtype=torch.bfloat16, device="cuda")
    h, g, u = X().gated(x, *w, activation=act, offsets=_offsets(ends), save=True, out=out[:, :n])
    again = X().gated(x, *w, activation=act, offsets=_offsets(ends))
    assert h.data_ptr() == out.data_ptr()
    hit = orc.rows_product(_np(x), _np(w[0]), ends)[2]
    assert _rows_kept(out, hit, 7.0) and (gap == 0 or bool((out[:, n:] == 7.0).all()))
    assert torch.equal(h[torch.from_numpy(hit).cuda()], again[torch.from_numpy(hit).cuda()])
    (gr, gs, _), (ur, us, _) = (orc.rows_product(_np(x), _np(v), ends) for v in w)
    eg, eu = sum_tol(k) * gs, sum_tol(k) * us
    _close(g[torch.from_numpy(hit).cuda()], gr[hit], (eg + H * np.abs(gr) + TINY)[hit], "gate")
    _close(u[torch.from_numpy(hit).cuda()], ur[hit], (eu + H * np.abs(ur) + TINY)[hit], "up")
    a, _ = orc.activation(gr, act)
    tol = 1.2 * eg * (np.abs(ur) + eu) + np.abs(a) * eu + (H + 160 * U) * np.abs(a * ur) + TINY
    _close(h[torch.from_numpy(hit).cuda()], (a * ur)[hit], tol[hit], "h")


def _int8(seed, *shape, stack_gap=0):
    """Random codes over the whole range, the padding zero, and scales."""
    *lead, rows, cols = shape
    codes = torch.zeros(*lead, rows + stack_gap, -(-cols // 128) * 128, dtype=torch.int8, device="cuda")[..., :rows, :]
    codes[..., :cols] = torch.randint(-128, 128, shape, device="cuda", generator=_gen(seed)).to(torch.int8)
    scales = torch.rand(*lead, rows, device="cuda", generator=_gen(seed + 50)) * 0.02 / math.sqrt(cols) + 1e-4
    return X().Int8(codes, scales, cols)


def _scaled(a, b, ends):
    """(product, rows covered): the sums of whole numbers, exact in float64, times the scales."""
    y, _, hit = orc.rows_product(_np(a.codes[..., :a.cols]), _np(b.codes[..., :b.cols]), ends)
    y *= _np(a.scales)[:, None]
    for g, lo, hi in orc.segments(ends, len(y)):
        y[lo:hi] *= _np(b.scales if g is None else b.scales[g])
    return y, hit


@pytest.mark.parametrize("m,n,k,ends,gap", SHAPES)
def test_product_int8(m, n, k, ends, gap):
    lead = () if ends is None else (len(ends) - 1,)
    a, b = _int8(3, m, k), _int8(4, *lead, n, k, stack_gap=gap)
    want, hit = _scaled(a, b, ends)
    pick = torch.from_numpy(hit).cuda()
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((m, n + gap), 7.0, dtype=dtype, device="cuda")
        X().product_int8(a, b, offsets=_offsets(ends), out=out[:, :n])
        assert _rows_kept(out, hit, 7.0) and (gap == 0 or bool((out[:, n:] == 7.0).all()))
        _close(out[:, :n][pick], want[hit], ((HALF[dtype] + 3 * U) * np.abs(want) + TINY)[hit], str(dtype))
        assert torch.equal(out[:, :n][pick], X().product_int8(a, b, offsets=_offsets(ends), dtype=dtype)[pick])


@pytest.mark.parametrize("m,n,k,ends,gap", SHAPES[::2] + SHAPES[-3:])
@pytest.mark.parametrize("act", ACTS)
def test_gated_int8(m, n, k, ends, gap, act):
    lead = () if ends is None else (len(ends) - 1,)
    x, g, u = _int8(5, m, k), _int8(6, *lead, n, k, stack_gap=gap), _int8(7, *lead, n, k, stack_gap=gap)
    x.scales.mul_(100)
    out = torch.full((m, n), 7.0, dtype=torch.bfloat16, device="cuda")
    h, pg, pu = X().gated(x, g, u, activation=act, offsets=_offsets(ends), save=True, out=out)
    (gr, hit), (ur, _) = _scaled(x, g, ends), _scaled(x, u, ends)
    pick = torch.from_numpy(hit).cuda()
    assert _rows_kept(out, hit, 7.0)
    eg, eu = 3 * U * np.abs(gr), 3 * U * np.abs(ur)
    _close(pg[pick], gr[hit], (eg + H * np.abs(gr) + TINY)[hit], "gate")
    _close(pu[pick], ur[hit], (eu + H * np.abs(ur) + TINY)[hit], "up")
    a, _ = orc.activation(gr, act)
    _close(h[pick], (a * ur)[hit], (1.2 * eg * (np.abs(ur) + eu) + np.abs(a) * eu + (H + 160 * U) * np.abs(a * ur) + TINY)[hit], "h")


@pytest.mark.parametrize("m,n,k,ends,gap", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_gated_backward(m, n, k, ends, gap, act):
    lead = () if ends is None else (len(ends) - 1,)
    x, w = _matrix(1, m, k, gap=gap), [_matrix(2 + i, *lead, n, k, std=1.5 / math.sqrt(k), gap=gap) for i in range(2)]
    d, g, u = (_matrix(8 + i, m, n, std=s, gap=-n % 64 if i else gap) for i, s in enumerate((0.1, 1.5, 1.0)))
    kept = [t.clone() for t in (g, u)]
    grad_x = torch.full((m, k + gap), 7.0, dtype=torch.bfloat16, device="cuda")
    _, w16g, w16u = X().gated_backward(d, x, *w, g, u, activation=act, offsets=_offsets(ends), grad_x=grad_x[:, :k])
    assert torch.equal(g, kept[0]) and torch.equal(u, kept[1])
    hit = orc.rows_product(_np(x), _np(w[0]), ends)[2]
    pick = torch.from_numpy(hit).cuda()
    assert _rows_kept(grad_x, hit, 7.0) and (gap == 0 or bool((grad_x[:, k:] == 7.0).all()))
    before = [torch.randn(w[0].shape, device="cuda", generator=_gen(20 + i)) for i in range(2)]
    acc = [t.clone() for t in before]
    again, *acc = X().gated_backward(d, x, *w, g, u, activation=act, offsets=_offsets(ends), grad_gate=acc[0], grad_up=acc[1],
                                     accumulate=True, reuse=True)
    assert torch.equal(again[pick], grad_x[:, :k][pick])
    # the pre-activations' gradients, as the call left them
    want = orc.gated_pre_grads(_np(d), _np(kept[0]), _np(kept[1]), act)
    value, slope = orc.activation(_np(kept[0]), act)
    # the slope is a sum whose terms are at most 1.2 + |g| / 4 in magnitude
    slack = 160 * U * np.abs(_np(d) * _np(kept[1])) * (1.2 + np.abs(_np(kept[0])) / 4), 160 * U * np.abs(_np(d) * value)
    for got, ref, extra, name in zip((g, u), want, slack, ("dg", "du")):
        _close(got[pick], ref[hit], (H * np.abs(ref) + extra + TINY)[hit], name)
    dg, du = _np(g), _np(u)
    ref, size = orc.gated_grad_x(dg, du, _np(w[0]), _np(w[1]), ends)
    _close(grad_x[:, :k][pick], ref[hit], (sum_tol(2 * n + 32) * size + H * np.abs(ref) + TINY)[hit], "grad_x")
    for got16, got32, start, dd, name in ((w16g, acc[0], before[0], dg, "gate"), (w16u, acc[1], before[1], du, "up")):
        ref, size = orc.gated_grad_w(dd, _np(x), ends)
        longest = max([hi - lo for _, lo, hi in orc.segments(ends, m)], default=1)
        tol = sum_tol(longest) * size
        _close(got16, ref, tol + H * np.abs(ref) + TINY, name)
        _close(got32, ref + _np(start), tol + U * (np.abs(ref) + np.abs(ref + _np(start))) + TINY, name + " added")


@pytest.mark.parametrize("ends", [None, [0, 0, 0]])
def test_gated_backward_without_rows(ends):
    lead = () if ends is None else (2,)
    x, w = _matrix(1, 0, 24), [_matrix(2 + i, *lead, 40, 24) for i in range(2)]
    d = _matrix(3, 0, 40)
    gx, gg, gu = X().gated_backward(d, x, *w, d, d, offsets=_offsets(ends), dtype=torch.float32)
    assert gx.shape == (0, 24) and not gg.any() and not gu.any() and gg.shape == w[0].shape
    assert X().gated(x, *w, offsets=_offsets(ends)).shape == (0, 40)


def test_gradients_against_differences():
    """Of the whole block in the oracle's float64: the formula's gradients are those of the formula, and the call's are the
    formula's (above)."""
    rng = np.random.Generator(np.random.PCG64(4))
    x, G, U_, d = rng.normal(size=(9, 12)), rng.normal(size=(2, 10, 12)), rng.normal(size=(2, 10, 12)), rng.normal(size=(9, 10))
    ends = [0, 4, 9]
    for act in ("silu", "gelu"):
        g, u = orc.rows_product(x, G, ends)[0], orc.rows_product(x, U_, ends)[0]
        dg, du = orc.gated_pre_grads(d, g, u, act)
        grads = (orc.gated_grad_x(dg, du, G, U_, ends)[0], orc.gated_grad_w(dg, x, ends)[0], orc.gated_grad_w(du, x, ends)[0])
        for which, grad in enumerate(grads):
            args = [x, G, U_]
            step = rng.normal(size=args[which].shape)
            loss = [(d * orc.gated(*[a + s * step if i == which else a for i, a in enumerate(args)], act, ends)).sum() for s in (1e-5, -1e-5)]
            assert abs((loss[0] - loss[1]) / 2e-5 - (grad * step).sum()) < 1e-5 * (1 + abs((grad * step).sum()))


def test_values_that_are_not_numbers_stay_in_their_rows():
    m, n, k = 140, 150, 96
    x, w = _matrix(1, m, k), [_matrix(2 + i, n, k, std=0.1) for i in range(2)]
    clean = X().gated(x, *w)
    x[3, 5], x[77, 0] = float("nan"), float("inf")
    h = X().gated(x, *w)
    other = torch.ones(m, dtype=torch.bool, device="cuda")
    other[[3, 77]] = False
    assert torch.equal(h[other], clean[other]) and bool(h[3].isnan().all()) and not bool(h[77].isfinite().any())
    # a weight's NaN stays in its column, a group's in its rows
    wn = [t.clone() for t in w]
    wn[1][10, 3] = float("nan")
    h = X().gated(_matrix(1, m, k), *wn)
    cols = torch.ones(n, dtype=torch.bool, device="cuda")
    cols[10] = False
    assert torch.equal(h[:, cols], clean[:, cols]) and bool(h[:, 10].isnan().all())
    # gradients: a NaN behind the last segment or in another group's rows reaches no weight
    x, ends = _matrix(1, m, k), [0, 50, 90, 120]
    W = [_matrix(2 + i, 3, n, k, std=0.1) for i in range(2)]
    d, g, u = (_matrix(8 + i, m, n) for i in range(3))
    want = X().gated_backward(d, x, *W, g, u, offsets=_offsets(ends))
    for t in (x, d, g, u):
        t[120:] = float("nan")
        t[60] = float("nan")
    got = X().gated_backward(d, x, *W, g, u, offsets=_offsets(ends))
    for grp in (0, 2):
        assert torch.equal(got[1][grp], want[1][grp]) and torch.equal(got[2][grp], want[2][grp])
    keep = [r for r in range(120) if r != 60]
    assert torch.equal(got[0][keep], want[0][keep]) and bool(got[0][60].isnan().all())


@pytest.mark.parametrize("act", ACTS)
def test_pre_gradients_at_the_ends(act):
    """Large, small and zero pre-activations: no overflow on the way to a finite result."""
    v = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3.0, -3.0, 9.0, -9.0, -12.0, 60.0, -60.0, -80.0, 100.0, -100.0, 1e4, -1e4, 3e38, -3e38],
                     device="cuda").to(torch.bfloat16)
    n = v.numel()
    g, u, d = _matrix(0, 2, n, gap=-n % 64), _matrix(1, 2, n, gap=-n % 64), _matrix(2, 2, n, std=0.1)
    g.copy_(v)
    x, w = _matrix(3, 2, 8), [_matrix(4 + i, n, 8) for i in range(2)]
    v, kept = _np(g), _np(u)
    X().gated_backward(d, x, *w, g, u, activation=act, reuse=True)
    value, slope = orc.activation(v, act)
    want = orc.gated_pre_grads(_np(d), v, kept, act)
    # the exponent's argument: 1.5 * 100 u (silu), 2.5 * 72 u (gelu; beyond 12 values are below 2^-120), and 40 u as above
    terms = {"silu": np.abs(slope) + 2 * np.exp(-np.abs(v)) * np.minimum(np.abs(v), 800), "gelu": np.abs(slope) + np.minimum(np.abs(v), 40) * np.exp(-0.5 * v * v),
             "relu": np.abs(slope)}[act]
    for got, ref, size in zip((g, u), want, (_np(d) * kept * terms, _np(d) * value)):
        _close(got, ref, H * np.abs(ref) + 220 * U * np.abs(size) + 2.0 ** -120, act)


# ---- 8-bit integer quantisation ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols,gap", [(1, 1, 0), (3, 7, 0), (5, 128, 0), (2, 129, 3), (17, 1000, 0), (300, 511, 1), (4, 4096, 0),
                                           (70, 2048, 8), (3, 8704, 0), (2, 16385, 0), (1, 40001, 0), (1025, 33, 0),
                                           (5000, 7, 0), (4100, 9, 1), (4099, 256, 0), (4097, 257, 0), (4096, 1000, 8), (4100, 2049, 0),
                                           (4101, 3999, 0), (4096, 4104, 0), (9, 10240, 0), (7, 16384, 0)])
def test_quantize_int8(dtype, rows, cols, gap):
    x = _matrix(1, rows, cols, dtype=dtype, gap=gap)
    x[0] = 0
    if rows > 2:
        x[1] = (torch.arange(cols, device="cuda") % 255 - 127).to(dtype) / 2      # ties
        x[2, 0] = 1e-44 if dtype == torch.float32 else 1e-40
    if rows > 4:
        x[3] *= 1e37
        x[4] *= 1e-38
    q = X().quantize_int8(x)
    codes, scales = orc.quantize_int8(_np(x))
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes[:, :cols].cpu().numpy(), codes) and not q.codes[:, cols:].any()


def test_quantize_int8_next_to_borders():
    """Values that are a code and a half of their scale, or one step of float32 beside that."""
    s = torch.tensor([1.0, 3.0, 0.7, 1e-20, 1e20, 1.1754944e-38, 1e-42], device="cuda")
    half = (torch.arange(-127, 127, device="cuda").double() + 0.5)
    x = torch.zeros(s.numel(), 3 * 254 + 1, device="cuda")
    x[:, 0] = s * 127
    scale = (x[:, 0].double() / 127).float()
    v = (half[None] * scale[:, None].double()).float()
    x[:, 1:255], x[:, 255:509], x[:, 509:763] = v, torch.nextafter(v, torch.full_like(v, 1e38)), torch.nextafter(v, torch.full_like(v, -1e38))
    q = X().quantize_int8(x)
    codes, scales = orc.quantize_int8(_np(x))
    assert np.array_equal(q.scales.cpu().numpy(), scales) and np.array_equal(q.codes[:, :763].cpu().numpy(), codes)


def test_quantize_int8_gathers_and_keeps():
    x = _matrix(1, 20, 200)
    rows = torch.tensor([3, -1, 39, 40, 0, 7, 2 ** 31 - 1, 5], dtype=torch.int32, device="cuda")
    out = X().Int8(torch.full((8, 256), 9, dtype=torch.int8, device="cuda"), torch.full((8,), 9.0, device="cuda"), 200)
    for limit in (7, 0, 100, -5):
        out.codes.fill_(9)
        out.scales.fill_(9)
        X().quantize_int8(x, rows=rows, per=2, limit=torch.tensor([limit], dtype=torch.int32, device="cuda"), out=out)
        codes, scales = orc.quantize_int8(orc.gather(_np(x), rows.cpu().numpy().astype(np.int64), 2))
        end = min(max(limit, 0), 8)
        assert np.array_equal(out.codes[:end, :200].cpu().numpy(), codes[:end]) and np.array_equal(out.scales[:end].cpu().numpy(), scales[:end])
        assert bool((out.codes[end:] == 9).all()) and bool((out.scales[end:] == 9).all()) and not out.codes[:end, 200:].any()


def test_quantize_int8_stacks_and_bad_rows():
    x = torch.randn(3, 50, 300, device="cuda", generator=_gen(1))[:, :40, 4:204]
    x[1, 2, 3], x[2, 0, 0] = float("nan"), float("inf")
    q = X().quantize_int8(x)
    codes, scales = orc.quantize_int8(_np(x))
    assert np.array_equal(q.codes[..., :200].cpu().numpy(), codes) and np.array_equal(q.scales.cpu().numpy(), scales, equal_nan=True)
    y = X().product_int8(X().Int8(q.codes[1], q.scales[1], 200), X().Int8(q.codes[0], q.scales[0], 200))
    assert bool(y[2].isnan().all()) and bool(y[torch.arange(40, device="cuda") != 2].isfinite().all())


# ---- rows to experts and back -----------------------------------------------------------------

def _grouped(tokens, top_k, experts, align, seed, drop=0):
    chosen = torch.rand(tokens, experts, device="cuda", generator=_gen(seed)).topk(top_k, dim=-1).indices.to(torch.int32)
    if drop:
        chosen[:drop] = -1
        chosen[-1, 0] = -1
    return X().group_rows(chosen, experts, align=align)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,top_k,experts,align,cols,gap,drop", [
    (1, 1, 1, 1, 1, 0, 0), (1, 4, 9, 16, 64, 0, 0), (5, 2, 7, 1, 33, 1, 1), (64, 7, 32, 16, 200, 0, 3), (300, 3, 16, 128, 513, 8, 0),
    (16, 7, 512, 1, 4096, 0, 2), (1000, 2, 4, 32, 1000, 0, 10), (3, 64, 64, 4, 40, 0, 0)])
def test_gather_combine_and_back(dtype, tokens, top_k, experts, align, cols, gap, drop):
    g = _grouped(tokens, top_k, experts, align, 5, drop)
    rows, position = g.rows.cpu().numpy(), g.position.cpu().numpy()
    used = int(g.offsets[-1])
    src = _matrix(1, tokens, cols, dtype=dtype, gap=gap)
    out = torch.full((rows.size, cols + gap), 7.0, dtype=dtype, device="cuda")
    X().gather_rows(src, g.rows, per=top_k, limit=g.limit, out=out[:, :cols])
    assert np.array_equal(_np(out[:used, :cols]), orc.gather(_np(src), rows, top_k)[:used])
    assert bool((out[used:] == 7.0).all()) and (gap == 0 or bool((out[:, cols:] == 7.0).all()))
    assert np.array_equal(_np(X().gather_rows(src, g.rows, per=top_k)), orc.gather(_np(src), rows, top_k))
    w = torch.rand(tokens, top_k, device="cuda", generator=_gen(3))
    y = _matrix(4, rows.size, cols, dtype=dtype, gap=gap)
    y[used:] = float("nan")
    for weights, residual, kind in itertools.product((w, None), (None, "in", "out"), (torch.float32, torch.bfloat16)):
        res = None if residual is None else _matrix(6, tokens, cols, dtype=kind, gap=gap)
        into = res if residual == "out" else None
        ref, size = orc.combine(_np(y), position, None if weights is None else _np(weights), None if res is None else _np(res))
        got = X().combine_rows(y, g.position, weights, residual=res, dtype=None if into is not None else kind, out=into)
        _close(got, ref, (top_k + 1) * 2 * U * size + HALF[kind] * np.abs(ref) + TINY, "combined")
    d = _matrix(7, tokens, cols, dtype=dtype, gap=gap)
    out.fill_(7.0)
    dy, dw = X().combine_rows_backward(d, y, g.rows, g.position, w, limit=g.limit, out=out[:, :cols])
    ref_y, ref_w, size = orc.combine_backward(_np(d), _np(y), rows, position, _np(w))
    assert bool((out[used:] == 7.0).all())
    _close(dy[:used], ref_y[:used], (HALF[dtype] * np.abs(ref_y) + TINY)[:used], "grad of rows")
    # 64 lanes' sums of cols / 64 products each, and 6 steps over the lanes
    _close(dw, ref_w, (-(-cols // 512) * 8 + 7) * 2 * U * size + TINY, "grad of weights")


def test_indices_of_another_grouping():
    """rows and position that are not each other's: every gradient as its formula says; indices outside go nowhere."""
    T, k, n, cols = 6, 3, 10, 70
    d, y, w = _matrix(1, T, cols), _matrix(2, n, cols), torch.rand(T, k, device="cuda", generator=_gen(3))
    rows = torch.tensor([0, 0, 17, 18, -1, 5, 5, -2 ** 31, 2 ** 31 - 1, 2], dtype=torch.int32, device="cuda")
    position = torch.randint(-2, n + 2, (T, k), device="cuda", generator=_gen(4)).to(torch.int32)
    dy, dw = X().combine_rows_backward(d, y, rows, position, w)
    ref_y, ref_w, size = orc.combine_backward(_np(d), _np(y), rows.cpu().numpy().astype(np.int64), position.cpu().numpy(), _np(w))
    _close(dy, ref_y, H * np.abs(ref_y) + TINY)
    _close(dw, ref_w, 40 * U * size + TINY)
    limit = torch.tensor([3], dtype=torch.int32, device="cuda")
    out = torch.full_like(dy, 7.0)
    dy, dw = X().combine_rows_backward(d, y, rows, position, w, limit=limit, out=out)
    _close(dw, ref_w, 40 * U * size + TINY)
    assert bool((out[3:] == 7.0).all())
    ref, size = orc.combine(_np(y), position.cpu().numpy(), _np(w))
    _close(X().combine_rows(y, position, w), ref, 8 * U * size + H * np.abs(ref) + TINY)


def test_rows_beyond_32_bits():
    """Rows whose byte and element offsets pass 2^32."""
    n, cols = 530000, 8200
    y = torch.empty(n, cols, dtype=torch.bfloat16, device="cuda")
    far = [0, n - 1, n - 2, 262000]
    y[far] = _matrix(1, 4, cols)
    position = torch.tensor([[n - 1, 0], [n - 2, -1], [262000, n]], dtype=torch.int32, device="cuda")
    got = X().combine_rows(y, position)
    want = torch.stack([y[n - 1].float() + y[0].float(), y[n - 2].float(), y[262000].float()]).bfloat16()
    assert torch.equal(got, want)
    rows = torch.tensor([n - 1, 262000], dtype=torch.int32, device="cuda")
    assert torch.equal(X().gather_rows(y, rows), y[[n - 1, 262000]])
    q = X().quantize_int8(y, rows=rows)
    codes, scales = orc.quantize_int8(_np(y[[n - 1, 262000]]))
    assert np.array_equal(q.codes[:, :cols].cpu().numpy(), codes) and np.array_equal(q.scales.cpu().numpy(), scales)


def _check_gated(h, x, gate, up):
    (g, gs, _), (u, us, _) = (orc.rows_product(_np(x), _np(v)) for v in (gate, up))
    eg, eu, a = sum_tol(x.shape[1]) * gs, sum_tol(x.shape[1]) * us, orc.activation(g, "silu")[0]
    _close(h, a * u, 1.2 * eg * (np.abs(u) + eu) + np.abs(a) * eu + (H + 160 * U) * np.abs(a * u) + TINY)


def test_products_beyond_32_bits():
    """Weights, rows and results whose offsets pass 2^32 bytes."""
    k, n, groups, m = 512, 1024, 4100, 60
    w = torch.empty(groups, n, k, dtype=torch.bfloat16, device="cuda")
    used = [0, 4096, groups - 1]
    for i, g in enumerate(used):
        w[g] = _matrix(10 + i, n, k, std=0.05)
    ends = np.zeros(1025, dtype=np.int64)
    x = _matrix(1, m, k)
    # at most 1024 groups: the last ones of the stack
    part = w[groups - 1024:]
    ends[4096 - (groups - 1024) + 1:] = 25
    ends[1024] = 60
    got = X().gated(x, part, part, offsets=_offsets(ends.tolist()))
    for g, lo, hi in ((4096 - (groups - 1024), 0, 25), (1023, 25, 60)):
        _check_gated(got[lo:hi], x[lo:hi], part[g], part[g])
    big = torch.empty(1100000, 2048, dtype=torch.bfloat16, device="cuda")
    y = X().gated(x, w[0][:512], w[0][512:], out=big[-m:, :512])
    _check_gated(y, x, w[0][:512], w[0][512:])
    q = X().quantize_int8(x)
    codes = torch.empty(groups, n, 1024, dtype=torch.int8, device="cuda")[groups - 1024:, :, :k]
    codes[1023] = X().quantize_int8(w[0]).codes
    ends[:1024] = 0
    got = X().product_int8(q, X().Int8(codes, torch.ones(1024, n, device="cuda"), k), offsets=_offsets(ends.tolist()), dtype=torch.float32)
    want = _np(q.codes) @ _np(codes[1023]).T * _np(q.scales)[:, None]
    _close(got, want, 3 * U * np.abs(want))


# ---- whole layers, streams, graphs ---------------------------------------------------------------

def _layer(T, E, k, d, n, seed):
    ex = X()
    tokens, logits = _matrix(seed, T, d), torch.randn(T, E, device="cuda", generator=_gen(seed + 1))
    W = [_matrix(seed + 2 + i, E, n, d, std=1 / math.sqrt(d)) for i in range(2)]
    down = _matrix(seed + 4, E, d, n, std=1 / math.sqrt(n))
    return ex, tokens, logits, W, down


@pytest.mark.parametrize("T,E,k,d,n,align", [(1, 4, 2, 64, 48, 1), (50, 8, 2, 136, 72, 1), (300, 16, 3, 256, 192, 16)])
def test_training_layer(T, E, k, d, n, align):
    """Route, group, gather, gated block, a product with the down projection, combine, and all the way back."""
    ex, tokens, logits, W, down = _layer(T, E, k, d, n, 40)
    chosen, weights = ex.route(logits, k, score="sigmoid")
    g = ex.group_rows(chosen, E, align=align)
    x = ex.gather_rows(tokens, g.rows, per=k, limit=g.limit, out=torch.zeros(g.rows.numel(), d, dtype=torch.bfloat16, device="cuda"))
    h, pg, pu = ex.gated(x, *W, offsets=g.offsets, save=True, out=torch.zeros(g.rows.numel(), n, dtype=torch.bfloat16, device="cuda"))
    ends = g.offsets.tolist()
    y = torch.zeros(g.rows.numel(), d, device="cuda")
    for e in range(E):
        y[ends[e]:ends[e + 1]] = h[ends[e]:ends[e + 1]].float() @ down[e].float().T
    y = y.bfloat16()
    out = ex.combine_rows(y, g.position, weights, residual=tokens)
    # forwards, token by token: bfloat16 roundings of h and y are in the sums, h of each of their terms
    xt, c, wt = _np(tokens), chosen.cpu().numpy(), _np(weights)
    want, size = xt.copy(), np.abs(xt)
    for t, j in itertools.product(range(T), range(k)):
        e = c[t, j]
        hh = orc.gated(xt[t:t + 1], _np(W[0][e]), _np(W[1][e]), "silu")[0]
        D = _np(down[e])
        want[t] += wt[t, j] * (D @ hh)
        size[t] += wt[t, j] * (np.abs(D) @ np.abs(hh) + np.abs(D @ hh))
    _close(out, want, (2 * H + 1e-4) * size, "layer")
    # back
    dout = _matrix(60, T, d)
    dy, dw = ex.combine_rows_backward(dout, y, g.rows, g.position, weights, limit=g.limit, out=torch.zeros_like(y))
    dh = torch.zeros(g.rows.numel(), n, device="cuda")
    for e in range(E):
        dh[ends[e]:ends[e + 1]] = dy[ends[e]:ends[e + 1]].float() @ down[e].float()
    dh = dh.bfloat16()
    dx, dG, dU = ex.gated_backward(dh, x, *W, pg, pu, offsets=g.offsets, dtype=torch.float32)
    dtokens = ex.combine_rows(dx, g.position, residual=dout)
    rows, position = g.rows.cpu().numpy(), g.position.cpu().numpy()
    used = ends[-1]
    pre = orc.gated_pre_grads(_np(dh), _np(pg), _np(pu), "silu")
    pre = [np.where(rows[:, None] >= 0, np.where(np.arange(len(rows))[:, None] < used, v, 0.0), 0.0) for v in pre]
    for got, dd in ((dG, pre[0]), (dU, pre[1])):
        ref, size = orc.gated_grad_w(dd[:used], _np(x)[:used], ends)
        _close(got, ref, (H + sum_tol(T * k)) * size + TINY, "weights")
    gx, size = orc.gated_grad_x(pre[0], pre[1], _np(W[0]), _np(W[1]), ends)
    ref, rsize = orc.combine(gx, position, None, _np(dout))
    tol = orc.combine(size, position)[0] * (H + sum_tol(2 * n + 32)) + (2 * H) * rsize
    _close(dtokens, ref, tol + TINY, "tokens")
    ref_w = orc.combine_backward(_np(dout), _np(y), rows, position, wt)
    _close(dw, ref_w[1], (-(-d // 512) * 8 + 7) * 2 * U * ref_w[2] + TINY, "routing weights")
    assert ex.route_backward(logits, chosen, dw, score="sigmoid").isfinite().all()


@pytest.mark.parametrize("T,E,k,d,n", [(1, 8, 2, 256, 128), (16, 64, 7, 512, 256), (200, 8, 2, 300, 140)])
def test_serving_layer(T, E, k, d, n):
    ex, tokens, logits, W, down = _layer(T, E, k, d, n, 70)
    Q = [ex.quantize_int8(w) for w in (*W, down)]
    chosen, weights = ex.route(logits, k)
    g = ex.group_rows(chosen, E)
    q = ex.quantize_int8(tokens, rows=g.rows, per=k, limit=g.limit)
    h = ex.gated(q, Q[0], Q[1], offsets=g.offsets)
    qh = ex.quantize_int8(h, limit=g.limit)
    y = ex.product_int8(qh, Q[2], offsets=g.offsets)
    out = ex.combine_rows(y, g.position, weights, residual=tokens)
    # with the layer's own codes as operands, each step as its formula says
    ends, used = g.offsets.tolist(), int(g.offsets[-1])
    q = ex.Int8(q.codes[:used], q.scales[:used], d)
    gr, ur = _scaled(q, Q[0], ends)[0], _scaled(q, Q[1], ends)[0]
    want = orc.activation(gr, "silu")[0] * ur
    _close(h[:used], want, (H + 166 * U) * np.abs(want) + 3.6 * U * np.abs(gr * ur) + TINY, "h")
    codes, scales = orc.quantize_int8(_np(h[:used]))
    assert np.array_equal(qh.codes[:used, :n].cpu().numpy(), codes) and np.array_equal(qh.scales[:used].cpu().numpy(), scales)
    ref = _scaled(ex.Int8(qh.codes[:used], qh.scales[:used], n), Q[2], ends)[0]
    _close(y[:used], ref, (H + 3 * U) * np.abs(ref) + TINY, "y")
    ref, size = orc.combine(_np(y), g.position.cpu().numpy(), _np(weights), _np(tokens))
    _close(out, ref, (k + 1) * 2 * U * size + H * np.abs(ref) + TINY, "out")


def test_two_graphs_and_streams():
    """A serving step and a training step captured, replayed in turn with eager work between, on streams of their own."""
    ex, tokens, logits, W, down = _layer(40, 8, 2, 256, 128, 90)
    Q = [ex.quantize_int8(w) for w in (*W, down)]
    zeros = lambda r, c: torch.zeros(r, c, dtype=torch.bfloat16, device="cuda")  # noqa: E731

    def serve():
        chosen, weights = ex.route(logits, 2)
        g = ex.group_rows(chosen, 8)
        q = ex.quantize_int8(tokens, rows=g.rows, per=2, limit=g.limit)
        y = ex.product_int8(ex.quantize_int8(ex.gated(q, Q[0], Q[1], offsets=g.offsets)), Q[2], offsets=g.offsets)
        return ex.combine_rows(y, g.position, weights)

    def train():
        chosen, weights = ex.route(logits, 2)
        g = ex.group_rows(chosen, 8, align=16)
        x = ex.gather_rows(tokens, g.rows, per=2)
        h, pg, pu = ex.gated(x, *W, offsets=g.offsets, save=True, out=zeros(g.rows.numel(), 128))
        return ex.gated_backward(h, x, *W, pg, pu, offsets=g.offsets, grad_x=zeros(g.rows.numel(), 256), dtype=torch.float32)

    graphs = []
    for f in (serve, train):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            f()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = f()
        graphs.append((graph, got))
    for turn in range(4):
        tokens.copy_(_matrix(100 + turn, 40, 256))
        logits.copy_(torch.randn(40, 8, device="cuda", generator=_gen(200 + turn)))
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][1], serve())
        for a, b in zip(graphs[1][1], train()):
            assert torch.equal(a, b)
    # a named stream: inputs may be dropped, the result belongs to it
    want = ex.gated(tokens, W[0][0], W[1][0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    copies = [t.clone() for t in (tokens, W[0][0], W[1][0])]
    side.wait_stream(torch.cuda.current_stream())
    got = ex.gated(*copies, stream=side)
    del copies
    torch.empty(1 << 20, device="cuda").fill_(float("nan"))
    side.synchronize()
    assert torch.equal(got, want)


def test_rows_in_two_launches_captured_and_side_by_side():
    """Sizes whose rows go in two launches: added to what is there, captured and replayed, and on two streams at once."""
    ex = X()
    x, w, d = _matrix(1, 96, 2000), [_matrix(2 + i, 5003, 2000, std=0.02) for i in range(2)], _matrix(4, 96, 5003)
    tall, narrow = _matrix(5, 16900, 128), [_matrix(6 + i, 512, 128, std=0.1) for i in range(2)]
    _, *pre = ex.gated(x, *w, save=True)
    grads = [torch.zeros(5003, 2000, device="cuda") for _ in range(2)]

    def both():
        dx, *_ = ex.gated_backward(d, x, *w, *pre, grad_gate=grads[0], grad_up=grads[1], accumulate=True)
        return dx, ex.gated(tall, *narrow)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for turn in range(3):
        d.copy_(_matrix(10 + turn, 96, 5003))
        tall.copy_(_matrix(20 + turn, 16900, 128))
        for g in grads:
            g.fill_(float(turn))
        graph.replay()
        torch.cuda.synchronize()
        ours = [g.clone() for g in grads]
        for g in grads:
            g.fill_(float(turn))
        want = both()
        assert all(torch.equal(a, b) for a, b in zip((*got, *ours), (*want, *grads)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[] for _ in streams]
    for _ in range(3):
        for at, st in zip(outs, streams):
            at.append(ex.gated(tall, *narrow, stream=st))
            at.append(ex.gated_backward(d, x, *w, *pre, stream=st)[1])
    torch.cuda.synchronize()
    for k, (h, g) in enumerate(zip(outs[0], outs[1])):
        assert torch.equal(h, g) and torch.equal(h, outs[0][k % 2])
    assert torch.equal(outs[0][0], want[1])


def test_wrapper_refuses():
    ex = X()
    x, w = _matrix(1, 4, 64), _matrix(2, 8, 64)
    st = _matrix(3, 2, 8, 64)
    off = _offsets([0, 2, 4])
    q, qw = ex.quantize_int8(x), ex.quantize_int8(w)
    bad = [
        lambda: ex.gated(x, w, w, activation="tanh"),
        lambda: ex.gated(x.float(), w, w),
        lambda: ex.gated(x, w, _matrix(2, 9, 64)),
        lambda: ex.gated(x, w, _matrix(2, 8, 65)),
        lambda: ex.gated(x, w, w, offsets=off),
        lambda: ex.gated(x, st, st),
        lambda: ex.gated(x, st, st, offsets=_offsets([0, 4])),
        lambda: ex.gated(x, st, st, offsets=off.long()),
        lambda: ex.gated(q, w, w),
        lambda: ex.gated(x, w.T.contiguous().T, w),
        lambda: ex.gated(x, w, w.cpu()),
        lambda: ex.gated(x.cpu(), w.cpu(), w.cpu()),
        lambda: ex.gated(x, w, w, out=torch.empty(4, 9, dtype=torch.bfloat16, device="cuda")),
        lambda: ex.gated(x, w, w, out=torch.empty(4, 8, device="cuda")),
        lambda: ex.product_int8(q, ex.quantize_int8(_matrix(1, 4, 65))),
        lambda: ex.product_int8(q, qw, dtype=torch.float16),
        lambda: ex.product_int8(q, ex.Int8(qw.codes, qw.scales[:4], 64)),
        lambda: ex.product_int8(q, ex.Int8(qw.codes, qw.scales, 200)),
        lambda: ex.gated_backward(x[:, :8], x, w, w, x[:, :8], x[:, 1:9], accumulate=True),
        lambda: ex.gated_backward(x[:3, :8], x, w, w, x[:, :8], x[:, :8]),
        lambda: ex.gated_backward(x[:, :8], x, w, w, x[:, :8], x[:, :8].contiguous()),
        lambda: ex.quantize_int8(x.half()),
        lambda: ex.quantize_int8(st, rows=off),
        lambda: ex.quantize_int8(x, out=ex.quantize_int8(w)),
        lambda: ex.gather_rows(x, off.view(1, 3)),
        lambda: ex.gather_rows(x.expand(2, 4, 64), off),
        lambda: ex.combine_rows(x, off),
        lambda: ex.combine_rows(x, off.view(1, 3), torch.ones(1, 2, device="cuda")),
        lambda: ex.combine_rows(x, off.view(1, 3), dtype=torch.float16),
        lambda: ex.combine_rows_backward(x, x, off, off.view(3, 1), torch.ones(3, 1, device="cuda")),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} is accepted")


def test_reuse_writes_no_other_tensor():
    """Saved values in a wider buffer, of rows apart from others by a column, and in a storage without the last row's padding."""
    ex, m, n, k = X(), 6, 40, 24
    x, w, d = _matrix(1, m, k), [_matrix(2 + i, n, k) for i in range(2)], _matrix(4, m, n)
    _, *saved = ex.gated(x, *w, save=True)
    for wide, first in ((128, 0), (64, 8)):
        buf = torch.full((2, m + 1, wide), 7.0, dtype=torch.bfloat16, device="cuda")
        pre = [b[:m, first:first + n] for b in buf]
        for p, v in zip(pre, saved):
            p.copy_(v)
        kept = buf.clone()
        with pytest.raises(ValueError):
            ex.gated_backward(d, x, *w, *pre, reuse=True)
        assert torch.equal(buf, kept)
    cut = [torch.empty((m - 1) * 64 + n, dtype=torch.bfloat16, device="cuda").as_strided((m, n), (64, 1)) for _ in range(2)]
    with pytest.raises(ValueError):
        ex.gated_backward(d, x, *w, *cut, reuse=True)
    want = ex.gated_backward(d, x, *w, *saved)
    some = ex.gated_backward(d[2:], x[2:].clone(), *w, saved[0][2:].contiguous(), saved[1][2:].contiguous())
    again = ex.gated_backward(d[2:], x[2:].clone(), *w, saved[0][2:], saved[1][2:], reuse=True)
    assert all(torch.equal(a, b) for a, b in zip(some, again)) and torch.equal(again[0], want[0][2:])
    assert not saved[0].as_strided((m, 64), (64, 1))[2:, n:].any()


@pytest.mark.parametrize("m,n,ends", [(1, 1, None), (70, 33, None), (5000, 5000, None), (70, 33, [3, 3, 20, 66]), (5000, 1030, [0, 300, 300, 4990])])
def test_products_without_depth(m, n, ends):
    """Rows without values: sums of nothing, so zeros, in the rows of the segments."""
    ex, lead, kinds = X(), () if ends is None else (len(ends) - 1,), (torch.bfloat16, torch.int8)
    hit = torch.zeros(m, dtype=torch.bool, device="cuda")
    for _, lo, hi in orc.segments(ends, m):
        hit[lo:hi] = True
    for kind in kinds:
        def operand(*shape):
            t = torch.empty(*shape, 0, dtype=kind, device="cuda")
            return t if kind is torch.bfloat16 else ex.Int8(t, torch.ones(shape, device="cuda"), 0)
        x, w = operand(m), operand(*lead, n)
        for act in ACTS:
            out = torch.full((m, n), 7.0, dtype=torch.bfloat16, device="cuda")
            got = ex.gated(x, w, w, activation=act, offsets=_offsets(ends), save=True, out=out)
            assert not any(bool(t[hit].any()) for t in got) and bool((out[~hit] == 7.0).all())
        if kind is torch.int8:
            for dtype in (torch.float32, torch.bfloat16):
                out = torch.full((m, n), 7.0, dtype=dtype, device="cuda")
                ex.product_int8(x, w, offsets=_offsets(ends), out=out)
                assert not out[hit].any() and bool((out[~hit] == 7.0).all())


@pytest.mark.parametrize("m,k,ends", [(1, 1, None), (70, 200, None), (70, 200, [3, 3, 20, 66]), (0, 24, None)])
@pytest.mark.parametrize("reuse", [False, True])
def test_gated_backward_without_features(m, k, ends, reuse):
    ex, lead = X(), () if ends is None else (len(ends) - 1,)
    x, w, d = _matrix(1, m, k), [_matrix(2 + i, *lead, 0, k) for i in range(2)], _matrix(4, m, 0)
    h, *pre = ex.gated(x, *w, offsets=_offsets(ends), save=True)
    out = torch.full((m, k), 7.0, dtype=torch.bfloat16, device="cuda")
    dx, dg, du = ex.gated_backward(d, x, *w, *pre, offsets=_offsets(ends), grad_x=out, reuse=reuse, dtype=torch.float32)
    hit = torch.zeros(m, dtype=torch.bool, device="cuda")
    for _, lo, hi in orc.segments(ends, m):
        hit[lo:hi] = True
    assert h.shape == (m, 0) and dg.shape == du.shape == w[0].shape and dx is out
    assert not dx[hit].any() and bool((dx[~hit] == 7.0).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gather_and_combine_without_rows_or_tokens(dtype):
    ex, cols = X(), 130
    ints = lambda *shape, value=-1: torch.full(shape, value, dtype=torch.int32, device="cuda")  # noqa: E731
    # no rows: no gradient of a row, zeros for the weights
    for T, k in ((1, 1), (70, 3)):
        d, y = _matrix(1, T, cols, dtype=dtype), _matrix(2, 0, cols, dtype=dtype)
        for at in (-1, 0):
            dy, dw = ex.combine_rows_backward(d, y, ints(0), ints(T, k, value=at), torch.ones(T, k, device="cuda"))
            assert dy.shape == (0, cols) and dw.shape == (T, k) and not dw.any()
        assert not ex.combine_rows(y, ints(T, k), torch.ones(T, k, device="cuda")).any()
        assert ex.gather_rows(d, ints(0)).shape == (0, cols)
    # no tokens: rows that pad segments only
    d, y = _matrix(1, 0, cols, dtype=dtype), _matrix(2, 40, cols, dtype=dtype)
    for value in (-1, 0, 5):
        dy, dw = ex.combine_rows_backward(d, y, ints(40, value=value), ints(0, 3), torch.ones(0, 3, device="cuda"))
        assert not dy.any() and dw.shape == (0, 3)
        assert not ex.gather_rows(d, ints(40, value=value), per=3).any()
    assert ex.combine_rows(y, ints(0, 3), torch.ones(0, 3, device="cuda")).shape == (0, cols)


# ---- offsets beyond 32 bits that the kernels form themselves ---------------------------------------

FAR_ROWS, FAR_N, FAR_STRIDE = 266000, 8104, 9 << 18        # rows of FAR_N values; 1024 groups' matrices FAR_STRIDE elements apart
FAR_BYTES, FAR_ELEMENTS = 2 ** 32, 2 ** 31


def _far(t, *index):
    """t, whose element at index lies beyond 2^31 elements and 2^32 bytes from its first."""
    away = sum(i * s for i, s in zip(index, t.stride()))
    assert away >= (FAR_ELEMENTS if t.element_size() > 1 else FAR_BYTES) and away * t.element_size() >= FAR_BYTES
    return t


def _far_stack(n, k, dtype, stride=FAR_STRIDE):
    return _far(torch.empty(1024 * stride, dtype=dtype, device="cuda").as_strided((1024, n, k), (stride, k, 1)), 1022)


def _last_two(m):
    """Offsets of 1024 groups of which the last two have rows: 25 and 35 before row m."""
    return [m - 60] * 1023 + [m - 35, m], ((1022, m - 60, m - 35), (1023, m - 35, m))


def _check_rows(h, g, u, x, gate, up, act):
    (gr, gs, _), (ur, us, _) = (orc.rows_product(_np(x), _np(v)) for v in (gate, up))
    eg, eu, a = sum_tol(x.shape[1]) * gs, sum_tol(x.shape[1]) * us, orc.activation(gr, act)[0]
    _close(h, a * ur, 1.2 * eg * (np.abs(ur) + eu) + np.abs(a) * eu + (H + 160 * U) * np.abs(a * ur) + TINY, "h")
    if g is not None:
        _close(g, gr, eg + H * np.abs(gr) + TINY, "gate")
        _close(u, ur, eu + H * np.abs(ur) + TINY, "up")


@pytest.mark.parametrize("m", [60, FAR_ROWS])
def test_gated_far_from_the_first_row_and_group(m):
    """Weights, rows, results, saved values and all gradients; 60 rows in the kernels for few, the others among 256 a tile."""
    ex, n, k = X(), FAR_N, 64
    ends, used = _last_two(m)
    w = [_far_stack(n, k, torch.bfloat16) for _ in range(2)]
    for i, v in enumerate(w):
        for g, _, _ in used:
            v[g] = _matrix(10 * i + g, n, k, std=1.5 / 8)
    wide = n if m > 60 else k
    x = torch.empty(m, wide, dtype=torch.bfloat16, device="cuda")[:, :k]
    x[-60:] = _matrix(1, 60, k)
    h, g, u = ex.gated(x, *w, offsets=_offsets(ends), save=True)
    d = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    d[-60:] = _matrix(2, 60, n, std=0.1)
    if m > 60:
        for t in (x, h, g, u, d):
            _far(t, m - 60)
    for grp, lo, hi in used:
        _check_rows(h[lo:hi], g[lo:hi], u[lo:hi], x[lo:hi], w[0][grp], w[1][grp], "silu")
    del h
    pre = _np(g[-60:]), _np(u[-60:])
    gx = torch.full((m, wide), 7.0, dtype=torch.bfloat16, device="cuda")[:, :k]
    grads = [_far_stack(n, k, torch.float32) for _ in range(2)]
    for v in grads:
        v[[0, 500, 1022, 1023]] = 7.0
    ex.gated_backward(d, x, *w, g, u, offsets=_offsets(ends), grad_x=gx, grad_gate=grads[0], grad_up=grads[1], reuse=True)
    for got, want, size in zip((g, u), orc.gated_pre_grads(_np(d[-60:]), *pre, "silu"),
                               (_np(d[-60:]) * pre[1] * (1.2 + np.abs(pre[0]) / 4), _np(d[-60:]) * orc.activation(pre[0], "silu")[0])):
        _close(got[-60:], want, H * np.abs(want) + 160 * U * np.abs(size) + TINY)
    assert m == 60 or bool((gx[:-60] == 7.0).all())
    for grp, lo, hi in used:
        ref, size = orc.gated_grad_x(_np(g[lo:hi]), _np(u[lo:hi]), _np(w[0][grp]), _np(w[1][grp]))
        _close(gx[lo:hi], ref, sum_tol(2 * n + 32) * size + H * np.abs(ref) + TINY, "grad_x")
        for got, dd in zip(grads, (g, u)):
            ref, size = orc.gated_grad_w(_np(dd[lo:hi]), _np(x[lo:hi]))
            _close(got[grp], ref, sum_tol(hi - lo) * size + U * np.abs(ref) + TINY, "weights")
    assert not any(bool(v[[0, 500]].any()) for v in grads)
    del w, x, d, g, u, gx, grads
    torch.cuda.empty_cache()


def test_dense_gated_far_from_the_first_row():
    """All rows in launches of whole tiles, and weight gradients over a depth whose rows end far away."""
    ex, m, n, k = X(), FAR_ROWS, FAR_N, 64
    w = [_matrix(2 + i, n, k, std=1.5 / 8) for i in range(2)]
    x = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")[:, :k]
    some = torch.tensor([0, 1, 255, 256, m // 2, *range(m - 60, m)], device="cuda")
    x[some] = _matrix(1, len(some), k)
    h, g, u = ex.gated(x, *w, activation="gelu", save=True)
    _check_rows(h[some], g[some], u[some], x[some], *w, "gelu")
    assert not h[1000:1100].any()
    d = h.zero_()
    d[some] = _matrix(4, len(some), n, std=0.1)
    for t in (x, g, u, d):
        _far(t, m - 60)
    gx, gg, gu = ex.gated_backward(d, x, *w, g, u, activation="gelu", grad_x=torch.empty_like(d)[:, :k], dtype=torch.float32, reuse=True)
    dg, du = _np(g[some]), _np(u[some])
    ref, size = orc.gated_grad_x(dg, du, *map(_np, w))
    _close(_far(gx, m - 60)[some], ref, sum_tol(2 * n + 32) * size + H * np.abs(ref) + TINY, "grad_x")
    for got, dd in ((gg, dg), (gu, du)):
        ref, size = orc.gated_grad_w(dd, _np(x[some]))
        # (the other rows add zeros, which round nothing)
        _close(got, ref, sum_tol(len(some) * 16) * size + U * np.abs(ref) + TINY, "weights")
    del x, h, g, u, d, gx
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m", [60, FAR_ROWS])
def test_int8_far_from_the_first_row_and_group(m):
    ex, n, k = X(), FAR_N, 100
    ends, used = _last_two(m)
    wide = 2 * FAR_N if m > 60 else 128                    # (a multiple of 16)
    a = ex.Int8(torch.empty(m, wide, dtype=torch.int8, device="cuda")[:, :128], torch.empty(m, device="cuda"), k)
    some = _int8(1, 60, k)
    a.codes[-60:], a.scales[-60:] = some.codes, some.scales
    codes = _far_stack(n, 128, torch.int8, 2 * FAR_STRIDE)
    b = ex.Int8(codes, _far(torch.empty(1024 * FAR_STRIDE, device="cuda").as_strided((1024, n), (FAR_STRIDE, 1)), 1022), k)
    for i, (grp, _, _) in enumerate(used):
        q = _int8(2 + i, n, k)
        b.codes[grp], b.scales[grp] = q.codes, q.scales
    y = ex.product_int8(a, b, offsets=_offsets(ends), dtype=torch.float32)
    h = ex.gated(a, b, b, activation="relu", offsets=_offsets(ends))
    if m > 60:
        for t in (a.codes, y, h):
            _far(t, m - 60)
    for grp, lo, hi in used:
        want, _ = _scaled(ex.Int8(a.codes[lo:hi], a.scales[lo:hi], k), ex.Int8(b.codes[grp], b.scales[grp], k), None)
        _close(y[lo:hi], want, 4 * U * np.abs(want) + TINY, "product")
        want = np.maximum(want, 0) * want
        _close(h[lo:hi], want, (H + 10 * U) * np.abs(want) + TINY, "gated")
    del a, b, codes, y, h
    torch.cuda.empty_cache()


def test_rows_written_far_from_the_first():
    """Gathered, combined and quantised rows, a residual, and rows whose weights' gradients are formed."""
    ex, T, cols = X(), 40, FAR_N
    src = _matrix(1, T, cols)
    rows = torch.full((FAR_ROWS,), -1, dtype=torch.int32, device="cuda")
    at = torch.tensor([0, 1000, FAR_ROWS // 2, *range(FAR_ROWS - 37, FAR_ROWS)], device="cuda")
    rows[at] = torch.arange(T, dtype=torch.int32, device="cuda")
    out = _far(ex.gather_rows(src, rows), FAR_ROWS - 37)
    assert torch.equal(out[at], src) and not out[2000:2100].any() and not out[-100:-37].any()
    # the gradients of a sum of single rows, each far away
    position, w = at.to(torch.int32).view(T, 1), torch.rand(T, 1, device="cuda", generator=_gen(3))
    d = _matrix(4, T, cols)
    dy, dw = ex.combine_rows_backward(d, out, rows, position, w)
    ref = _np(w) * _np(d)
    _close(_far(dy, FAR_ROWS - 37)[at], ref, H * np.abs(ref) + TINY, "rows")
    _close(dw[:, 0], (_np(d) * _np(src)).sum(-1), (-(-cols // 512) * 8 + 7) * 2 * U * np.abs(_np(d) * _np(src)).sum(-1) + TINY, "weights")
    del dy
    # single rows to tokens far away, in place of their residual
    position = rows.view(-1, 1).clone()
    out.fill_(1.0)
    assert ex.combine_rows(src, position, residual=out, out=out) is out
    ref = 1.0 + _np(src)
    _close(out[at], ref, 4 * U * (1 + np.abs(_np(src))) + H * np.abs(ref) + TINY, "combined")
    assert bool((out[2000:2100] == 1.0).all())
    del out
    n = 2 * FAR_ROWS                                       # (codes of one byte)
    rows = torch.cat([rows[:FAR_ROWS // 2], torch.full((FAR_ROWS,), -1, dtype=torch.int32, device="cuda"), rows[FAR_ROWS // 2:]])
    q = ex.quantize_int8(src, rows=rows)
    at = torch.nonzero(rows >= 0)[:, 0]
    codes, scales = orc.quantize_int8(_np(src))
    assert q.codes.shape[0] == n and np.array_equal(_far(q.codes, n - 37)[at, :cols].cpu().numpy(), codes)
    assert np.array_equal(q.scales[at].cpu().numpy(), scales) and not q.codes[n - 100:n - 37].any() and not q.codes[at, cols:].any()
    del q
    torch.cuda.empty_cache()


# ---- outputs left out, and the deepest sums ------------------------------------------------------

@pytest.mark.parametrize("m,n,k,ends", [(70, 40, 96, None), (300, 136, 264, [0, 1, 2, 130, 130, 280, 290]), (16900, 512, 128, None), (9, 5, 7, [2, 2, 8]), (70, 40, 0, None)])
def test_gated_backward_of_some_outputs(m, n, k, ends):
    """Each subset of the nullable outputs holds what the whole call writes, and what a subset does not read may be NULL."""
    import ctypes as C

    from muon_newton_schulz_momentum_amd import binding as L
    ex, lead = X(), () if ends is None else (len(ends) - 1,)
    x, w = _matrix(1, m, k), [_matrix(2 + i, *lead, n, k, std=0.1) for i in range(2)]
    d, *pre = (_matrix(8 + i, m, n, std=0.5) for i in range(3))
    hit = torch.from_numpy(orc.rows_product(_np(x), _np(w[0]), ends)[2]).cuda()
    offsets, width = _offsets(ends), -(-n // 64) * 64
    want = ex.gated_backward(d, x, *w, *pre, offsets=offsets, dtype=torch.float32)
    for rows, weights in itertools.product((False, True), repeat=2):
        work = torch.full((2, m, width), 5.0, dtype=torch.bfloat16, device="cuda")
        gx = torch.full((m, k), 7.0, dtype=torch.bfloat16, device="cuda")
        gw = [torch.full(w[0].shape, 7.0, device="cuda") for _ in range(2)]
        operand = lambda t: L.muon_operand(t.data_ptr(), None, k, n * k, 0)  # noqa: E731
        c = L.muon_gated_backward_config(
            L.MUON_PRODUCT_DENSE if ends is None else L.MUON_PRODUCT_ROWS, lead[0] if lead else 1, L.MUON_ACT_SILU, L.MUON_DTYPE_F32, 0, 0, m, n, k,
            operand(x) if weights else L.muon_operand(), operand(w[0]) if rows else L.muon_operand(), operand(w[1]) if rows else L.muon_operand(),
            None if ends is None else offsets.data_ptr(), d.data_ptr(), n, pre[0].data_ptr(), pre[1].data_ptr(), n,
            work[0].data_ptr(), work[1].data_ptr(), width, gx.data_ptr() if rows else None, k,
            gw[0].data_ptr() if weights else None, gw[1].data_ptr() if weights else None, k, n * k)
        L.check(L.muon_gated_backward(C.byref(c), torch.cuda.current_stream().cuda_stream), "muon_gated_backward")
        ref, there = [_np(v) for v in (d, *pre)], hit.cpu().numpy()
        slack = np.abs(ref[0] * ref[2]) * (1.2 + np.abs(ref[1]) / 4), np.abs(ref[0] * orc.activation(ref[1], "silu")[0])
        for got, v, size in zip(work, orc.gated_pre_grads(*ref, "silu"), slack):
            _close(got[hit][:, :n], v[there], (H * np.abs(v) + 160 * U * size + TINY)[there])
            assert not got[hit][:, n:].any() and bool((got[~hit] == 5.0).all())
        assert torch.equal(gx[hit], want[0][hit]) if rows else bool((gx == 7.0).all())
        assert bool((gx[~hit] == 7.0).all())
        assert all(torch.equal(a, b) if weights else bool((a == 7.0).all()) for a, b in zip(gw, want[1:]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,top_k,experts,align,cols", [(1, 1, 1, 1, 3), (64, 7, 32, 16, 200), (300, 3, 16, 128, 513)])
def test_gather_rows_of_the_weights_gradients_alone(dtype, tokens, top_k, experts, align, cols):
    import ctypes as C

    from muon_newton_schulz_momentum_amd import binding as L
    ex, g = X(), _grouped(tokens, top_k, experts, align, 5, 2)
    n, kind = g.rows.numel(), L.MUON_DTYPE_F32 if dtype is torch.float32 else L.MUON_DTYPE_BF16
    d, y = _matrix(1, tokens, cols, dtype=dtype), _matrix(2, n, cols, dtype=dtype)
    w = torch.rand(tokens, top_k, device="cuda", generator=_gen(3))
    _, want = ex.combine_rows_backward(d, y, g.rows, g.position, w, limit=g.limit)
    got = torch.full_like(w, 7.0)
    c = L.muon_gather_rows_config(d.data_ptr(), tokens, cols, cols, kind, top_k, g.rows.data_ptr(), n, g.limit.data_ptr(), None, 0, None,
                                  y.data_ptr(), cols, g.position.data_ptr(), got.data_ptr())
    L.check(L.muon_gather_rows(C.byref(c), torch.cuda.current_stream().cuda_stream), "muon_gather_rows")
    assert torch.equal(got, want)


@pytest.mark.parametrize("m,n,ends", [(1, 33, None), (300, 520, None), (300, 136, [0, 100, 100, 290])])
def test_deepest_sums_of_8_bit_integers(m, n, ends):
    """131071 products of 16384 each, the largest sum that 32 bits hold, and of -128 by 127."""
    ex, k, lead = X(), 131071, () if ends is None else (len(ends) - 1,)
    a, b = ex.Int8.empty(m, k), ex.Int8.empty(n, k, stack=lead[0] if lead else None)
    for q in (a, b):
        q.codes.fill_(-128)
        q.codes[..., k:] = 0
        q.scales.fill_(1.0)
    b.codes[..., 1::2, :k] = 127
    got = ex.product_int8(a, b, offsets=_offsets(ends), dtype=torch.float32)
    want = np.where(np.arange(n) % 2, -128.0 * 127 * k, 128.0 * 128 * k)
    for _, lo, hi in orc.segments(ends, m):
        _close(got[lo:hi], np.broadcast_to(want, (hi - lo, n)), U * np.abs(want))
    # (relu(g) u with g = u: 0 where the sum is negative; a scale keeps the square within the type)
    a.scales.fill_(2.0 ** -20)
    got = ex.gated(a, b, b, activation="relu", offsets=_offsets(ends))
    want = np.maximum(want, 0) * want * 2.0 ** -40
    for _, lo, hi in orc.segments(ends, m):
        _close(got[lo:hi], np.broadcast_to(want, (hi - lo, n)), (H + 4 * U) * np.abs(want))


@pytest.mark.parametrize("m,n,k,ends", [(1, 130, 72, None), (2, 40, 96, [0, 2, 2]), (448, 200, 264, None), (900, 128, 192, [0, 10, 520, 890]), (8191, 64, 40, None)])
@pytest.mark.parametrize("act", ACTS)
def test_gated_backward_end_to_end(m, n, k, ends, act):
    """The whole call against the definition of unrounded terms: each term is off by dg's or du's rounding, h of itself, and by what
    these were off before it (as above); float32 results by no more than that and their sums."""
    lead = () if ends is None else (len(ends) - 1,)
    x, w = _matrix(1, m, k), [_matrix(2 + i, *lead, n, k, std=1.5 / math.sqrt(k)) for i in range(2)]
    d, g, u = (_matrix(8 + i, m, n, std=s) for i, s in enumerate((0.1, 1.5, 1.0)))
    hit = orc.rows_product(_np(x), _np(w[0]), ends)[2]
    pick = torch.from_numpy(hit).cuda()
    dg, du = orc.gated_pre_grads(_np(d), _np(g), _np(u), act)
    off = (H * np.abs(dg) + 160 * U * np.abs(_np(d) * _np(u)) * (1.2 + np.abs(_np(g)) / 4) + TINY,
           H * np.abs(du) + 160 * U * np.abs(_np(d) * orc.activation(_np(g), act)[0]) + TINY)
    ref_x, size = orc.gated_grad_x(dg, du, _np(w[0]), _np(w[1]), ends)
    off_x = orc.gated_grad_x(*off, *(np.abs(_np(v)) for v in w), ends)[0]
    tol_x = off_x + sum_tol(2 * n + 32) * (size + off_x)
    longest = max([hi - lo for _, lo, hi in orc.segments(ends, m)], default=1)
    for dtype in (torch.float32, torch.bfloat16):
        gx, *gw = X().gated_backward(d, x, *w, g, u, activation=act, offsets=_offsets(ends), dtype=dtype)
        _close(gx[pick], ref_x[hit], (tol_x + H * (np.abs(ref_x) + tol_x) + TINY)[hit], "grad_x")
        for got, dd, o, name in zip(gw, (dg, du), off, ("gate", "up")):
            ref, size = orc.gated_grad_w(dd, _np(x), ends)
            tol = orc.gated_grad_w(o, np.abs(_np(x)), ends)[0]
            tol = tol + sum_tol(longest) * (size + tol)
            _close(got, ref, tol + HALF[dtype] * (np.abs(ref) + tol) + TINY, name)
