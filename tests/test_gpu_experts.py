"""The routed-expert operators on the GPU against their float64 definitions (oracle/experts_oracle.py).

Tolerances.  u = 2^-24 is float32's half step, 2^-8 bfloat16's.
  * choices, groups, scales and codes are compared for equality;
  * sigmoid weights: expf is off by 4 u at most, 1 + e and the quotient by u, a sum of 64 and its quotient by 65 u: 80 u;
    softmax weights: the argument's rounding (|x - max| <= 40 here) 40 u, twice for the chosen and the sum, the sum's
    1024 terms in 16 lanes 68 u and its exponentials' 62 u: 256 u; beside 1e-32 where terms are denormal;
  * the routing gradient is off by the rounding of g = grad * scale (u each, in the terms g and mean of
    at most max|g|, with their products: 8 u B, B = (weight or score) * max|g|) and its own
    rounding; the unnormalised softmax works in float32: its exponent's argument (|x - max| <= 40 here)
    is off by 40 u, expf by 2 steps, a sum of 16 + 6 terms by 22 u, three such factors: 256 u B;
  * a product sums ceil(k / 128) blocks of 128 exact products: one rounding a block and at most 16 within it, each of
    at most 2 u (a sum that cuts off rather than rounds) of the sum of magnitudes, and out's rounding;
  * for a bfloat16 out the matrix instruction adds 8 neighbouring products after cutting each to a multiple of 2^-13 of
    the largest one's power of two (256 * 256 - 256 * 256 + 1 gives 0 in one such group and 1 across two): the largest is a
    product of two 4-bit significands and loses nothing, the 7 others lose at most that step each, so a group is off by
    at most 7 * 2^-13 of its largest product.
"""
import ctypes as C
import itertools

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from oracle import experts_oracle as orc  # noqa: E402

U = 2.0 ** -24
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def X():
    from muon_newton_schulz_momentum_amd import experts
    return experts


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _np(t):
    return t.detach().double().cpu().numpy()


# ---- routing ---------------------------------------------------------------------------------

def _logits(T, E, seed, dtype, kind):
    x = torch.randn(T, E, device="cuda", generator=_gen(seed)) * 2
    if kind == "masked":
        x[torch.rand(T, E, device="cuda", generator=_gen(seed + 1)) < 0.5] = -float("inf")
        x[0] = -float("inf")                                   # a row that is empty
        x[T // 2, 1:] = -float("inf")                          # a row with one expert
    elif kind == "lowest":
        x[:, ::3] = torch.finfo(dtype).min                     # the type's lowest value is finite: it may fill up
        x[0] = torch.finfo(dtype).min
    elif kind == "wild":
        x[:, 0] = float("nan")
        x[T // 2, E // 2] = float("inf")
        x[0] = float("nan")
    elif kind == "ties":
        x = (x * 2).round() / 2
    return x.to(dtype)


def _check_route(x, experts, weights, want, k):
    e_ref, w_ref = want
    assert np.array_equal(experts.cpu().numpy(), e_ref)
    w = _np(weights)
    assert (np.abs(w - w_ref) <= 256 * U * np.abs(w_ref) + 1e-32).all()


ROUTES = [
    # tokens, experts, top_k, dtype, kind, options
    (1, 1, 1, torch.float32, "plain", dict(score="softmax")),
    (3, 7, 7, torch.float32, "plain", dict(score="sigmoid", bias=True)),
    (5, 64, 2, torch.bfloat16, "ties", dict(score="softmax")),
    (257, 65, 6, torch.float32, "masked", dict(score="softmax", renormalize=False)),
    (33, 128, 8, torch.bfloat16, "lowest", dict(score="softmax", bias=True)),
    (9, 129, 4, torch.float32, "wild", dict(score="sigmoid", bias=True, scale=2.5)),
    (9, 129, 4, torch.float32, "wild", dict(score="softmax", renormalize=False)),
    (130, 512, 7, torch.bfloat16, "ties", dict(score="sigmoid", bias=True, groups=8, top_groups=4, scale=2.5)),
    (31, 512, 8, torch.float32, "masked", dict(score="softmax", groups=8, top_groups=3)),
    (31, 512, 12, torch.float32, "masked", dict(score="sigmoid", groups=64, top_groups=2)),
    (17, 513, 64, torch.float32, "plain", dict(score="sigmoid", renormalize=False)),
    (17, 1000, 40, torch.bfloat16, "masked", dict(score="softmax", bias=True, groups=4, top_groups=2)),
    (6, 1024, 64, torch.float32, "plain", dict(score="softmax", bias=True, renormalize=False)),
    (6, 96, 5, torch.float32, "plain", dict(score="sigmoid", groups=96 // 3 // 2, top_groups=3)),
    (4, 256, 3, torch.float32, "lowest", dict(score="sigmoid")),
    (1003, 512, 7, torch.float32, "plain", dict(score="sigmoid", bias=True)),
    (1003, 512, 8, torch.bfloat16, "ties", dict(score="softmax")),
    (301, 512, 8, torch.float32, "ties", dict(score="softmax", groups=8, top_groups=4)),
    (301, 256, 8, torch.bfloat16, "ties", dict(score="sigmoid", groups=8, top_groups=4, bias=True)),
    (65, 256, 15, torch.float32, "masked", dict(score="softmax", groups=4, top_groups=2, bias=True)),
    (65, 160, 6, torch.float32, "plain", dict(score="softmax", groups=10, top_groups=3)),
    (65, 1024, 6, torch.bfloat16, "masked", dict(score="sigmoid", groups=4, top_groups=1)),
    (65, 1024, 9, torch.float32, "plain", dict(score="softmax", groups=64, top_groups=5, bias=True)),
    (5, 100, 15, torch.float32, "masked", dict(score="sigmoid", bias=True)),
    (2051, 300, 7, torch.bfloat16, "masked", dict(score="sigmoid", bias=True)),
    (2051, 512, 15, torch.float32, "ties", dict(score="softmax", renormalize=False)),
    (2050, 65, 4, torch.bfloat16, "lowest", dict(score="softmax", bias=True)),
    (2048, 128, 8, torch.float32, "wild", dict(score="softmax")),
    (7, 20, 15, torch.bfloat16, "wild", dict(score="softmax")),
]


@pytest.mark.parametrize("T,E,k,dtype,kind,opt", ROUTES)
def test_route_and_backward(T, E, k, dtype, kind, opt):
    x = _logits(T, E, 100 + E + k, dtype, kind)
    bias = torch.randn(E, device="cuda", generator=_gen(7)) * 0.1 if opt.get("bias") else None
    kw = {n: v for n, v in opt.items() if n != "bias"}
    experts, weights = X().route(x, k, bias=bias, **kw)
    want = orc.route(_np(x), k, None if bias is None else _np(bias), **kw)
    _check_route(x, experts, weights, want, k)
    grad = torch.randn(T, k, device="cuda", generator=_gen(8))
    bk = {n: v for n, v in kw.items() if n in ("score", "renormalize", "scale")}
    dx = X().route_backward(x, experts, grad, **bk)
    assert dx.dtype == dtype
    _check_backward(x, want[0], grad, dx, bk)


def _check_backward(x, e_ref, grad, dx, bk):
    ref = orc.route_backward(_np(x), e_ref, _np(grad), **bk)
    s, _ = orc.scores(_np(x), bk["score"])
    renorm, raw = bk.get("renormalize", True), bk["score"] == "softmax" and not bk.get("renormalize", True)
    size = s.copy()
    if renorm:
        for t in range(s.shape[0]):
            sel = [int(e) for e in e_ref[t] if 0 <= e < s.shape[1]]
            total = s[t, sel].sum() if sel else 0.0
            size[t] = np.where(total > 0, s[t] / max(total, 1e-300), 0.0)
    gmax = np.abs(_np(grad)).max(axis=1, keepdims=True) * abs(bk.get("scale", 1.0)) * (1 + grad.shape[1] * 0)
    err = np.abs(_np(dx) - ref)
    tol = (256 if raw else 8) * U * size * gmax + HALF[dx.dtype] * np.abs(ref) * (1 + 1e-3) + 1e-40
    assert (err <= tol).all(), float((err / tol).max())


def test_route_keeps_near_ties_apart():
    """Keys that differ by less than float32 resolves: the choice follows the float64 values."""
    E = 64
    x = torch.full((1, E), 3.0, device="cuda")
    ulp = 2.0 ** -22
    x[0, 40] = 3.0 + ulp                  # sigmoid differs by about 4.5e-2 * 2.4e-7, below float32's step near 1
    bias = torch.zeros(E, device="cuda")
    experts, _ = X().route(x, 2, bias=bias, score="sigmoid")
    assert experts.cpu().tolist() == [[40, 0]]
    s = torch.sigmoid(x)
    assert s[0, 40] == s[0, 0]            # which is why float32 keys would not do


def test_route_low_scores_and_crowded_lanes():
    """Scores that underflow in float32, and the chosen experts side by side (one lane's)."""
    x = torch.randn(40, 512, device="cuda", generator=_gen(2)) - 120.0
    for kw in (dict(score="sigmoid"), dict(score="sigmoid", renormalize=False), dict(score="softmax")):
        experts, weights = X().route(x, 6, **kw)
        e_ref, w_ref = orc.route(_np(x), 6, **kw)
        assert np.array_equal(experts.cpu().numpy(), e_ref)
        # e^-120 is below float32's normal range: half its least denormal, 2^-150
        assert (np.abs(_np(weights) - w_ref) <= 256 * U * w_ref + 2.0 ** -149).all()
    x = torch.randn(40, 512, device="cuda", generator=_gen(3))
    x[:, 4:8] += 20.0
    x[:, 68:72] += 18.0
    for bias in (None, torch.zeros(512, device="cuda")):
        for dtype in (torch.float32, torch.bfloat16):
            y = x.to(dtype)
            experts, weights = X().route(y, 7, bias=bias)
            _check_route(y, experts, weights, orc.route(_np(y), 7, None if bias is None else _np(bias)), 7)


@pytest.mark.parametrize("T", [5, 2050])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_zeros_of_both_signs_are_equal(T, dtype):
    x = torch.zeros(T, 64, device="cuda")
    x[:, 1::3] = -0.0
    x[:, ::2] *= -1.0
    x[:, 5] = -1.0
    x = x.to(dtype)
    for kw in (dict(score="softmax"), dict(score="sigmoid"), dict(score="sigmoid", groups=4, top_groups=2)):
        experts, weights = X().route(x, 6, **kw)
        _check_route(x, experts, weights, orc.route(_np(x), 6, **kw), 6)


@pytest.mark.parametrize("T", [300, 2100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_near_ties_with_bias(T, score):
    """Keys that agree to 1e-7 and to 1e-5 in some of the chosen: float64 decides, for 16 experts or for the row."""
    E, k = 512, 7
    base = torch.randn(1, E, device="cuda", generator=_gen(21))
    x = base + 1e-6 * torch.randn(T, E, device="cuda", generator=_gen(22))
    s = torch.from_numpy(orc.scores(_np(base), score)[0][0]).cuda()
    for near, spread in ((10, 1e-7), (10, 1e-5), (10, 0.0), (500, 1e-7)):
        bias = torch.randn(E, device="cuda", generator=_gen(23)).double().abs() * -0.1
        at = torch.randperm(E, device="cuda", generator=_gen(24))[:near]
        bias[at] = 0.5 + spread * torch.randn(near, device="cuda", generator=_gen(25)).double()
        bias = (bias - s).float()
        experts, weights = X().route(x, k, bias=bias, score=score)
        _check_route(x, experts, weights, orc.route(_np(x), k, _np(bias), score=score), k)


@pytest.mark.parametrize("E,groups,top", [(512, 8, 4), (256, 16, 3), (512, 16, 15), (512, 4, 1), (512, 2, 1), (128, 4, 4),
                                          (304, 8, 5), (160, 2, 1), (22, 2, 1), (60, 20, 7), (64, 64, 9), (512, 64, 20), (350, 50, 33)])
@pytest.mark.parametrize("score,biased", [("sigmoid", False), ("softmax", False), ("sigmoid", True), ("softmax", True)])
def test_route_groups_at_the_border(E, groups, top, score, biased):
    """Group sums that are equal (coarse logits) or agree to 1e-7 (two groups alike but for their noise)."""
    T, k, per = 2100, 5, E // groups
    coarse = ((torch.randn(T, E, device="cuda", generator=_gen(31)) * 4).round() / 4).bfloat16()
    alike = torch.randn(T, per, device="cuda", generator=_gen(32)).repeat(1, groups)
    alike = alike + 1e-6 * torch.randn(T, E, device="cuda", generator=_gen(33))
    alike[:, per:2 * per] += 1.0
    if groups > 3:
        alike[:, 3 * per:] -= 1.0
    bias = None
    if biased:
        bias = (torch.randn(per, device="cuda", generator=_gen(34)) * 0.1).repeat(groups)
    for x in (coarse, alike):
        kw = dict(score=score, groups=groups, top_groups=top)
        experts, weights = X().route(x, k, bias=bias, **kw)
        e_ref, w_ref = orc.route(_np(x), k, None if bias is None else _np(bias), **kw)
        got = experts.cpu().numpy()
        for t in np.nonzero((got != e_ref).any(axis=1))[0]:
            assert biased
            e_ref[t], w_ref[t] = _either_group(_np(x[t:t + 1]), got[t], _np(bias), score, groups, top)
        _check_route(x, experts, weights, (e_ref, w_ref), k)


def _either_group(x, got, bias, score, groups, top):
    """got, if it is the choice for some order of the groups whose sums are equal but for rounding.

    Coarse logits and a bias that repeats give groups like (s_a + b_0) + (s_c + b_1) and (s_c + b_0) + (s_a + b_1): equal in
    exact arithmetic, and in float64 off by their roundings.  Those are at most 2^-53 for each of the three
    sums (of at most 1) and, for either score, 2^-52 of exp and 2^-53 of the quotient (what the softmax's sum is off
    by is a factor common to both): below 2^-50 in all."""
    s = orc.scores(x, score)[0][0]
    key, per = s + bias, len(bias) // groups
    worth = np.array([np.sort(key[g * per:(g + 1) * per])[-2:].sum() for g in range(groups)])
    border = np.sort(worth)[::-1][top - 1]
    sure = [g for g in range(groups) if worth[g] > border + 2.0 ** -50]
    level = [g for g in range(groups) if abs(worth[g] - border) <= 2.0 ** -50]
    for some in itertools.combinations(level, top - len(sure)):
        kept = set(sure) | set(some)
        order = sorted((e for e in range(len(bias)) if e // per in kept), key=lambda e: (-key[e], e))[:len(got)]
        if list(got) == order:
            return np.array(order), s[order] / s[order].sum()
    raise AssertionError((got, worth))


def test_route_nan_bias_counts_in_no_group():
    x = torch.randn(2100, 128, device="cuda", generator=_gen(41))
    bias = torch.zeros(128, device="cuda")
    bias[40::3] = float("nan")
    bias[20:32] = -float("inf")
    for groups in (8, 4, 2):
        kw = dict(groups=groups, top_groups=1, score="sigmoid")
        experts, weights = X().route(x, 4, bias=bias, **kw)
        _check_route(x, experts, weights, orc.route(_np(x), 4, _np(bias), **kw), 4)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_lowest_bias_and_empty_groups(score):
    """A bias of float32's lowest value leaves its experts in, behind all others; groups without an expert come last."""
    T, E, groups = 2100, 64, 8
    x = torch.randn(T, E, device="cuda", generator=_gen(51))
    x[:, :8] = -float("inf")                                   # group 0: nobody
    x[::2, 16:24] = float("nan")
    bias = torch.full((E,), torch.finfo(torch.float32).min, device="cuda")
    bias[60:] = 0.1
    bias[40] = 0.2                                             # one such expert in its group
    for top in (1, 2, 3, 7, 8):
        kw = dict(score=score, groups=groups, top_groups=top)
        experts, weights = X().route(x, 12, bias=bias, **kw)
        _check_route(x, experts, weights, orc.route(_np(x), 12, _np(bias), **kw), 12)
    experts, weights = X().route(x, 9, bias=bias, score=score)
    _check_route(x, experts, weights, orc.route(_np(x), 9, _np(bias), score=score), 9)
    x, bias = x[:, 6:22].clone(), bias[48:].clone()            # pairs: one empty, six of the lowest value, one above them
    bias[:-2] = torch.finfo(torch.float32).min
    for top in (1, 2, 3):
        kw = dict(score=score, groups=8, top_groups=top)
        experts, weights = X().route(x, 6, bias=bias, **kw)
        _check_route(x, experts, weights, orc.route(_np(x), 6, _np(bias), **kw), 6)


def test_route_bias_infinite_and_nan():
    x = torch.randn(9, 64, device="cuda", generator=_gen(4))
    bias = torch.zeros(64, device="cuda")
    bias[3], bias[5], bias[7] = float("inf"), -float("inf"), float("nan")
    for groups, top in ((1, 1), (2, 1), (4, 2)):
        kw = dict(groups=groups, top_groups=top, score="sigmoid")
        experts, weights = X().route(x, 4, bias=bias, **kw)
        _check_route(x, experts, weights, orc.route(_np(x), 4, _np(bias), **kw), 4)
        assert (experts[:, 0] == 3).all() and not ((experts == 5) | (experts == 7)).any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("power", [8, 16, 20, 30])
def test_route_groups_whose_keys_cancel(score, power):
    """Large biases of both signs in a group: its sum is small, the rounding of its float32 keys is not."""
    for E, groups, top in ((4, 2, 1), (8, 4, 2), (64, 8, 3), (160, 40, 7)):
        T, per = 600, E // groups
        x = torch.randn(T, E, device="cuda", generator=_gen(61 + E))
        bias = torch.full((E,), -2.0 ** power, device="cuda")
        bias[::per] = 2.0 ** power                              # one forced, the others banned
        bias[per * (groups - 1):] = 0.25                         # but for one group, whose sum is like theirs
        for b in (bias, bias.where(torch.arange(E, device="cuda") >= E // 2, torch.zeros_like(bias))):
            kw = dict(score=score, groups=groups, top_groups=top)
            experts, weights = X().route(x, 2, bias=b, **kw)
            e_ref, w_ref = orc.route(_np(x), 2, _np(b), **kw)
            got = experts.cpu().numpy()
            # at 2^power float64's own step is 2^(power - 52): sums nearer than 4 of them fall by their rounding
            key = orc.scores(_np(x), score)[0] + _np(b)
            worth = np.sort(key.reshape(T, groups, per), axis=2)[:, :, -2:].sum(axis=2)
            border = np.sort(worth, axis=1)[:, ::-1]
            sure = border[:, top - 1] - border[:, top] > 2.0 ** (power - 50)
            assert sure.mean() > 0.9 or power == 30
            assert np.array_equal(got[sure], e_ref[sure])
            w, w_ref = _np(weights)[sure], w_ref[sure]
            assert (np.abs(w - w_ref) <= 256 * U * np.abs(w_ref) + 1e-32).all()


def test_route_groups_at_the_softmax_sums_rounding():
    """A row whose float32 exponentials are lost one by one as they are added to the largest: the sum is 2.08e-6 short,
    and a group whose keys are biases lies in between."""
    E, ulp = 512, 2.0 ** -23
    x = np.zeros(E)
    for e in range(1, E):
        lane = e % 64 // 4                                      # of 16; lane 0 has the largest
        beside = 1 if lane < 2 else 2 if lane < 4 else 4 if lane < 8 else 8
        x[e] = np.log((0.4999 if lane == 0 else 0.49 / (32 * beside)) * ulp)
    x = torch.tensor(x, dtype=torch.float32, device="cuda").repeat(5, 1)
    kept = set()
    for j in range(50, 80):
        bias = torch.zeros(E, device="cuda")
        bias[64], bias[65] = 0.5, 0.5 - j * 2.0 ** -25
        kw = dict(score="softmax", groups=8, top_groups=1)
        experts, weights = X().route(x, 1, bias=bias, **kw)
        want = orc.route(_np(x), 1, _np(bias), **kw)
        _check_route(x, experts, weights, want, 1)
        kept.add(int(want[0][0, 0]) // 64)
    assert kept == {0, 1}                                       # both sides of the border


def test_route_infinite_biases_in_groups():
    """A forced expert makes its group's sum infinite; groups of equal infinite sums stay by lowest index."""
    x = torch.randn(300, 64, device="cuda", generator=_gen(71))
    bias = torch.zeros(64, device="cuda")
    bias[[3, 40, 41, 50]] = float("inf")
    bias[48], bias[56:60] = -float("inf"), torch.finfo(torch.float32).max
    for score in ("softmax", "sigmoid"):
        for top in (1, 2, 3, 4, 5):
            kw = dict(score=score, groups=8, top_groups=top)
            experts, weights = X().route(x, 6, bias=bias, **kw)
            _check_route(x, experts, weights, orc.route(_np(x), 6, _np(bias), **kw), 6)


@pytest.mark.parametrize("T", [6, 4200])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_route_infinity_is_float32s_largest_value(T, dtype):
    """+inf comes before bfloat16's largest value and is equal to float32's, whichever kernel takes the token."""
    x = torch.randn(T, 64, device="cuda", generator=_gen(81))
    x[:, [5, 9]] = torch.finfo(dtype).max
    x[:, [8, 11, 60]] = float("inf")
    x[::2, 1] = torch.finfo(dtype).min
    x = x.to(dtype)
    for k in (1, 4, 20):                                       # 20: the float64 kernel
        for kw in (dict(score="softmax", renormalize=False), dict(score="softmax"), dict(score="sigmoid"),
                   dict(score="softmax", groups=8, top_groups=3)):
            experts, weights = X().route(x, k, **kw)
            for rows in (slice(0, 6), slice(T - 6, T)):
                _check_route(x[rows], experts[rows], weights[rows], orc.route(_np(x[rows]), k, **kw), k)
        first = X().route(x, 1)[0]
        assert (first == (8 if dtype == torch.bfloat16 else 5)).all()


@pytest.mark.parametrize("k", [2, 5, 20])
@pytest.mark.parametrize("T", [3, 4099])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ratios_of_scores_that_underflow(k, T, score):
    """A bias chooses experts far below the row's largest logit, or all logits are far below zero: renormalised weights are
    the ratios that they are of larger scores, and the gradient is that of those weights."""
    x = torch.randn(T, 40, device="cuda", generator=_gen(91))
    x[:, 20:] += 800.0 if score == "softmax" else 0.0
    x[1::3] -= 700.0                                            # about where exp(-x) overflows
    x[2::3] -= 20000.0
    bias = torch.zeros(40, device="cuda")
    bias[:20] = 3.0
    at = np.r_[0:3, T - 3:T]
    for b in (bias, None):
        kw = dict(score=score, scale=1.5)
        experts, weights = X().route(x, k, bias=b, **kw)
        e_ref, w_ref = orc.route(_np(x[at]), k, None if b is None else _np(b), **kw)
        assert (np.abs(w_ref.sum(axis=1) - 1.5) < 1e-12).all()
        _check_route(x[at], experts[at], weights[at], (e_ref, w_ref), k)
        grad = torch.randn(T, k, device="cuda", generator=_gen(92))
        dx = _np(X().route_backward(x, experts, grad, **kw)[at])
        ref = orc.route_backward(_np(x[at]), e_ref, _np(grad[at]), **kw)
        size = np.zeros_like(ref)                                # the weights (of scale 1) bound the terms
        np.put_along_axis(size, e_ref, w_ref / 1.5, axis=1)
        gmax = 1.5 * np.abs(_np(grad[at])).max(axis=1, keepdims=True)
        assert (np.abs(dx - ref) <= 8 * U * size * gmax + U * (1 + 1e-3) * np.abs(ref) + 1e-40).all()
        assert np.abs(ref).max(axis=1).min() > 1e-4


@pytest.mark.parametrize("T", [40, 4200])
def test_route_small_sigmoids_keep_their_digits(T):
    """Down to float32's least number: e^-103 is 2^-149, and exp(-x) overflows at x = -88.8."""
    x = -86.0 - 18.0 * torch.rand(T, 64, device="cuda", generator=_gen(95))
    experts, weights = X().route(x, 6, score="sigmoid", renormalize=False)
    e_ref, w_ref = orc.route(_np(x), 6, score="sigmoid", renormalize=False)
    assert np.array_equal(experts.cpu().numpy(), e_ref)
    # a number below 2^-126 is rounded to a multiple of 2^-149: once by exp, which may be a step off, and once by the quotient
    assert (np.abs(_np(weights) - w_ref) <= 256 * U * w_ref + 2.5 * 2.0 ** -149).all()
    assert (w_ref < 2.0 ** -126).any() and (w_ref > 2.0 ** -126).any()


@pytest.mark.parametrize("E,k", [(40, 4), (300, 7), (512, 16), (512, 20), (1024, 33)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_softmax_gradient_near_one(E, k, dtype):
    """The plain softmax's gradient where one score is nearly 1, or the chosen ones are nearly all: its terms cancel, and the
    result is compared by what is left of them.

    dx_e = s_e (g_e (1 - s_e) - sum over i != e of g_i s_i) for a chosen e, -s_e sum_i g_i s_i for another.  The exponentials of
    experts that are not chosen are float32's: (|x - max| <= 45 here) the argument off by 45 u, its product with log2 e by as
    much again, exp2 by 2 u, and other factors by 4 u: 100 u of them, and 1 - s_e = (sum of the others) / z with them.  g_e (1 - s_e)
    less the chosen others' part is the others' part and a difference of exact terms; so 128 u of the terms."""
    x = torch.randn(64, E, device="cuda", generator=_gen(E + k))
    x[::2, 3] += 15.0
    x[1::4, :k] += 16.0
    x = x.to(dtype)
    experts, _ = X().route(x, k, renormalize=False)
    grad = torch.randn(64, k, device="cuda", generator=_gen(6))
    grad[3::4] = 1.0                                            # all alike: what is left is the part of those not chosen
    dx = _np(X().route_backward(x, experts, grad, renormalize=False, scale=1.5))
    s, _ = orc.scores(_np(x), "softmax")
    e, g = experts.cpu().numpy().astype(np.int64), 1.5 * _np(grad)
    sel = np.take_along_axis(s, e, axis=1)
    rest = np.ones_like(s)
    np.put_along_axis(rest, e, 0.0, axis=1)
    rest = (s * rest).sum(axis=1, keepdims=True)                # of the experts not chosen, without a difference
    ref, size = -s * (g * sel).sum(axis=1, keepdims=True), s * (np.abs(g) * sel).sum(axis=1, keepdims=True)
    for j in range(k):
        # g_j - sum g_i s_i = g_j rest + sum (g_j - g_i) s_i, as rest + sum s_i = 1
        left = g[:, j:j + 1] * rest + ((g[:, j:j + 1] - g) * sel).sum(axis=1, keepdims=True)
        terms = np.abs(g[:, j:j + 1]) * rest + (np.abs(g[:, j:j + 1] - g) * sel).sum(axis=1, keepdims=True)
        np.put_along_axis(ref, e[:, j:j + 1], sel[:, j:j + 1] * left, axis=1)
        np.put_along_axis(size, e[:, j:j + 1], sel[:, j:j + 1] * terms, axis=1)
    err = np.abs(dx - ref)
    tol = 128 * U * size + HALF[dtype] * (1 + 1e-3) * np.abs(ref) + 1e-40
    assert (err <= tol).all(), float((err / tol).max())
    assert (rest < 1e-4).any()


@pytest.mark.parametrize("T", [50, 4150])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_saturated_scores(T, score):
    """All keys equal or within 2^-16: nothing that float32 could decide, so every token goes the float64 way."""
    at = np.r_[0:20, T - 20:T]
    x = torch.randn(T, 128, device="cuda", generator=_gen(97)) + 45.0       # sigmoids of 1 in float64
    flat = 1e-6 * torch.randn(T, 128, device="cuda", generator=_gen(98))
    bias = 1e-7 * torch.randn(128, device="cuda", generator=_gen(99))
    for y in (x, flat):
        for b in (torch.zeros_like(bias), bias):
            for kw in (dict(score=score), dict(score=score, groups=8, top_groups=3)):
                experts, weights = X().route(y, 7, bias=b, **kw)
                want = orc.route(_np(y[at]), 7, _np(b), **kw)
                _check_route(y[at], experts[at], weights[at], want, 7)


def test_route_strided_and_large_rows():
    base = torch.randn(70, 200, device="cuda", generator=_gen(3))
    x = base[:, 3:100]                                        # neither aligned rows nor contiguous
    x = base[:, 4:101]                                        # the base pointer is 16-byte aligned, 97 experts
    experts, weights = X().route(x, 5)
    want = orc.route(_np(x), 5)
    _check_route(x, experts, weights, want, 5)
    out = torch.full((70, 300), 9.0, device="cuda")
    grad = torch.randn(70, 5, device="cuda", generator=_gen(4))
    X().route_backward(x, experts, grad, out=out[:, :97])
    _check_backward(x, want[0], grad, out[:, :97], dict(score="softmax"))
    assert (out[:, 97:] == 9.0).all()
    from muon_newton_schulz_momentum_amd import binding as L
    with pytest.raises(L.MuonError, match="16-byte"):
        X().route(base[:, 3:100], 5)


def test_route_backward_repeated_and_foreign_experts():
    """Equal entries add up; entries outside the experts pass nothing on."""
    x = torch.randn(4, 20, device="cuda", generator=_gen(5))
    experts = torch.tensor([[3, 3, 3], [-1, 7, 25], [0, 19, 0], [-1, -1, -1]], dtype=torch.int32, device="cuda")
    grad = torch.randn(4, 3, device="cuda", generator=_gen(6))
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            bk = dict(score=score, renormalize=renorm)
            _check_backward(x, experts.cpu().numpy(), grad, X().route_backward(x, experts, grad, **bk), bk)


@pytest.mark.parametrize("E,k", [(40, 4), (512, 7), (300, 20), (1024, 8)])
@pytest.mark.parametrize("kw", [dict(score="softmax"), dict(score="softmax", renormalize=False), dict(score="sigmoid")])
def test_route_backward_in_place(E, k, kw):
    x = torch.randn(67, E, device="cuda", generator=_gen(11))
    experts, _ = X().route(x, k, **kw)
    grad = torch.randn(67, k, device="cuda", generator=_gen(12))
    want = X().route_backward(x, experts, grad, **kw)
    assert X().route_backward(x, experts, grad, out=x, **kw) is x
    assert torch.equal(x, want)


def test_route_gradient_is_the_difference_quotient():
    """d sum(w * grad) / dx by central differences of the kernel's own weights (float32: the quotient of
    weights rounded at 2^-24 over 2 * 2^-6 is off by k * 2^-24 * 2^5, the third derivative adds h^2)."""
    x = torch.randn(2, 24, device="cuda", generator=_gen(9))
    grad = torch.randn(2, 4, device="cuda", generator=_gen(10))
    h = 2.0 ** -6
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            bias = torch.zeros(24, device="cuda")
            bias[[2, 5, 11, 17]] = 10.0                       # the choice stays put
            kw = dict(bias=bias, score=score, renormalize=renorm)
            e0, _ = X().route(x, 4, **kw)
            dx = X().route_backward(x, e0, grad, score=score, renormalize=renorm)
            order = e0.long()

            def loss(y):
                e, w = X().route(y, 4, **kw)
                full = torch.zeros(2, 24, device="cuda", dtype=torch.float64).scatter_(1, e.long(), w.double())
                return (full.gather(1, order) * grad.double()).sum(1)
            for e in range(24):
                up, dn = x.clone(), x.clone()
                up[:, e] += h
                dn[:, e] -= h
                q = (loss(up) - loss(dn)) / (up[:, e] - dn[:, e]).double()
                gmax = grad.abs().sum(1).double()
                assert ((q - dx[:, e].double()).abs() <= gmax * (4 * U * 2 ** 5 + h * h) + 1e-6).all()


# ---- grouping ---------------------------------------------------------------------------------

@pytest.mark.parametrize("T,k,E,align", [
    (1, 1, 1, 1), (1, 7, 512, 1), (16, 7, 512, 128), (5, 3, 2, 16), (100, 64, 1024, 8), (1170, 7, 512, 128),
    (1171, 7, 512, 1), (3000, 3, 1, 128), (2000, 5, 1024, 32), (4097, 4, 65, 128), (30000, 2, 300, 1),
])
def test_group_rows(T, k, E, align):
    ex = torch.randint(0, E, (T, k), device="cuda", generator=_gen(T + E), dtype=torch.int32)
    ex = torch.where(torch.rand(T, k, device="cuda", generator=_gen(T)) < 0.5, ex, ex // 3)   # uneven
    if T > 4:
        ex[T // 2] = -1
        ex[1, 0] = E                                           # no such expert: goes nowhere
    for _ in range(2):
        g = X().group_rows(ex, E, align=align)
        want = orc.group_rows(ex.cpu().numpy().reshape(-1), E, align)
        for name, t, ref in zip(("counts", "offsets", "rows", "position"), (g.counts, g.offsets, g.rows, g.position), want):
            assert np.array_equal(t.cpu().numpy().reshape(-1), ref), name
    assert g.position.shape == ex.shape and int(g.limit) == want[1][-1]


def test_group_rows_of_nothing():
    g = X().group_rows(torch.empty(0, 3, dtype=torch.int32, device="cuda"), 5, align=128)
    assert g.counts.tolist() == [0] * 5 and g.offsets.tolist() == [0] * 6 and g.rows.numel() == 0
    g = X().group_rows(torch.full((4, 3), -1, dtype=torch.int32, device="cuda"), 5, align=4)
    assert g.offsets.tolist() == [0] * 6 and (g.rows == -1).all() and (g.position == -1).all()


def test_balance_step():
    counts = torch.tensor([5, 0, 3, 2, 2, 6], dtype=torch.int32, device="cuda")       # mean 3
    bias = torch.randn(6, device="cuda", generator=_gen(1))
    out = X().balance_step(bias, counts, 0.01)
    sign = torch.tensor([-1, 1, 0, 1, 1, -1], device="cuda", dtype=torch.float32)
    assert torch.equal(out, bias + sign * torch.tensor(0.01, device="cuda"))
    X().balance_step(bias, counts, 0.01, out=bias)
    assert torch.equal(out, bias)
    # 3 * 2^31 - 3 choices in all: the sum and the comparison are not float32's
    big = torch.tensor([2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 2], dtype=torch.int64).to(torch.int32).cuda()
    out = X().balance_step(torch.zeros(4, device="cuda"), big, 1.0)
    assert out.tolist() == [-1, -1, -1, 1]


# ---- quantisation -----------------------------------------------------------------------------

def _check_fp8(q, ref, fmt, rows=None):
    codes, exps = ref
    got, gs = _np(q.codes.float()), q.scales.view(torch.uint8).cpu().numpy().astype(np.int64) - 127
    if rows is not None:
        got, gs, codes, exps = got[rows], gs[rows], codes[rows], exps[rows]
    assert np.array_equal(gs, exps)
    assert np.array_equal(got, codes, equal_nan=True)


def _source(rows, cols, dtype, seed, kind="plain"):
    x = torch.randn(rows, cols, device="cuda", generator=_gen(seed))
    x *= torch.exp(2 * torch.randn(rows, 1, device="cuda", generator=_gen(seed + 1)))
    if kind == "edges":
        flat = x.view(-1)
        special = torch.tensor([0.0, -0.0, 448.0, 449.0, 1e-45, -1e-45, 1.17e-38, 3.4e38, -3.4e38, 57344.0, 464.0, 2.0 ** -126])
        flat[:special.numel()] = special.cuda()[:flat.numel()]
        x[rows // 2] = 0.0
        x[:, cols // 2] = 0.0
    elif kind == "wild":
        x[0, 0] = float("inf")
        x[rows // 2, cols // 2] = float("nan")
        x[rows - 1] = -float("inf")
    elif kind == "midpoints":
        # halves between codes at every power of two, so that ties decide
        x = torch.randint(-63, 64, (rows, cols), device="cuda", generator=_gen(seed)).float() * 2.0 ** -3
    return x.to(dtype)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 130), (128, 128), (129, 257), (40, 1000), (300, 515), (5, 640)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", ["plain", "edges", "wild", "midpoints"])
def test_quantize(rows, cols, fmt, kind):
    dtype = torch.float32 if (rows + cols) % 2 else torch.bfloat16
    x = _source(rows, cols, dtype, rows + cols, kind)
    for block in ("row", "square"):
        q, qt = X().quantize(x, block=block, format=fmt, transpose=True)
        assert q.codes.dtype == FP8[fmt]
        _check_fp8(q, orc.quantize(_np(x), fmt, block == "square"), fmt)
        _check_fp8(qt, orc.quantize(_np(x).T, fmt, block == "square"), fmt)
        alone = X().quantize(x, block=block, format=fmt)
        assert torch.equal(alone.codes.view(torch.uint8), q.codes.view(torch.uint8))
        assert torch.equal(alone.scales.view(torch.uint8), q.scales.view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_stack_and_strides(dtype):
    base = _source(3 * 200, 400, dtype, 5).view(3, 200, 400)
    x = base[:, :150, 8:301]                                   # strided rows and matrices, odd columns
    for block in ("row", "square"):
        q, qt = X().quantize(x, block=block, transpose=True)
        for i in range(3):
            sub = X().Fp8(q.codes[i], q.scales[i], q.cols, q.square)
            _check_fp8(sub, orc.quantize(_np(x[i]), "e4m3", block == "square"), "e4m3")
            sub = X().Fp8(qt.codes[i], qt.scales[i], qt.cols, qt.square)
            _check_fp8(sub, orc.quantize(_np(x[i]).T, "e4m3", block == "square"), "e4m3")
    odd = base[0, :, 8:301].contiguous()                       # ld 293: rows on no 16-byte boundary
    _check_fp8(X().quantize(odd), orc.quantize(_np(odd), "e4m3", False), "e4m3")


def test_quantize_gather_and_limit():
    tokens, cols, per = 50, 300, 3
    x = _source(tokens, cols, torch.bfloat16, 11)
    rows = torch.randint(0, tokens * per, (390,), device="cuda", generator=_gen(12), dtype=torch.int32)
    rows[::7] = -1
    rows[5], rows[6] = tokens * per, 2 ** 31 - 1               # past the source: zeros, not a read
    r = rows.cpu().numpy().astype(np.int64)
    full = np.where(((r >= 0) & (r < tokens * per))[:, None], _np(x)[np.clip(r // per, 0, tokens - 1)], 0.0)
    q, qt = X().quantize(x, rows=rows, per=per, transpose=True)
    _check_fp8(q, orc.quantize(full, "e4m3", False), "e4m3")
    _check_fp8(qt, orc.quantize(full.T, "e4m3", False), "e4m3")
    for used in (0, 1, 128, 200, 390, 1000):
        outs = [X().Fp8.empty(390, cols), X().Fp8.empty(cols, 390)]
        for o in outs:
            o.codes.view(torch.uint8).fill_(0x55)
            o.scales.view(torch.uint8).fill_(0x33)
        limit = torch.tensor([used], dtype=torch.int32, device="cuda")
        X().quantize(x, rows=rows, per=per, limit=limit, transpose=True, out=outs)
        n = min(used, 390)
        cut = full.copy()
        cut[n:] = 0.0
        _check_fp8(outs[0], orc.quantize(cut, "e4m3", False), "e4m3", rows=slice(0, n))
        assert (outs[0].codes.view(torch.uint8)[n:] == 0x55).all() and (outs[0].scales.view(torch.uint8)[n:] == 0x33).all()
        nb = -(-n // 128)
        ref_c, ref_e = orc.quantize(cut.T, "e4m3", False)
        assert np.array_equal(_np(outs[1].codes.float())[:, :nb * 128], ref_c[:, :nb * 128])
        assert (outs[1].codes.view(torch.uint8)[:, nb * 128:] == 0x55).all()
        got = outs[1].scales.view(torch.uint8).cpu().numpy().astype(np.int64)
        assert np.array_equal(got[:, :nb] - 127, ref_e[:, :nb])
        if nb < 4:
            assert (got[:, nb:] == 0x33).all()


def test_quantize_empty_rows():
    q, qt = X().quantize(torch.empty(0, 200, device="cuda"), transpose=True)
    assert q.codes.shape == (0, 256) and qt.codes.shape == (200, 0)
    q = X().quantize(torch.randn(4, 200, device="cuda"), rows=torch.empty(0, dtype=torch.int32, device="cuda"))
    assert q.codes.shape == (0, 256)
    none = X().quantize(torch.empty(0, 200, device="cuda"), rows=torch.zeros(5, dtype=torch.int32, device="cuda"))
    assert (none.codes.view(torch.uint8) == 0).all()


def test_route_and_quantize_beyond_32_bits():
    """Logits, sources and copies of more than 2^32 bytes: the last rows are those of a call on them alone."""
    x = torch.empty(4_300_000, 512, dtype=torch.bfloat16, device="cuda").normal_(generator=_gen(1))
    tail = x[-2051:]
    for got, want in zip(X().route(x, 7, score="sigmoid"), X().route(tail, 7, score="sigmoid")):
        assert torch.equal(got[-2051:], want)
    experts, _ = X().route(tail, 7)
    grad = torch.randn(len(x), 7, device="cuda", generator=_gen(2))
    every = torch.zeros(len(x), 7, dtype=torch.int32, device="cuda")
    every[-2051:] = experts
    want = X().route_backward(tail, experts, grad[-2051:].clone())
    assert torch.equal(X().route_backward(x, every, grad, out=x)[-2051:], want)
    del every, grad
    x.normal_(generator=_gen(3))
    x = x.view(-1, 4096)                                     # 537500 rows, not a multiple of 128
    cut = 537500 // 128 * 128
    q, qt = X().quantize(x[:, :4090], transpose=True)
    part, part_t = X().quantize(x[cut:, :4090], transpose=True)
    assert torch.equal(q.codes[cut:].view(torch.uint8), part.codes.view(torch.uint8))
    assert torch.equal(q.scales[cut:].view(torch.uint8), part.scales.view(torch.uint8))
    assert torch.equal(qt.codes[:, cut:].view(torch.uint8), part_t.codes.view(torch.uint8))
    assert torch.equal(qt.scales[:, cut // 128].view(torch.uint8), part_t.scales[:, 0].view(torch.uint8))


# ---- products ---------------------------------------------------------------------------------

def _random_fp8(rows, cols, fmt, square, seed, stack=None):
    x = torch.randn(*(() if stack is None else (stack,)), rows, cols, device="cuda", generator=_gen(seed))
    x *= torch.exp(torch.randn(*x.shape[:-1], 1, device="cuda", generator=_gen(seed + 1)))
    return X().quantize(x, block="square" if square else "row", format=fmt)


def _largest_of_8(a, b):
    """Sum over groups of 8 neighbouring k of the largest product in the group."""
    x, y = (torch.from_numpy(np.abs(np.pad(v, ((0, 0), (0, -v.shape[1] % 8))))).cuda() for v in (a, b))
    total = torch.zeros(len(x), len(y), dtype=torch.float64, device="cuda")
    for q in range(0, x.shape[1], 8):
        total += (x[:, None, q:q + 8] * y[None, :, q:q + 8]).amax(-1)
    return total.cpu().numpy()


def _check_product(out, a, b, k, rows=slice(None), before=0.0):
    """out against a b^T in float64 from the float64 values a, b (numpy)."""
    ref = a @ b.T
    mag = np.abs(a) @ np.abs(b).T
    err = np.abs(_np(out) - (ref + before))
    tol = 2 * U * (-(-k // 128) + 16) * mag + HALF[out.dtype] * (1 + 1e-3) * np.abs(ref + before) + 1e-37
    if out.dtype == torch.bfloat16:
        tol = tol + 7 * 2.0 ** -13 * _largest_of_8(a, b)
    assert (err <= tol).all(), float((err / tol).max())


SIZES = [(1, 1, 1), (1, 128, 128), (16, 16, 256), (17, 100, 300), (128, 128, 128), (129, 255, 1000), (300, 513, 640),
         (5, 2000, 130), (257, 129, 2048)]
# enough tiles for the 256 x 256 kernel; last tiles of 5, 100 and 190 rows, and more tiles than workgroups
SIZES += [(2053, 1100, 640), (2148, 1280, 1), (2238, 1025, 129), (4500, 4300, 400)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_product_dense(m, n, k, fmt):
    a, b = _random_fp8(m, k, fmt, False, m + k), _random_fp8(n, k, "e4m3", True, n + k)
    va, vb = _np(a.dequantize()), _np(b.dequantize())
    for dtype in (torch.bfloat16, torch.float32):
        _check_product(X().product(a, b, dtype=dtype), va, vb, k)
    sq, row = _random_fp8(m, k, fmt, True, m), _random_fp8(n, k, "e4m3", False, n)
    _check_product(X().product(sq, row, dtype=torch.float32), _np(sq.dequantize()), _np(row.dequantize()), k)
    # into a strided, wider matrix, and added to what is there
    wide = torch.randn(m, n + 7, device="cuda", generator=_gen(1))
    before = wide.clone()
    X().product(a, b, out=wide[:, :n], accumulate=True)
    _check_product(wide[:, :n], va, vb, k, before=_np(before[:, :n]))
    assert torch.equal(wide[:, n:], before[:, n:])


GROUPS = [
    # sizes of the segments, n, k
    ([5], 70, 200),
    ([0, 3, 0, 0, 1, 16, 0], 130, 256),
    ([1] * 40, 64, 128),
    ([129, 0, 128, 300, 1, 127], 200, 384),
    ([2, 40, 17, 64, 33, 8, 100, 0], 256, 1000),
    ([0] * 600 + [7] + [0] * 300 + [20], 33, 130),
    ([600, 500], 257, 256),
    # enough tiles for the 256 x 256 kernel: segments of every number of row blocks, some empty
    ([(37 * i * i) % 290 if i % 7 else 0 for i in range(40)], 1000, 400),
    ([300, 0, 513, 64, 65, 1000, 1, 129, 192, 193, 255, 256], 2100, 900),
    ([20] * 150 + [0] * 50 + [21] * 100, 2060, 300),
]


@pytest.mark.parametrize("sizes,n,k", GROUPS)
@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.bfloat16), ("e5m2", torch.float32)])
def test_product_rows(sizes, n, k, fmt, dtype):
    m, E = sum(sizes), len(sizes)
    tail = 3                                                   # rows behind the last segment
    a, b = _random_fp8(m + tail, k, fmt, False, m), _random_fp8(n, k, "e4m3", True, n, stack=E)
    ends = np.concatenate([[0], np.cumsum(sizes)])
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    out = torch.full((m + tail, n), 7.5, dtype=dtype, device="cuda")
    X().product(a, b, offsets=offsets, group="rows", out=out)
    va, vb = _np(a.dequantize()), _np(b.dequantize())
    for g in range(E):
        if sizes[g]:
            s = slice(ends[g], ends[g + 1])
            _check_product(out[s], va[s], vb[g], k)
    assert (out[m:] == 7.5).all()
    again = torch.full_like(out, 7.5)
    X().product(a, b, offsets=offsets, group="rows", out=again)
    assert torch.equal(again, out)


@pytest.mark.parametrize("sizes,m,n", [([3], 20, 30), ([0, 128, 5, 0], 130, 128), ([300, 1, 256], 100, 515), ([0, 0], 8, 8),
                                       ([600, 0, 1, 128, 300, 0], 700, 1100), ([130, 0, 0, 0, 20, 1, 513, 128, 0], 1030, 2060)])
@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float32), ("e5m2", torch.bfloat16)])
def test_product_depth(sizes, m, n, fmt, dtype):
    ends = np.concatenate([[0], np.cumsum([-(-s // 128) * 128 for s in sizes])])
    total = int(ends[-1]) + 128                                # columns behind the last segment
    xa = torch.randn(total, m, device="cuda", generator=_gen(m))
    xb = torch.randn(total, n, device="cuda", generator=_gen(n))
    for g, s in enumerate(sizes):
        xa[ends[g] + s:ends[g + 1]] = 0.0
    _, a = X().quantize(xa, format=fmt, transpose=True)
    _, b = X().quantize(xb, transpose=True)
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    out = X().product(a, b, offsets=offsets, group="depth", dtype=dtype)
    va, vb = _np(a.dequantize()), _np(b.dequantize())
    for g in range(len(sizes)):
        s = slice(ends[g], ends[g + 1])
        _check_product(out[g], va[:, s], vb[:, s], ends[g + 1] - ends[g])
    if dtype == torch.float32:
        acc = torch.randn_like(out)
        before = acc.clone()
        X().product(a, b, offsets=offsets, group="depth", out=acc, accumulate=True)
        for g in range(len(sizes)):
            s = slice(ends[g], ends[g + 1])
            _check_product(acc[g], va[:, s], vb[:, s], ends[g + 1] - ends[g], before=_np(before[g]))


def _check_full_sums(out, a, b, k, more=0.0):
    """As _check_product, without what the 8-bit instruction drops."""
    ref, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = 2 * U * (-(-k // 128) + 16) * mag + HALF[out.dtype] * (1 + 1e-3) * np.abs(ref) + 1e-37 + more
    err = np.abs(_np(out) - ref)
    assert (err <= tol).all(), float((err / tol).max())


def test_product_full_sums_where_products_cancel():
    """256 * 256 - 256 * 256 + 1 in one group of 8: the 1 is there with full sums."""
    for rows, cols, k in ((1, 1, 128), (40, 70, 384), (2100, 2300, 256)):
        x, y = torch.zeros(rows, k, device="cuda"), torch.zeros(cols, k, device="cuda")
        x[:, 0], x[:, 1], x[:, 2] = 256.0, 256.0, 1.0
        y[:, 0], y[:, 1], y[:, 2] = 256.0, -256.0, 1.0
        a, b = X().quantize(x), X().quantize(y)
        assert (X().product(a, b, full_sums=True) == 1.0).all()
        assert (X().product(a, b, dtype=torch.float32) == 1.0).all()
        assert ((X().product(a, b) - 1.0).abs() <= 7 * 2.0 ** -13 * 65536).all()


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (17, 100, 300), (129, 255, 1000), (300, 513, 640), (2053, 1100, 640), (4500, 4300, 400)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_product_full_sums_dense(m, n, k, fmt):
    a, b = _random_fp8(m, k, fmt, False, m + k), _random_fp8(n, k, "e4m3", True, n + k)
    got = X().product(a, b, full_sums=True)
    _check_full_sums(got, _np(a.dequantize()), _np(b.dequantize()), k)
    assert torch.equal(got, X().product(a, b, dtype=torch.float32).bfloat16())      # the same sums, rounded once


def test_product_full_sums_in_groups():
    sizes, n, k = [300, 0, 513, 64, 65, 1000, 1, 129, 192, 193, 255, 256], 2100, 900
    ends = np.concatenate([[0], np.cumsum(sizes)])
    a, b = _random_fp8(int(ends[-1]) + 3, k, "e4m3", False, 1), _random_fp8(n, k, "e4m3", True, 2, stack=len(sizes))
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    out = torch.full((int(ends[-1]) + 3, n + 1), 7.5, dtype=torch.bfloat16, device="cuda")
    X().product(a, b, offsets=offsets, group="rows", out=out[:, :n], full_sums=True)
    va, vb = _np(a.dequantize()), _np(b.dequantize())
    for g, s in enumerate(sizes):
        if s:
            _check_full_sums(out[ends[g]:ends[g + 1], :n], va[ends[g]:ends[g + 1]], vb[g], k)
    assert (out[ends[-1]:] == 7.5).all() and (out[:, n] == 7.5).all()
    cols = [300, 0, 128, 5, 640]
    ends = np.concatenate([[0], np.cumsum([-(-s // 128) * 128 for s in cols])])
    a, b = _random_fp8(130, int(ends[-1]), "e5m2", False, 3), _random_fp8(515, int(ends[-1]), "e4m3", False, 4)
    out = X().product(a, b, offsets=torch.tensor(ends, dtype=torch.int32, device="cuda"), group="depth", full_sums=True)
    va, vb = _np(a.dequantize()), _np(b.dequantize())
    for g in range(len(cols)):
        s = slice(ends[g], ends[g + 1])
        _check_full_sums(out[g], va[:, s], vb[:, s], max(1, int(ends[g + 1] - ends[g])))


def test_product_offsets_are_clamped():
    """Offsets outside the operand reach neither past it nor past out."""
    a, b = _random_fp8(40, 128, "e4m3", False, 1), _random_fp8(32, 128, "e4m3", True, 2, stack=3)
    va, vb = _np(a.dequantize()), _np(b.dequantize())
    guard = torch.full((60, 32), 3.0, device="cuda")
    X().product(a, b, offsets=torch.tensor([-5, 10, 10, 1000], dtype=torch.int32, device="cuda"), group="rows", out=guard[:40])
    _check_product(guard[:10], va[:10], vb[0], 128)
    _check_product(guard[10:40], va[10:], vb[2], 128)
    assert (guard[40:] == 3.0).all()
    xa = torch.randn(256, 16, device="cuda", generator=_gen(3))
    _, t = X().quantize(xa, transpose=True)
    out = X().product(t, t, offsets=torch.tensor([-128, 128, 1024], dtype=torch.int32, device="cuda"), group="depth",
                      dtype=torch.float32)
    vt = _np(t.dequantize())
    _check_product(out[0], vt[:, :128], vt[:, :128], 128)
    _check_product(out[1], vt[:, 128:], vt[:, 128:], 128)


def test_product_large_with_bad_offsets_and_odd_rows():
    """256 x 256 tiles: offsets outside the operand, rows of out that are not 16-byte aligned, sums onto out."""
    m, n, k, E = 3001, 2045, 300, 4
    a, b = _random_fp8(m, k, "e4m3", False, 5), _random_fp8(n, k, "e4m3", True, 6, stack=E)
    va, vb = _np(a.dequantize()), _np(b.dequantize())
    offsets = torch.tensor([-7, 1000, 1000, 2500, 1 << 30], dtype=torch.int32, device="cuda")
    ends = [0, 1000, 1000, 2500, m]
    for accumulate in (False, True):
        wide = torch.randn(m + 5, n + 2, device="cuda", generator=_gen(7))   # rows of 8188 bytes
        before = wide.clone()
        X().product(a, b, offsets=offsets, group="rows", out=wide[:m, :n], accumulate=accumulate)
        for g in range(E):
            s = slice(ends[g], ends[g + 1])
            if s.stop > s.start:
                _check_product(wide[s, :n], va[s], vb[g], k, before=_np(before[s, :n]) if accumulate else 0.0)
        assert torch.equal(wide[m:], before[m:]) and torch.equal(wide[:, n:], before[:, n:])
    half = torch.full((m, n + 1), 3.0, dtype=torch.bfloat16, device="cuda")
    X().product(a, b, offsets=offsets, group="rows", out=half[:, :n])
    for g in (0, 2, 3):
        s = slice(ends[g], ends[g + 1])
        _check_product(half[s, :n], va[s], vb[g], k)
    assert (half[:, n] == 3.0).all()
    # depth: bounds below, between blocks (rounded down) and behind the operand
    xa, xb = (torch.randn(1024, c, device="cuda", generator=_gen(c)) for c in (1500, 2000))
    ta, tb = X().quantize(xa, transpose=True)[1], X().quantize(xb, transpose=True)[1]
    out = X().product(ta, tb, offsets=torch.tensor([-1, 300, 640, 640, 9999], dtype=torch.int32, device="cuda"),
                      group="depth", dtype=torch.float32)
    va, vb = _np(ta.dequantize()), _np(tb.dequantize())
    for g, (lo, hi) in enumerate([(0, 256), (256, 640), (640, 640), (640, 1024)]):
        _check_product(out[g], va[:, lo:hi], vb[:, lo:hi], hi - lo)


def test_product_beyond_32_bits():
    """Operands and results of more than 2^32 bytes: their last rows and groups."""
    def random_fp8(rows, cols, stack=None):
        q = X().Fp8.empty(rows, cols, stack=stack)
        q.codes.view(torch.uint8).random_(0, 0x78, generator=_gen(rows))             # finite
        q.scales.view(torch.uint8).random_(120, 130, generator=_gen(cols))
        return q

    def last(q, n):
        return X().Fp8(q.codes[..., -n:, :], q.scales[..., -n:, :], q.cols, q.square)

    a, b = random_fp8(1_100_000, 4096), random_fp8(2100, 4096)
    out = X().product(a, b)                                   # 4.5 and 4.6 GB
    _check_product(out[-300:], _np(last(a, 300).dequantize()), _np(b.dequantize()), 4096)
    del out
    b = random_fp8(2048, 4096, stack=520)                     # 4.4 GB
    offsets = torch.arange(521, dtype=torch.int32, device="cuda") * 2
    a = last(a, 1040)
    one = X().Fp8(b.codes[519], b.scales[519], 4096, False)
    _check_product(X().product(a, b, offsets=offsets, group="rows")[-2:], _np(last(a, 2).dequantize()),
                   _np(one.dequantize()), 4096)
    del b
    a, b = random_fp8(4096, 8192), random_fp8(4300, 8192)
    offsets = torch.arange(65, dtype=torch.int32, device="cuda") * 128
    out = X().product(a, b, offsets=offsets, group="depth", dtype=torch.float32)     # 4.5 GB
    _check_product(out[63][:, -300:], _np(a.dequantize())[:, -128:], _np(last(b, 300).dequantize())[:, -128:], 128)


@pytest.mark.parametrize("m,n,groups,dtype,deep", [
    (1100, 3400, 9, torch.float32, 1), (2048, 2048, 20, torch.bfloat16, 1), (2000, 2050, 300, torch.bfloat16, 1),
    (2048, 64, 9, torch.float32, 6),                           # 32 x 64 tiles
])
def test_product_depth_groups_of_many_tiles(m, n, groups, dtype, deep):
    """Groups whose tiles are dealt to all XCDs, deepest first (or, from 257 groups on, as they come)."""
    blocks = [(5 * g * g + 3 * g) % 4 * deep for g in range(groups)]
    ends = np.concatenate([[0], np.cumsum(blocks)]) * 128
    a, b = _random_fp8(m, int(ends[-1]), "e4m3", False, m), _random_fp8(n, int(ends[-1]), "e4m3", False, n)
    out = torch.full((groups, m, n), float("nan"), dtype=dtype, device="cuda")
    X().product(a, b, offsets=torch.tensor(ends, dtype=torch.int32, device="cuda"), group="depth", out=out)
    assert not torch.isnan(out).any()
    va, vb = _np(a.dequantize()), _np(b.dequantize())
    for g in range(groups) if groups < 10 else (0, 1, 2, groups // 2, groups - 2, groups - 1):
        s = slice(ends[g], ends[g + 1])
        _check_product(out[g], va[:, s], vb[:, s], ends[g + 1] - ends[g])


def test_product_large_captured_and_replayed():
    """Rows-grouped and depth-grouped products in 256 x 256 tiles, their offsets changed between replays."""
    E, n, k = 5, 1300, 512
    a, b = _random_fp8(2560, k, "e4m3", False, 1), _random_fp8(n, k, "e4m3", True, 2, stack=E)
    ta, tb = _random_fp8(1000, 2560, "e4m3", False, 3), _random_fp8(n, 2560, "e4m3", False, 4)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    y = torch.zeros(2560, n, dtype=torch.bfloat16, device="cuda")
    dw = torch.zeros(E, 1000, n, device="cuda")

    def run(y, dw):
        X().product(a, b, offsets=offsets, group="rows", out=y)
        X().product(ta, tb, offsets=offsets, group="depth", out=dw)

    run(y, dw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(y, dw)
    for bounds in ([0, 512, 512, 1024, 2432, 2560], [0, 0, 0, 0, 0, 128], [0, 128, 1280, 1408, 1536, 2304]):
        offsets.copy_(torch.tensor(bounds, dtype=torch.int32))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        y2, dw2 = torch.zeros_like(y), torch.zeros_like(dw)
        run(y2, dw2)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(dw, dw2)
        assert (y[bounds[-1]:] == 0).all()


def test_product_no_depth():
    a, b = X().Fp8.empty(5, 0), X().Fp8.empty(9, 0)
    assert (X().product(a, b, dtype=torch.float32) == 0).all()
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert (X().product(a, b, offsets=off, group="depth", dtype=torch.float32) == 0).all()
    assert X().product(X().Fp8.empty(0, 128), _random_fp8(9, 128, "e4m3", True, 1)).shape == (0, 9)


def test_product_nan_stays_in_its_row():
    x = torch.randn(20, 256, device="cuda", generator=_gen(1))
    x[3, 200] = float("nan")
    x[4, 0] = float("inf")
    a, b = X().quantize(x), _random_fp8(64, 256, "e4m3", True, 2)
    out = X().product(a, b, dtype=torch.float32)
    bad = torch.isnan(out).all(dim=1)
    assert bad.nonzero().flatten().tolist() == [3, 4] and torch.isfinite(out[~bad]).all()


def _carve(*sizes):
    """Tensors directly behind one another, in one allocation: of (shape, dtype)."""
    bytes_of = [int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size() for shape, dtype in sizes]
    assert all(b % 16 == 0 for b in bytes_of[:-1])             # every one begins on a 16-byte boundary
    block, at, out = torch.empty(sum(bytes_of), dtype=torch.uint8, device="cuda"), 0, []
    for (shape, dtype), b in zip(sizes, bytes_of):
        out.append(block[at:at + b].view(dtype).view(shape))
        at += b
    return out


def test_column_slices_beside_their_outputs():
    """Columns away from the left end with their rows' last column: what follows is another buffer's, and may be written."""
    R, K, n = 512, 2048, 256
    e8 = torch.float8_e8m0fnu
    base, codes, scales = _carve(((R, K), torch.bfloat16), ((R, K // 2), torch.float8_e4m3fn), ((R, 8), e8))
    base.normal_(generator=_gen(1))
    half = base[:, K // 2:]
    q = X().Fp8(codes, scales, K // 2, False)
    X().quantize(half, out=q)
    _check_fp8(q, orc.quantize(_np(half), "e4m3", False), "e4m3")
    stack, codes, scales = _carve(((3, 64, 512), torch.float32), ((3, 64, 256), torch.float8_e4m3fn), ((3, 1, 4), e8))
    stack.normal_(generator=_gen(2))
    q = X().Fp8(codes, scales, 256, True)
    X().quantize(stack[:, :, 256:], block="square", out=q)
    for i in range(3):
        _check_fp8(X().Fp8(codes[i], scales[i], 256, True), orc.quantize(_np(stack[i, :, 256:]), "e4m3", True), "e4m3")
    # both halves of a gate / up result, the operands right behind it
    y, ac, asc, bc, bsc = _carve(((R, 2 * n), torch.bfloat16), ((R, 512), torch.float8_e4m3fn), ((R, 4), e8), ((n, 512), torch.float8_e4m3fn),
                                 ((n // 128, 4), e8))
    a, b = X().Fp8(ac, asc, 512, False), X().Fp8(bc, bsc, 512, True)
    for q, src, block in ((a, _source(R, 512, torch.float32, 3), "row"), (b, _source(n, 512, torch.float32, 4), "square")):
        X().quantize(src, block=block, out=q)
    y.fill_(3.0)
    X().product(a, b, out=y[:, n:])
    assert (y[:, :n] == 3.0).all()
    right = y[:, n:].clone()
    X().product(a, b, out=y[:, :n])
    va, vb = _np(a.dequantize()), _np(b.dequantize())
    _check_product(y[:, :n], va, vb, 512)
    assert torch.equal(y[:, n:], right) and torch.equal(y[:, :n], right)


def test_column_ranges_of_one_buffer():
    """A result in the columns beside its input's: the rows of one lie in the gaps of the other's."""
    both = torch.zeros(70, 128, device="cuda")
    both[:, :64].normal_(generator=_gen(5))
    x = both[:, :64].clone()
    experts, _ = X().route(both[:, :64], 4)
    grad = torch.randn(70, 4, device="cuda", generator=_gen(6))
    X().route_backward(both[:, :64], experts, grad, out=both[:, 64:])
    assert torch.equal(both[:, 64:], X().route_backward(x, experts, grad)) and torch.equal(both[:, :64], x)
    codes = torch.zeros(40, 512, dtype=torch.uint8, device="cuda")
    src = _source(40, 128, torch.float32, 7)
    q = X().quantize(src)
    codes[:, :128] = q.codes.view(torch.uint8)
    a = X().Fp8(codes[:, :128].view(torch.float8_e4m3fn), q.scales, 128, False)
    out = codes.view(torch.float32)[:, 64:104]                 # bytes 256 to 416 of rows of 512
    X().product(a, q, out=out)
    assert torch.equal(out, X().product(q, q, dtype=torch.float32))
    assert torch.equal(codes[:, :128], q.codes.view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_gather_into_squares(dtype):
    """Rows gathered into 128 x 128 squares, both orientations; -1 and rows past the source are zeros."""
    tokens, cols, per = 70, 333, 2
    x = _source(tokens, cols, dtype, 21)
    rows = torch.randint(0, tokens * per, (301,), device="cuda", generator=_gen(22), dtype=torch.int32)
    rows[::9], rows[4] = -1, tokens * per
    rows[128:256] = -1                                         # a square of zeros
    r = rows.cpu().numpy().astype(np.int64)
    full = np.where(((r >= 0) & (r < tokens * per))[:, None], _np(x)[np.clip(r // per, 0, tokens - 1)], 0.0)
    for fmt in ("e4m3", "e5m2"):
        q, qt = X().quantize(x, rows=rows, per=per, block="square", format=fmt, transpose=True)
        _check_fp8(q, orc.quantize(full, fmt, True), fmt)
        _check_fp8(qt, orc.quantize(full.T, fmt, True), fmt)


@pytest.mark.parametrize("sizes,n,k", [([5, 0, 130, 7], 70, 300), ([300, 1, 513, 0, 640, 90] * 3, 1030, 400)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product_rows_of_squares(sizes, n, k, dtype):
    """a in squares, whose 128 rows straddle the segments, and b in rows."""
    m, E = sum(sizes), len(sizes)
    a, b = _random_fp8(m, k, "e5m2", True, m), _random_fp8(n, k, "e4m3", False, n, stack=E)
    ends = np.concatenate([[0], np.cumsum(sizes)])
    out = X().product(a, b, offsets=torch.tensor(ends, dtype=torch.int32, device="cuda"), group="rows", dtype=dtype)
    va, vb = _np(a.dequantize()), _np(b.dequantize())
    for g in range(E):
        if sizes[g]:
            _check_product(out[ends[g]:ends[g + 1]], va[ends[g]:ends[g + 1]], vb[g], k)


@pytest.mark.parametrize("blocks,m,n", [([1, 0, 2, 3], 100, 260), ([3, 1, 0, 5, 2, 1], 1030, 2060)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product_depth_of_squares(blocks, m, n, dtype):
    """Both operands as square copies' transposes."""
    ends = 128 * np.concatenate([[0], np.cumsum(blocks)])
    xa, xb = (_source(int(ends[-1]), c, torch.float32, c) for c in (m, n))
    a, b = X().quantize(xa, block="square", transpose=True)[1], X().quantize(xb, block="square", transpose=True)[1]
    out = X().product(a, b, offsets=torch.tensor(ends, dtype=torch.int32, device="cuda"), group="depth", dtype=dtype)
    va, vb = _np(a.dequantize()), _np(b.dequantize())
    for g in range(len(blocks)):
        s = slice(ends[g], ends[g + 1])
        _check_product(out[g], va[:, s], vb[:, s], max(1, int(ends[g + 1] - ends[g])))


@pytest.mark.parametrize("magnitude", [3e38, 1e30, 2e-36, 1e-37])
def test_product_of_extreme_scales(magnitude):
    """Scale bytes at both ends of their range.

    Full float32 sums take the values as bfloat16: one below 2^-126 is rounded to a multiple of 2^-133, by at most half of that, and its
    products are off by as much of the other factor."""
    def step(v):
        return np.where((np.abs(v) < 2.0 ** -126) & (v != 0), 2.0 ** -134, 0.0)

    x = _source(40, 256, torch.float32, 31).sign() * magnitude * (0.5 + 0.4 * torch.rand(40, 256, device="cuda", generator=_gen(32)))
    y = torch.randn(70, 256, device="cuda", generator=_gen(33)) / magnitude
    for fmt in ("e4m3", "e5m2"):
        a, b = X().quantize(x, format=fmt), X().quantize(y)
        _check_fp8(a, orc.quantize(_np(x), fmt, False), fmt)
        va, vb = _np(a.dequantize()), _np(b.dequantize())
        assert np.isfinite(va).all()
        _check_product(X().product(a, b), va, vb, 256)
        more = step(va) @ np.abs(vb).T + np.abs(va) @ step(vb).T + step(va) @ step(vb).T
        _check_full_sums(X().product(a, b, dtype=torch.float32), va, vb, 256, more)
        _check_full_sums(X().product(a, b, full_sums=True), va, vb, 256, more * (1 + HALF[torch.bfloat16]))
        assert ((step(va) > 0).any() or (step(vb) > 0).any()) == (magnitude == 3e38)


def test_stream_argument_captured():
    """Calls that name their stream, captured on it and replayed."""
    s = torch.cuda.Stream()
    x = torch.randn(300, 64, device="cuda", generator=_gen(1))
    w = X().quantize(torch.randn(48, 64, device="cuda", generator=_gen(2)), block="square")

    def run():
        e, weights = X().route(x, 3, stream=s)
        g = X().group_rows(e, 64, stream=s)
        q = X().quantize(x, rows=g.rows, per=3, limit=g.limit, stream=s)
        return e, weights, g.rows, X().product(q, w, dtype=torch.float32, stream=s)

    torch.cuda.synchronize()
    run()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = run()
    for replay in range(3):
        x.copy_(torch.randn(300, 64, device="cuda", generator=_gen(10 + replay)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_wrapper_refusals_on_the_gpu():
    a, b = _random_fp8(4, 128, "e4m3", False, 1), _random_fp8(8, 128, "e5m2", True, 2)
    with pytest.raises(ValueError, match="dtype"):
        X().product(a, b)
    c = _random_fp8(8, 256, "e4m3", True, 2)
    with pytest.raises(ValueError, match="columns"):
        X().product(a, c)
    with pytest.raises(ValueError, match="offsets"):
        X().product(a, a, group="depth")
    with pytest.raises(ValueError, match="accumulate"):
        X().product(a, a, accumulate=True)
    with pytest.raises(ValueError, match="shape"):
        X().product(a, a, out=torch.empty(4, 5, device="cuda"))
    wrong = X().Fp8(a.codes, a.scales[:, :2], a.cols, False)
    with pytest.raises(ValueError, match="scales"):
        X().product(wrong, a)
    with pytest.raises(ValueError, match="out"):
        X().quantize(torch.zeros(4, 128, device="cuda"), out=[a, a])
    with pytest.raises(ValueError, match="dtype"):
        X().route(torch.zeros(4, 8, device="cuda"), 2, bias=torch.zeros(8, device="cuda", dtype=torch.float64))


# ---- streams, graphs, and a run of them together ------------------------------------------------

def _layer(tokens, logits, bias, W, grad_y, top_k, E, G=None):
    """The routed part of a training step up to the weights' gradients; also what a serving step does (its first half)."""
    x = X()
    chosen, weights = x.route(logits, top_k, bias=bias, score="sigmoid", groups=4, top_groups=2, scale=2.0)
    g = x.group_rows(chosen, E, align=128)
    w, w_t = x.quantize(W, block="square", transpose=True)
    xq, xq_t = x.quantize(tokens, rows=g.rows, per=top_k, limit=g.limit, transpose=True)
    y = x.product(xq, w, offsets=g.offsets, group="rows")
    dy, dy_t = x.quantize(grad_y, rows=g.rows, per=1, limit=g.limit, format="e5m2", transpose=True)
    dx = x.product(dy, w_t, offsets=g.offsets, group="rows")
    dW = x.product(dy_t, xq_t, offsets=g.offsets, group="depth", out=G, dtype=torch.float32)
    y_at = y.float()[g.position.clamp(min=0).long()]                        # (tokens, top_k, out)
    dw = (y_at * grad_y.float().view(*chosen.shape, -1)).sum(-1)
    dlogits = x.route_backward(logits, chosen, dw.contiguous(), score="sigmoid", scale=2.0)
    new_bias = x.balance_step(bias, g.counts, 0.01)
    return dict(chosen=chosen, weights=weights, g=g, w=w, w_t=w_t, xq=xq, xq_t=xq_t, y=y, dy=dy, dy_t=dy_t, dx=dx,
                dW=dW, dw=dw, dlogits=dlogits, bias=new_bias)


def _layer_inputs(T, E, k, d, n, seed):
    g = _gen(seed)
    return dict(tokens=torch.randn(T, d, device="cuda", generator=g).bfloat16(),
                logits=torch.randn(T, E, device="cuda", generator=g) * 2,
                bias=torch.randn(E, device="cuda", generator=g) * 0.1,
                W=torch.randn(E, n, d, device="cuda", generator=g) * 0.02,
                grad_y=torch.randn(T * k, n, device="cuda", generator=g).bfloat16())


def test_layer_and_optimizer_step_together():
    """Route, group, quantise, multiply, go back, and step the experts' weights with the plan: each stage
    against its definition on that stage's inputs, then the weights, requantised, are the next step's."""
    from muon_newton_schulz_momentum_amd.harness import ParamTensors, Plan
    T, E, k, d, n = 90, 16, 3, 192, 144
    inp = _layer_inputs(T, E, k, d, n, 3)
    G, M = torch.zeros(E, n, d, device="cuda"), torch.zeros(E, n, d, device="cuda")
    plan = Plan([ParamTensors(inp["W"][e], M[e], G[e]) for e in range(E)])
    for step in range(2):
        W0 = inp["W"].clone()
        r = _layer(**inp, top_k=k, E=E, G=G)
        kw = dict(score="sigmoid", groups=4, top_groups=2, scale=2.0)
        e_ref, w_ref = orc.route(_np(inp["logits"]), k, _np(inp["bias"]), **kw)
        _check_route(inp["logits"], r["chosen"], r["weights"], (e_ref, w_ref), k)
        counts, offsets, rows, position = orc.group_rows(e_ref.reshape(-1), E, 128)
        assert np.array_equal(r["g"].rows.cpu().numpy(), rows)
        used = int(offsets[-1])
        src = np.where(rows[:used, None] >= 0, _np(inp["tokens"])[np.maximum(rows[:used], 0) // k], 0.0)
        _check_fp8(r["xq"], orc.quantize(src, "e4m3", False), "e4m3", rows=slice(0, used))
        for e in range(E):
            _check_fp8(X().Fp8(r["w"].codes[e], r["w"].scales[e], d, True), orc.quantize(_np(W0[e]), "e4m3", True), "e4m3")
        vx, vw, vdy = _np(r["xq"].dequantize()), _np(r["w"].dequantize()), _np(r["dy"].dequantize())
        vwt, vdyt, vxt = _np(r["w_t"].dequantize()), _np(r["dy_t"].dequantize()), _np(r["xq_t"].dequantize())
        assert np.array_equal(vwt, vw.transpose(0, 2, 1))
        for e in range(E):
            s = slice(offsets[e], offsets[e + 1])
            if counts[e]:
                _check_product(r["y"][s], vx[s], vw[e], d)
                _check_product(r["dx"][s], vdy[s], vwt[e], n)
            _check_product(r["dW"][e], vdyt[:, s], vxt[:, s], max(1, offsets[e + 1] - offsets[e]))
            if not counts[e]:
                assert (r["dW"][e] == 0).all()
        _check_backward(inp["logits"], e_ref, r["dw"], r["dlogits"], dict(score="sigmoid", scale=2.0))
        # the step reads those gradients: bitwise the step of a plan on copies
        copies = [ParamTensors(W0[e].clone(), M[e].clone(), r["dW"][e].clone()) for e in range(E)]
        other = Plan(copies)
        other.step(0.95, 0.02, 0.1)
        plan.step(0.95, 0.02, 0.1)
        torch.cuda.synchronize()
        for e in range(E):
            assert torch.equal(inp["W"][e], copies[e].weight)
        assert not torch.equal(inp["W"], W0)
        inp["bias"] = r["bias"]
        other.close()
    plan.close()


def _flat(r):
    used = int(r["g"].limit)
    for name in ("chosen", "weights", "dW", "dw", "dlogits", "bias"):
        yield name, r[name]
    for name in ("y", "dx"):
        yield name, r[name][:used]
    for name in ("counts", "offsets", "rows", "position"):
        yield name, getattr(r["g"], name)


def test_layer_captured_and_replayed():
    """The whole layer in one graph, replayed with new inputs and with eager work in between: every replay is
    bitwise the eager result."""
    T, E, k, d, n = 700, 24, 4, 256, 128                       # 2800 choices
    static = _layer_inputs(T, E, k, d, n, 50)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for _ in range(2):
            _layer(**static, top_k=k, E=E)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        res = _layer(**static, top_k=k, E=E)
    for replay in range(4):
        fresh = _layer_inputs(T, E, k, d, n, 60 + replay)
        for name, t in fresh.items():
            static[name].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        want = _layer(**fresh, top_k=k, E=E)
        torch.cuda.synchronize()
        for (name, got), (_, ref) in zip(_flat(res), _flat(want)):
            assert torch.equal(got, ref), (replay, name)


def test_large_group_rows_captured():
    """The three-launch grouping in a graph: its workspace is the graph's own."""
    ex = torch.randint(0, 100, (5000, 6), device="cuda", generator=_gen(1), dtype=torch.int32)
    X().group_rows(ex, 100, align=16)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = X().group_rows(ex, 100, align=16)
    for replay in range(3):
        ex.copy_(torch.randint(-1, 100, (5000, 6), device="cuda", generator=_gen(replay), dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = orc.group_rows(ex.cpu().numpy().reshape(-1), 100, 16)
        for t, ref in zip((g.counts, g.offsets, g.rows, g.position), want):
            assert np.array_equal(t.cpu().numpy().reshape(-1), ref)


def test_two_streams_at_once():
    """Two layers on two streams at the same time: neither shares anything with the other."""
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    inputs = [_layer_inputs(600, 16, 3, 384, 256, s) for s in (1, 2)]
    want = [_layer(**i, top_k=3, E=16) for i in inputs]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = _layer(**inputs[i], top_k=3, E=16)
    torch.cuda.synchronize()
    for i in range(2):
        for (name, a), (_, b) in zip(_flat(got[i]), _flat(want[i])):
            assert torch.equal(a, b), name


def test_stream_of_another_device_is_refused():
    class Elsewhere:
        device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="stream is on"):
        X().route(torch.zeros(4, 8, device="cuda"), 2, stream=Elsewhere())


def test_stream_argument():
    s = torch.cuda.Stream()
    x = torch.randn(300, 64, device="cuda", generator=_gen(1))
    torch.cuda.synchronize()
    e, w = X().route(x, 3, stream=s)
    g = X().group_rows(e, 64, stream=s)
    q = X().quantize(x, stream=s)
    y = X().product(q, q, dtype=torch.float32, stream=s)
    s.synchronize()
    e2, w2 = X().route(x, 3)
    assert torch.equal(e, e2) and torch.equal(w, w2) and torch.equal(g.rows, X().group_rows(e2, 64).rows)
    assert torch.equal(y, X().product(q, q, dtype=torch.float32))


@pytest.mark.parametrize("name", ["route", "route_backward", "group_rows", "balance_step", "quantize", "product"])
def test_tensors_dropped_behind_a_stream(name):
    """A tensor that the caller drops after a call on another stream is not handed out again before that stream is done."""
    x, s = X(), torch.cuda.Stream()
    q = x.quantize(torch.randn(512, 4096, device="cuda", generator=_gen(1)))
    logits = torch.randn(4096, 256, device="cuda", generator=_gen(2))
    experts, weights = x.route(logits, 8)
    off = torch.tensor([0, 128, 1024], dtype=torch.int32, device="cuda")
    made = {
        "route": (lambda a, b: x.route(a, 8, bias=b, stream=s), lambda: [logits.clone(), torch.randn(256, device="cuda", generator=_gen(3))]),
        "route_backward": (lambda a, b, c: x.route_backward(a, b, c, stream=s), lambda: [logits.clone(), experts.clone(), weights.clone()]),
        "group_rows": (lambda a: x.group_rows(a, 256, align=16, stream=s), lambda: [experts.clone()]),
        "balance_step": (lambda a, b: x.balance_step(a, b, 0.5, stream=s),
                         lambda: [torch.randn(1024, device="cuda", generator=_gen(4)), torch.arange(1024, dtype=torch.int32, device="cuda")]),
        "quantize": (lambda a, b: x.quantize(a, rows=b, per=2, stream=s),
                     lambda: [logits.clone(), torch.arange(8191, -1, -1, dtype=torch.int32, device="cuda")]),
        "product": (lambda a, b, c, d, e: x.product(x.Fp8(a, b, 4096, False), x.Fp8(c, d, 4096, False), dtype=torch.float32, stream=s,
                                                    offsets=e, group="depth"),
                    lambda: [q.codes.clone(), q.scales.clone(), q.codes.clone(), q.scales.clone(), off.clone()]),
    }
    call, inputs = made[name]
    flat = lambda r: [t for t in (vars(r).values() if isinstance(r, x.Groups) else r if isinstance(r, tuple) else    # noqa: E731
                                  [r.codes, r.scales] if isinstance(r, x.Fp8) else [r])]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)                         # longer than the host takes for what follows
    given = inputs()
    sizes = [(t.shape, t.dtype) for t in given]
    s.wait_stream(torch.cuda.current_stream())
    got = call(*given)
    del given
    again = [torch.zeros(shape, dtype=torch.uint8 if dtype.itemsize == 1 else dtype, device="cuda") for shape, dtype in sizes]
    torch.cuda.synchronize()
    del again
    for a, b in zip(flat(got), flat(call(*inputs()))):
        torch.cuda.synchronize()
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
