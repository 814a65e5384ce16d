"""CPU tests of the routed-expert entry points: what they refuse, what they do with empty sizes, their size
queries, and the oracle's own pins.  Device pointers are fake, aligned addresses: every call here ends before a launch.
"""
import ctypes as C

import numpy as np
import pytest
import torch

from muon_newton_schulz_momentum_amd import binding as L
from oracle import experts_oracle as orc

MEM = 1 << 40                      # fake, 256-byte aligned addresses, far apart
A, B, S, T, O, W = (MEM + i * (1 << 36) for i in range(6))


def _route(**kw):
    c = L.muon_route_config(4, 8, 8, 2, L.MUON_DTYPE_F32, L.MUON_SCORE_SOFTMAX, 1, 1, 1, 1.0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("kw,status", [
    (dict(n_experts=0), L.MUON_ERR_SHAPE), (dict(n_experts=1025, ld=2000), L.MUON_ERR_SHAPE),
    (dict(top_k=0), L.MUON_ERR_SHAPE), (dict(top_k=9), L.MUON_ERR_SHAPE),
    (dict(n_experts=100, ld=100, top_k=65), L.MUON_ERR_SHAPE), (dict(tokens=-1), L.MUON_ERR_SHAPE),
    (dict(tokens=1 << 31), L.MUON_ERR_SHAPE), (dict(tokens=1 << 26, top_k=1), L.MUON_ERR_SHAPE), (dict(tokens=1 << 30), L.MUON_ERR_SHAPE), (dict(ld=7), L.MUON_ERR_SHAPE),
    (dict(dtype=2), L.MUON_ERR_INVALID_ARG), (dict(score=2), L.MUON_ERR_INVALID_ARG),
    (dict(n_groups=3), L.MUON_ERR_INVALID_ARG), (dict(n_groups=0), L.MUON_ERR_INVALID_ARG),
    (dict(n_experts=130, ld=130, n_groups=65), L.MUON_ERR_INVALID_ARG),
    (dict(n_groups=2, top_groups=3), L.MUON_ERR_INVALID_ARG), (dict(top_groups=0), L.MUON_ERR_INVALID_ARG),
    (dict(renormalize=2), L.MUON_ERR_INVALID_ARG), (dict(scale=float("nan")), L.MUON_ERR_INVALID_ARG),
    (dict(scale=float("inf")), L.MUON_ERR_INVALID_ARG),
])
def test_route_refuses(kw, status):
    c = _route(**kw)
    assert L.muon_route(C.byref(c), A, None, B, S, None) == status
    assert b"muon_route" in L.muon_last_error()
    assert L.muon_route_backward(C.byref(c), A, B, S, O, 4096, None) == status


def test_route_refuses_buffers():
    c = _route()
    assert L.muon_route(None, A, None, B, S, None) == L.MUON_ERR_INVALID_ARG
    for bad in ((None, None, B, S), (A, None, None, S), (A, None, B, None)):
        assert L.muon_route(C.byref(c), *bad, None) == L.MUON_ERR_INVALID_ARG
    for bad in ((A + 4, None, B, S), (A, T + 8, B, S), (A, None, B + 4, S), (A, None, B, S + 4)):
        assert L.muon_route(C.byref(c), *bad, None) == L.MUON_ERR_ALIGNMENT
    assert L.muon_route_backward(C.byref(c), A, B, S, O, 7, None) == L.MUON_ERR_SHAPE
    for bad in ((None, B, S, O), (A, None, S, O), (A, B, None, O), (A, B, S, None)):
        assert L.muon_route_backward(C.byref(c), *bad, 8, None) == L.MUON_ERR_INVALID_ARG
    for bad in ((A + 4, B, S, O), (A, B + 4, S, O), (A, B, S + 4, O), (A, B, S, O + 8)):
        assert L.muon_route_backward(C.byref(c), *bad, 8, None) == L.MUON_ERR_ALIGNMENT
    none = _route(tokens=0)
    assert L.muon_route(C.byref(none), None, None, None, None, None) == L.MUON_OK
    assert L.muon_route_backward(C.byref(none), None, None, None, None, 8, None) == L.MUON_OK


@pytest.mark.parametrize("n,e,align", [(0, 5, 128), (1, 5, 128), (3, 512, 16), (9000, 512, 128), (100, 7, 1)])
def test_group_rows_sizes(n, e, align):
    rows, ws = C.c_int64(), C.c_uint64()
    assert L.muon_group_rows_capacity(n, e, align, C.byref(rows)) == L.MUON_OK
    assert rows.value == orc.capacity(n, e, align) and rows.value % align == 0 and rows.value >= n
    assert L.muon_group_rows_workspace(n, e, C.byref(ws)) == L.MUON_OK
    if ws.value:
        bad = L.muon_group_rows(A, n, e, align, B, S, T, O, W, ws.value - 1, None)
        assert bad == L.MUON_ERR_WORKSPACE_TOO_SMALL
        assert L.muon_group_rows(A, n, e, align, B, S, T, O, None, ws.value, None) == L.MUON_ERR_INVALID_ARG
        assert L.muon_group_rows(A, n, e, align, B, S, T, O, W + 8, ws.value, None) == L.MUON_ERR_ALIGNMENT


def test_capacity_holds_the_worst_case():
    for n in (1, 4, 5, 37):
        worst = 0
        for spread in range(1, 6):
            counts = np.bincount(np.arange(n) % spread, minlength=5)
            worst = max(worst, int((-(-counts // 16) * 16).sum()))
        assert worst <= orc.capacity(n, 5, 16)


def test_group_rows_refuses():
    rows = C.c_int64()
    for n, e, align, st in ((-1, 4, 1, L.MUON_ERR_SHAPE), (4, 0, 1, L.MUON_ERR_SHAPE), (4, 1025, 1, L.MUON_ERR_SHAPE),
                            ((1 << 31) - 4, 4, 1, L.MUON_ERR_SHAPE), (4, 4, 0, L.MUON_ERR_INVALID_ARG),
                            (4, 4, 3, L.MUON_ERR_INVALID_ARG), (4, 4, 256, L.MUON_ERR_INVALID_ARG)):
        assert L.muon_group_rows_capacity(n, e, align, C.byref(rows)) == st
        assert L.muon_group_rows(A, n, e, align, B, S, T, O, None, 0, None) == st
    assert L.muon_group_rows_capacity(4, 4, 1, None) == L.MUON_ERR_INVALID_ARG
    assert L.muon_group_rows_workspace(4, 4, None) == L.MUON_ERR_INVALID_ARG
    good = [A, 4, 4, 1, B, S, T, O, None, 0, None]
    for i in (0, 4, 5, 6, 7):
        args = list(good)
        args[i] = None
        assert L.muon_group_rows(*args) == L.MUON_ERR_INVALID_ARG
        args[i] = good[i] + 4
        assert L.muon_group_rows(*args) == L.MUON_ERR_ALIGNMENT


def test_balance_refuses():
    assert L.muon_balance_step(A, B, 0, 0.1, S, None) == L.MUON_ERR_SHAPE
    assert L.muon_balance_step(A, B, 1025, 0.1, S, None) == L.MUON_ERR_SHAPE
    assert L.muon_balance_step(A, B, 8, float("nan"), S, None) == L.MUON_ERR_INVALID_ARG
    for bad in ((None, B, S), (A, None, S), (A, B, None)):
        assert L.muon_balance_step(bad[0], bad[1], 8, 0.1, bad[2], None) == L.MUON_ERR_INVALID_ARG
    assert L.muon_balance_step(A, B + 4, 8, 0.1, S, None) == L.MUON_ERR_ALIGNMENT


def _quant(**kw):
    c = L.muon_fp8_quantize_config()
    c.src, c.batch, c.rows, c.cols, c.ld, c.per = A, 1, 4, 200, 200, 1
    c.codes, c.scales, c.codes_t, c.scales_t = B, S, T, O
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("kw,status", [
    (dict(src_dtype=2), L.MUON_ERR_INVALID_ARG), (dict(format=2), L.MUON_ERR_INVALID_ARG),
    (dict(square=2), L.MUON_ERR_INVALID_ARG), (dict(cols=0), L.MUON_ERR_SHAPE), (dict(rows=-1), L.MUON_ERR_SHAPE),
    (dict(batch=-1), L.MUON_ERR_SHAPE), (dict(ld=199), L.MUON_ERR_SHAPE), (dict(ld=1 << 31), L.MUON_ERR_SHAPE),
    (dict(batch=2, batch_stride=799), L.MUON_ERR_SHAPE), (dict(batch=2, batch_stride=800, gather=W), L.MUON_ERR_INVALID_ARG),
    (dict(batch=2, batch_stride=800, limit=W), L.MUON_ERR_INVALID_ARG), (dict(square=1, limit=W), L.MUON_ERR_INVALID_ARG),
    (dict(gather=W, per=0, src_rows=4), L.MUON_ERR_INVALID_ARG), (dict(gather=W, src_rows=-1), L.MUON_ERR_INVALID_ARG),
    (dict(codes=None, scales=None, codes_t=None, scales_t=None), L.MUON_ERR_INVALID_ARG),
    (dict(scales=None), L.MUON_ERR_INVALID_ARG), (dict(codes_t=None), L.MUON_ERR_INVALID_ARG),
    (dict(src=None), L.MUON_ERR_INVALID_ARG), (dict(src=A + 4), L.MUON_ERR_ALIGNMENT),
    (dict(codes=B + 8), L.MUON_ERR_ALIGNMENT), (dict(scales_t=O + 4), L.MUON_ERR_ALIGNMENT),
    (dict(gather=W + 4, src_rows=4), L.MUON_ERR_ALIGNMENT), (dict(limit=W + 2), L.MUON_ERR_ALIGNMENT),
    (dict(codes=A + 1024), L.MUON_ERR_INVALID_ARG), (dict(codes_t=A - 256), L.MUON_ERR_INVALID_ARG),
    (dict(rows=(1 << 31) - 128, cols=(1 << 31) - 128, ld=(1 << 31) - 128), L.MUON_ERR_SHAPE),
    (dict(batch=1 << 24, rows=1, cols=1, batch_stride=1), L.MUON_ERR_SHAPE),
])
def test_quantize_refuses(kw, status):
    c = _quant(**kw)
    assert L.muon_fp8_quantize(C.byref(c), None) == status
    assert b"muon_fp8_quantize" in L.muon_last_error()


def test_quantize_empty():
    assert L.muon_fp8_quantize(None, None) == L.MUON_ERR_INVALID_ARG
    assert L.muon_fp8_quantize(C.byref(_quant(rows=0)), None) == L.MUON_OK
    assert L.muon_fp8_quantize(C.byref(_quant(batch=0)), None) == L.MUON_OK


def _product(mode=0, **kw):
    c = L.muon_fp8_product_config()
    c.mode, c.groups, c.m, c.n, c.k = mode, (3 if mode else 1), 8, 200, 256
    for o, codes, scales in ((c.a, A, S), (c.b, B, T)):
        o.codes, o.scales, o.ld, o.ld_scales = codes, scales, 256, 4
    c.b.stride, c.b.stride_scales = 200 * 256, 200 * 4
    c.out, c.ld_out, c.out_stride = O, 200, 8 * 200
    c.offsets = W if mode else None
    for k, v in kw.items():
        t = c
        *path, last = k.split("__")
        for x in path:
            t = getattr(t, x)
        setattr(t, last, v)
    return c


@pytest.mark.parametrize("mode,kw,status", [
    (3, {}, L.MUON_ERR_INVALID_ARG), (0, dict(groups=2), L.MUON_ERR_INVALID_ARG), (1, dict(groups=0), L.MUON_ERR_INVALID_ARG),
    (1, dict(groups=1025), L.MUON_ERR_INVALID_ARG), (0, dict(m=-1), L.MUON_ERR_SHAPE), (0, dict(n=1 << 31), L.MUON_ERR_SHAPE),
    (0, dict(k=-1), L.MUON_ERR_SHAPE), (0, dict(a__format=2), L.MUON_ERR_INVALID_ARG),
    (0, dict(b__format=1), L.MUON_ERR_INVALID_ARG), (0, dict(out_dtype=2), L.MUON_ERR_INVALID_ARG),
    (0, dict(accumulate=1, out_dtype=1), L.MUON_ERR_INVALID_ARG), (0, dict(accumulate=2), L.MUON_ERR_INVALID_ARG),
    (0, dict(ld_out=199), L.MUON_ERR_SHAPE), (2, dict(out_stride=1599), L.MUON_ERR_SHAPE),
    (0, dict(out=None), L.MUON_ERR_INVALID_ARG), (1, dict(offsets=None), L.MUON_ERR_INVALID_ARG),
    (0, dict(out=O + 8), L.MUON_ERR_ALIGNMENT), (1, dict(offsets=W + 2), L.MUON_ERR_ALIGNMENT),
    (0, dict(a__codes=None), L.MUON_ERR_INVALID_ARG), (0, dict(b__scales=None), L.MUON_ERR_INVALID_ARG),
    (0, dict(a__codes=A + 8), L.MUON_ERR_ALIGNMENT), (0, dict(b__scales=T + 4), L.MUON_ERR_ALIGNMENT),
    (0, dict(a__ld=255), L.MUON_ERR_SHAPE), (0, dict(a__ld=240), L.MUON_ERR_SHAPE), (0, dict(b__ld_scales=6), L.MUON_ERR_SHAPE),
    (0, dict(a__ld=1 << 23), L.MUON_ERR_SHAPE), (0, dict(b__ld_scales=1 << 23), L.MUON_ERR_SHAPE),
    (0, dict(k=600, a__ld=640, b__ld=640), L.MUON_ERR_SHAPE), (0, dict(a__square=2), L.MUON_ERR_INVALID_ARG),
    (1, dict(b__stride=200 * 256 - 16), L.MUON_ERR_SHAPE), (1, dict(b__stride_scales=200 * 4 - 4), L.MUON_ERR_SHAPE),
    (1, dict(b__stride=-16), L.MUON_ERR_SHAPE), (0, dict(out=A), L.MUON_ERR_INVALID_ARG),
    (1, dict(out=B + 2 * 200 * 256), L.MUON_ERR_INVALID_ARG),
    (2, dict(groups=1024, m=1 << 17, n=1 << 20, ld_out=1 << 20, out_stride=1 << 37, offsets=W), L.MUON_ERR_SHAPE),
])
def test_product_refuses(mode, kw, status):
    c = _product(mode, **kw)
    assert L.muon_fp8_product(C.byref(c), None) == status
    assert b"muon_fp8_product" in L.muon_last_error()


def test_product_empty():
    assert L.muon_fp8_product(None, None) == L.MUON_ERR_INVALID_ARG
    for mode in (0, 1, 2):
        assert L.muon_fp8_product(C.byref(_product(mode, m=0)), None) == L.MUON_OK
        assert L.muon_fp8_product(C.byref(_product(mode, n=0)), None) == L.MUON_OK


def test_wrapper_refuses_host_tensors():
    from muon_newton_schulz_momentum_amd import experts as X
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        X.route(x, 2)
    with pytest.raises(ValueError, match="score"):
        X.route(x, 2, score="relu")
    with pytest.raises(ValueError, match="GPU"):
        X.quantize(x)
    with pytest.raises(ValueError, match="block"):
        X.quantize(x, block="col")
    with pytest.raises(ValueError, match="overlap"):
        X.route(torch.zeros(8).expand(4, 8), 2)
    q = X.Fp8.empty(4, 200, device="cpu")
    assert q.codes.shape == (4, 256) and q.scales.shape == (4, 4) and q.rows == 4
    with pytest.raises(ValueError, match="GPU"):
        X.product(q, q)


# ---- the oracle ------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_oracle_rounding_is_the_formats(fmt, dtype):
    codes = torch.arange(256, dtype=torch.uint8).view(dtype).double()
    codes = codes[torch.isfinite(codes)].unique().numpy()
    assert codes.max() == orc.MAX[fmt]
    assert np.array_equal(orc.round_fp8(codes, fmt), codes)
    mid = (codes[1:] + codes[:-1]) / 2
    for nudge, want in ((-1e-9, codes[:-1]), (1e-9, codes[1:])):
        assert np.array_equal(orc.round_fp8(mid + nudge * np.maximum(np.abs(mid), 1e-6), fmt), want)
    even = orc.round_fp8(mid, fmt)
    assert np.array_equal(even, torch.tensor(mid).float().to(dtype).double().numpy())


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_oracle_block_exponent(fmt):
    rng = np.random.default_rng(3)
    amax = np.concatenate([2.0 ** rng.uniform(-100, 100, 500), orc.MAX[fmt] * 2.0 ** np.arange(-20, 20.0)])
    e = orc.block_exponents(amax, fmt).astype(np.float64)
    assert (amax <= orc.MAX[fmt] * 2.0 ** e).all() and (amax > orc.MAX[fmt] * 2.0 ** (e - 1)).all()
    assert orc.block_exponents(np.zeros(1), fmt)[0] == -127


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_oracle_route_gradient_is_the_difference_quotient(score, renormalize):
    rng = np.random.default_rng(5)
    x = rng.normal(0, 1.5, (3, 9))
    x[1, 4] = -np.inf
    g = rng.normal(size=(3, 4))
    kw = dict(score=score, renormalize=renormalize, scale=1.7)
    experts, _ = orc.route(x, 4, **kw)
    dx = orc.route_backward(x, experts, g, **kw)

    def loss(y):
        s, _ = orc.scores(y, score)
        w = np.take_along_axis(s, experts, 1)
        if renormalize:
            w = w / w.sum(1, keepdims=True)
        return (w * g).sum() * 1.7
    for t in range(3):
        for e in range(9):
            if not np.isfinite(x[t, e]):
                assert dx[t, e] == 0
                continue
            up, dn = x.copy(), x.copy()
            up[t, e] += 1e-6
            dn[t, e] -= 1e-6
            # central difference: error of order 1e-12 * third derivative + 1e-16 / 1e-6
            assert abs((loss(up) - loss(dn)) / 2e-6 - dx[t, e]) < 1e-8


# ---- sizes near the ends of their types --------------------------------------------------------

@pytest.mark.parametrize("n", [(1 << 63) - 1, (1 << 63) - 512, 1 << 62, (1 << 31) - 1 - 4 * 128])
def test_group_rows_refuses_a_capacity_that_is_no_int32(n):
    rows, ws = C.c_int64(), C.c_uint64()
    assert L.muon_group_rows_capacity(n, 4, 128, C.byref(rows)) == L.MUON_ERR_SHAPE
    assert L.muon_group_rows_workspace(n, 4, C.byref(ws)) == L.MUON_ERR_SHAPE
    assert L.muon_group_rows(A, n, 4, 128, B, S, T, O, W, (1 << 64) - 1, None) == L.MUON_ERR_SHAPE


def test_group_rows_takes_the_largest_size():
    rows = C.c_int64()
    n = (1 << 31) - 1 - 127 - 4 * 128
    assert L.muon_group_rows_capacity(n, 4, 128, C.byref(rows)) == L.MUON_OK
    assert n <= rows.value < 1 << 31


def test_route_launches_stay_below_2_32_threads():
    """64 lanes a token, 4 tokens a workgroup: 2^26 - 3 tokens would be 2^24 workgroups of 256."""
    for tokens in ((1 << 26) - 3, (1 << 26) - 1):
        c = _route(tokens=tokens, top_k=1)
        assert L.muon_route(C.byref(c), A, None, B, S, None) == L.MUON_ERR_SHAPE
        assert L.muon_route_backward(C.byref(c), A, B, S, O, 8, None) == L.MUON_ERR_SHAPE
    # the last size that is taken: refused for a buffer only
    c = _route(tokens=(1 << 26) - 4, top_k=1)
    assert -(-c.tokens // 4) * 256 < 1 << 32
    assert L.muon_route(C.byref(c), A + 4, None, B, S, None) == L.MUON_ERR_ALIGNMENT
    assert L.muon_route_backward(C.byref(c), A + 4, B, S, O, 8, None) == L.MUON_ERR_ALIGNMENT


# ---- buffers that overlap -----------------------------------------------------------------------

# 4 x 200 float32 in (3200 bytes), codes 4 x 256, scales 4 x 4, transposed codes 200 x 128, scales 200 x 4
@pytest.mark.parametrize("kw", [
    dict(codes=A + 3184), dict(codes=A - 1008), dict(scales=A + 3184), dict(scales=A), dict(codes_t=A + 3184), dict(scales_t=A - 784),
    dict(scales=B + 1008), dict(codes_t=B + 1008), dict(codes_t=B - 25584), dict(scales_t=B - 784), dict(codes_t=S), dict(scales_t=S),
    dict(scales_t=T + 25584), dict(codes_t=B, scales_t=S),
    dict(gather=W, src_rows=4, codes=W), dict(gather=W, src_rows=4, scales=W), dict(gather=W, src_rows=4, scales_t=W - 784),
    dict(limit=B + 1020), dict(limit=S + 12), dict(limit=O + 796),
    dict(square=1, codes=None, scales=None, scales_t=A + 3184), dict(square=1, scales=T + 25584, scales_t=S),
    dict(batch=3, batch_stride=1000, codes=A + 4 * 2784), dict(batch=3, batch_stride=1000, scales=A + 4 * 2784),
])
def test_quantize_refuses_every_overlap(kw):
    c = _quant(**kw)
    assert L.muon_fp8_quantize(C.byref(c), None) == L.MUON_ERR_INVALID_ARG
    assert b"overlap" in L.muon_last_error()


# a 8 x 256 codes and 8 x 4 scales, b (of 3 groups) 200 x 256 and 200 x 4, out 8 x 200 float32
@pytest.mark.parametrize("mode,kw", [
    (0, dict(out=A + 2032)), (0, dict(out=A - 6384)), (0, dict(out=S + 16)), (0, dict(out=S - 6384)), (0, dict(out=B + 51184)),
    (0, dict(out=T + 784)), (1, dict(out=T + 2384)), (1, dict(out=B + 153584)), (1, dict(out=W)), (1, dict(out=W - 6384)),
    (2, dict(out=W)), (2, dict(out=T + 784)), (2, dict(out=S - 3 * 6400 + 16)), (0, dict(out=T - 6384, b__square=1)),
])
def test_product_refuses_every_overlap(mode, kw):
    c = _product(mode, **kw)
    assert L.muon_fp8_product(C.byref(c), None) == L.MUON_ERR_INVALID_ARG
    assert b"overlap" in L.muon_last_error()


# 4 tokens of 8 float32 logits (128 bytes), 2 choices each (32 bytes)
def test_routing_refuses_every_overlap():
    c = _route(ld=16)                                           # logits: 3 * 64 + 32 bytes
    for bad in ((A, None, A + 208, S), (A, None, B, A - 16), (A, None, B, B + 16), (A, B, B + 16, S), (A, B, O, B - 16)):
        assert L.muon_route(C.byref(c), *bad, None) == L.MUON_ERR_INVALID_ARG
        assert b"overlap" in L.muon_last_error()
    # logits, experts, grad_weights, grad_logits, ld_grad
    for *bad, ld in ((A, B, S, A + 16, 16), (A, B, S, A, 8), (A, B, S, A - 208, 16), (A, B, S, B + 16, 8), (A, B, S, S - 112, 8),
                     (A, B, S, A + 208, 8), (A, B, S, A + 48, 16), (A, B, S, A + 16, 16), (A, B, S, A - 48, 16)):
        assert L.muon_route_backward(C.byref(c), *bad, ld, None) == L.MUON_ERR_INVALID_ARG
        assert b"overlap" in L.muon_last_error()


def test_grouping_refuses_every_overlap():
    # 9000 choices of 5 experts: experts, counts, offsets, rows, position, workspace
    rows, ws = C.c_int64(), C.c_uint64()
    assert L.muon_group_rows_capacity(9000, 5, 16, C.byref(rows)) == L.MUON_OK
    assert L.muon_group_rows_workspace(9000, 5, C.byref(ws)) == L.MUON_OK
    last = lambda size: (size - 1) // 16 * 16                    # noqa: E731  the last 16-byte step inside
    good = dict(experts=A, counts=B, offsets=S, rows=T, position=O, work=W)
    for kw in (dict(position=A), dict(counts=A + last(36000)), dict(offsets=B + 16), dict(rows=A + last(36000)),
               dict(position=T + last(4 * rows.value)), dict(work=A), dict(work=O + last(36000)), dict(offsets=W + last(ws.value))):
        a = dict(good, **kw)
        st = L.muon_group_rows(a["experts"], 9000, 5, 16, a["counts"], a["offsets"], a["rows"], a["position"], a["work"], ws.value, None)
        assert st == L.MUON_ERR_INVALID_ARG and b"overlap" in L.muon_last_error()
    for out in (B, A + 16, B - 16, B + 16):
        assert L.muon_balance_step(A, B, 8, 0.1, out, None) == L.MUON_ERR_INVALID_ARG and b"overlap" in L.muon_last_error()


@pytest.mark.parametrize("mode", [8, 32, 16 + 3, 16 + 4, -1])
def test_product_refuses_modes_that_it_does_not_know(mode):
    c = _product(mode, groups=1)
    assert L.muon_fp8_product(C.byref(c), None) == L.MUON_ERR_INVALID_ARG and b"unknown mode" in L.muon_last_error()


@pytest.mark.parametrize("mode,kw,status", [
    (0, dict(groups=2), L.MUON_ERR_INVALID_ARG), (1, dict(offsets=None), L.MUON_ERR_INVALID_ARG),
    (1, dict(b__stride=200 * 256 - 16), L.MUON_ERR_SHAPE), (2, dict(out_stride=1599), L.MUON_ERR_SHAPE),
    (0, dict(out=A), L.MUON_ERR_INVALID_ARG),
])
def test_full_sums_are_checked_like_the_mode_they_go_with(mode, kw, status):
    c = _product(mode, **kw)
    c.mode |= L.MUON_PRODUCT_FULL_SUMS
    assert L.muon_fp8_product(C.byref(c), None) == status


def test_product_config_has_its_size():
    """Programs built against the header pass it by its layout."""
    assert C.sizeof(L.muon_fp8_product_config) == 184
