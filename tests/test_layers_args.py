"""CPU tests of the expert layers' entry points: what they refuse and what they do with empty sizes.  Device pointers are
fake, aligned addresses: every call here ends before a launch."""
import ctypes as C

import numpy as np
import pytest

from muon_newton_schulz_momentum_amd import binding as L
from oracle import layers_oracle as orc

MEM = 1 << 40                      # fake, 256-byte aligned addresses, far apart
P = [MEM + i * (1 << 36) for i in range(16)]
INVALID, SHAPE, ALIGN = L.MUON_ERR_INVALID_ARG, L.MUON_ERR_SHAPE, L.MUON_ERR_ALIGNMENT


def _set(c, kw):
    for name, v in kw.items():
        o, *field = name.split("__")
        if field:
            setattr(getattr(c, o), field[0], v)
        else:
            setattr(c, name, v)
    return c


def _operand(data, scales=None, ld=256, stride=1 << 20, stride_scales=1 << 10):
    return L.muon_operand(data, scales, ld, stride, stride_scales)


def _quantize(**kw):
    c = L.muon_int8_quantize_config(P[0], L.MUON_DTYPE_F32, 2, 1, 10, 100, 100, 0, None, 0, None, P[1], P[2])
    return _set(c, kw)


def _product(**kw):
    c = L.muon_int8_product_config(L.MUON_PRODUCT_ROWS, 4, 10, 20, 200, _operand(P[0], P[1]), _operand(P[2], P[3]), P[4], P[5], 20,
                                   L.MUON_DTYPE_F32, 0)
    return _set(c, kw)


def _gated(i8=False, **kw):
    s = (lambda p: p) if i8 else (lambda p: None)
    c = L.muon_gated_config(L.MUON_PRODUCT_ROWS, 4, 1 if i8 else 0, L.MUON_ACT_GELU, 10, 20, 200, _operand(P[0], s(P[1])),
                            _operand(P[2], s(P[3])), _operand(P[4], s(P[5])), P[6], P[7], 20, P[8], P[9], 20)
    return _set(c, kw)


def _backward(**kw):
    c = L.muon_gated_backward_config(L.MUON_PRODUCT_ROWS, 4, L.MUON_ACT_SILU, L.MUON_DTYPE_F32, 0, 0, 10, 20, 200, _operand(P[0]),
                                     _operand(P[1]), _operand(P[2]), P[3], P[4], 20, P[5], P[6], 64, P[7], P[8], 64, P[9], 200,
                                     P[10], P[11], 200, 4000)
    return _set(c, kw)


def _gather(**kw):
    c = L.muon_gather_rows_config(P[0], 10, 100, 100, L.MUON_DTYPE_BF16, 2, P[1], 30, P[2], P[3], 100, P[4], P[5], 100, P[6], P[7])
    return _set(c, kw)


def _combine(**kw):
    c = L.muon_combine_rows_config(P[0], 30, 100, 100, L.MUON_DTYPE_BF16, L.MUON_DTYPE_F32, 10, 2, 0, P[1], P[2], P[3], 100, P[4], 100)
    return _set(c, kw)


CALLS = {"int8_quantize": _quantize, "int8_product": _product, "gated": _gated, "gated_backward": _backward,
         "gather_rows": _gather, "combine_rows": _combine}
BIG = 1 << 31

REFUSED = [
    *[("int8_quantize", kw, st) for kw, st in [
        (dict(src_dtype=2), INVALID), (dict(batch=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(cols=BIG), SHAPE),
        (dict(rows=1 << 20, batch=1 << 12, batch_stride=1 << 40), SHAPE), (dict(ld=99), SHAPE), (dict(ld=BIG), SHAPE),
        (dict(batch=2, batch_stride=999), SHAPE), (dict(batch=2, batch_stride=1000, limit=P[5]), INVALID),
        (dict(batch=2, batch_stride=1000, gather=P[5]), INVALID), (dict(gather=P[5], per=0), INVALID), (dict(gather=P[5], src_rows=-1), INVALID),
        (dict(src=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(src=P[0] + 4), ALIGN),
        (dict(codes=P[1] + 8), ALIGN), (dict(scales=P[2] + 4), ALIGN), (dict(limit=P[5] + 2), ALIGN), (dict(gather=P[5] + 4, src_rows=4), ALIGN),
        (dict(codes=P[0] + 16), INVALID), (dict(scales=P[0] + 3984), INVALID), (dict(scales=P[1] + 1264), INVALID), (dict(limit=P[2] + 36), INVALID),
        (dict(gather=P[1], src_rows=4), INVALID)]],
    *[("int8_product", kw, st) for kw, st in [
        (dict(mode=L.MUON_PRODUCT_DEPTH), INVALID), (dict(mode=L.MUON_PRODUCT_ROWS | L.MUON_PRODUCT_FULL_SUMS), INVALID),
        (dict(mode=L.MUON_PRODUCT_DENSE), INVALID), (dict(groups=0), INVALID), (dict(groups=1025), INVALID), (dict(out_dtype=2), INVALID),
        (dict(m=-1), SHAPE), (dict(n=BIG, ld_out=BIG), SHAPE), (dict(k=131072, a__ld=1 << 18, b__ld=1 << 18), SHAPE), (dict(ld_out=19), SHAPE),
        (dict(ld_out=BIG), SHAPE), (dict(offsets=None), INVALID), (dict(offsets=P[4] + 2), ALIGN), (dict(out=None), INVALID), (dict(out=P[5] + 4), ALIGN),
        (dict(a__data=None), INVALID), (dict(a__scales=None), INVALID), (dict(b__scales=None), INVALID), (dict(a__data=P[0] + 8), ALIGN),
        (dict(b__scales=P[3] + 2), ALIGN), (dict(a__ld=255), SHAPE), (dict(a__ld=240), SHAPE), (dict(b__ld=1 << 23), SHAPE),
        (dict(b__stride=4000), SHAPE), (dict(b__stride=(1 << 20) + 8), SHAPE), (dict(b__stride_scales=19), SHAPE),
        (dict(out=P[0] + 256), INVALID), (dict(out=P[1]), INVALID), (dict(out=P[2] + 3 * (1 << 20) + 4800), INVALID), (dict(out=P[4] + 16), INVALID),
        (dict(m=2 ** 31 - 200, n=2 ** 31 - 200, ld_out=2 ** 31 - 1), SHAPE)]],
    *[("gated", kw, st) for kw, st in [
        (dict(operands=2), INVALID), (dict(activation=3), INVALID), (dict(activation=-1), INVALID), (dict(mode=2), INVALID), (dict(groups=0), INVALID),
        (dict(pre_up=None), INVALID), (dict(pre_gate=None), INVALID), (dict(k=-1), SHAPE), (dict(ld_out=19), SHAPE), (dict(ld_pre=19), SHAPE),
        (dict(x__ld=199), SHAPE), (dict(x__ld=1 << 22), SHAPE), (dict(gate__ld=199), SHAPE), (dict(up__stride=19 * 256 + 199), SHAPE),
        (dict(up__ld=264), SHAPE), (dict(gate__stride=(1 << 20) + 8), SHAPE), (dict(x__scales=P[1]), INVALID), (dict(up__data=None), INVALID), (dict(up__data=P[4] + 2), ALIGN), (dict(out=P[7] + 8), ALIGN),
        (dict(pre_up=P[9] + 8), ALIGN), (dict(out=P[0]), INVALID), (dict(pre_gate=P[7] + 384), INVALID), (dict(pre_up=P[8]), INVALID),
        (dict(out=P[4] + 6 * (1 << 20)), INVALID), (dict(pre_up=P[6]), INVALID), (dict(offsets=None), INVALID)]],
    *[("gated_backward", kw, st) for kw, st in [
        (dict(activation=3), INVALID), (dict(grad_dtype=2), INVALID), (dict(accumulate=2), INVALID),
        (dict(accumulate=1, grad_dtype=L.MUON_DTYPE_BF16), INVALID), (dict(grad_up=None), INVALID), (dict(ld_grad=19), SHAPE), (dict(ld_pre=19), SHAPE),
        (dict(ld_grad_pre=0), SHAPE), (dict(ld_grad_pre=96), SHAPE), (dict(ld_grad_pre=1 << 22), SHAPE), (dict(ld_grad_x=199), SHAPE), (dict(ld_grad_w=199), SHAPE),
        (dict(n=0), SHAPE),
        (dict(stride_grad_w=3999), SHAPE), (dict(x__ld=199), SHAPE), (dict(gate__ld=199), SHAPE), (dict(x__data=None), INVALID),
        (dict(up__ld=264), SHAPE), (dict(up__stride=(1 << 20) + 8), SHAPE), (dict(up__data=None), INVALID), (dict(grad=None), INVALID), (dict(grad_pre_up=None), INVALID), (dict(pre_gate=P[5] + 2), ALIGN),
        (dict(offsets=None), INVALID), (dict(grad_x=P[0]), INVALID), (dict(grad_pre_gate=P[4]), INVALID),
        (dict(grad_pre_gate=P[5]), INVALID), (dict(grad_pre_gate=P[6], grad_pre_up=P[5]), INVALID),
        (dict(grad_pre_gate=P[5], grad_pre_up=P[6], ld_grad_pre=128), INVALID), (dict(grad_up=P[10] + 64), INVALID), (dict(grad_x=P[7]), INVALID),
        (dict(grad_gate=P[1]), INVALID)]],
    *[("gather_rows", kw, st) for kw, st in [
        (dict(dtype=2), INVALID), (dict(per=0), INVALID), (dict(src_rows=-1), SHAPE), (dict(src_rows=1 << 30, per=3), SHAPE), (dict(n_rows=(1 << 30) + 1), SHAPE),
        (dict(cols=0), SHAPE), (dict(ld=99), SHAPE), (dict(ld_out=99), SHAPE), (dict(ld_y=99), SHAPE), (dict(y=None), INVALID), (dict(position=None), INVALID),
        (dict(grad_weights=None), INVALID), (dict(out=None, y=None, position=None, grad_weights=None), INVALID), (dict(src=None), INVALID),
        (dict(rows=None), INVALID), (dict(rows=P[1] + 4), ALIGN), (dict(limit=P[2] + 2), ALIGN), (dict(weights=P[4] + 4), ALIGN), (dict(out=P[3] + 2), ALIGN),
        (dict(out=P[0]), INVALID), (dict(out=P[5]), INVALID), (dict(grad_weights=P[4]), INVALID), (dict(grad_weights=P[3]), INVALID),
        (dict(limit=P[3] + 4), INVALID)]],
    *[("combine_rows", kw, st) for kw, st in [
        (dict(dtype=2), INVALID), (dict(out_dtype=-1), INVALID), (dict(top_k=0), SHAPE), (dict(top_k=65), SHAPE), (dict(tokens=-1), SHAPE),
        (dict(tokens=1 << 30), SHAPE), (dict(n_rows=BIG), SHAPE), (dict(cols=0), SHAPE), (dict(ld=99), SHAPE), (dict(ld_out=99), SHAPE),
        (dict(ld_residual=99), SHAPE), (dict(src=None), INVALID), (dict(out=None), INVALID), (dict(position=None), INVALID), (dict(position=P[1] + 8), ALIGN),
        (dict(residual=P[3] + 4), ALIGN), (dict(out=P[0]), INVALID), (dict(out=P[1]), INVALID), (dict(out=P[3] + 16), INVALID),
        (dict(out=P[3], ld_out=104), INVALID)]],
]


@pytest.mark.parametrize("name,kw,status", REFUSED, ids=[f"{n}-{'-'.join(map(str, kw))}-{i}" for i, (n, kw, _) in enumerate(REFUSED)])
def test_refuses(name, kw, status):
    assert getattr(L, f"muon_{name}")(C.byref(CALLS[name](**kw)), None) == status
    assert f"muon_{name}".encode() in L.muon_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(x__scales=None), INVALID), (dict(up__scales=None), INVALID), (dict(k=131072, x__ld=1 << 18, gate__ld=1 << 18, up__ld=1 << 18), SHAPE),
    (dict(x__ld=255), SHAPE), (dict(gate__ld=128), SHAPE), (dict(gate__stride=(1 << 20) + 4), SHAPE), (dict(up__stride_scales=4), SHAPE),
    (dict(out=P[5]), INVALID)])
def test_gated_of_8_bit_integers_refuses(kw, status):
    assert L.muon_gated(C.byref(_gated(True, **kw)), None) == status


def test_null_and_empty():
    for name in CALLS:
        assert getattr(L, f"muon_{name}")(None, None) == INVALID
    none = None
    assert L.muon_int8_quantize(C.byref(_quantize(rows=0, src=none, codes=none, scales=none)), None) == L.MUON_OK
    assert L.muon_int8_quantize(C.byref(_quantize(batch=0)), None) == L.MUON_OK
    assert L.muon_int8_product(C.byref(_product(m=0, out=none, offsets=none, a__data=none)), None) == L.MUON_OK
    assert L.muon_gated(C.byref(_gated(m=0, out=none, offsets=none, x__data=none)), None) == L.MUON_OK
    assert L.muon_gated(C.byref(_gated(n=0)), None) == L.MUON_OK
    assert L.muon_gated_backward(C.byref(_backward(m=0, grad_gate=none, grad_up=none, offsets=none, grad=none)), None) == L.MUON_OK
    assert L.muon_gated_backward(C.byref(_backward(n=0, grad_x=None)), None) == L.MUON_OK
    assert L.muon_gather_rows(C.byref(_gather(n_rows=0, src_rows=0, src=none, rows=none)), None) == L.MUON_OK
    assert L.muon_combine_rows(C.byref(_combine(tokens=0, out=none)), None) == L.MUON_OK


def test_oracle_of_int8_quantisation():
    x = np.array([[0.0, 0.0, 0.0], [127.0, 0.5, -1.5], [254.0, 3.0, 1.0], [np.nan, 1.0, 2.0], [1.0, -np.inf, 2.0]])
    codes, scales = orc.quantize_int8(x)
    assert codes.tolist() == [[0, 0, 0], [127, 0, -2], [127, 2, 0], [0, 0, 0], [0, 0, 0]]
    assert scales[:3].tolist() == [0.0, 1.0, 2.0] and np.isnan(scales[3:]).all()


def test_oracle_of_activations():
    for kind in ("silu", "gelu", "relu"):
        v = np.array([-30.0, -5.0, -1.3, -0.2, 0.4, 2.0, 40.0])
        value, slope = orc.activation(v, kind)
        ends = [orc.activation(v + s, kind)[0] for s in (1e-6, -1e-6)]
        assert np.allclose((ends[0] - ends[1]) / 2e-6, slope, atol=1e-8)
        assert np.allclose(orc.activation(np.array([40.0, 0.0, -800.0]), kind)[0], [40.0, 0.0, 0.0])


def test_oracle_combines_what_it_gathers():
    rng = np.random.Generator(np.random.PCG64(1))
    src, w = rng.normal(size=(5, 4)), rng.normal(size=(5, 2))
    position = np.array([[3, 0], [7, 9], [-1, 2], [1, -1], [8, 4]])
    rows = np.full(10, -1)
    for c, p in enumerate(position.reshape(-1)):
        if p >= 0:
            rows[p] = c
    y = orc.gather(src, rows, 2)
    there = (position >= 0).sum(1)
    assert np.allclose(orc.combine(y, position)[0], src * there[:, None])
    d = rng.normal(size=(5, 4))
    dy, dw, _ = orc.combine_backward(d, y, rows, position, w)
    step_y, step_w = rng.normal(size=y.shape), rng.normal(size=w.shape)
    f = lambda s: (d * orc.combine(y + s * step_y, position, w + s * step_w)[0]).sum()  # noqa: E731
    assert abs((f(1e-4) - f(-1e-4)) / 2e-4 - (dy * step_y).sum() - (dw * step_w).sum()) < 1e-8


def test_reuse_takes_rows_whose_padding_is_their_own():
    """Tensors that gated_backward(reuse=True) may write into, up to a multiple of 64 columns in every row, and those where
    that would be another tensor's memory or none."""
    import torch

    from muon_newton_schulz_momentum_amd.experts import _padded_rows
    saved = torch.empty(2, 5, 64, dtype=torch.bfloat16)[:, :, :40]
    flat = torch.empty(5 * 128, dtype=torch.bfloat16)
    good = [saved[0], saved[1], saved[1, 2:], saved[1, 4:], saved[0, :0], torch.empty(2, 0, 64)[1, :, :40], flat.view(5, 128), flat.view(10, 64),
            flat.view(5, 128)[:, :64]]
    for t in good:
        assert _padded_rows("t", t) == t.stride(0) and t.stride(0) % 64 == 0
    bad = [flat.view(5, 128)[:, :40],                      # a wider buffer's columns behind them
           flat.view(10, 64)[:, 8:48],                     # into the next row
           flat[:9 * 64 + 40].clone().as_strided((10, 40), (64, 1)),    # the storage ends with the last row's values
           flat[:40].clone().view(1, 40),
           torch.empty(5, 40, dtype=torch.bfloat16)]
    for i, t in enumerate(bad):
        with pytest.raises(ValueError, match="reuse needs t"):
            _padded_rows("t", t)
            pytest.fail(f"tensor {i} is accepted")


@pytest.mark.parametrize("name,kw", [
    ("int8_product", dict(a__data=None, b__data=None, a__ld=1, b__ld=7, b__stride=3, out=P[4])),
    ("gated", dict(x__data=None, gate__data=None, up__data=None, x__ld=1, gate__ld=3, up__ld=5, gate__stride=0, up__stride=1, out=P[6])),
    ("gated", dict(x__data=P[7], gate__data=P[7] + 2, up__data=P[8], out=P[6]))])
def test_without_depth_data_is_not_looked_at(name, kw):
    """Only what is wrong besides is refused: here out, which overlaps offsets."""
    assert getattr(L, f"muon_{name}")(C.byref(CALLS[name](k=0, **kw)), None) == INVALID and b"overlaps" in L.muon_last_error()


def test_without_depth_scales_are():
    for kw, status in ((dict(a__scales=None), INVALID), (dict(b__scales=P[3] + 2), ALIGN), (dict(b__stride_scales=19), SHAPE)):
        assert L.muon_int8_product(C.byref(_product(k=0, **kw)), None) == status
    assert L.muon_gated(C.byref(_gated(True, k=0, up__stride_scales=64)), None) == SHAPE


def test_gather_rows_without_rows_or_choices():
    """Buffers of 0 elements are NULL: only what is wrong besides is refused, here an output over an input."""
    none = dict.fromkeys(("rows", "out", "y"))
    for kw in (dict(n_rows=0, grad_weights=P[4], **none), dict(n_rows=0, grad_weights=P[6] + 64, **none),
               dict(src_rows=0, src=None, weights=None, position=None, grad_weights=None, out=P[1])):
        assert L.muon_gather_rows(C.byref(_gather(**kw)), None) == INVALID and b"overlaps" in L.muon_last_error(), kw
    # nothing to write
    for kw in (dict(n_rows=0, position=None, grad_weights=None, **none), dict(src_rows=0, src=None, position=None, grad_weights=None, out=None)):
        assert L.muon_gather_rows(C.byref(_gather(**kw)), None) == L.MUON_OK, kw
    for kw in (dict(n_rows=0, position=None, **none), dict(n_rows=0, grad_weights=None, **none)):
        assert L.muon_gather_rows(C.byref(_gather(**kw)), None) == INVALID, kw
