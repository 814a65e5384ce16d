"""Torch-side wrapper of the routed-expert operators of libmuon: routing, grouping rows by expert, 8-bit
block quantisation and 8-bit products; the gated block and its gradients, 8-bit integer products, and rows gathered to
the experts and combined back.

One layer's matrices in a training step, with the optimizer's `harness.Plan` at its end:

    chosen, weights = route(logits, top_k, bias=bias, score="sigmoid")
    g = group_rows(chosen, n_experts, align=128)
    w, w_t = quantize(W, block="square", transpose=True)             # after each step: W (experts, out, in)
    x, x_t = quantize(tokens, rows=g.rows, per=top_k, limit=g.limit, transpose=True)
    y = product(x, w, offsets=g.offsets, group="rows")               # rows of g, each by its expert
    ...
    dy, dy_t = quantize(grad_y, limit=g.limit, transpose=True)       # grad_y: zeros in the rows that pad a segment
    dx = product(dy, w_t, offsets=g.offsets, group="rows")
    product(dy_t, x_t, offsets=g.offsets, group="depth", out=G)      # the gradients that the plan reads
    bias = balance_step(bias, g.counts, rate)

The same layer in bfloat16 between its ends, and back:

    x = gather_rows(tokens, g.rows, per=top_k, limit=g.limit)
    h, pre_gate, pre_up = gated(x, W_gate, W_up, offsets=g.offsets, save=True)
    ...                                                              # y: h through the experts' third matrices, by the caller
    out = combine_rows(y, g.position, weights, residual=tokens)
    ...
    dy, dweights = combine_rows_backward(dout, y, g.rows, g.position, weights, limit=g.limit)
    ...                                                              # dh: dy through the third matrices, and their gradient
    dx, *_ = gated_backward(dh, x, W_gate, W_up, pre_gate, pre_up, offsets=g.offsets, grad_gate=G_gate, grad_up=G_up)
    dtokens = combine_rows(dx, g.position)
    dlogits = route_backward(logits, chosen, dweights, score="sigmoid")

and in 8-bit integers for serving (weights quantised once, a scale for each output channel):

    q = quantize_int8(tokens, rows=g.rows, per=top_k, limit=g.limit)
    h = gated(q, Q_gate, Q_up, offsets=g.offsets)
    y = product_int8(quantize_int8(h, limit=g.limit), Q_down, offsets=g.offsets)
    out = combine_rows(y, g.position, weights, residual=tokens)

Every operator runs in libmuon's HIP kernels on the current stream of its tensors' device; this module
checks tensors, allocates outputs and marshals arguments.  Sizes that only the device knows (segments, the
number of grouped rows) are never read back.

With `stream` it runs there instead: that stream has to come after the work that makes the inputs (wait_stream), and
whoever uses the outputs elsewhere waits for it.  Tensors passed in may be dropped after the call (their memory is
kept until the stream is done with them); outputs made by the call belong to the stream, like all that is allocated
under torch.cuda.stream.
"""
from __future__ import annotations

import contextlib
import ctypes as C
from dataclasses import dataclass
from typing import Optional

import torch

from . import binding as L

BLOCK = 128
_SCORES = {"softmax": L.MUON_SCORE_SOFTMAX, "sigmoid": L.MUON_SCORE_SIGMOID}
_FORMATS = {"e4m3": (L.MUON_FP8_E4M3, torch.float8_e4m3fn), "e5m2": (L.MUON_FP8_E5M2, torch.float8_e5m2)}
_GROUPS = {None: L.MUON_PRODUCT_DENSE, "rows": L.MUON_PRODUCT_ROWS, "depth": L.MUON_PRODUCT_DEPTH}
_ACTIVATIONS = {"silu": L.MUON_ACT_SILU, "gelu": L.MUON_ACT_GELU, "relu": L.MUON_ACT_RELU}
_DTYPES = {torch.float32: L.MUON_DTYPE_F32, torch.bfloat16: L.MUON_DTYPE_BF16}


def _up(v: int, step: int) -> int:
    return -(-v // step) * step


_AS_IT_IS = contextlib.nullcontext()


@contextlib.contextmanager
def _switched(device: torch.device, stream: Optional[torch.cuda.Stream], tensors):
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield
        if stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)


def _on(t: torch.Tensor, stream: Optional[torch.cuda.Stream], *others: Optional[torch.Tensor]):
    """The device of t, and the stream if one is given, made current: outputs are then allocated for the stream that the
    kernels run on.  t and the others are kept from reuse until that stream is done with them."""
    if not t.is_cuda:
        raise ValueError("tensors must be on a GPU")
    if stream is None:
        if t.device.index == torch._C._cuda_getDevice():
            return _AS_IT_IS
    elif stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, expected {t.device}")
    return _switched(t.device, stream, (t, *others))


def _stream_ptr(t: torch.Tensor) -> int:
    # the current stream of t's device, without the Stream object that torch.cuda.current_stream makes (7 us)
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _tensor(name: str, t: torch.Tensor, like: torch.Tensor, dtype, shape=None, contiguous=True) -> torch.Tensor:
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, expected {like.device}")
    if t.dtype not in (dtype if isinstance(dtype, (tuple, dict)) else (dtype,)):
        raise ValueError(f"{name} has dtype {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _rows(name: str, t: torch.Tensor) -> int:
    """Row stride of a matrix whose rows are contiguous and do not overlap."""
    shape, strides = t.shape, t.stride()
    cols = shape[-1]
    if cols > 1 and strides[-1] != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    ld = strides[-2] if shape[-2] > 1 else cols
    if ld < cols:
        raise ValueError(f"{name}'s rows overlap")
    return ld


def _route_config(logits, top_k, score, groups, top_groups, renormalize, scale):
    if logits.dim() != 2 or logits.dtype not in _DTYPES:
        raise ValueError("logits must be a float32 or bfloat16 matrix (tokens, experts)")
    if score not in _SCORES:
        raise ValueError(f"score must be one of {', '.join(_SCORES)}")
    tokens, n = logits.shape
    return L.muon_route_config(tokens, _rows("logits", logits), n, top_k, _DTYPES[logits.dtype], _SCORES[score],
                               groups, top_groups, 1 if renormalize else 0, scale)


def route(logits: torch.Tensor, top_k: int, *, bias: Optional[torch.Tensor] = None, score: str = "softmax",
          groups: int = 1, top_groups: int = 1, renormalize: bool = True, scale: float = 1.0, stream=None):
    """The top_k experts of each token and their weights: (int32, float32) of (tokens, top_k).

    muon_route: an expert with a logit of -inf or NaN is out; the bias moves the choice and not the weights; a
    token with fewer experts gets -1 and weight 0 in the remaining places.
    """
    k = _route_config(logits, top_k, score, groups, top_groups, renormalize, scale)
    with _on(logits, stream, bias):
        if bias is not None:
            _tensor("bias", bias, logits, torch.float32, (logits.shape[1],))
        size = (k.tokens, max(int(top_k), 0))
        experts = torch.empty(size, dtype=torch.int32, device=logits.device)
        weights = torch.empty(size, dtype=torch.float32, device=logits.device)
        L.check(L.muon_route(C.byref(k), logits.data_ptr(), None if bias is None else bias.data_ptr(),
                             experts.data_ptr(), weights.data_ptr(), _stream_ptr(logits)), "muon_route")
    return experts, weights


def route_backward(logits: torch.Tensor, experts: torch.Tensor, grad_weights: torch.Tensor, *,
                   score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient of `route`'s weights with respect to the logits (in `out` if given, which may be `logits`), the
    choice held fixed."""
    if experts.dim() != 2:
        raise ValueError("experts must be route's (tokens, top_k)")
    k = _route_config(logits, experts.shape[1], score, 1, 1, renormalize, scale)
    with _on(logits, stream, experts, grad_weights, out):
        size = (k.tokens, k.top_k)
        _tensor("experts", experts, logits, torch.int32, size)
        _tensor("grad_weights", grad_weights, logits, torch.float32, size)
        if out is None:
            out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        else:
            _tensor("out", out, logits, logits.dtype, logits.shape, contiguous=False)
        L.check(L.muon_route_backward(C.byref(k), logits.data_ptr(), experts.data_ptr(), grad_weights.data_ptr(),
                                      out.data_ptr(), _rows("out", out), _stream_ptr(logits)), "muon_route_backward")
    return out


@dataclass
class Groups:
    """Choices grouped by expert (muon_group_rows)."""
    counts: torch.Tensor     # (experts,) choices of each expert
    offsets: torch.Tensor    # (experts + 1,) segments of the grouped rows, padded to `align`
    rows: torch.Tensor       # (capacity,) choice in each grouped row, -1 in padding
    position: torch.Tensor   # grouped row of each choice, -1 where it has no expert

    @property
    def limit(self) -> torch.Tensor:
        """How many grouped rows there are, on the device."""
        return self.offsets[-1:]


def group_rows(experts: torch.Tensor, n_experts: int, *, align: int = 1, stream=None) -> Groups:
    """Groups route's choices (any shape) by expert in stable order, each segment padded to a multiple of align."""
    with _on(experts, stream):
        _tensor("experts", experts, experts, torch.int32)
        n, dev = experts.numel(), experts.device
        cap, ws = C.c_int64(), C.c_uint64()
        L.check(L.muon_group_rows_capacity(n, n_experts, align, C.byref(cap)), "muon_group_rows_capacity")
        L.check(L.muon_group_rows_workspace(n, n_experts, C.byref(ws)), "muon_group_rows_workspace")
        g = Groups(torch.empty(n_experts, dtype=torch.int32, device=dev),
                   torch.empty(n_experts + 1, dtype=torch.int32, device=dev),
                   torch.empty(cap.value, dtype=torch.int32, device=dev), torch.empty_like(experts))
        work = torch.empty(ws.value, dtype=torch.uint8, device=dev) if ws.value else None
        L.check(L.muon_group_rows(experts.data_ptr(), n, n_experts, align, g.counts.data_ptr(), g.offsets.data_ptr(),
                                  g.rows.data_ptr(), g.position.data_ptr(), None if work is None else work.data_ptr(), ws.value,
                                  _stream_ptr(experts)),
                "muon_group_rows")
    return g


def balance_step(bias: torch.Tensor, counts: torch.Tensor, rate: float, *, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """The selection bias after one step: + rate where an expert had fewer choices than the mean, - rate where
    more.  `out` may be `bias`."""
    with _on(bias, stream, counts, out):
        if bias.dim() != 1:
            raise ValueError("bias must be (experts,)")
        _tensor("bias", bias, bias, torch.float32)
        _tensor("counts", counts, bias, torch.int32, bias.shape)
        if out is None:
            out = torch.empty_like(bias)
        else:
            _tensor("out", out, bias, torch.float32, bias.shape)
        L.check(L.muon_balance_step(bias.data_ptr(), counts.data_ptr(), bias.numel(), rate, out.data_ptr(),
                                    _stream_ptr(bias)), "muon_balance_step")
    return out


@dataclass
class Fp8:
    """An 8-bit matrix, or a stack of them: codes (.., rows, cols rounded up to 128) and the power-of-two scales
    (.., rows or ceil(rows / 128) if square, blocks rounded up to 4)."""
    codes: torch.Tensor
    scales: torch.Tensor
    cols: int
    square: bool

    @property
    def rows(self) -> int:
        return self.codes.shape[-2]

    @staticmethod
    def empty(rows: int, cols: int, *, format: str = "e4m3", square: bool = False, stack: Optional[int] = None,
              device="cuda") -> "Fp8":
        lead = () if stack is None else (stack,)
        srows = -(-rows // BLOCK) if square else rows
        return Fp8(torch.empty(*lead, rows, _up(cols, BLOCK), dtype=_FORMATS[format][1], device=device),
                   torch.empty(*lead, srows, _up(-(-cols // BLOCK), 4), dtype=torch.float8_e8m0fnu, device=device),
                   cols, square)

    def dequantize(self) -> torch.Tensor:
        """The float32 values (with torch operations; for looking at them)."""
        kb = self.codes.shape[-1] // BLOCK
        s = self.scales[..., :kb].float()
        if self.square:
            s = s.repeat_interleave(BLOCK, dim=-2)[..., :self.rows, :]
        v = self.codes.float().unflatten(-1, (kb, BLOCK)) * s.unsqueeze(-1)
        return v.flatten(-2)[..., :self.cols]


def _layout(name: str, q: Fp8):
    """The shape and strides of q's codes and the strides of its scales, after checking that the two go together."""
    shape, strides, sshape, sstrides = q.codes.shape, q.codes.stride(), q.scales.shape, q.scales.stride()
    kb = -(-q.cols // BLOCK)
    srows = -(-shape[-2] // BLOCK) if q.square else shape[-2]
    if q.cols < 0 or shape[-1] != kb * BLOCK or sshape[-1] != -(-kb // 4) * 4 or sshape[-2] != srows or shape[:-2] != sshape[:-2]:
        raise ValueError(f"{name}: codes {tuple(shape)} and scales {tuple(sshape)} are not those of {q.cols} columns, "
                         f"square={q.square}")
    if q.codes.device != q.scales.device or q.scales.dtype != torch.float8_e8m0fnu:
        raise ValueError(f"{name}.scales must be float8_e8m0fnu on the codes' device")
    if kb and (strides[-1] != 1 or sstrides[-1] != 1):
        raise ValueError(f"{name}'s rows must be contiguous")
    return shape, strides, sshape, sstrides


def quantize(src: torch.Tensor, *, block: str = "row", format: str = "e4m3", transpose: bool = False,
             rows: Optional[torch.Tensor] = None, per: int = 1, limit: Optional[torch.Tensor] = None, out=None,
             stream=None):
    """8-bit copy of a float32 or bfloat16 matrix (or stack of them): an Fp8, or with `transpose` the pair of
    it and the Fp8 of the transposed matrix, from one pass over src (muon_fp8_quantize).

    block "row": a scale per 128 values of a row; "square": per 128 x 128.  With `rows` (int32), quantised row
    r is src row rows[r] // per, or zeros for -1.  `limit` (one int32 on the device): rows from there on are
    left as they were.  `out`: an Fp8, or with transpose a pair, to write into.
    """
    if block not in ("row", "square"):
        raise ValueError("block must be 'row' or 'square'")
    if format not in _FORMATS:
        raise ValueError(f"format must be one of {', '.join(_FORMATS)}")
    if src.dim() not in (2, 3) or src.dtype not in _DTYPES:
        raise ValueError("src must be a float32 or bfloat16 matrix or stack of matrices")
    square, (fmt, ftype) = block == "square", _FORMATS[format]
    stack = src.shape[0] if src.dim() == 3 else None
    if rows is not None and stack is not None:
        raise ValueError("rows goes with one matrix")
    cols, n = src.shape[-1], src.shape[-2] if rows is None else rows.numel()
    kept = [] if out is None else [t for q in (out if isinstance(out, (tuple, list)) else [out]) for t in (q.codes, q.scales)]
    with _on(src, stream, rows, limit, *kept):
        if rows is not None:
            _tensor("rows", rows, src, torch.int32, (n,))
        if limit is not None:
            _tensor("limit", limit, src, torch.int32, (1,))
        want = [(n, cols)] + ([(cols, n)] if transpose else [])
        if out is None:
            got = [Fp8.empty(r, c, format=format, square=square, stack=stack, device=src.device) for r, c in want]
        else:
            got = list(out) if isinstance(out, (tuple, list)) else [out]
            if len(got) != len(want):
                raise ValueError("out must be an Fp8, or with transpose a pair of them")
            for name, q, (r, c) in zip(("out", "transposed out"), got, want):
                if q.codes.device != src.device or q.codes.dtype != ftype or q.codes.dim() != src.dim():
                    raise ValueError(f"{name} must be {ftype} with {src.dim()} dimensions on {src.device}")
                _layout(name, q)
                if (q.rows, q.cols, q.square) != (r, c, square) or (stack is not None and q.codes.shape[0] != stack):
                    raise ValueError(f"{name} must hold {(r, c)}, square={square}")
                if not q.codes.is_contiguous() or not q.scales.is_contiguous():
                    raise ValueError(f"{name} must be contiguous")
        k = L.muon_fp8_quantize_config()
        k.src, k.src_dtype, k.format, k.square = src.data_ptr(), _DTYPES[src.dtype], fmt, 1 if square else 0
        k.batch, k.rows, k.cols, k.ld = 1 if stack is None else stack, n, cols, _rows("src", src)
        k.batch_stride = src.stride(0) if stack is not None and stack > 1 else 0
        if rows is not None:
            k.gather, k.per, k.src_rows = rows.data_ptr(), per, src.shape[0]
        if limit is not None:
            k.limit = limit.data_ptr()
        k.codes, k.scales = got[0].codes.data_ptr(), got[0].scales.data_ptr()
        if transpose:
            k.codes_t, k.scales_t = got[1].codes.data_ptr(), got[1].scales.data_ptr()
        # without rows there is nothing to write (and torch gives an empty tensor no address)
        if n > 0 and k.batch > 0:
            L.check(L.muon_fp8_quantize(C.byref(k), _stream_ptr(src)), "muon_fp8_quantize")
    return (got[0], got[1]) if transpose else got[0]


def _operand(o: L.muon_fp8_operand, name: str, q: Fp8, stacked: bool) -> torch.Size:
    """Fills o with q, checked; the shape of its codes."""
    shape, strides, sshape, sstrides = _layout(name, q)
    dtype = q.codes.dtype
    if len(shape) != (3 if stacked else 2):
        raise ValueError(f"{name} must be {'a stack of matrices' if stacked else 'one matrix'}")
    if dtype == torch.float8_e5m2:
        o.format = L.MUON_FP8_E5M2
    elif dtype != torch.float8_e4m3fn:
        raise ValueError(f"{name} has dtype {dtype}")
    o.codes, o.scales, o.square = q.codes.data_ptr(), q.scales.data_ptr(), 1 if q.square else 0
    o.ld = strides[-2] if shape[-2] > 1 else shape[-1]
    o.ld_scales = sstrides[-2] if sshape[-2] > 1 else sshape[-1]
    if stacked and shape[0] > 1:
        o.stride, o.stride_scales = strides[0], sstrides[0]
    return shape


def product(a: Fp8, b: Fp8, *, offsets: Optional[torch.Tensor] = None, group: Optional[str] = None,
            out: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16, accumulate: bool = False,
            full_sums: bool = False, stream=None) -> torch.Tensor:
    """a times the transpose of b in 8 bits (muon_fp8_product).

    group None: (m, n) of a (m, k) and b (n, k).  "rows": b is a stack (groups, n, k), and the rows offsets[g] to
    offsets[g + 1] of a go by b[g]; rows outside every segment are not written.
    "depth": out (groups, m, n), group g's over columns offsets[g] to offsets[g + 1] (multiples of 128) of both;
    with `accumulate` added to a float32 `out`.  a is e4m3 or e5m2, b e4m3.

    A float32 result has full float32 sums.  A bfloat16 one is summed by the 8-bit matrix instruction, which of 8
    neighbouring products drops what is below 2^-13 of the largest; with `full_sums` it has full float32 sums, too, at
    half the rate.
    """
    if group not in _GROUPS:
        raise ValueError("group must be None, 'rows' or 'depth'")
    if (group is None) != (offsets is None):
        raise ValueError("offsets go with group 'rows' or 'depth'")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    codes = a.codes
    with _on(codes, stream, a.scales, b.codes, b.scales, offsets, out):
        k = L.muon_fp8_product_config()
        k.mode, k.groups = _GROUPS[group] | (L.MUON_PRODUCT_FULL_SUMS if full_sums else 0), 1
        (m, _), (*stack, n, _) = _operand(k.a, "a", a, False), _operand(k.b, "b", b, group == "rows")
        if b.codes.device != codes.device or b.codes.dtype != torch.float8_e4m3fn:
            raise ValueError(f"b must have dtype float8_e4m3fn on {codes.device}")
        if a.cols != b.cols:
            raise ValueError(f"a has {a.cols} columns, b {b.cols}")
        k.m, k.n, k.k = m, n, a.cols
        if offsets is not None:
            _tensor("offsets", offsets, codes, torch.int32)
            k.groups, k.offsets = offsets.numel() - 1, offsets.data_ptr()
            if offsets.dim() != 1 or (stack and stack[0] != k.groups):
                raise ValueError("offsets must be (groups + 1,)")
        shape = (k.groups, m, n) if group == "depth" else (m, n)
        if out is None:
            if dtype not in _DTYPES:
                raise ValueError("dtype must be float32 or bfloat16")
            out = torch.empty(shape, dtype=dtype, device=codes.device)
            k.ld_out, k.out_stride = n, m * n
        else:
            _tensor("out", out, codes, _DTYPES, shape, contiguous=False)
            k.ld_out = _rows("out", out)
            k.out_stride = out.stride(0) if group == "depth" and k.groups > 1 else m * k.ld_out
        k.out, k.out_dtype, k.accumulate = out.data_ptr(), _DTYPES[out.dtype], 1 if accumulate else 0
        L.check(L.muon_fp8_product(C.byref(k), _stream_ptr(codes)), "muon_fp8_product")
    return out


@dataclass
class Int8:
    """A matrix of 8-bit integers, or a stack of them: codes (.., rows, cols rounded up to 128, zeros behind cols) and a
    float32 scale for each row (.., rows)."""
    codes: torch.Tensor
    scales: torch.Tensor
    cols: int

    @property
    def rows(self) -> int:
        return self.codes.shape[-2]

    @staticmethod
    def empty(rows: int, cols: int, *, stack: Optional[int] = None, device="cuda") -> "Int8":
        lead = () if stack is None else (stack,)
        return Int8(torch.empty(*lead, rows, _up(cols, BLOCK), dtype=torch.int8, device=device),
                    torch.empty(*lead, rows, dtype=torch.float32, device=device), cols)

    def dequantize(self) -> torch.Tensor:
        """The float32 values (with torch operations; for looking at them)."""
        return self.codes[..., :self.cols].float() * self.scales.unsqueeze(-1)


def _check_int8(name: str, q: Int8, like: torch.Tensor) -> tuple:
    codes, scales, cols, device = q.codes, q.scales, q.cols, like.device
    shape = tuple(codes.shape)             # (a torch.Size is slow to slice)
    if cols < 0 or len(shape) < 2 or shape[-1] != -(-cols // BLOCK) * BLOCK or tuple(scales.shape) != shape[:-1]:
        raise ValueError(f"{name}: codes {shape} and scales {tuple(scales.shape)} are not those of {cols} columns")
    if codes.dtype != torch.int8 or scales.dtype != torch.float32:
        raise ValueError(f"{name} must have int8 codes and float32 scales")
    if (codes is not like and codes.device != device) or scales.device != device:
        raise ValueError(f"{name} is on {codes.device}, expected {device}")
    return shape


def quantize_int8(src: torch.Tensor, *, rows: Optional[torch.Tensor] = None, per: int = 1,
                  limit: Optional[torch.Tensor] = None, out: Optional[Int8] = None, stream=None) -> Int8:
    """8-bit integer copy of a float32 or bfloat16 matrix (or stack of them), with a scale for each row: tokens of
    activations, output channels of weights (muon_int8_quantize).

    With `rows` (int32), quantised row r is src row rows[r] // per, or zeros for -1.  `limit` (one int32 on the
    device): rows from there on are left as they were.  `out`: an Int8 to write into.
    """
    if src.dim() not in (2, 3) or src.dtype not in _DTYPES:
        raise ValueError("src must be a float32 or bfloat16 matrix or stack of matrices")
    stack = src.shape[0] if src.dim() == 3 else None
    if stack is not None and (rows is not None or limit is not None):
        raise ValueError("rows and limit go with one matrix")
    cols, n = src.shape[-1], src.shape[-2] if rows is None else rows.numel()
    with _on(src, stream, rows, limit, *(() if out is None else (out.codes, out.scales))):
        if rows is not None:
            _tensor("rows", rows, src, torch.int32, (n,))
        if limit is not None:
            _tensor("limit", limit, src, torch.int32, (1,))
        if out is None:
            out = Int8.empty(n, cols, stack=stack, device=src.device)
        else:
            shape = _check_int8("out", out, src)
            if tuple(shape[:-1]) != ((n,) if stack is None else (stack, n)) or out.cols != cols:
                raise ValueError(f"out must hold {(n, cols)}")
            if not out.codes.is_contiguous() or not out.scales.is_contiguous():
                raise ValueError("out must be contiguous")
        k = L.muon_int8_quantize_config()
        k.src, k.src_dtype = src.data_ptr(), _DTYPES[src.dtype]
        k.batch, k.rows, k.cols, k.ld = 1 if stack is None else stack, n, cols, _rows("src", src)
        k.batch_stride = src.stride(0) if stack is not None and stack > 1 else 0
        if rows is not None:
            k.gather, k.per, k.src_rows = rows.data_ptr(), per, src.shape[0]
        if limit is not None:
            k.limit = limit.data_ptr()
        k.codes, k.scales = out.codes.data_ptr(), out.scales.data_ptr()
        L.check(L.muon_int8_quantize(C.byref(k), _stream_ptr(src)), "muon_int8_quantize")
    return out


def _layer_operand(o: L.muon_operand, name: str, t, like: torch.Tensor, stacked: bool):
    """Fills o with a bfloat16 tensor or an Int8, checked; (groups or None, rows, columns)."""
    if isinstance(t, Int8):
        shape, cols, data, scales = _check_int8(name, t, like), t.cols, t.codes, t.scales
        strides = scales.stride()
        if shape[-2] > 1 and strides[-1] != 1:
            raise ValueError(f"{name}.scales must be contiguous")
        o.scales = scales.data_ptr()
        if stacked and shape[0] > 1:
            o.stride_scales = strides[0]
    else:
        data = _tensor(name, t, like, torch.bfloat16, contiguous=False)
        shape, cols = t.shape, t.shape[-1] if t.dim() else 0
    if len(shape) != (3 if stacked else 2):
        raise ValueError(f"{name} must be {'a stack of matrices' if stacked else 'one matrix'}")
    o.data, o.ld = data.data_ptr(), _rows(name, data)
    if stacked and shape[0] > 1:
        o.stride = data.stride(0)
    return (shape[0] if stacked else None), shape[-2], cols


def _tensors(*operands):
    return [t for o in operands for t in ((o.codes, o.scales) if isinstance(o, Int8) else (o,))]


def _by_group(k, offsets: Optional[torch.Tensor], like: torch.Tensor, *groups) -> None:
    """Mode, groups and offsets of k, checked against the stacks'."""
    k.mode, k.groups = L.MUON_PRODUCT_DENSE, 1
    if offsets is not None:
        _tensor("offsets", offsets, like, torch.int32)
        k.mode, k.groups, k.offsets = L.MUON_PRODUCT_ROWS, offsets.numel() - 1, offsets.data_ptr()
        if offsets.dim() != 1 or any(g != k.groups for g in groups):
            raise ValueError("offsets must be (groups + 1,)")


def _result(name: str, out: Optional[torch.Tensor], like: torch.Tensor, shape, dtype) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    return _tensor(name, out, like, dtype, shape, contiguous=False)


def product_int8(a: Int8, b: Int8, *, offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """a times the transpose of b in 8-bit integers (muon_int8_product): exact sums, times both rows' scales.

    (m, n) of a (m, k) and b (n, k), or with `offsets` of a stack b (groups, n, k), the rows offsets[g] to
    offsets[g + 1] of a by b[g]; rows outside every segment are not written.
    """
    codes = a.codes
    with _on(codes, stream, *_tensors(a, b), offsets, out):
        k = L.muon_int8_product_config()
        _, m, ka = _layer_operand(k.a, "a", a, codes, False)
        groups, n, kb = _layer_operand(k.b, "b", b, codes, offsets is not None)
        if ka != kb:
            raise ValueError(f"a has {ka} columns, b {kb}")
        k.m, k.n, k.k = m, n, ka
        _by_group(k, offsets, codes, groups)
        if dtype not in _DTYPES:
            raise ValueError("dtype must be float32 or bfloat16")
        out = _result("out", out, codes, (m, n), dtype if out is None else _DTYPES)
        k.out, k.ld_out, k.out_dtype = out.data_ptr(), _rows("out", out), _DTYPES[out.dtype]
        L.check(L.muon_int8_product(C.byref(k), _stream_ptr(codes)), "muon_int8_product")
    return out


def gated(x, gate, up, *, activation: str = "silu", offsets: Optional[torch.Tensor] = None, save: bool = False,
          out: Optional[torch.Tensor] = None, stream=None):
    """The gated block act(x gate^T) * (x up^T) in one pass (muon_gated), in bfloat16.

    x (rows, k) and gate, up (n, k), or with `offsets` stacks (groups, n, k), the rows offsets[g] to offsets[g + 1] by
    gate[g] and up[g]; rows outside every segment are not written.  All three are bfloat16 or all three Int8.
    activation: "silu", "gelu" or "relu".  With `save` the triple of the result, x gate^T and x up^T, which
    gated_backward takes (their rows are padded to multiples of 64).
    """
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(_ACTIVATIONS)}")
    i8 = isinstance(x, Int8)
    if isinstance(gate, Int8) != i8 or isinstance(up, Int8) != i8:
        raise ValueError("x, gate and up must be of one kind")
    like = x.codes if i8 else x
    with _on(like, stream, *_tensors(x, gate, up), offsets, out):
        k = L.muon_gated_config()
        k.operands, k.activation = L.MUON_OPERANDS_INT8 if i8 else L.MUON_OPERANDS_BF16, _ACTIVATIONS[activation]
        _, k.m, k.k = _layer_operand(k.x, "x", x, like, False)
        groups, k.n, kg = _layer_operand(k.gate, "gate", gate, like, offsets is not None)
        shape_up = _layer_operand(k.up, "up", up, like, offsets is not None)
        if kg != k.k or shape_up != (groups, k.n, kg):
            raise ValueError("x, gate and up must agree in their columns, gate and up in their shape")
        _by_group(k, offsets, like, groups)
        size = (k.m, k.n)
        out = _result("out", out, like, size, torch.bfloat16)
        k.out, k.ld_out = out.data_ptr(), _rows("out", out)
        if save:
            pre = torch.empty(2, k.m, _up(k.n, 64), dtype=torch.bfloat16, device=like.device)
            k.pre_gate, k.pre_up, k.ld_pre = pre[0].data_ptr(), pre[1].data_ptr(), pre.shape[2]
            pre = pre[:, :, :k.n]
        L.check(L.muon_gated(C.byref(k), _stream_ptr(like)), "muon_gated")
    return (out, pre[0], pre[1]) if save else out


def _padded_rows(name: str, t: torch.Tensor) -> int:
    """Row stride of a matrix (rows, n) that `gated` saved, or of some of its rows, each padded to a multiple of 64.  Where n is none
    itself the padding is written: every row's has to be its own, the last row's inside the storage as well."""
    n, ld, first = t.shape[1], t.stride(0), t.storage_offset()
    own = ld % 64 == 0 or n == 0
    if n % 64:
        end = (first + t.shape[0] * ld) * t.element_size() if t.shape[0] else 0
        own = ld == _up(n, 64) and first % ld == 0 and end <= t.untyped_storage().nbytes()
    if not own:
        raise ValueError(f"reuse needs {name} as gated saved it, its rows padded to multiples of 64")
    return ld


def gated_backward(grad: torch.Tensor, x: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, pre_gate: torch.Tensor,
                   pre_up: torch.Tensor, *, activation: str = "silu", offsets: Optional[torch.Tensor] = None,
                   grad_x: Optional[torch.Tensor] = None, grad_gate: Optional[torch.Tensor] = None,
                   grad_up: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16, accumulate: bool = False,
                   reuse: bool = False, stream=None):
    """The gradients of `gated` with respect to x, gate and up (muon_gated_backward), from the gradient of its result and
    what it saved.

    grad_x is bfloat16; grad_gate and grad_up are of `dtype` or go into the given tensors (float32 ones are added to
    with `accumulate`).  Rows outside every segment of offsets are not written in grad_x and have no part in the others.
    The products' terms are the pre-activations' gradients rounded to bfloat16, float32 results are sums of those too.
    Without features (n = 0) grad_x is zeros.
    With `reuse` the saved tensors (as `gated` made them, or some of their rows) serve as the workspace and do not keep
    their values; zeros are written behind each row's n values, to the multiple of 64 that it is padded to.
    """
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(_ACTIVATIONS)}")
    if accumulate and (grad_gate is None or grad_up is None):
        raise ValueError("accumulate needs grad_gate and grad_up")
    with _on(x, stream, grad, gate, up, pre_gate, pre_up, offsets, grad_x, grad_gate, grad_up):
        k = L.muon_gated_backward_config()
        k.activation, k.accumulate = _ACTIVATIONS[activation], 1 if accumulate else 0
        _, k.m, k.k = _layer_operand(k.x, "x", x, x, False)
        groups, k.n, kg = _layer_operand(k.gate, "gate", gate, x, offsets is not None)
        shape_up = _layer_operand(k.up, "up", up, x, offsets is not None)
        if kg != k.k or shape_up != (groups, k.n, kg):
            raise ValueError("x, gate and up must agree in their columns, gate and up in their shape")
        _by_group(k, offsets, x, groups)
        size = (k.m, k.n)
        _tensor("grad", grad, x, torch.bfloat16, size, contiguous=False)
        k.grad, k.ld_grad = grad.data_ptr(), _rows("grad", grad)
        for name, t in (("pre_gate", pre_gate), ("pre_up", pre_up)):
            _tensor(name, t, x, torch.bfloat16, size, contiguous=False)
        k.pre_gate, k.pre_up, k.ld_pre = pre_gate.data_ptr(), pre_up.data_ptr(), _rows("pre_gate", pre_gate)
        if _rows("pre_up", pre_up) != k.ld_pre:
            raise ValueError("pre_gate and pre_up must have the same row stride")
        if reuse:
            k.ld_pre = k.ld_grad_pre = _padded_rows("pre_gate", pre_gate)
            if _padded_rows("pre_up", pre_up) != k.ld_pre:
                raise ValueError("pre_gate and pre_up must have the same row stride")
            work = (pre_gate, pre_up)
        else:
            work = torch.empty(2, k.m, _up(k.n, 64), dtype=torch.bfloat16, device=x.device)
            k.ld_grad_pre = work.shape[2]
        k.grad_pre_gate, k.grad_pre_up = work[0].data_ptr(), work[1].data_ptr()
        grad_x = _result("grad_x", grad_x, x, (k.m, k.k), torch.bfloat16)
        k.grad_x, k.ld_grad_x = grad_x.data_ptr(), _rows("grad_x", grad_x)
        if dtype not in _DTYPES:
            raise ValueError("dtype must be float32 or bfloat16")
        if (grad_gate is None) != (grad_up is None):
            raise ValueError("grad_gate and grad_up go together")
        shape = tuple(gate.shape)
        dtype = dtype if grad_gate is None else grad_gate.dtype
        if dtype not in _DTYPES:
            raise ValueError("grad_gate must be float32 or bfloat16")
        grad_gate, grad_up = _result("grad_gate", grad_gate, x, shape, dtype), _result("grad_up", grad_up, x, shape, dtype)
        k.grad_gate, k.grad_up, k.grad_dtype = grad_gate.data_ptr(), grad_up.data_ptr(), _DTYPES[dtype]
        k.ld_grad_w = _rows("grad_gate", grad_gate)
        if groups is not None and groups > 1:
            k.stride_grad_w = grad_gate.stride(0)
        if _rows("grad_up", grad_up) != k.ld_grad_w or (k.groups > 1 and grad_up.stride(0) != k.stride_grad_w):
            raise ValueError("grad_gate and grad_up must have the same strides")
        if k.n == 0:
            # sums of nothing: muon_gated_backward refuses this grad_x, muon_gated writes it from rows without values
            gated(x[:, :0], gate.transpose(-1, -2), up.transpose(-1, -2), offsets=offsets, out=grad_x)
            k.grad_x = None
        L.check(L.muon_gated_backward(C.byref(k), _stream_ptr(x)), "muon_gated_backward")
    return grad_x, grad_gate, grad_up


def _gather(src, rows, per, limit, out, stream, weights=None, y=None, position=None):
    if src.dim() != 2 or src.dtype not in _DTYPES:
        raise ValueError("the source must be a float32 or bfloat16 matrix")
    with _on(src, stream, rows, limit, out, weights, y, position):
        _tensor("rows", rows, src, torch.int32)
        if rows.dim() != 1:
            raise ValueError("rows must be (rows,)")
        if limit is not None:
            _tensor("limit", limit, src, torch.int32, (1,))
        n, cols = rows.numel(), src.shape[1]
        out = _result("out", out, src, (n, cols), src.dtype)
        k = L.muon_gather_rows_config()
        k.src, k.src_rows, k.cols, k.ld = src.data_ptr(), src.shape[0], cols, _rows("source", src)
        k.dtype, k.per, k.rows, k.n_rows = _DTYPES[src.dtype], per, rows.data_ptr(), n
        k.limit = None if limit is None else limit.data_ptr()
        k.out, k.ld_out = out.data_ptr(), _rows("out", out)
        grad = None
        if weights is not None:
            _tensor("weights", weights, src, torch.float32, (src.shape[0], per))
            _tensor("position", position, src, torch.int32, weights.shape)
            _tensor("y", y, src, src.dtype, (n, cols), contiguous=False)
            grad = torch.empty_like(weights)
            k.weights, k.y, k.ld_y, k.position, k.grad_weights = (weights.data_ptr(), y.data_ptr(), _rows("y", y),
                                                                  position.data_ptr(), grad.data_ptr())
        if n > 0 or (grad is not None and grad.numel() > 0):
            L.check(L.muon_gather_rows(C.byref(k), _stream_ptr(src)), "muon_gather_rows")
    return out, grad


def gather_rows(src: torch.Tensor, rows: torch.Tensor, *, per: int = 1, limit: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Tokens in expert order: row r is src row rows[r] // per, or zeros for -1 (muon_gather_rows).  `limit` (one int32
    on the device): rows from there on are left as they were.  Its gradient is `combine_rows` without weights."""
    return _gather(src, rows, per, limit, out, stream)[0]


def combine_rows(src: torch.Tensor, position: torch.Tensor, weights: Optional[torch.Tensor] = None, *,
                 residual: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
                 out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Experts' rows back to their tokens: out[t] = residual[t] + the sum over j of weights[t, j] * src[position[t, j]]
    (muon_combine_rows); positions of -1 add nothing.  The result is of `dtype` (src's if not given).  `residual`
    may be `out`."""
    if src.dim() != 2 or src.dtype not in _DTYPES or position.dim() != 2:
        raise ValueError("src must be a float32 or bfloat16 matrix, position (tokens, top_k)")
    with _on(src, stream, position, weights, residual, out):
        _tensor("position", position, src, torch.int32)
        size = (position.shape[0], src.shape[1])
        if weights is not None:
            _tensor("weights", weights, src, torch.float32, position.shape)
        dtype = out.dtype if out is not None else src.dtype if dtype is None else dtype
        if dtype not in _DTYPES:
            raise ValueError("dtype must be float32 or bfloat16")
        out = _result("out", out, src, size, dtype)
        k = L.muon_combine_rows_config()
        k.src, k.n_rows, k.cols, k.ld, k.dtype = src.data_ptr(), src.shape[0], src.shape[1], _rows("src", src), _DTYPES[src.dtype]
        k.tokens, k.top_k, k.position = position.shape[0], position.shape[1], position.data_ptr()
        k.weights = None if weights is None else weights.data_ptr()
        if residual is not None:
            _tensor("residual", residual, src, dtype, size, contiguous=False)
            k.residual, k.ld_residual = residual.data_ptr(), _rows("residual", residual)
        k.out, k.ld_out, k.out_dtype = out.data_ptr(), _rows("out", out), _DTYPES[dtype]
        L.check(L.muon_combine_rows(C.byref(k), _stream_ptr(src)), "muon_combine_rows")
    return out


def combine_rows_backward(grad: torch.Tensor, src: torch.Tensor, rows: torch.Tensor, position: torch.Tensor,
                          weights: torch.Tensor, *, limit: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None, stream=None):
    """The gradients of `combine_rows` with respect to src and weights, from the gradient of its result (of src's dtype):
    zeros in the rows that pad a segment; rows from `limit` on are left as they were; 0 for a weight without a row."""
    if position.dim() != 2:
        raise ValueError("position must be (tokens, top_k)")
    return _gather(grad, rows, position.shape[1], limit, out, stream, weights, src, position)
