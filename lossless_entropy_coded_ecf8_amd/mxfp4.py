"""Microscaled 4-bit weights beside the lossless FP8 ones (include/ecf8x.h).

A compressed weight keeps every bit of its FP8 form.  Where a layer may lose some, its weight is kept in MXFP4: E2M1
values of 4 bits in blocks of 32 with a power of two each, 0.53 bytes a value.  Here are the conversion, the product
with activations of 16 bits or of the same 4 bits, the gradient that a frozen 4-bit weight passes to its input, and
``MXFP4Linear``, which stands beside ``ECF8Linear`` and takes the same adapters.  Every step is a HIP kernel of libecf8;
this module checks arguments, supplies device memory and passes the current stream.
"""
from __future__ import annotations

import ctypes
import warnings
from typing import Optional, Tuple

import torch

from .adapters import (_TYPES, AdapterBank, AdapterPlan, _apart, _empty, _Launch, _ptr, _rows, _scratch, adapter_add, adapter_grads)
from .binding import _check, lib

_HALF = (torch.bfloat16, torch.float16)
BLOCK, PITCH, _MX4 = 32, 128, 5


class MatrixX(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("factors", ctypes.c_void_p)]


class ExpertsX(ctypes.Structure):
    _fields_ = [("gate", MatrixX), ("up", MatrixX), ("down", MatrixX), ("features", ctypes.c_uint64), ("inner", ctypes.c_uint64),
                ("experts", ctypes.c_uint32), ("type", ctypes.c_uint32)]


EXPORTS_X = ["ecf8x_quantize", "ecf8x_dequantize", "ecf8x_linear_bytes", "ecf8x_linear", "ecf8x_input_grad_bytes",
             "ecf8x_input_grad", "ecf8x_route", "ecf8x_moe_bytes", "ecf8x_moe"]

_ready = None


def _lib() -> ctypes.CDLL:
    global _ready
    if _ready is not None:
        return _ready
    L = lib()
    vp, u32, u64, i, f = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int, ctypes.c_float
    matrix, experts = ctypes.POINTER(MatrixX), ctypes.POINTER(ExpertsX)
    sig = {
        "ecf8x_quantize": (i, [vp, u64, u32, vp, u64, u64, vp, vp, vp]),
        "ecf8x_dequantize": (i, [vp, vp, u64, u64, u32, vp, u64, vp]),
        "ecf8x_linear_bytes": (u64, [u64, u64, u64, u32]),
        "ecf8x_linear": (i, [vp, vp, u64, u32, u64, u64, u64, matrix, vp, u32, vp, u64, vp, u64, vp]),
        "ecf8x_input_grad_bytes": (u64, [u64, u64, u64, u32]),
        "ecf8x_input_grad": (i, [vp, u64, u32, u64, u64, u64, matrix, vp, u64, vp, u64, vp]),
        "ecf8x_route": (i, [vp, u64, u32, u64, u32, u32, u32, u32, f, vp, vp, vp]),
        "ecf8x_moe_bytes": (u64, [u64, u32, experts]),
        "ecf8x_moe": (i, [vp, u64, u32, u64, u32, vp, vp, experts, vp, u64, vp, u64, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _ready = L
    return L


class MXFP4:
    """Values in microscaled 4-bit floating point: ``data`` (..., Kp / 2) holds two codes a byte, the first in the low
    half, ``scales`` (..., Kp / 32) a byte s for each block of 32 values, which stands for 2^(s - 127) (255: NaN).
    ``features`` is K, a multiple of 32; Kp is K rounded up to 128, and what lies past K is zero."""

    def __init__(self, data: torch.Tensor, scales: torch.Tensor, features: int):
        wide = -(-features // PITCH) * PITCH
        if features < BLOCK or features % BLOCK:
            raise ValueError("features must be a multiple of %d, got %d" % (BLOCK, features))
        for t, what, n in ((data, "data", wide // 2), (scales, "scales", wide // BLOCK)):
            if t.dtype != torch.uint8 or not t.is_contiguous() or t.dim() < 2 or t.shape[-1] != n:
                raise ValueError("%s must be contiguous uint8 rows of %d bytes, got %s %s" % (what, n, t.dtype, tuple(t.shape)))
        if data.shape[:-1] != scales.shape[:-1] or data.device != scales.device:
            raise ValueError("data %s on %s and scales %s on %s do not go together"
                             % (tuple(data.shape), data.device, tuple(scales.shape), scales.device))
        if data.data_ptr() % 16 or scales.data_ptr() % 4:
            raise ValueError("data must start on a 16-byte border, scales on a 4-byte one")
        self.data, self.scales, self.features = data, scales, features

    @classmethod
    def _of(cls, data, scales, features) -> "MXFP4":
        """Of tensors made for it, which need no checks."""
        q = cls.__new__(cls)
        q.data, q.scales, q.features = data, scales, features
        return q

    @property
    def shape(self) -> Tuple[int, ...]:
        return tuple(self.data.shape[:-1]) + (self.features,)

    @property
    def device(self) -> torch.device:
        return self.data.device

    def nbytes(self) -> int:
        return self.data.numel() + self.scales.numel()

    def dequantize(self, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
        """The values, a new tensor of this shape: exact in float32 and bfloat16 (but for magnitudes that bfloat16
        rounds to infinity), rounded in float16."""
        if dtype not in (torch.bfloat16, torch.float16, torch.float32):
            raise ValueError("dtype must be bfloat16, float16 or float32, got %s" % dtype)
        _on_gpu(self.data, "the values")
        with _Launch(self.device, stream) as st:
            out = _empty(self.shape, dtype, self.device, stream)
            _check(_lib().ecf8x_dequantize(self.data.data_ptr(), self.scales.data_ptr(), out.numel() // self.features,
                                           self.features, _TYPES[dtype], out.data_ptr(), self.features, st), "ecf8x_dequantize")
        return out

    def _c(self) -> MatrixX:
        return MatrixX(self.data.data_ptr(), self.scales.data_ptr(), None)


_warned = set()


def _no_graph(name: str, *operands):
    """Says once that a result carries no gradient where one may be expected."""
    if name not in _warned and torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in operands):
        _warned.add(name)
        warnings.warn("%s keeps no gradients%s; when serving, torch.no_grad() or requires_grad_(False) says that none are wanted"
                      % (name, ": MXFP4Linear.adapted is the differentiable layer" if "mxfp4" in name else ""), stacklevel=3)


def _on_gpu(t, what: str):
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU, got %s" % (what, t.device))


def quantize_mxfp4(x: torch.Tensor, x_scale: Optional[torch.Tensor] = None, *, out: Optional[MXFP4] = None, stream=None) -> MXFP4:
    """x (..., K), K a multiple of 32, in 4 bits (ecf8x_quantize): each block of 32 over the power of two that brings its
    largest magnitude into [4, 8), rounded to the nearest value (ties to the even code, over 6 to 6).  A block that
    holds an infinity or NaN is all NaN.

    x: bfloat16, float16, float32, or float8_e4m3fn with a float32 x_scale (default 1); a matrix's rows may lie apart, a
    tensor of more dimensions must be contiguous.  out: an MXFP4 of x's shape to write into.  Not differentiable (it warns
    once where an operand requires gradients).
    """
    if x.requires_grad or (x_scale is not None and x_scale.requires_grad):
        _no_graph("quantize_mxfp4", x, x_scale)
    return _quantize(x, x_scale, out, stream)


def _quantize(x, x_scale=None, out=None, stream=None) -> MXFP4:
    _on_gpu(x, "x")
    if x.dtype not in _TYPES:
        raise ValueError("x must be bfloat16, float16, float32 or float8_e4m3fn, got %s" % x.dtype)
    if x.dim() < 2:
        raise ValueError("x must have rows, got %s" % (tuple(x.shape),))
    if x.dim() > 2 and not x.is_contiguous():
        raise ValueError("x of %d dimensions must be contiguous" % x.dim())
    dev, K = x.device, x.shape[-1]
    if K < BLOCK or K % BLOCK:
        raise ValueError("the last dimension must be a multiple of %d, got %d" % (BLOCK, K))
    rows = x.numel() // K
    ld = _rows(x, "x", rows, K, (x.dtype,), dev) if x.dim() == 2 else K
    if x_scale is not None:
        if x.dtype != torch.float8_e4m3fn:
            raise ValueError("x_scale goes with a float8_e4m3fn x")
        if x_scale.dtype != torch.float32 or x_scale.numel() != 1 or x_scale.device != dev:
            raise ValueError("x_scale must be one float32 value on %s" % dev)
    with _Launch(dev, stream) as st:
        if out is None:
            wide, lead = -(-K // PITCH) * PITCH, tuple(x.shape[:-1])
            out = MXFP4._of(_empty(lead + (wide // 2,), torch.uint8, dev, stream), _empty(lead + (wide // BLOCK,), torch.uint8, dev, stream), K)
        else:
            if out.shape != tuple(x.shape) or out.device != dev:
                raise ValueError("out is %s on %s, x %s on %s" % (out.shape, out.device, tuple(x.shape), dev))
            for t, what in ((out.data, "out.data"), (out.scales, "out.scales")):
                _apart(t, [("x", x), ("x_scale", x_scale)], what)
            _apart(out.data, [("out.scales", out.scales)], "out.data")
        _check(_lib().ecf8x_quantize(x.data_ptr(), ld, _TYPES[x.dtype], _ptr(x_scale), rows, K, out.data.data_ptr(),
                                     out.scales.data_ptr(), st), "ecf8x_quantize")
    return out


def _weight_ok(w, what="w"):
    if not isinstance(w, MXFP4):
        raise TypeError("%s must be an MXFP4, got %s" % (what, type(w).__name__))
    if w.data.dim() != 2:
        raise ValueError("%s must be (N, K), got %s" % (what, w.shape))
    _on_gpu(w.data, what)
    return w.shape


def linear_mxfp4(x, w: MXFP4, bias: Optional[torch.Tensor] = None, *, out_dtype: Optional[torch.dtype] = None,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = x w^T + bias with a weight (N, K) in 4 bits (ecf8x_linear); (T, N), summed in float32 and rounded once.

    x: (T, K) bfloat16 or float16, rows on 16-byte borders (y has its type), or an MXFP4 (y is out_dtype, bfloat16
    unless given).  bias: (N,) in y's type.  out: where y goes.  Not differentiable by itself (it warns once where an operand
    requires gradients): MXFP4Linear.adapted is.
    """
    four = isinstance(x, MXFP4)
    _no_graph("linear_mxfp4", None if four else x, bias)
    N, K = _weight_ok(w)
    dev = w.device
    if len(x.shape) != 2 or x.shape[1] != K:
        raise ValueError("x must be (T, %d), got %s" % (K, tuple(x.shape)))
    T = x.shape[0]
    if four:
        if x.device != dev:
            raise ValueError("x is on %s, w on %s" % (x.device, dev))
        dtype, ldx, xp, xs = out_dtype or torch.bfloat16, K, x.data.data_ptr(), x.scales.data_ptr()
        if dtype not in _HALF:
            raise ValueError("out_dtype must be bfloat16 or float16, got %s" % dtype)
    else:
        ldx = _rows(x, "x", T, K, _HALF, dev)
        dtype, xp, xs = x.dtype, x.data_ptr(), None
        if out_dtype not in (None, dtype):
            raise ValueError("out_dtype is x's type, %s, unless x is an MXFP4" % dtype)
        if xp % 16 or (T > 1 and ldx % 8):
            raise ValueError("x must have its rows on 16-byte borders (address %% 16 = %d, %d values between rows)" % (xp % 16, ldx))
    if bias is not None and (bias.shape != (N,) or bias.dtype != dtype or bias.device != dev or not bias.is_contiguous()):
        raise ValueError("bias must be %d contiguous %s values on %s" % (N, dtype, dev))
    fresh = out is None
    with _Launch(dev, stream) as st:
        reads = None
        if not fresh or workspace is not None:
            reads = [("x", x.data if four else x), ("x.scales", x.scales if four else None), ("w", w.data), ("w.scales", w.scales), ("bias", bias)]
        if fresh:
            out, ld_out = _empty((T, N), dtype, dev, stream), N
        else:
            ld_out = _rows(out, "out", T, N, (dtype,), dev)
            _apart(out, reads, "out")
        L, kind = _lib(), _MX4 if four else _TYPES[dtype]
        need = L.ecf8x_linear_bytes(T, N, K, kind)
        ws = _scratch(need, workspace, dev, stream, reads and reads + [("out", out)]) if need else None
        _check(L.ecf8x_linear(xp, xs, ldx, kind, T, N, K, ctypes.byref(w._c()), _ptr(bias), _TYPES[dtype], out.data_ptr(), ld_out,
                              _ptr(ws), 0 if ws is None else ws.numel(), st), "ecf8x_linear")
    return out


def linear_mxfp4_input_grad(dy: torch.Tensor, w: MXFP4, *, out: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dx = dy w: the gradient that linear_mxfp4's frozen weight passes to its input (ecf8x_input_grad).

    dy: (T, N) bfloat16 or float16, rows on 16-byte borders.  Returns (T, K) in dy's type.  Not differentiable itself (it
    warns once where dy requires gradients).
    """
    if dy.requires_grad:
        _no_graph("linear_mxfp4_input_grad", dy)
    N, K = _weight_ok(w)
    if dy.dim() != 2:
        raise ValueError("dy must be (T, N), got %s" % (tuple(dy.shape),))
    T, dev = dy.shape[0], w.device
    ld_dy = _rows(dy, "dy", T, N, _HALF, dev)
    fresh = out is None
    with _Launch(dev, stream) as st:
        if fresh:
            out = _empty((T, K), dy.dtype, dev, stream)
        ld_dx = _rows(out, "out", T, K, (dy.dtype,), dev)
        for t, what, ld in ((dy, "dy", ld_dy), (out, "out", ld_dx)):
            if t.data_ptr() % 16 or (T > 1 and ld % 8):
                raise ValueError("%s must have its rows on 16-byte borders (address %% 16 = %d, %d values between rows)"
                                 % (what, t.data_ptr() % 16, ld))
        reads = [("dy", dy), ("w", w.data), ("w.scales", w.scales)]
        if not fresh:
            _apart(out, reads, "out")
        L = _lib()
        need = L.ecf8x_input_grad_bytes(T, N, K, _TYPES[dy.dtype])
        ws = _scratch(need, workspace, dev, stream, reads + [("out", out)]) if need else None
        _check(L.ecf8x_input_grad(dy.data_ptr(), ld_dy, _TYPES[dy.dtype], T, N, K, ctypes.byref(w._c()), out.data_ptr(), ld_dx,
                                  _ptr(ws), 0 if ws is None else ws.numel(), st), "ecf8x_input_grad")
    return out


class MXFP4Linear(torch.nn.Module):
    """A linear layer whose frozen weight is kept in 4 bits: ``data``, ``scales`` and ``bias`` are buffers,
    0.53 bytes a weight.

    ``forward`` takes 16-bit activations, or quantises them to 4 bits first where ``four_bit_input`` is set (the product
    then runs on the scaled matrix instruction); adapters and index add low-rank adapters as ECF8Linear.forward does.
    ``adapted`` is the differentiable layer.
    """

    def __init__(self, weight: MXFP4, bias: Optional[torch.Tensor] = None, four_bit_input: bool = False):
        super().__init__()
        self.out_features, self.in_features = _weight_ok(weight, "weight")
        self.four_bit_input = four_bit_input
        self.register_buffer("data", weight.data)
        self.register_buffer("scales", weight.scales)
        self.register_buffer("bias", None if bias is None else bias.detach().to(weight.device))

    @classmethod
    def from_linear(cls, linear: torch.nn.Linear, device="cuda", four_bit_input: bool = False) -> "MXFP4Linear":
        """Quantises an nn.Linear weight."""
        w = linear.weight.detach().to(device)
        if w.dtype not in _TYPES:
            w = w.float()
        return cls(quantize_mxfp4(w.contiguous()), linear.bias, four_bit_input)

    @classmethod
    def from_ecf8(cls, layer, four_bit_input: bool = False) -> "MXFP4Linear":
        """Decodes an ECF8Linear's weight and quantises it: the lossy form of the same layer."""
        w = layer.decoded_weight().view(torch.float8_e4m3fn)
        return cls(quantize_mxfp4(w, layer.w_scale), layer.bias, four_bit_input)

    @property
    def weight(self) -> MXFP4:
        return MXFP4._of(self.data, self.scales, self.in_features)

    def _bias(self, dtype):
        return None if self.bias is None else self.bias.to(dtype)

    def forward(self, x: torch.Tensor, adapters: Optional[AdapterBank] = None, index=None) -> torch.Tensor:
        if adapters is not None and index is None:
            raise ValueError("adapters need the index of each token's adapter")
        if self.four_bit_input:
            _no_graph("linear_mxfp4", x)
            y = linear_mxfp4(_quantize(x), self.weight, self._bias(x.dtype), out_dtype=x.dtype)
        else:
            y = linear_mxfp4(x, self.weight, self._bias(x.dtype))
        return y if adapters is None else adapters.add_(y, x, index)

    def adapted(self, x: torch.Tensor, adapters: Optional[AdapterBank] = None, index=None) -> torch.Tensor:
        """The layer for training: differentiable in x and, with adapters, in their parameters.  The frozen product takes
        x's 16 bits, forward and backward, whatever four_bit_input says; the weight and the bias get no gradient.  The
        gradient of x is the frozen part's, rounded to x's type, plus the adapters' part, rounded again."""
        if adapters is None:
            return _Frozen.apply(x, self)
        if index is None:
            raise ValueError("adapters need the index of each token's adapter")
        plan = index if isinstance(index, AdapterPlan) else AdapterPlan(index, adapters.n_adapters)
        return _AdaptedMX.apply(x, adapters.down, adapters.up, self, adapters, plan)


def _whole(dy):
    """A gradient as the kernels take it (a sum's is one value, expanded)."""
    dy = dy.contiguous()
    if dy.data_ptr() % 16:
        dy = dy.clone()
    if dy.shape[0] > 1 and dy.shape[1] % 8:                   # rows on 16-byte borders
        wide = dy.new_zeros(dy.shape[0], -(-dy.shape[1] // 8) * 8)
        wide[:, :dy.shape[1]] = dy
        dy = wide[:, :dy.shape[1]]
    return dy


class _Frozen(torch.autograd.Function):
    """MXFP4Linear.adapted without adapters."""

    @staticmethod
    def forward(ctx, x, layer):
        ctx.save_for_backward(layer.data, layer.scales)
        ctx.features = layer.in_features
        return linear_mxfp4(x, layer.weight, layer._bias(x.dtype))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        if not ctx.needs_input_grad[0]:
            return None, None
        return linear_mxfp4_input_grad(_whole(dy), MXFP4._of(*ctx.saved_tensors, ctx.features)), None


class _AdaptedMX(torch.autograd.Function):
    """MXFP4Linear.adapted: y = frozen(x) + adapters(x)."""

    @staticmethod
    def forward(ctx, x, down, up, layer, bank, plan):
        y = linear_mxfp4(x, layer.weight, layer._bias(x.dtype))
        hidden = plan.hidden(bank.rank) if ctx.needs_input_grad[1] or ctx.needs_input_grad[2] else None
        adapter_add(y, x, down, up, bank.scaling, plan, ranks=bank.ranks, out=y, hidden=hidden)
        ctx.save_for_backward(x, down, up, bank.scaling, bank.ranks, hidden, layer.data, layer.scales)
        ctx.plan, ctx.features = plan, layer.in_features
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, down, up, scaling, ranks, hidden, data, scales = ctx.saved_tensors
        dy = _whole(dy)
        want_x, want_factors = ctx.needs_input_grad[0], ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        # In x's 16 bits, to which the adapters' part is added and rounded again, as where the two are layers of their own.
        dx = linear_mxfp4_input_grad(dy, MXFP4._of(data, scales, ctx.features)) if want_x else None
        dx, d_down, d_up = adapter_grads(dy, x, down, up, scaling, ctx.plan, hidden=hidden, ranks=ranks, dx_base=dx, dx=dx,
                                         want=(want_x, want_factors))
        return dx, d_down, d_up, None, None, None
