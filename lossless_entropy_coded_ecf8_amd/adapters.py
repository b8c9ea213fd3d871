"""Low-rank adapters and gradients beside a compressed weight (include/ecf8a.h).

A weight kept ECF8-compressed is frozen.  These are the operators a user needs
next to its product: the adapters of many requests added to the projection's
output (serving: single tokens and prompts in one batch), their gradients, the
gradient that the frozen weight passes to its input, and the clipping of many
gradients by their global norm.  Every step is a HIP kernel of libecf8; this
module checks arguments, supplies device memory and passes the current stream.

Shapes: T tokens, K inputs, N outputs, L adapters of up to R rows.  ``down`` is
(L, R, K) and ``up`` (L, R, N), both stored by rank row: the update that
adapter a adds to the weight is ``scaling[a] * up[a].T @ down[a]``.

Sums are held in float32 and results rounded once; between an adapter's two products its hidden values keep 16
significant bits (include/ecf8a.h says what that comes to).
"""
from __future__ import annotations

import ctypes
import threading
import warnings
from typing import List, Optional, Sequence, Tuple

import torch

from . import binding
from .binding import _check, lib

_TYPES = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3, torch.float8_e4m3fn: 4}
_INDEX_BYTES = {torch.int32: 4, torch.int64: 8}


class PlanA(ctypes.Structure):
    _fields_ = [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_uint64), ("tokens", ctypes.c_uint64),
                ("adapters", ctypes.c_uint32), ("max_slots", ctypes.c_uint32), ("max_chunks", ctypes.c_uint32),
                ("max_units", ctypes.c_uint32), ("unit_slots", ctypes.c_uint32)]


class BankA(ctypes.Structure):
    _fields_ = [("down", ctypes.c_void_p), ("up", ctypes.c_void_p), ("scaling", ctypes.c_void_p),
                ("ranks", ctypes.c_void_p), ("in_features", ctypes.c_uint64), ("out_features", ctypes.c_uint64),
                ("adapters", ctypes.c_uint32), ("rank", ctypes.c_uint32), ("type", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class GradA(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_uint64)]


class ClipPlanA(ctypes.Structure):
    _fields_ = [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_uint64), ("pieces", ctypes.c_uint64),
                ("count", ctypes.c_uint32), ("type", ctypes.c_uint32), ("grid", ctypes.c_uint32),
                ("in_place", ctypes.c_uint32)]


EXPORTS_A = ["ecf8a_plan_bytes", "ecf8a_plan_prepare", "ecf8a_hidden_bytes", "ecf8a_add_bytes", "ecf8a_grads_bytes",
             "ecf8a_add", "ecf8a_few", "ecf8a_add_few_bytes", "ecf8a_add_few", "ecf8a_grads", "ecf8a_input_grad_bytes", "ecf8a_input_grad", "ecf8a_clip_bytes",
             "ecf8a_clip_prepare", "ecf8a_clip_run"]

_ready = None


def _lib() -> ctypes.CDLL:
    global _ready
    if _ready is not None:
        return _ready
    L = lib()
    vp, u32, u64, i, f = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int, ctypes.c_float
    plan, bank, clip, grad = (ctypes.POINTER(t) for t in (PlanA, BankA, ClipPlanA, GradA))
    sig = {
        "ecf8a_plan_bytes": (u64, [u64, u32]),
        "ecf8a_plan_prepare": (i, [vp, u32, u64, u32, vp, u64, vp, plan]),
        "ecf8a_hidden_bytes": (u64, [plan, u32]),
        "ecf8a_add_bytes": (u64, [plan, bank]),
        "ecf8a_grads_bytes": (u64, [plan, bank]),
        "ecf8a_add": (i, [plan, bank, vp, u64, u32, vp, vp, u64, vp, u64, vp, vp, u64, vp]),
        "ecf8a_few": (i, [u64, bank]),
        "ecf8a_add_few_bytes": (u64, [u64, bank]),
        "ecf8a_add_few": (i, [vp, u32, u64, bank, vp, u64, u32, vp, vp, u64, vp, u64, vp, u64, vp]),
        "ecf8a_grads": (i, [plan, bank, vp, u64, vp, u64, vp, vp, u64, vp, u64, vp, vp, vp, u64, vp]),
        "ecf8a_input_grad_bytes": (u64, [u64, u64, u64]),
        "ecf8a_input_grad": (i, [vp, u64, u64, u64, vp, u64, vp, u32, vp, u64, vp, u64, vp]),
        "ecf8a_clip_bytes": (u64, [grad, u32]),
        "ecf8a_clip_prepare": (i, [grad, u32, u32, vp, u64, vp, clip]),
        "ecf8a_clip_run": (i, [clip, f, vp, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _ready = L
    return L


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


class _Launch:
    """The device of the operands made current for the launches; gives the handle of the stream to launch on."""

    def __init__(self, device, stream):
        if stream is not None and stream.device != device:
            raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, device))
        self.device, self.stream = device, stream

    def __enter__(self):
        self.before = torch.cuda.current_device()
        if self.before != self.device.index:
            torch.cuda.set_device(self.device)
        if self.stream is not None:
            return self.stream.cuda_stream
        return torch._C._cuda_getCurrentRawStream(self.device.index)

    def __exit__(self, *exc):
        if self.before != self.device.index:
            torch.cuda.set_device(self.before)


def _stream_of(device, stream):
    return torch.cuda.current_stream(device) if stream is None else stream


def _capturing(stream) -> bool:
    """Whether the launch stream (None: the current one) is being captured into a graph."""
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _empty(bytes_or_shape, dtype, device, stream):
    """Device memory of the launch stream, so that the allocator does not hand it on before the launch ends."""
    if stream is None:
        return torch.empty(bytes_or_shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(bytes_or_shape, dtype=dtype, device=device)


def _rows(t, what: str, rows: int, cols: int, dtypes, device) -> int:
    """A (rows, cols) operand whose rows are contiguous; returns the elements between rows."""
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError("%s must be (%d, %d), got %s" % (what, rows, cols, tuple(t.shape)))
    if t.dtype not in dtypes:
        raise ValueError("%s must be %s, got %s" % (what, " or ".join(str(d) for d in dtypes), t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, the index on %s" % (what, t.device, device))
    ld, step = t.stride()
    if rows <= 1:
        ld = cols                                       # no second row: whatever its stride says
    if (cols > 1 and step != 1) or ld < cols:
        raise ValueError("%s must have contiguous rows that do not overlap (strides %s)" % (what, t.stride()))
    return ld


def _span(t) -> Tuple[int, int]:
    """First and past-the-last byte a tensor touches."""
    if t.numel() == 0:
        return (t.data_ptr(), t.data_ptr())
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return (t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size())


def _apart(out, others, what: str):
    """out must not share memory with any of others, unless rows of one buffer lie side by side."""
    a0, a1 = _span(out)
    for name, o in others:
        if o is None:
            continue
        b0, b1 = _span(o)
        if a0 >= b1 or b0 >= a1:
            continue
        if out.dim() == 2 and o.dim() == 2 and out.shape[0] > 1 and out.stride(0) == o.stride(0) \
                and out.element_size() == o.element_size():
            pitch = out.stride(0) * out.element_size()
            d = (b0 - a0) % pitch                       # columns of one buffer: apart if neither reaches the other
            if d >= out.shape[1] * out.element_size() and pitch - d >= o.shape[1] * o.element_size():
                continue
        raise ValueError("%s overlaps %s" % (what, name))


def _index_ok(index):
    if index.dim() != 1 or index.dtype not in _INDEX_BYTES or not index.is_contiguous():
        raise ValueError("index must be a contiguous int32 or int64 vector")
    if not index.is_cuda:
        raise ValueError("index must be on the GPU, got %s" % index.device)


class AdapterPlan:
    """The tokens of a batch grouped by adapter (ecf8a_plan_prepare): one launch, shared by every projection that
    the batch passes through.

    index: (T,) int32 or int64 on the GPU, the adapter of each token; a value outside [0, n_adapters) means none.
    It is read by this call's launch only.  A call that uses the plan on another stream first waits for what the
    plan's stream has been given so far; a call that is being captured into a graph does not, so the replay has to be
    ordered after the plan, and the plan kept as long as the graph.  A plan made in a capture is filled by the replay,
    and calls outside of that graph have to be ordered after it.
    """

    def __init__(self, index: torch.Tensor, n_adapters: int, workspace: Optional[torch.Tensor] = None, stream=None):
        _index_ok(index)
        L = _lib()
        self.tokens, self.adapters, self.device = index.numel(), int(n_adapters), index.device
        need = L.ecf8a_plan_bytes(self.tokens, self.adapters) if self.adapters > 0 else 0
        if need == 0:
            raise binding.Ecf8Error(-2, "ecf8a_plan_prepare")
        with _Launch(self.device, stream) as st:
            if workspace is None:
                workspace = _empty(need, torch.uint8, self.device, stream)
            else:
                binding._check_buffer(workspace, self.device, "workspace")
                _apart(workspace, [("index", index)], "workspace")
            self.workspace, self.c = workspace, PlanA()
            _check(L.ecf8a_plan_prepare(index.data_ptr(), _INDEX_BYTES[index.dtype], self.tokens, self.adapters,
                                        workspace.data_ptr(), workspace.numel(), st, ctypes.byref(self.c)),
                   "ecf8a_plan_prepare")
            # The stream is kept by its identity: its handle does not give it back where it is the default stream's, 0.
            # (A Stream object of the current one would cost 2 us here; it is made when it is needed.)
            self._made_on = torch._C._cuda_getCurrentStream(self.device.index) if stream is None else stream
            self._handle, self._event = st, None
            self._captured = _capturing(stream)

    def _order(self, handle, stream):
        """Makes a launch on another stream than the plan's own wait for the grouping.

        The event is recorded by the first such launch: recorded with every plan it adds 4 us to each of them on the
        host (8 -> 12) and 5 to a short training pass (77 tokens, rank 6: 49 -> 54), and few plans leave their stream."""
        if handle == self._handle or self._captured or _capturing(stream):
            return
        event = self._event
        if event is None:
            made_on = self._made_on
            if isinstance(made_on, tuple):
                made_on = torch.cuda.Stream(stream_id=made_on[0], device_index=made_on[1], device_type=made_on[2])
            if _capturing(made_on):
                raise RuntimeError("the plan's stream is being captured: use the plan on another stream before that")
            event = torch.cuda.Event()
            event.record(made_on)
            self._event = event                         # seen by other threads only once it is recorded
        stream = _stream_of(self.device, stream)
        stream.wait_event(event)
        self.workspace.record_stream(stream)            # not handed on before that stream is done with it

    def hidden(self, rank: int, stream=None) -> torch.Tensor:
        """A buffer that carries h from adapter_add to adapter_grads (opaque bytes)."""
        n = _lib().ecf8a_hidden_bytes(ctypes.byref(self.c), int(rank))
        if n == 0 and self.tokens:
            raise binding.Ecf8Error(-2, "ecf8a_hidden_bytes")
        return _empty(max(n, 16), torch.uint8, self.device, stream)


def _bank(down, up, scaling, ranks, dev) -> BankA:
    if down.dim() != 3 or up.dim() != 3 or down.shape[:2] != up.shape[:2]:
        raise ValueError("down must be (L, R, K) and up (L, R, N), got %s and %s" % (tuple(down.shape), tuple(up.shape)))
    if down.dtype not in (torch.bfloat16, torch.float16) or up.dtype != down.dtype:
        raise ValueError("down and up must both be bfloat16 or float16, got %s and %s" % (down.dtype, up.dtype))
    if not (down.is_contiguous() and up.is_contiguous()):
        raise ValueError("down and up must be contiguous")
    L, R, K = down.shape
    if scaling.dtype != torch.float32 or scaling.shape != (L,) or not scaling.is_contiguous():
        raise ValueError("scaling must be %d contiguous float32 values" % L)
    if ranks is not None and (ranks.dtype != torch.int32 or ranks.shape != (L,) or not ranks.is_contiguous()):
        raise ValueError("ranks must be %d contiguous int32 values" % L)
    if down.device != dev or up.device != dev or scaling.device != dev or (ranks is not None and ranks.device != dev):
        raise ValueError("the adapters and the index must be on one device")
    return BankA(down.data_ptr(), up.data_ptr(), scaling.data_ptr(), _ptr(ranks), K, up.shape[2], L, R,
                 _TYPES[down.dtype], 0)


def _hidden_ok(hidden, plan, rank):
    if hidden.dtype != torch.uint8 or not hidden.is_contiguous() or hidden.device != plan.device:
        raise ValueError("hidden must be a plan.hidden() buffer on %s" % plan.device)
    if hidden.numel() < _lib().ecf8a_hidden_bytes(ctypes.byref(plan.c), rank):
        raise ValueError("hidden is smaller than plan.hidden(%d)" % rank)


def _scratch(need, workspace, device, stream, others):
    """The workspace of a call: a new one, or the caller's, which must lie apart from the call's operands (the kernels
    find row and adapter numbers in it)."""
    if workspace is None:
        return _empty(max(need, 256), torch.uint8, device, stream)
    binding._check_buffer(workspace, device, "workspace")
    _apart(workspace, others, "workspace")
    return workspace


_warned = False


def _no_graph(base, x, down, up):
    """Says once that a result carries no gradient where one may be expected."""
    global _warned
    if not _warned and (down.requires_grad or up.requires_grad or x.requires_grad or (base is not None and base.requires_grad)) \
            and torch.is_grad_enabled():
        _warned = True
        warnings.warn("adapters were added to an output that keeps no gradients: ECF8Linear.adapted is the differentiable "
                      "layer; when serving, torch.no_grad() or requires_grad_(False) says that none are wanted", stacklevel=3)


def adapter_add(base: Optional[torch.Tensor], x: torch.Tensor, down: torch.Tensor, up: torch.Tensor,
                scaling: torch.Tensor, index, *, ranks: Optional[torch.Tensor] = None,
                x_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                hidden: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """base + scaling[a] * x_scale * (x down[a]^T) up[a] for each token's adapter a (ecf8a_add).

    base: (T, N) in the factors' type, the shared projection's output (None: 0); x: (T, K) in the factors' type or
    float8_e4m3fn with a float32 x_scale; rows may lie apart (a column slice of a wider buffer).  index: the adapter
    of each token, or an AdapterPlan of it.  ranks: rows of each adapter that take part (default: all).  out: where
    the result goes (default: a new tensor); out=base adds in place and leaves tokens without an adapter untouched.
    hidden: a plan.hidden(R) buffer that keeps h for adapter_grads.  Not differentiable by itself (it warns once where
    an operand requires gradients): see ECF8Linear.adapted.
    """
    _no_graph(base, x, down, up)
    plan = index if isinstance(index, AdapterPlan) else None
    if plan is None:
        _index_ok(index)
        if hidden is not None:
            raise ValueError("hidden goes with an AdapterPlan")
    dev, T = index.device, index.tokens if plan is not None else index.numel()
    bank = _bank(down, up, scaling, ranks, dev)
    K, N = bank.in_features, bank.out_features
    ldx = _rows(x, "x", T, K, (down.dtype, torch.float8_e4m3fn), dev)
    if x_scale is not None:
        if x.dtype != torch.float8_e4m3fn:
            raise ValueError("x_scale goes with a float8_e4m3fn x")
        if x_scale.dtype != torch.float32 or x_scale.numel() != 1 or x_scale.device != dev:
            raise ValueError("x_scale must be one float32 value on %s" % dev)
    ld_base = _rows(base, "base", T, N, (down.dtype,), dev) if base is not None else 0
    fresh = out is None
    if fresh:
        out = _empty((T, N), down.dtype, dev, stream)
    ld_out = _rows(out, "out", T, N, (down.dtype,), dev)
    if not fresh:
        same = base is not None and out.data_ptr() == base.data_ptr() and ld_out == ld_base
        _apart(out, [("x", x), ("down", down), ("up", up), ("scaling", scaling), ("ranks", ranks), ("x_scale", x_scale),
                     ("hidden", hidden), ("base", None if same else base)], "out")
    L = _lib()
    operands = None
    if workspace is not None:
        operands = [("out", out), ("x", x), ("base", base), ("down", down), ("up", up), ("scaling", scaling), ("ranks", ranks),
                    ("x_scale", x_scale), ("hidden", hidden), ("index", index if plan is None else plan.workspace)]
    if plan is None:
        if L.ecf8a_few(T, ctypes.byref(bank)):
            with _Launch(dev, stream) as st:
                need = L.ecf8a_add_few_bytes(T, ctypes.byref(bank))
                ws = _scratch(need, workspace, dev, stream, operands) if need else None
                _check(L.ecf8a_add_few(index.data_ptr(), _INDEX_BYTES[index.dtype], T, ctypes.byref(bank), x.data_ptr(), ldx,
                                       _TYPES[x.dtype], _ptr(x_scale), _ptr(base), ld_base, out.data_ptr(), ld_out,
                                       _ptr(ws), 0 if ws is None else ws.numel(), st), "ecf8a_add_few")
            return out
        plan = AdapterPlan(index, bank.adapters, stream=stream)
    if plan.adapters != bank.adapters:
        raise ValueError("a plan of %d adapters with a bank of %d" % (plan.adapters, bank.adapters))
    if hidden is not None:
        _hidden_ok(hidden, plan, bank.rank)
    with _Launch(dev, stream) as st:
        plan._order(st, stream)
        need = L.ecf8a_add_bytes(ctypes.byref(plan.c), ctypes.byref(bank))
        ws = _scratch(need, workspace, dev, stream, operands) if need else None
        _check(L.ecf8a_add(ctypes.byref(plan.c), ctypes.byref(bank), x.data_ptr(), ldx, _TYPES[x.dtype], _ptr(x_scale),
                           _ptr(base), ld_base, out.data_ptr(), ld_out, _ptr(hidden), _ptr(ws),
                           0 if ws is None else ws.numel(), st), "ecf8a_add")
    return out


def adapter_grads(dy: torch.Tensor, x: Optional[torch.Tensor], down: torch.Tensor, up: torch.Tensor,
                  scaling: torch.Tensor, plan: AdapterPlan, *, hidden: Optional[torch.Tensor] = None,
                  ranks: Optional[torch.Tensor] = None, dx_base: Optional[torch.Tensor] = None,
                  dx: Optional[torch.Tensor] = None, want: Tuple[bool, bool] = (True, True),
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """The gradients of adapter_add for dy = d loss / d out (ecf8a_grads): (dx, d_down, d_up).

    dx (T, K) = dx_base (None: 0) + the adapters' part; dx=dx_base adds in place.  d_down and d_up have the factors'
    shape and type, zero for adapters without a token and for rows past ranks.  hidden: what adapter_add kept for the
    same batch (None: h is computed again from x).  want: whether dx, and the factors' gradients, are wanted; what is
    not comes back as None.  x must be in the factors' type; it may be None if only dx is wanted.
    """
    T, dev = plan.tokens, plan.device
    bank = _bank(down, up, scaling, ranks, dev)
    K, N = bank.in_features, bank.out_features
    if plan.adapters != bank.adapters:
        raise ValueError("a plan of %d adapters with a bank of %d" % (plan.adapters, bank.adapters))
    ty = (down.dtype,)
    ld_dy = _rows(dy, "dy", T, N, ty, dev)
    want_dx, want_factors = want
    if want_factors and x is None:
        raise ValueError("the factors' gradients need x")
    ldx = _rows(x, "x", T, K, ty, dev) if want_factors else K
    ld_b = ld_dx = 0
    if want_dx:
        if dx_base is not None:
            ld_b = _rows(dx_base, "dx_base", T, K, ty, dev)
        fresh = dx is None
        if fresh:
            dx = _empty((T, K), down.dtype, dev, stream)
        ld_dx = _rows(dx, "dx", T, K, ty, dev)
        if not fresh:
            same = dx_base is not None and dx.data_ptr() == dx_base.data_ptr() and ld_dx == ld_b
            _apart(dx, [("x", x), ("dy", dy), ("down", down), ("up", up), ("scaling", scaling), ("ranks", ranks),
                        ("hidden", hidden), ("dx_base", None if same else dx_base)], "dx")
    else:
        dx = dx_base = None
    if hidden is not None:
        _hidden_ok(hidden, plan, bank.rank)
    d_down = _empty(down.shape, down.dtype, dev, stream) if want_factors else None
    d_up = _empty(up.shape, up.dtype, dev, stream) if want_factors else None
    L = _lib()
    with _Launch(dev, stream) as st:
        plan._order(st, stream)
        ws = _scratch(L.ecf8a_grads_bytes(ctypes.byref(plan.c), ctypes.byref(bank)), workspace, dev, stream,
                      workspace is not None and [
                          ("dx", dx), ("dy", dy), ("x", x), ("dx_base", dx_base), ("down", down), ("up", up), ("scaling", scaling),
                          ("ranks", ranks), ("hidden", hidden), ("the plan's workspace", plan.workspace)])
        _check(L.ecf8a_grads(ctypes.byref(plan.c), ctypes.byref(bank), dy.data_ptr(), ld_dy,
                             _ptr(x) if want_factors else None, ldx, _ptr(hidden), _ptr(dx_base), ld_b, _ptr(dx), ld_dx,
                             _ptr(d_down), _ptr(d_up), ws.data_ptr(), ws.numel(), st), "ecf8a_grads")
    return dx, d_down, d_up


def linear_fp8_input_grad(dy: torch.Tensor, w_u8: torch.Tensor, w_scale: torch.Tensor, *,
                          out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """dx = w_scale * dy w: the gradient that linear_fp8's frozen weight passes to its input (ecf8a_input_grad).

    dy: (T, N) bfloat16 or float16, rows 16-byte aligned; w_u8: (N, K) uint8 E4M3 bytes (a decoded weight), N and K
    multiples of 16 as the forward product asks; w_scale: one float32 value.  Returns (T, K) in dy's type.
    """
    if w_u8.dim() != 2 or w_u8.dtype != torch.uint8 or not w_u8.is_contiguous() or not w_u8.is_cuda:
        raise ValueError("w_u8 must be a contiguous 2-D uint8 tensor of FP8 E4M3 bytes on the GPU")
    if dy.dim() != 2:
        raise ValueError("dy must be (T, N), got %s" % (tuple(dy.shape),))
    (N, K), T, dev = w_u8.shape, dy.shape[0], w_u8.device
    ty = (torch.bfloat16, torch.float16)
    ld_dy = _rows(dy, "dy", T, N, ty, dev)
    if w_scale.dtype != torch.float32 or w_scale.numel() != 1 or w_scale.device != dev:
        raise ValueError("w_scale must be one float32 value on %s" % dev)
    fresh = out is None
    if fresh:
        out = _empty((T, K), dy.dtype, dev, stream)
    ld_dx = _rows(out, "out", T, K, (dy.dtype,), dev)
    if not fresh:
        _apart(out, [("dy", dy), ("w_u8", w_u8), ("w_scale", w_scale)], "out")
    L = _lib()
    with _Launch(dev, stream) as st:
        need = L.ecf8a_input_grad_bytes(T, N, K)
        ws = _scratch(need, workspace, dev, stream, [("out", out), ("dy", dy), ("w_u8", w_u8), ("w_scale", w_scale)]) if need else None
        _check(L.ecf8a_input_grad(dy.data_ptr(), ld_dy, T, N, w_u8.data_ptr(), K, w_scale.data_ptr(), _TYPES[dy.dtype],
                                  out.data_ptr(), ld_dx, _ptr(ws), 0 if ws is None else ws.numel(), st),
               "ecf8a_input_grad")
    return out


class GradClip:
    """Many gradients scaled to a largest global norm (ecf8a_clip_prepare / ecf8a_clip_run).

    grads: contiguous tensors of one type (bfloat16, float16 or float32) on one GPU, none overlapping another; out:
    where the scaled values go (default: in place).  The list is put on the GPU once and run() reads the gradients'
    values anew each time, so a plan serves as long as the tensors stay where they are.  It has to be made before a
    capture (the list comes from the host); run() can be captured.
    """

    def __init__(self, grads: Sequence[torch.Tensor], out: Optional[Sequence[torch.Tensor]] = None, stream=None):
        self.grads = list(grads)
        self.out: List[torch.Tensor] = self.grads if out is None else list(out)
        if not self.grads:
            raise ValueError("no gradients")
        if len(self.out) != len(self.grads):
            raise ValueError("%d outputs for %d gradients" % (len(self.out), len(self.grads)))
        first = self.grads[0]
        if first.dtype not in (torch.bfloat16, torch.float16, torch.float32) or not first.is_cuda:
            raise ValueError("gradients must be bfloat16, float16 or float32 on the GPU")
        arr = (GradA * len(self.grads))()
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            for t, what in ((g, "gradient"), (o, "output")):
                if t.dtype != first.dtype or t.device != first.device or not t.is_contiguous():
                    raise ValueError("%s %d must be a contiguous %s tensor on %s" % (what, i, first.dtype, first.device))
            if o.numel() != g.numel():
                raise ValueError("output %d has %d values, its gradient %d" % (i, o.numel(), g.numel()))
            arr[i] = GradA(g.data_ptr(), o.data_ptr(), g.numel())
        self.device = first.device
        L = _lib()
        need = L.ecf8a_clip_bytes(arr, len(self.grads))
        with _Launch(self.device, stream) as st:
            if _capturing(stream):
                raise RuntimeError("a GradClip cannot be made while its stream is captured: make it before, and capture its run()")
            self.workspace = _empty(max(need, 256), torch.uint8, self.device, stream)
            self.c = ClipPlanA()
            _check(L.ecf8a_clip_prepare(arr, len(self.grads), _TYPES[first.dtype], self.workspace.data_ptr(),
                                        self.workspace.numel(), st, ctypes.byref(self.c)),
                   "ecf8a_clip_prepare")
            self._last, self._handle, self._lock = _stream_of(self.device, stream), st, threading.Lock()

    def run(self, max_norm: float, stream=None) -> torch.Tensor:
        """Scales every gradient by min(1, max_norm / (norm + 1e-6)) and returns the norm before (0-d float32).

        All runs share the workspace's partial sums, so one on another stream than the last one's first waits for what
        that stream has been given so far.  A captured run does not, and is not waited for: its replays have to be
        ordered with the plan's other runs, and the plan kept as long as the graph."""
        with _Launch(self.device, stream) as st, self._lock:
            captured = st != self._handle and _capturing(stream)
            if st != self._handle and not captured:
                if _capturing(self._last):
                    raise RuntimeError("the stream of the plan's last run is being captured: run it on another one before that")
                event, other = torch.cuda.Event(), _stream_of(self.device, stream)
                event.record(self._last)
                other.wait_event(event)
                self.workspace.record_stream(other)     # not handed on before that stream is done with it
                self._last, self._handle = other, st
            norm = _empty((), torch.float32, self.device, stream)
            _check(_lib().ecf8a_clip_run(ctypes.byref(self.c), float(max_norm), norm.data_ptr(), st),
                   "ecf8a_clip_run")
        return norm


def clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: float, out: Optional[Sequence[torch.Tensor]] = None,
                   stream=None) -> torch.Tensor:
    """GradClip(grads, out).run(max_norm): for lists whose tensors change from step to step.  Not in a capture: a
    captured step makes its GradClip beforehand."""
    return GradClip(grads, out, stream).run(max_norm, stream)


FEW_TOKENS, FEW_RANK = 512, 64          # up to here a batch needs no AdapterPlan (ECF8A_FEW_TOKENS, ECF8A_FEW_RANK)


class AdapterBank(torch.nn.Module):
    """The low-rank adapters of one projection: ``n_adapters`` pairs of up to ``rank`` rows, as trainable parameters
    ``down`` (L, R, K) and ``up`` (L, R, N), with a float32 ``scaling`` (L,) and, where ranks differ, int32 ``ranks``.

    Adapter a adds scaling[a] * up[a].T @ down[a] to the weight of the tokens that name it.  ``up`` starts at 0, so a
    new adapter changes nothing.
    """

    def __init__(self, n_adapters: int, rank: int, in_features: int, out_features: int, scaling=1.0, ranks=None,
                 dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("adapters are bfloat16 or float16, got %s" % dtype)
        if n_adapters < 1 or rank < 1:
            raise ValueError("need at least one adapter of rank 1 or more")
        self.down = torch.nn.Parameter((torch.randn(n_adapters, rank, in_features, device=device) / in_features ** 0.5).to(dtype))
        self.up = torch.nn.Parameter(torch.zeros(n_adapters, rank, out_features, dtype=dtype, device=device))
        scaling = torch.as_tensor(scaling, dtype=torch.float32, device=device).expand(n_adapters).contiguous()
        self.register_buffer("scaling", scaling)
        if ranks is not None:
            ranks = torch.as_tensor(ranks, dtype=torch.int32, device=device).expand(n_adapters).contiguous()
        self.register_buffer("ranks", ranks)

    @property
    def n_adapters(self) -> int:
        return self.down.shape[0]

    @property
    def rank(self) -> int:
        return self.down.shape[1]

    def add_(self, y: torch.Tensor, x: torch.Tensor, index, x_scale: Optional[torch.Tensor] = None) -> torch.Tensor:
        """adapter_add into y, the shared projection's output; no gradients are kept (it warns once where the bank's
        parameters require them)."""
        _no_graph(y, x, self.down, self.up)
        return adapter_add(y, x, self.down.detach(), self.up.detach(), self.scaling, index, ranks=self.ranks,
                           x_scale=x_scale, out=y)


def clip_adapter_grads(banks, max_norm: float, stream=None) -> torch.Tensor:
    """clip_grad_norm over the gradients of these banks' parameters, in place; returns the norm before.  Not in a
    capture: there a GradClip of the same gradients, made before it, takes its place."""
    grads = [p.grad for b in banks for p in (b.down, b.up) if p.grad is not None]
    return clip_grad_norm(grads, max_norm, stream=stream)
