"""A mixture-of-experts layer for a few tokens (include/ecf8x.h).

A decode dispatch fills the weights of a whole expert layer at once; these are the operators that read them when
serving: the choice of experts from the router's logits, and the chosen experts' gated products with the weighted sum,
in two launches, with weights in E4M3 (decoded) or in 4 bits.  ``ECF8Experts`` keeps the layer compressed.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple

import torch

from . import binding
from .adapters import _TYPES, _apart, _capturing, _empty, _Launch, _ptr, _rows, _scratch
from .binding import _check
from .mxfp4 import _HALF, _MX4, MXFP4, ExpertsX, MatrixX, _lib, _no_graph, _on_gpu, quantize_mxfp4

_SCORES = {"softmax": 0, "sigmoid": 1}
MAX_PAIRS = 512                          # tokens * top of one moe_few (ECF8X_MAX_PAIRS)


def moe_route(logits: torch.Tensor, top: int, *, score: str = "softmax", normalise: bool = True, scale: float = 1.0,
              stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The `top` largest logits of each token (ecf8x_route): ids (T, top) int32, largest first and of equal ones the
    lowest, and weights (T, top) float32.

    logits: (T, E) float32, bfloat16 or float16.  A weight is exp(v - max) (softmax) or 1 / (1 + exp(-v)) (sigmoid) of
    the chosen logit v, over the sum of the chosen ones (normalise), else softmax's over the sum over all experts;
    times scale.  An expert with logit -inf is never chosen: where fewer than `top` are left the ids are -1 and the
    weights 0, which moe_few leaves out.  Serving only: no gradients (it warns once where the logits require them).
    """
    _no_graph("moe_route", logits)
    _on_gpu(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be (T, E), got %s" % (tuple(logits.shape),))
    if score not in _SCORES:
        raise ValueError("score must be softmax or sigmoid, got %r" % (score,))
    T, E = logits.shape
    dev = logits.device
    ld = _rows(logits, "logits", T, E, (torch.float32, torch.bfloat16, torch.float16), dev)
    if not 1 <= top <= min(E, 32) or E > 1024:
        raise ValueError("top %d of %d experts: 1 to 32, no more than there are, of up to 1024" % (top, E))
    with _Launch(dev, stream) as st:
        ids, weights = _empty((T, top), torch.int32, dev, stream), _empty((T, top), torch.float32, dev, stream)
        _check(_lib().ecf8x_route(logits.data_ptr(), ld, _TYPES[logits.dtype], T, E, top, _SCORES[score], int(normalise), scale,
                                  ids.data_ptr(), weights.data_ptr(), st), "ecf8x_route")
    return ids, weights


def _stack(w, scale, what: str, dev) -> Tuple[MatrixX, tuple, bool]:
    """One of the three stacks of weights, its shape, and whether it is in 4 bits."""
    if isinstance(w, MXFP4):
        if scale is not None:
            raise ValueError("%s_scale goes with E4M3 weights" % what)
        if w.data.dim() != 3:
            raise ValueError("%s must be (E, rows, columns), got %s" % (what, w.shape))
        c, shape, four = w._c(), w.shape, True
    else:
        if w.dim() != 3 or w.dtype != torch.uint8 or not w.is_contiguous():
            raise ValueError("%s must be an MXFP4 or contiguous (E, rows, columns) uint8 E4M3 bytes, got %s %s"
                             % (what, w.dtype, tuple(w.shape)))
        if scale is not None and (scale.shape != (w.shape[0],) or scale.dtype != torch.float32 or not scale.is_contiguous()
                                  or scale.device != dev):
            raise ValueError("%s_scale must be %d contiguous float32 values on %s" % (what, w.shape[0], dev))
        c, shape, four = MatrixX(w.data_ptr(), None, _ptr(scale)), tuple(w.shape), False
    if w.device != dev:
        raise ValueError("%s is on %s, x on %s" % (what, w.device, dev))
    return c, shape, four


def moe_few(x: torch.Tensor, gate, up, down, ids: torch.Tensor, weights: torch.Tensor, *,
            gate_scale: Optional[torch.Tensor] = None, up_scale: Optional[torch.Tensor] = None,
            down_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y[t] = sum over j of weights[t, j] * down_e (silu(gate_e x[t]) * up_e x[t]), e = ids[t, j] (ecf8x_moe).

    x: (T, K) bfloat16 or float16, rows on 16-byte borders.  gate, up: (E, I, K), down: (E, K, I), all three MXFP4, or
    all three uint8 E4M3 bytes (K and I multiples of 16) with a float32 scale for each expert (default 1).  ids: (T, top)
    int32, a value outside [0, E) adds nothing; weights: (T, top) float32; both contiguous.  T * top is at most 512.  A chosen
    expert's weights are read once for every 8, 16 or 32 of its pairs, as the pairs an expert has on average; that reading
    is what bounds few tokens, so that batches far from even routing take longer.  Returns (T, K) in x's type.  Serving
    only: no gradients (it warns once where an operand requires them).
    """
    _no_graph("moe_few", x, weights, gate_scale, up_scale, down_scale)
    _on_gpu(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be (T, K), got %s" % (tuple(x.shape),))
    dev, (T, K) = x.device, x.shape
    cg, shape, four = _stack(gate, gate_scale, "gate", dev)
    E, inner = shape[:2]
    cu, shape_u, four_u = _stack(up, up_scale, "up", dev)
    cd, shape_d, four_d = _stack(down, down_scale, "down", dev)
    if shape != (E, inner, K) or shape_u != shape or shape_d != (E, K, inner):
        raise ValueError("gate %s, up %s and down %s do not go with x %s" % (shape, shape_u, shape_d, tuple(x.shape)))
    if four_u != four or four_d != four:
        raise ValueError("gate, up and down must all be MXFP4 or all E4M3 bytes")
    ldx = _rows(x, "x", T, K, _HALF, dev)
    if x.data_ptr() % 16 or (T > 1 and ldx % 8):
        raise ValueError("x must have its rows on 16-byte borders (address %% 16 = %d, %d values between rows)" % (x.data_ptr() % 16, ldx))
    if ids.dim() != 2 or ids.shape[0] != T or ids.dtype != torch.int32 or not ids.is_contiguous() or ids.device != dev:
        raise ValueError("ids must be contiguous (%d, top) int32 on %s, got %s %s" % (T, dev, ids.dtype, tuple(ids.shape)))
    if weights.shape != ids.shape or weights.dtype != torch.float32 or not weights.is_contiguous() or weights.device != dev:
        raise ValueError("weights must be contiguous %s float32 on %s" % (tuple(ids.shape), dev))
    top = ids.shape[1]
    if T * top > MAX_PAIRS:
        raise ValueError("%d tokens with %d experts each: moe_few takes up to %d pairs" % (T, top, MAX_PAIRS))
    fresh = out is None
    with _Launch(dev, stream) as st:
        if fresh:
            out, ld_out = _empty((T, K), x.dtype, dev, stream), K
        else:
            ld_out = _rows(out, "out", T, K, (x.dtype,), dev)
        layer = ExpertsX(cg, cu, cd, K, inner, E, _MX4 if four else _TYPES[torch.float8_e4m3fn])
        need = _lib().ecf8x_moe_bytes(T, top, ctypes.byref(layer))
        reads = None
        if not fresh or workspace is not None:
            reads = [("x", x), ("ids", ids), ("weights", weights), ("gate_scale", gate_scale), ("up_scale", up_scale), ("down_scale", down_scale)]
            for w, what in ((gate, "gate"), (up, "up"), (down, "down")):
                reads += [(what, w.data), (what + ".scales", w.scales)] if four else [(what, w)]
        if not fresh:
            _apart(out, reads, "out")
        ws = _scratch(need, workspace, dev, stream, None if workspace is None else reads + [("out", out)])
        _check(_lib().ecf8x_moe(x.data_ptr(), ldx, _TYPES[x.dtype], T, top, ids.data_ptr(), weights.data_ptr(), ctypes.byref(layer),
                                out.data_ptr(), ld_out, ws.data_ptr(), ws.numel(), st), "ecf8x_moe")
    return out


class ECF8Experts(torch.nn.Module):
    """A mixture-of-experts layer whose FP8 E4M3 weights are kept ECF8-compressed on the GPU.

    gate, up: E tensors (inner, features), down: E tensors (features, inner), uint8 E4M3 bytes, each encoded with a
    codebook of its own, with a scale each.  One dispatch decodes the layer, or the experts that a caller names, into one
    pool, each expert at its own place; ``forward`` then routes and runs ``moe_few`` on it.
    """

    def __init__(self, gate: Sequence[torch.Tensor], up: Sequence[torch.Tensor], down: Sequence[torch.Tensor], scales,
                 device="cuda", max_code_len: int = 11):
        """scales: (3, E) values: gate, up and down of each expert."""
        super().__init__()
        self.experts = len(gate)
        if not self.experts or len(up) != self.experts or len(down) != self.experts:
            raise ValueError("gate, up and down must hold one matrix for each expert, got %d, %d and %d" % (len(gate), len(up), len(down)))
        self.inner, self.features = (int(n) for n in gate[0].shape)
        self.device = torch.device(device)
        self.shapes = [(self.inner, self.features), (self.inner, self.features), (self.features, self.inner)]
        self.encs = []                   # gate, up, down; expert by expert
        for stack, shape in zip((gate, up, down), self.shapes):
            for w in stack:
                if w.dtype != torch.uint8 or tuple(w.shape) != shape:
                    raise ValueError("an expert's weight must be %s uint8 E4M3 bytes, got %s %s" % (shape, w.dtype, tuple(w.shape)))
                self.encs.append(binding.encode(w.contiguous().cpu(), max_len=max_code_len).to(self.device))
        scales = torch.as_tensor(scales, dtype=torch.float32, device=self.device)
        if scales.shape != (3, self.experts):
            raise ValueError("scales must be (3, %d), got %s" % (self.experts, tuple(scales.shape)))
        self.device = scales.device                             # with its number
        self.register_buffer("scales", scales.contiguous())
        self._pool: Optional[torch.Tensor] = None
        self._whole: Optional[binding.DecodePlan] = None        # of the whole layer
        self._named: tuple = ((), None)                         # the experts last named, and their plan
        self._captured: dict = {}                               # plans of named experts that a capture used, whose graphs read them

    def _apply(self, fn, *args, **kwargs):
        """Module.to and its like: the scales stay float32, as the weights stay bytes, whatever type the module is brought to."""
        scales = self.scales
        super()._apply(fn, *args, **kwargs)
        self.scales = scales.to(self.scales.device)
        return self

    def compressed_bytes(self) -> int:
        return sum(e.compressed_bytes() for e in self.encs)

    def _plan(self, experts: Optional[Tuple[int, ...]], stream):
        if experts is None and self._whole is not None:
            return self._whole
        if experts is not None and self._named[0] == experts:
            return self._named[1]
        if experts in self._captured:
            return self._captured[experts]
        if _capturing(stream):
            raise RuntimeError("a plan cannot be made while its stream is captured: decode the same experts once before")
        if self._pool is None:
            self._pool = _empty(3 * self.experts * self.inner * self.features, torch.uint8, self.device, stream)
        named = range(self.experts) if experts is None else experts
        at = [m * self.experts + e for m in range(3) for e in named]
        size = self.inner * self.features
        plan = binding.DecodePlan([self.encs[i] for i in at], out=self._pool, offsets=[i * size for i in at], stream=stream)
        if experts is None:
            self._whole = plan
        else:
            self._named = (experts, plan)
        return plan

    def decode(self, experts: Optional[Sequence[int]] = None, stream=None):
        """Decodes the layer, or the experts named, into the layer's pool; returns gate, up and down as moe_few takes them.
        Other experts' places are left as they are.  The plan of the whole layer is kept, and that of the experts last named:
        naming others costs their plan, which is made on the host.  A plan that was run in a capture is kept with the layer,
        which has to live as long as the graph.  All calls write the one pool: on several streams the caller orders them, and
        what reads it."""
        if experts is not None:
            experts = tuple(sorted({int(e) for e in experts}))
            if not experts or experts[0] < 0 or experts[-1] >= self.experts:
                raise ValueError("experts must be some of 0 .. %d" % (self.experts - 1))
        with _Launch(self.device, stream):               # also where another device is current
            plan = self._plan(experts, stream)
            if experts is not None and _capturing(stream):
                self._captured[experts] = plan
            plan.run(stream)
        size = self.experts * self.inner * self.features
        return tuple(self._pool[m * size:(m + 1) * size].view(self.experts, *self.shapes[m]) for m in range(3))

    def forward(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, decoded=None) -> torch.Tensor:
        """moe_few on the decoded layer.  decoded: what decode() has returned, if it holds the experts of ids already (they
        were named, or nothing has changed since); else the whole layer is decoded first.  ids and weights as moe_route
        gives them."""
        gate, up, down = self.decode() if decoded is None else decoded
        return moe_few(x, gate, up, down, ids, weights, gate_scale=self.scales[0], up_scale=self.scales[1], down_scale=self.scales[2])

    def in_four_bits(self) -> Tuple[MXFP4, MXFP4, MXFP4]:
        """The layer's weights in MXFP4, for moe_few: decoded, scaled and quantised expert by expert."""
        stacks = []
        for m, w in enumerate(self.decode()):
            each = [quantize_mxfp4(w[e].view(torch.float8_e4m3fn), self.scales[m, e]) for e in range(self.experts)]
            stacks.append(MXFP4(torch.stack([q.data for q in each]), torch.stack([q.scales for q in each]), w.shape[2]))
        return tuple(stacks)
