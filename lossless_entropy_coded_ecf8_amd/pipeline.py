"""Decode-on-use of ECF8-compressed linear layers.

ECF8 technical blog (codearts.csdn.net):
  * §3.2.2 memory management: a pool sized for the largest layer is
    allocated once, a layer's weights are decoded into it when the layer is
    about to run, and the pool is reused with no further allocation;
  * §3.3: layer-wise pipelining (and, on large GPUs, resident compressed
    weights with batched decode);
  * deployment notes: while layer N computes, the weights of layer N + 2 are
    decoded in the background;
  * integration notes: an ``ECF8Linear`` wrapper replaces a linear layer and
    decodes its weight when it is used.

Every decode is the library's HIP kernel (``DecodePlan``) and every product is
a library GEMM (``torch._scaled_mm`` on FP8 operands, i.e. hipBLASLt); this
module only allocates the pool once and orders launches on two HIP streams
with events.

A compressed weight is frozen.  What varies per request, or is trained, is a bank
of low-rank adapters beside it (adapters.py): ``ECF8Linear.forward`` and
``DecodePipeline.run`` add them when serving, ``ECF8Linear.adapted`` is the
differentiable layer for training them.
"""
from __future__ import annotations

from typing import List, Optional, Sequence

import torch

from . import binding
from .adapters import FEW_RANK, FEW_TOKENS, AdapterBank, AdapterPlan, adapter_add, adapter_grads, linear_fp8_input_grad

E4M3_MAX = 448.0


def fp8_e4m3_bytes(w: torch.Tensor) -> "tuple[torch.Tensor, float]":
    """Per-tensor max-abs scaling of a float weight to FP8 E4M3 bytes.

    Returns (uint8 bytes, scale) with w ~= e4m3(bytes) * scale; values are
    clamped to +-448 before the round-to-nearest-even cast.
    """
    amax = float(w.detach().abs().max())
    scale = amax / E4M3_MAX if amax > 0 else 1.0
    q = (w.detach().float() / scale).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), scale


def _scaled_mm_ok(device) -> bool:
    """Whether torch._scaled_mm runs FP8 E4M3 here (probed once per device)."""
    key = str(device)
    if key not in _SCALED_MM_OK:
        try:
            a = torch.zeros(16, 32, dtype=torch.float8_e4m3fn, device=device)
            b = torch.zeros(16, 32, dtype=torch.float8_e4m3fn, device=device)
            one = torch.ones((), dtype=torch.float32, device=device)
            torch._scaled_mm(a, b.t(), scale_a=one, scale_b=one, out_dtype=torch.bfloat16)
            _SCALED_MM_OK[key] = True
        except (RuntimeError, TypeError, AttributeError):
            _SCALED_MM_OK[key] = False
    return _SCALED_MM_OK[key]


_SCALED_MM_OK: dict = {}


def linear_fp8(x_fp8: torch.Tensor, x_scale: torch.Tensor, w_u8: torch.Tensor, w_scale: torch.Tensor,
               bias: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16) -> torch.Tensor:
    """y = (x * x_scale) @ (w * w_scale)^T + bias for FP8 E4M3 x (T x K) and w (N x K).

    The FP8 GEMM is hipBLASLt's, through torch._scaled_mm.  There is no other
    GEMM path: where torch._scaled_mm does not run FP8 E4M3 this raises.
    """
    w = w_u8.view(torch.float8_e4m3fn)
    if not _scaled_mm_ok(x_fp8.device):
        raise RuntimeError("torch._scaled_mm does not run FP8 E4M3 GEMMs on %s" % x_fp8.device)
    y = torch._scaled_mm(x_fp8, w.t(), scale_a=x_scale, scale_b=w_scale, out_dtype=out_dtype)
    if bias is not None:
        y = y + bias.to(out_dtype)
    return y


def check_decode(plan: binding.DecodePlan, stream=None):
    """Checked mode: synchronize `stream` and raise if a run of `plan` since the
    previous check flagged any block (its decoded symbol count disagreed with
    blk_off); each check restarts the count."""
    bad = plan.status(stream)
    if bad:
        raise binding.Ecf8Error(-5, "ECF8 decode (%d corrupt blocks)" % bad)


class ECF8Linear(torch.nn.Module):
    """A linear layer whose FP8 E4M3 weight is kept ECF8-compressed on the GPU.

    ``weight_u8`` is the (out_features x in_features) weight as E4M3 bytes and
    ``scale`` its per-tensor scale.  The compressed form (stream, nibble plane,
    gaps, block offsets) is device resident; ``forward`` decodes it (into a
    buffer the caller passes, or one the layer allocates on first use) and runs
    the FP8 GEMM.
    """

    def __init__(self, weight_u8: torch.Tensor, scale: float, bias: Optional[torch.Tensor] = None,
                 device="cuda", checked: bool = False, max_code_len: int = 11):
        """checked: after each decode into the layer's own buffer, synchronize
        and raise if the decode's block check flagged a block (a corrupt
        stream, gap or block offset) instead of feeding the GEMM.
        max_code_len: the code length limit of the weight's encoding; at 11
        every codeword fits the decode table's 11-bit index, so the decode
        takes its one-shift form (the limit costs a few hundredths of a
        percent of the stream on typical weights); 16 is plain Huffman."""
        super().__init__()
        self.checked = checked
        if weight_u8.dim() != 2 or weight_u8.dtype != torch.uint8:
            raise ValueError("weight_u8 must be a 2-D uint8 tensor of FP8 E4M3 bytes")
        self.out_features, self.in_features = (int(s) for s in weight_u8.shape)
        self.device = torch.device(device)
        self.enc = binding.encode(weight_u8.contiguous().cpu(), max_len=max_code_len).to(self.device)
        self.register_buffer("w_scale", torch.tensor(float(scale), dtype=torch.float32, device=self.device))
        self.bias = None if bias is None else bias.detach().to(self.device)
        self._own: Optional[torch.Tensor] = None
        self._own_plan: Optional[binding.DecodePlan] = None

    @classmethod
    def from_linear(cls, linear: torch.nn.Linear, device="cuda") -> "ECF8Linear":
        """Quantize an nn.Linear weight to FP8 E4M3 (per-tensor max-abs scale) and compress it."""
        q, scale = fp8_e4m3_bytes(linear.weight.detach().cpu())
        return cls(q, scale, linear.bias, device)

    @property
    def numel(self) -> int:
        return self.out_features * self.in_features

    def compressed_bytes(self) -> int:
        return self.enc.compressed_bytes()

    def plan_into(self, out_u8: torch.Tensor, workspace=None, stream=None,
                  workgroups: Optional[int] = None) -> binding.DecodePlan:
        """A decode plan writing this layer's weight bytes into out_u8[:numel]."""
        return binding.DecodePlan([self.enc], out=out_u8, offsets=[0], workspace=workspace, stream=stream,
                                  workgroups=workgroups)

    def decoded_weight(self, stream=None) -> torch.Tensor:
        """Decode into the layer's own buffer (allocated on first use) and return it (uint8, out x in)."""
        if self._own is None:
            self._own = torch.empty(self.numel, dtype=torch.uint8, device=self.device)
            self._own_plan = self.plan_into(self._own, stream=stream)
        self._own_plan.run(stream)
        if self.checked:
            check_decode(self._own_plan, stream)
        return self._own.view(self.out_features, self.in_features)

    def forward(self, x_fp8: torch.Tensor, x_scale: torch.Tensor, weight_u8: Optional[torch.Tensor] = None,
                adapters: Optional[AdapterBank] = None, index=None) -> torch.Tensor:
        """adapters, index: low-rank adapters added to the output, and the adapter of each token (a vector on the GPU,
        -1 for none, or an AdapterPlan of it).  The output then has the adapters' type, and no gradients: adapted trains
        them."""
        w = self.decoded_weight() if weight_u8 is None else weight_u8.view(self.out_features, self.in_features)
        if adapters is None:
            return linear_fp8(x_fp8, x_scale, w, self.w_scale, self.bias)
        if index is None:
            raise ValueError("adapters need the index of each token's adapter")
        y = linear_fp8(x_fp8, x_scale, w, self.w_scale, self.bias, out_dtype=adapters.down.dtype)
        return adapters.add_(y, x_fp8, index, x_scale)

    def adapted(self, x: torch.Tensor, adapters: AdapterBank, index, x_scale: Optional[torch.Tensor] = None,
                weight_u8: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The layer with adapters for training: differentiable in x and in the adapters' parameters.

        x: (T, in_features) in the adapters' type.  The frozen product takes x in E4M3 with x_scale (default: the
        largest magnitude of x over 448), which its gradient passes through as if it were exact; the adapters take x
        itself.  The gradient of x is the frozen part's, rounded to x's type, plus the adapters' part, rounded again.  The
        weight is decoded for the forward pass and again for the backward pass.  weight_u8: a decoded weight
        that is kept instead, and holds this weight until the backward pass: one that torch has written, or a pipeline's
        slot that has taken another layer, is refused there (a DecodePlan's own run into it is not seen).  The weight and
        the bias get no gradient.  index as in forward.
        """
        plan = index if isinstance(index, AdapterPlan) else AdapterPlan(index, adapters.n_adapters)
        return _Adapted.apply(x, adapters.down, adapters.up, self, adapters, plan, x_scale, weight_u8)


def quantize_e4m3(x: torch.Tensor, scale: Optional[torch.Tensor] = None) -> "tuple[torch.Tensor, torch.Tensor]":
    """x as float8_e4m3fn and its float32 scale, on the device and without a synchronisation (scale None: the largest
    magnitude over 448, 1 for an all-zero x)."""
    v = x.detach().float()
    if scale is None:
        amax = v.abs().amax() if v.numel() else v.new_zeros(())
        scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    return (v / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


class _Adapted(torch.autograd.Function):
    """ECF8Linear.adapted: y = frozen(x) + adapters(x)."""

    @staticmethod
    def forward(ctx, x, down, up, layer, bank, plan, x_scale, weight_u8):
        xq, scale = quantize_e4m3(x, x_scale)
        w = layer.decoded_weight() if weight_u8 is None else weight_u8.view(layer.out_features, layer.in_features)
        y = linear_fp8(xq, scale, w, layer.w_scale, layer.bias, out_dtype=down.dtype)
        hidden = plan.hidden(bank.rank) if ctx.needs_input_grad[1] or ctx.needs_input_grad[2] else None
        adapter_add(y, x, down, up, bank.scaling, plan, ranks=bank.ranks, out=y, hidden=hidden)
        # Saved as a tensor, a kept weight that is written before the backward pass is refused there.  One made in
        # inference mode has no version to go by, and autograd does not take it.
        plain = weight_u8 is not None and weight_u8.is_inference()
        ctx.save_for_backward(x, down, up, bank.scaling, bank.ranks, hidden, None if plain else weight_u8)
        ctx.layer, ctx.plan, ctx.plain_weight = layer, plan, weight_u8 if plain else None
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, down, up, scaling, ranks, hidden, w = ctx.saved_tensors
        layer, w = ctx.layer, ctx.plain_weight if w is None else w
        dy = dy.contiguous()                                  # a sum's gradient is one value, expanded
        if dy.data_ptr() % 16:
            dy = dy.clone()
        want_x, want_factors = ctx.needs_input_grad[0], ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        dx = None
        if want_x:
            w = layer.decoded_weight() if w is None else w.view(layer.out_features, layer.in_features)
            # In x's 16 bits, to which the adapters' part is added and rounded again: half a step more, as where the two
            # are layers of their own; a float32 sum between them would be four bytes a value more to write and read.
            dx = linear_fp8_input_grad(dy, w, layer.w_scale)
        dx, d_down, d_up = adapter_grads(dy, x, down, up, scaling, ctx.plan, hidden=hidden, ranks=ranks, dx_base=dx, dx=dx,
                                         want=(want_x, want_factors))
        return dx, d_down, d_up, None, None, None, None, None


class DecodePipeline:
    """Runs ECF8Linear layers in order, decoding each layer's weight ahead of use.

    One pool of ``slots`` weight buffers (each the size of the largest layer)
    is allocated at construction; layer i decodes into slot i % slots on a side
    stream, ``ahead`` layers before it runs on the caller's stream.  Events
    order the two streams: layer i's GEMM waits for its decode, and the decode
    that reuses a slot waits for the GEMM that last read it.  ``ahead`` = 0
    decodes each layer on the caller's stream right before its GEMM (no
    overlap).  ``workgroups`` caps the decode grid so that GEMMs keep compute
    units while a decode runs beside them.
    """

    def __init__(self, layers: Sequence[ECF8Linear], slots: int = 3, ahead: int = 2,
                 workgroups: Optional[int] = None, checked: bool = False):
        """checked: at the end of each run, synchronize and raise if any layer's
        decode flagged a block (every plan has its own workspace, so each
        layer's block check is read separately)."""
        self.checked = checked
        if not layers:
            raise ValueError("no layers")
        if ahead < 0 or (ahead > 0 and ahead > slots - 1) or slots < 1:
            raise ValueError("need 0 <= ahead <= slots - 1")
        self.layers = list(layers)
        self.slots, self.ahead = slots, ahead
        dev = self.layers[0].device
        self.slot_bytes = (max(l.numel for l in self.layers) + 255) // 256 * 256
        self.pool = torch.empty(slots * self.slot_bytes, dtype=torch.uint8, device=dev)
        # .data: each slot has a version of its own, by which autograd sees that it has taken another layer.
        self._slots = [self.pool[k * self.slot_bytes: (k + 1) * self.slot_bytes].data for k in range(slots)]
        self._holds: List[Optional[ECF8Linear]] = [None] * slots
        self.side = torch.cuda.Stream(device=dev) if ahead > 0 else None
        self.plans: List[binding.DecodePlan] = []
        for i, layer in enumerate(self.layers):
            self.plans.append(layer.plan_into(self.slot(i), stream=self.side, workgroups=workgroups))
        if self.side is not None:
            self.side.synchronize()
        self.decoded = [torch.cuda.Event() for _ in self.layers]
        self.used = [torch.cuda.Event() for _ in self.layers]

    def slot(self, i: int) -> torch.Tensor:
        return self._slots[i % self.slots][: self.layers[i].numel]

    def _decode(self, i: int, stream):
        """Decodes layer i into its slot."""
        self.plans[i].run(stream)
        k = i % self.slots
        if self._holds[k] is not self.layers[i]:
            self._holds[k] = self.layers[i]
            torch.autograd.graph.increment_version(self._slots[k])

    def pool_bytes(self) -> int:
        return self.pool.numel()

    def run(self, xs: Sequence[torch.Tensor], x_scales: Sequence[torch.Tensor],
            adapters: Optional[Sequence[Optional[AdapterBank]]] = None, index=None) -> List[torch.Tensor]:
        """Layer i computes on xs[i]; returns the outputs (caller's stream order).

        adapters: a bank (or None) for each layer, added to the layer's output as ECF8Linear.forward does; index: the
        adapter of each token, the same for all layers.  It is grouped once for all banks of one number of adapters
        (few tokens and small ranks need no grouping)."""
        L = len(self.layers)
        main = torch.cuda.current_stream(self.layers[0].device)
        outs = []
        banks = list(adapters) if adapters is not None else [None] * L
        if len(banks) != L:
            raise ValueError("%d adapter banks for %d layers" % (len(banks), L))
        indexes = [index] * L
        if any(b is not None for b in banks):
            if index is None:
                raise ValueError("adapters need the index of each token's adapter")
            grouped = {}                # number of adapters: the plan
            for i, b in enumerate(banks):
                if b is None:
                    continue
                if isinstance(index, AdapterPlan):
                    if index.adapters != b.n_adapters:
                        raise ValueError("a plan of %d adapters with a bank of %d" % (index.adapters, b.n_adapters))
                elif index.numel() > FEW_TOKENS or b.rank > FEW_RANK:
                    if b.n_adapters not in grouped:
                        grouped[b.n_adapters] = AdapterPlan(index, b.n_adapters)
                    indexes[i] = grouped[b.n_adapters]
        if self.ahead == 0:
            for i in range(L):
                self._decode(i, main)
                outs.append(self.layers[i](xs[i], x_scales[i], weight_u8=self.slot(i), adapters=banks[i], index=indexes[i]))
            self._check(main)
            return outs
        side = self.side
        side.wait_stream(main)          # inputs and the pool are ready on the caller's stream
        for j in range(min(self.ahead, L)):
            self._decode(j, side)
            self.decoded[j].record(side)
        for i in range(L):
            j = i + self.ahead
            if j < L:
                if j - self.slots >= 0:
                    side.wait_event(self.used[j - self.slots])
                self._decode(j, side)
                self.decoded[j].record(side)
            main.wait_event(self.decoded[i])
            outs.append(self.layers[i](xs[i], x_scales[i], weight_u8=self.slot(i), adapters=banks[i], index=indexes[i]))
            self.used[i].record(main)
        main.wait_stream(side)
        self._check(main)
        return outs

    def _check(self, stream):
        if self.checked:
            for p in self.plans:
                check_decode(p, stream)
