"""The dense side of a routed-experts layer, and the whole layer, through the C ABI.

``Router`` turns tokens into expert ids and weights (moe_gate, moe_route),
``SharedExpertI8`` is a SwiGLU MLP on every token in 8-bit integers (moe_quant_i8,
moe_linear_i8), and ``MoeBlock`` runs them around a ``MoeLayer``: router, routed experts,
weighted combine, shared expert added last.  Each owns its device buffers for up to B_max
tokens and reuses them from call to call, so calls of one object must be ordered (one
stream, or ordered streams), and follow its construction, which enqueues on the current stream.
torch only allocates memory and supplies the stream.

A call runs on the current stream, or on `stream` (a torch stream or a raw handle): there it
allocates too, as it would under torch.cuda.stream(stream), so that no buffer it drops is
handed on before the stream is done with it.  What it returns is recorded on the caller's current
stream: after the usual wait for `stream` it may be read there and dropped at any time.
"""
from __future__ import annotations

import contextlib

import torch

from . import _lib
from .layer import MoeLayer


@contextlib.contextmanager
def _on(stream, device):
    """Work and allocate on `stream` of `device` (None: its current one); yields a function that hands tensors on to
    the caller's stream."""
    if stream is None:
        yield lambda t: t
        return
    caller = torch.cuda.current_stream(device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    elif stream.device_index != device.index:
        raise ValueError("the stream belongs to another GPU than the tensors")

    def give(t):
        t.record_stream(caller)
        return t

    with torch.cuda.stream(stream):
        yield give


class Router:
    def __init__(self, weight, *, topk: int, B_max: int, bias=None, score: str = "softmax", groups: int = 0,
                 topk_groups: int = 0, group_score: str = "max", renorm: bool = True, scale: float = 1.0,
                 device="cuda"):
        """weight: BF16 or FP32 [E, D]; the other arguments as moe_route's."""
        self.device, self.B_max, self.topk = torch.device(device), int(B_max), int(topk)
        w = torch.as_tensor(weight).to(self.device).contiguous()
        self.E, self.D = map(int, w.shape)
        n = _lib.moe_gate_packed_bytes(self.E, self.D, w.dtype)
        if n == 0:
            raise ValueError("unsupported shape or type of the router's weight")
        self.device = w.device  # with its index: "cuda" would mean another GPU where another is current
        self.packed = torch.empty(n, dtype=torch.uint8, device=self.device)
        self.gate = _lib.moe_gate_pack(w, self.packed)
        self.bias = None if bias is None else torch.as_tensor(bias).to(self.device, torch.float32).contiguous()
        self.opts = dict(score=score, groups=groups, topk_groups=topk_groups, group_score=group_score, renorm=renorm,
                         scale=scale)
        self.logits = torch.empty(self.B_max, self.E, device=self.device)

    def forward(self, x: torch.Tensor, *, stream=None):
        """x: BF16 [B, D] -> (ids int32 [B, topk], weights FP32 [B, topk])."""
        B = x.shape[0]
        if B > self.B_max:
            raise ValueError("batch larger than B_max")
        with _on(stream, x.device) as give:
            ids = torch.empty(B, self.topk, dtype=torch.int32, device=self.device)
            weights = torch.empty(B, self.topk, device=self.device)
            logits = self.logits[:B]
            _lib.moe_gate(self.gate, x, logits)
            _lib.moe_route(logits, ids, weights, bias=self.bias, **self.opts)
            return give(ids), give(weights)


class SharedExpertI8:
    def __init__(self, w13, s13, w2, s2, *, B_max: int, device="cuda"):
        """w13 int8 [2I, D] (gate rows, then up rows) with FP32 scales [2I], w2 int8 [D, I] with scales [D].  Codes of
        another type are taken where int8 holds them; quantize() takes weights that are not codes yet."""
        self.device, self.B_max = torch.device(device), int(B_max)
        self.w13, self.w2 = (self._codes(t).to(self.device).contiguous() for t in (w13, w2))
        self.s13, self.s2 = (torch.as_tensor(t).to(self.device, torch.float32).contiguous() for t in (s13, s2))
        self.device = self.w2.device  # with its index: "cuda" would mean another GPU where another is current
        self.D, self.I = map(int, self.w2.shape)
        if self.w13.shape != (2 * self.I, self.D) or self.s13.shape != (2 * self.I,) or self.s2.shape != (self.D,):
            raise ValueError("shared expert: weights or scales of the wrong shape")
        B = self.B_max
        self.codes = torch.empty(B, max(self.D, self.I), dtype=torch.int8, device=self.device)
        self.scales = torch.empty(B, device=self.device)
        self.hidden = torch.empty(B, self.I, dtype=torch.bfloat16, device=self.device)

    @staticmethod
    def _codes(t) -> torch.Tensor:
        t = torch.as_tensor(t)
        if t.dtype == torch.int8:
            return t
        codes = t.to(torch.int8)
        if not torch.equal(codes.double(), t.double()):
            raise ValueError(f"shared expert: weights of {t.dtype} that are no int8 codes (see quantize)")
        return codes

    @classmethod
    def quantize(cls, w13, w2, *, B_max: int, device="cuda") -> "SharedExpertI8":
        """From FP32, BF16 or FP16 weights: a scale for each output channel (moe_quant_i8 on their rows)."""
        parts = []
        for w in (w13, w2):
            w = torch.as_tensor(w).to(device).contiguous()
            q = torch.empty(w.shape, dtype=torch.int8, device=device)
            s = torch.empty(w.shape[0], device=device)
            _lib.moe_quant_i8(w, q, s)
            parts += [q, s]
        return cls(*parts, B_max=B_max, device=device)

    def forward(self, x: torch.Tensor, *, add: torch.Tensor | None = None, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
        """x: BF16 [B, D] -> BF16 [B, D], plus `add` if given (which may be out itself).  The hidden is rounded to
        BF16 between the products."""
        B = x.shape[0]
        if B > self.B_max:
            raise ValueError("batch larger than B_max")
        with _on(stream, x.device) as give:
            if out is None:
                out = give(torch.empty(B, self.D, dtype=torch.bfloat16, device=self.device))
            # rows of the code buffers are packed for each product, so that they stay 16-byte aligned
            flat = self.codes.view(-1)
            scales, hidden = self.scales[:B], self.hidden[:B]
            q = flat[:B * self.D].view(B, self.D)
            _lib.moe_quant_i8(x, q, scales)
            _lib.moe_linear_i8(q, scales, self.w13, self.s13, hidden, act="swiglu")
            q = flat[:B * self.I].view(B, self.I)
            _lib.moe_quant_i8(hidden, q, scales)
            _lib.moe_linear_i8(q, scales, self.w2, self.s2, out, add=add)
        return out


class MoeBlock:
    def __init__(self, router: Router, layer: MoeLayer, shared: SharedExpertI8 | None = None):
        if (router.E, router.D, router.topk) != (layer.E, layer.D, layer.topk):
            raise ValueError("router and experts differ in E, D or topk")
        if shared is not None and shared.D != layer.D:
            raise ValueError("shared expert and experts differ in D")
        self.router, self.layer, self.shared = router, layer, shared

    def forward(self, x: torch.Tensor, *, stream=None, path: str = "auto") -> torch.Tensor:
        """x: BF16 [B, D], contiguous -> the layer's output BF16 [B, D]: the weighted sum of the routed experts'
        rows, rounded to BF16, plus the shared expert's."""
        if x.dtype != torch.bfloat16 or not x.is_contiguous():
            raise ValueError("x: expected contiguous BF16 [B, D]")
        with torch.cuda.device(x.device), _on(stream, x.device) as give:
            return give(self._forward(x, path))

    def _forward(self, x, path):
        ids, weights = self.router.forward(x)
        rows = self.layer.forward(x, ids, path=path)
        y = self.layer.combine(rows, weights)
        if self.shared is not None:
            self.shared.forward(x, add=y, out=y)
        return y
