"""The dense side of a routed-experts layer, and the whole layer, through the C ABI.

``Router`` turns tokens into expert ids and weights (moe_gate, moe_route),
``SharedExpertI8`` is a SwiGLU MLP on every token in 8-bit integers (moe_quant_i8,
moe_linear_i8), and ``MoeBlock`` runs them around a ``MoeLayer``: router, routed experts,
weighted combine, shared expert added last.  ``ExpertsF8`` and ``SharedExpertF8`` are the routed
experts (moe_lists, moe_grouped_f8) and the shared one (moe_linear_f8) in block-scaled FP8, for
batches from one token to prompts, and ``Norm`` (moe_rms_norm) stands in front of the layer.  Each owns its device buffers for up to B_max
tokens and reuses them from call to call, so calls of one object must be ordered (one
stream, or ordered streams), and follow its construction, which enqueues on the current stream.
torch only allocates memory and supplies the stream.

A call runs on the current stream, or on `stream` (a torch stream or a raw handle): there it
allocates too, as it would under torch.cuda.stream(stream), so that no buffer it drops is
handed on before the stream is done with it.  What it returns is recorded on the caller's current
stream: after the usual wait for `stream` it may be read there and dropped at any time.
"""
from __future__ import annotations

import torch

from . import _lib
from .layer import MoeLayer, _on

_F8 = torch.float8_e4m3fn


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
        """x: BF16 [B, D], or its codes and scales (as moe_quant_i8 or moe_rms_norm made them) -> BF16 [B, D], plus `add`
        if given (which may be out itself).  The hidden is rounded to BF16 between the products."""
        given = isinstance(x, (tuple, list))
        first = x[0] if given else x
        B = first.shape[0]
        if B > self.B_max:
            raise ValueError("batch larger than B_max")
        with _on(stream, first.device) as give:
            if out is None:
                out = give(torch.empty(B, self.D, dtype=torch.bfloat16, device=self.device))
            # rows of the code buffers are packed for each product, so that they stay 16-byte aligned
            flat = self.codes.view(-1)
            scales, hidden = self.scales[:B], self.hidden[:B]
            if given:
                q, first_scales = x
            else:
                q, first_scales = flat[:B * self.D].view(B, self.D), scales
                _lib.moe_quant_i8(x, q, scales)
            _lib.moe_linear_i8(q, first_scales, self.w13, self.s13, hidden, act="swiglu")
            q = flat[:B * self.I].view(B, self.I)
            _lib.moe_quant_i8(hidden, q, scales)
            _lib.moe_linear_i8(q, scales, self.w2, self.s2, out, add=add)
        return out


def f8_weight_blocks(w, *, halves: bool = False):
    """Weights [.., N, K] of a float type -> (codes float8_e4m3fn [.., N, K], scales FP32 [.., row blocks, K blocks])
    with scale = amax / 448 for each 128 x 128; halves: gate and up rows, each half with blocks of its own (the
    first product's weight).  For loading, in torch."""
    w = torch.as_tensor(w)
    if halves:
        if w.shape[-2] % 2:
            raise ValueError("gate and up rows: expected an even number of rows")
        parts = [f8_weight_blocks(p) for p in w.chunk(2, dim=-2)]
        return torch.cat([p[0].view(torch.uint8) for p in parts], -2).view(_F8), torch.cat([p[1] for p in parts], -2)
    *lead, N, K = w.shape
    nb, kb = (N + 127) // 128, (K + 127) // 128
    v = torch.nn.functional.pad(w.float(), (0, kb * 128 - K, 0, nb * 128 - N)).view(*lead, nb, 128, kb, 128)
    amax = v.abs().amax((-3, -1))
    scales = amax / 448
    # among subnormals the quotient's rounding is coarse: up, or v / scale could pass 448
    scales = torch.where((amax > 0) & (scales < 2.0 ** -126), torch.nextafter(scales, torch.full_like(scales, 1.0)), scales)
    v = v / torch.where(scales > 0, scales, 1.0)[..., :, None, :, None]
    return v.view(*lead, nb * 128, kb * 128)[..., :N, :K].to(_F8).contiguous(), scales.contiguous()


def _f8_weight(w, s, device, shape, name):
    """Codes and scales of a block-scaled weight, on the device."""
    w, s = torch.as_tensor(w), torch.as_tensor(s)
    if w.dtype != _F8 or w.shape != shape[0] or s.shape != shape[1]:
        raise ValueError(f"{name}: expected float8_e4m3fn {list(shape[0])} with scales {list(shape[1])} (see "
                         f"f8_weight_blocks), got {w.dtype} {list(w.shape)} with {list(s.shape)}")
    return w.to(device).contiguous(), s.to(device, torch.float32).contiguous()


class _CodesF8:
    """Codes and scales of up to `rows` rows of `cols` features."""

    def __init__(self, rows: int, cols: int, device):
        self.codes = torch.empty(rows, cols, dtype=_F8, device=device)
        self.scales = torch.empty(rows, (cols + 127) // 128, device=device)

    def of(self, x):
        # rows that moe_quant_f8 takes; the experts' routes may be more
        n, most = x.shape[0], min(1 << 22, ((1 << 27) - 1) // ((self.codes.shape[1] + 511) // 512))
        codes, scales = self.codes[:n], self.scales[:n]
        if n <= most:
            _lib.moe_quant_f8(x, codes, scales)
        else:
            for i in range(0, n, most):
                _lib.moe_quant_f8(x[i:i + most], codes[i:i + most], scales[i:i + most])
        return codes, scales


class ExpertsF8:
    """Routed experts in block-scaled FP8, for batches from one token to prompts; in MoeLayer's place in a MoeBlock."""

    def __init__(self, w13, s13, w2, s2, *, topk: int, B_max: int, exact: bool = True, device="cuda"):
        """w13 float8_e4m3fn [E, 2I, D] (gate rows, then up rows) with FP32 scales [E, 2 ceil(I / 128), ceil(D / 128)],
        w2 [E, D, I] with [E, ceil(D / 128), ceil(I / 128)]; D and I multiples of 16.  f8_weight_blocks makes them of
        other weights.  exact: the first product's sums, as moe_linear_f8's; its result is quantized again, so that
        without it the rows' error grows by a fifth, while a prompt takes a fifth less time."""
        w2 = torch.as_tensor(w2)
        if w2.dim() != 3:
            raise ValueError("experts: w2: expected [E, D, I]")
        self.E, self.D, self.I = map(int, w2.shape)
        self.B_max, self.topk, self.exact = int(B_max), int(topk), bool(exact)
        if self.D % 16 or self.I % 16 or not 1 <= self.E <= 1024 or self.topk < 1 or self.B_max < 1:
            raise ValueError("experts: D and I must be multiples of 16, E at most 1024")
        R = self.B_max * self.topk
        if max(self.D, self.I) > 65536 or R > 1 << 26 or R * max(2 * self.I, self.D) > 1 << 40 or self.B_max * self.D >= 1 << 31:
            raise ValueError("experts: D and I up to 65536 and batches up to topk * B_max = 2^26 routes, 2^40 values of a product "
                             "and B_max * D < 2^31 are taken")
        E, D, I, b = self.E, self.D, self.I, lambda n: (n + 127) // 128
        self.w13, self.s13 = _f8_weight(w13, s13, device, ((E, 2 * I, D), (E, 2 * b(I), b(D))), "experts: w13")
        self.w2, self.s2 = _f8_weight(w2, s2, device, ((E, D, I), (E, b(D), b(I))), "experts: w2")
        self.device = self.w2.device  # with its index: "cuda" would mean another GPU where another is current
        self.x = _CodesF8(self.B_max, D, self.device)
        self.hidden = torch.empty(R, I, dtype=torch.bfloat16, device=self.device)
        self.h = _CodesF8(R, I, self.device)
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device=self.device)
        self.pairs = torch.empty(R, dtype=torch.int32, device=self.device)
        self.ws = torch.empty(_lib.moe_lists_ws_bytes(R, E), dtype=torch.uint8, device=self.device)

    def out_buffer(self, B: int) -> torch.Tensor:
        return torch.empty(B * self.topk, self.D, dtype=torch.bfloat16, device=self.device)

    def forward(self, x, ids: torch.Tensor, out: torch.Tensor | None = None, *, stream=None,
                path: str = "auto") -> torch.Tensor:
        """x: BF16 [B, D], or its codes and scales (as moe_quant_f8 or moe_rms_norm made them); ids: int32 [B, topk]
        -> rows BF16 [B * topk, D] in the order of the ids, no routing weight applied.  Ids outside [0, E) have no
        expert here: their rows of `out` are left as they were.  Without `out` they are zeros, which costs filling them all
        (940 MB of 8192 tokens' rows): where every id has an expert, pass out_buffer(B).  The hidden is rounded to BF16
        between the products.
        path: "auto" (there is one)."""
        given = isinstance(x, (tuple, list))
        B = (x[0] if given else x).shape[0]
        if B > self.B_max or ids.shape != (B, self.topk):
            raise ValueError("batch larger than B_max or ids of the wrong shape")
        if path != "auto":
            raise ValueError(f"unknown path {path!r}")
        R = B * self.topk
        if out is not None and (out.dim() != 2 or out.shape[0] < R or out.shape[1] != self.D):
            raise ValueError(f"out: expected [{R}, {self.D}], got {list(out.shape)}")
        with _on(stream, self.device) as give:
            if out is None:
                out = give(torch.zeros(R, self.D, dtype=torch.bfloat16, device=self.device))
            pairs, hidden = self.pairs[:R], self.hidden[:R]
            codes, scales = x if given else self.x.of(x)
            _lib.moe_lists(ids, self.offsets, pairs, ws=self.ws)
            _lib.moe_grouped_f8(codes, scales, self.w13, self.s13, self.offsets, hidden, act="swiglu", pairs=pairs,
                                gather=self.topk, exact=self.exact)
            codes, scales = self.h.of(hidden)
            _lib.moe_grouped_f8(codes, scales, self.w2, self.s2, self.offsets, out, pairs=pairs, scatter=True)
        return out

    def combine(self, rows: torch.Tensor, weights: torch.Tensor, y: torch.Tensor | None = None, *, stream=None):
        """Weighted top-k combine of the rows, as MoeLayer's."""
        with torch.cuda.device(self.device), _on(stream, self.device) as give:
            if y is None:
                y = give(torch.empty(weights.shape[0], self.D, dtype=torch.bfloat16, device=self.device))
            _lib.moe_combine(rows, weights, y)
        return y


class SharedExpertF8:
    def __init__(self, w13, s13, w2, s2, *, B_max: int, exact: bool = True, device="cuda"):
        """w13 float8_e4m3fn [2I, D] (gate rows, then up rows) with FP32 scales [2 ceil(I / 128), ceil(D / 128)], w2
        [D, I] with [ceil(D / 128), ceil(I / 128)]; D and I multiples of 16.  exact: as ExpertsF8's."""
        w2 = torch.as_tensor(w2)
        if w2.dim() != 2:
            raise ValueError("shared expert: w2: expected [D, I]")
        self.D, self.I = map(int, w2.shape)
        self.B_max, self.exact = int(B_max), bool(exact)
        if self.D % 16 or self.I % 16 or self.B_max < 1:
            raise ValueError("shared expert: D and I must be multiples of 16")
        if max(self.D, self.I) > 65536 or self.B_max > 1 << 22 or self.B_max * max(2 * self.I, self.D) > 1 << 34:
            raise ValueError("shared expert: D and I up to 65536 and batches up to 2^22 tokens and 2^34 values of a product are "
                             "taken")
        D, I, b = self.D, self.I, lambda n: (n + 127) // 128
        self.w13, self.s13 = _f8_weight(w13, s13, device, ((2 * I, D), (2 * b(I), b(D))), "shared expert: w13")
        self.w2, self.s2 = _f8_weight(w2, s2, device, ((D, I), (b(D), b(I))), "shared expert: w2")
        self.device = self.w2.device  # with its index: "cuda" would mean another GPU where another is current
        self.x = _CodesF8(self.B_max, D, self.device)
        self.hidden = torch.empty(self.B_max, I, dtype=torch.bfloat16, device=self.device)
        self.h = _CodesF8(self.B_max, I, self.device)

    def forward(self, x, *, add: torch.Tensor | None = None, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
        """x: BF16 [B, D], or its codes and scales -> BF16 [B, D], plus `add` if given (which may be out itself).  The
        hidden is rounded to BF16 between the products."""
        given = isinstance(x, (tuple, list))
        B = (x[0] if given else x).shape[0]
        if B > self.B_max:
            raise ValueError("batch larger than B_max")
        with _on(stream, self.device) as give:
            if out is None:
                out = give(torch.empty(B, self.D, dtype=torch.bfloat16, device=self.device))
            codes, scales = x if given else self.x.of(x)
            hidden = self.hidden[:B]
            _lib.moe_linear_f8(codes, scales, self.w13, self.s13, hidden, act="swiglu", exact=self.exact)
            codes, scales = self.h.of(hidden)
            _lib.moe_linear_f8(codes, scales, self.w2, self.s2, out, add=add)
        return out


class Norm:
    """The root-mean-square norm in front of a layer, and the residual stream's addition before it."""

    def __init__(self, weight, *, eps: float = 1e-6, device="cuda"):
        """weight: [D], kept in FP32."""
        self.weight = torch.as_tensor(weight).to(device, torch.float32).contiguous()
        if self.weight.dim() != 1:
            raise ValueError("norm: expected a weight [D]")
        self.device, self.D, self.eps = self.weight.device, int(self.weight.shape[0]), float(eps)

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None, *, codes=None, stream=None):
        """x: [B, D] (BF16, FP16 or FP32) -> the norm of x + residual, of x's type; `residual` is overwritten with the
        sum.  codes: None, torch.int8 or torch.float8_e4m3fn; with it (norm, codes, scales) is returned."""
        B = x.shape[0]
        with _on(stream, self.device) as give:
            out = torch.empty(B, self.D, dtype=x.dtype, device=self.device)
            q = s = None
            if codes is not None:
                q = torch.empty(B, self.D, dtype=codes, device=self.device)
                s = torch.empty(*((B,) if codes == torch.int8 else (B, (self.D + 127) // 128)), device=self.device)
            _lib.moe_rms_norm(x, self.weight, out=out, residual=residual, total=residual, codes=q, scales=s, eps=self.eps)
            return give(out) if codes is None else (give(out), give(q), give(s))


class MoeBlock:
    def __init__(self, router: Router, layer: MoeLayer | ExpertsF8,
                 shared: SharedExpertI8 | SharedExpertF8 | None = None, norm: Norm | None = None):
        """norm: None, or the norm in front of the layer; its 8-bit codes then go straight to the parts in FP8, or to an
        int8 shared expert beside experts that are not."""
        if (router.E, router.D, router.topk) != (layer.E, layer.D, layer.topk):
            raise ValueError("router and experts differ in E, D or topk")
        if shared is not None and shared.D != layer.D:
            raise ValueError("shared expert and experts differ in D")
        if norm is not None and norm.D != layer.D:
            raise ValueError("norm and experts differ in D")
        self.router, self.layer, self.shared, self.norm = router, layer, shared, norm

    def forward(self, x: torch.Tensor, *, residual: torch.Tensor | None = None, stream=None,
                path: str = "auto") -> torch.Tensor:
        """x: BF16 [B, D], contiguous -> the layer's output BF16 [B, D]: the weighted sum of the routed experts'
        rows, rounded to BF16, plus the shared expert's.  With a norm the layer sees the norm of x + residual, and
        `residual`, where it is given, is overwritten with that sum."""
        if x.dtype != torch.bfloat16 or not x.is_contiguous():
            raise ValueError("x: expected contiguous BF16 [B, D]")
        if residual is not None and self.norm is None:
            raise ValueError("a residual without a norm")
        with torch.cuda.device(x.device), _on(stream, x.device) as give:
            return give(self._forward(x, residual, path))

    def _forward(self, x, residual, path):
        f8 = isinstance(self.layer, ExpertsF8), isinstance(self.shared, SharedExpertF8)
        x8, codes = x, None
        if self.norm is not None:
            # (one kind of codes a norm: e4m3 where a part takes them, else int8 for an int8 shared expert)
            codes = _F8 if any(f8) else torch.int8 if isinstance(self.shared, SharedExpertI8) else None
            if codes is None:
                x = self.norm.forward(x, residual)
            else:
                x, *x8 = self.norm.forward(x, residual, codes=codes)
        ids, weights = self.router.forward(x)
        if f8[0]:  # (every id of the router has an expert)
            rows = self.layer.forward(x8, ids, self.layer.out_buffer(len(ids)), path=path)
        else:
            rows = self.layer.forward(x, ids, path=path)
        y = self.layer.combine(rows, weights)
        if self.shared is not None:
            self.shared.forward(x8 if f8[1] or codes == torch.int8 else x, add=y, out=y)
        return y
