"""Choices and refusals of the block-scaled FP8 layer that hold without a GPU, beside those of test_f8_checks.py."""
import contextlib
import ctypes
import types

import pytest
import torch

import moe_routed_expert_mx_amd as m
from moe_routed_expert_mx_amd import block
from moe_routed_expert_mx_amd.layer import MoeLayer

L, EINVAL = m._lib.lib, m._lib.MOE_EINVAL
FAKE = ctypes.c_void_p(0x1000)
BF, F32, F8, I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32


def _z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


def _experts(E=4, D=64, I=48, **k):
    w13, s13 = block.f8_weight_blocks(torch.ones(E, 2 * I, D), halves=True)
    w2, s2 = block.f8_weight_blocks(torch.ones(E, D, I))
    return block.ExpertsF8(w13, s13, w2, s2, **{"topk": 2, "B_max": 4, "device": "cpu", **k})


def _shared(D=64, I=48, **k):
    w13, s13 = block.f8_weight_blocks(torch.ones(2 * I, D), halves=True)
    w2, s2 = block.f8_weight_blocks(torch.ones(D, I))
    return block.SharedExpertF8(w13, s13, w2, s2, **{"B_max": 4, "device": "cpu", **k})


def test_exact_is_0_or_1():
    for exact in (-1, 2):
        o = m.moe_linear_opts_t(exact=exact)
        assert L.moe_linear_f8(FAKE, 128, FAKE, 1, FAKE, 128, FAKE, 1, 8, 128, ctypes.byref(o), FAKE, 0, 8, None) == EINVAL
        o = m.moe_grouped_opts_t(exact=exact)
        assert L.moe_grouped_f8(FAKE, 128, FAKE, 1, 4, FAKE, 128, 8 * 128, FAKE, FAKE, 4, 2, 8, 128, ctypes.byref(o), FAKE, 0, 8, 4,
                                None) == EINVAL


def test_exact_reaches_both_ways_of_a_call(monkeypatch):
    """The native binding takes it as its last argument, ctypes as a field of the options."""
    seen = []
    for name in ("linear_f8", "grouped_f8"):
        monkeypatch.setattr(m._lib._dense, name, lambda *a: seen.append(a[-1]) or -100)
    fields = {"moe_linear_f8": (m._lib._LINEAR_OPTS, 1), "moe_grouped_f8": (m._lib._GROUPED_OPTS, 3)}

    def enqueue(name, fn, stream, tensors, *a):
        opts, i = fields[name]
        seen.append(opts.unpack(next(b for b in a if isinstance(b, bytes)))[i])

    monkeypatch.setattr(m._lib, "_enqueue", enqueue)
    q, s, o = _z(4, 256, dtype=F8), _z(4, 2), _z(3, dtype=I32)
    for exact in (False, True):
        m.moe_linear_f8(q, s, q, _z(1, 2), _z(4, 4), exact=exact)
        m.moe_grouped_f8(q, s, q[None], _z(1, 1, 2), o[:2], _z(4, 4), exact=exact)
        assert seen == [exact] * 4
        seen.clear()


@pytest.mark.parametrize("exact", [True, False])
def test_first_product_of_the_experts_is_exact_unless_told(monkeypatch, exact):
    """Its result is quantized again; the second one's is not."""
    calls = []
    for name in ("moe_quant_f8", "moe_lists", "moe_grouped_f8", "moe_linear_f8"):
        monkeypatch.setattr(m._lib, name, lambda *a, **k: calls.append(k) if "act" in k or "scatter" in k or "add" in k else None)
    opts = {} if exact else dict(exact=False)
    _experts(**opts).forward(_z(3, 64, dtype=BF), _z(3, 2, dtype=I32))
    _shared(**opts).forward(_z(3, 64, dtype=BF))
    assert [bool(k.get("exact")) for k in calls] == [exact, False] * 2


class _Streams:
    """Stand-ins for the streams and devices: where tensors are allocated, library calls made and results recorded."""

    def __init__(self, monkeypatch):
        self.here, self.side = types.SimpleNamespace(name="here"), types.SimpleNamespace(name="side", cuda_stream=7, device_index=None)
        self.current, self.device, self.allocated, self.calls, self.recorded = self.here, None, [], [], []
        empty, streams = torch.empty, self

        class Tensors(torch.Tensor):
            def record_stream(self, s):
                streams.recorded.append(s)

        def allocate(*a, **k):
            self.allocated.append(self.current)
            return empty(*a, **k).as_subclass(Tensors)

        @contextlib.contextmanager
        def entered(name, value):
            before = getattr(self, name)
            setattr(self, name, value)
            yield
            setattr(self, name, before)

        monkeypatch.setattr(torch, "empty", allocate)
        monkeypatch.setattr(torch.cuda, "stream", lambda s: entered("current", s))
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: self.current)
        monkeypatch.setattr(torch.cuda, "device", lambda d: entered("device", torch.device(d)))
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: self.side if h == 7 else None)

    def called(self, *a, stream=None, **k):
        self.calls.append((self.device, self.current if stream is None else self.side if stream == 7 else stream))

    def clear(self):
        for record in (self.allocated, self.calls, self.recorded):
            record.clear()


@pytest.mark.parametrize("stream", [None, "side", 7])
def test_combine_allocates_and_runs_on_its_stream(monkeypatch, stream):
    """On `stream` and on the experts' GPU, whichever is current; what it returns is recorded on the caller's stream."""
    ex = _experts()
    s = _Streams(monkeypatch)
    monkeypatch.setattr(m._lib, "moe_combine", s.called)
    named = s.side if stream == "side" else stream
    ran = s.here if stream is None else s.side
    y = ex.combine(_z(6, 64, dtype=BF), _z(3, 2), stream=named)
    assert y.shape == (3, 64) and s.allocated == [ran] and s.calls == [(ex.device, ran)]
    assert s.recorded == ([] if stream is None else [s.here]) and s.current is s.here and s.device is None
    s.clear()
    mine = _z(3, 64, dtype=BF)
    assert ex.combine(_z(6, 64, dtype=BF), _z(3, 2), mine, stream=named) is mine
    assert s.allocated == [] and s.calls == [(ex.device, ran)]


@pytest.mark.parametrize("stream", [None, "side", 7])
def test_fp4_layer_allocates_on_the_stream_it_runs_on(monkeypatch, stream):
    layer = object.__new__(MoeLayer)
    layer.E, layer.D, layer.I, layer.B_max, layer.topk, layer.device = 4, 64, 48, 8, 2, torch.device("cpu")
    layer.structs, layer.ws, layer.plan, layer.units = [None], None, None, None
    s = _Streams(monkeypatch)
    for name in ("moe_decode_run", "moe_plan_group", "moe_experts_run", "moe_combine"):
        monkeypatch.setattr(m._lib, name, s.called)
    named = s.side if stream == "side" else stream
    ran = s.here if stream is None else s.side
    for path, calls in (("decode", 1), ("grouped", 2)):
        rows = layer.forward(_z(3, 64, dtype=BF), _z(3, 2, dtype=I32), path=path, stream=named)
        assert rows.shape == (6, 64) and s.allocated == [ran] and [c[1] for c in s.calls] == [ran] * calls
        assert s.recorded == ([] if stream is None else [s.here]) and s.current is s.here
        s.clear()
    y = layer.combine(rows, _z(3, 2), stream=named)
    assert y.shape == (3, 64) and s.allocated == [ran] and [c[1] for c in s.calls] == [ran]
    assert s.recorded == ([] if stream is None else [s.here])


# --------------------------------------------------------------- sizes
def test_experts_refuse_batches_that_a_step_would_refuse():
    """When they are made, not between two launches: B_max * topk and B_max * D beyond what each step takes."""
    meta = dict(device="meta", topk=2)
    for I, D, k in ((48, 64, dict(topk=64, B_max=(1 << 20) + 1)),      # more routes than the lists take
                    (48, 64, dict(B_max=(1 << 25) + 1)),               # (both: B_max * D = 2^31 too)
                    (48, 8192, dict(B_max=1 << 18)),                   # rows gathered beyond 2^31
                    (32768, 64, dict(B_max=1 << 24)),                  # the first product beyond 2^40
                    (65552, 64, {}), (48, 65552, {})):
        w13, w2 = torch.empty(1, 2 * I, D, dtype=F8, device="meta"), torch.empty(1, D, I, dtype=F8, device="meta")
        b = lambda n: (n + 127) // 128
        s13, s2 = torch.empty(1, 2 * b(I), b(D), device="meta"), torch.empty(1, b(D), b(I), device="meta")
        with pytest.raises(ValueError, match="batch|65536"):
            block.ExpertsF8(w13, s13, w2, s2, **{**meta, "B_max": 4, **k})
    for I, D, B in ((48, 64, (1 << 22) + 1), (8192, 64, (1 << 20) + 1), (65552, 64, 4), (48, 65552, 4)):
        w13, w2 = torch.empty(2 * I, D, dtype=F8, device="meta"), torch.empty(D, I, dtype=F8, device="meta")
        with pytest.raises(ValueError, match="batch|65536"):
            block.SharedExpertF8(w13, torch.empty(2 * b(I), b(D), device="meta"), w2, torch.empty(b(D), b(I), device="meta"),
                                 B_max=B, device="meta")


def test_rows_are_quantized_in_parts_that_the_library_takes(monkeypatch):
    """A hidden of more than 2^22 rows (routes): in order, whole, no part longer."""
    parts = []
    monkeypatch.setattr(m._lib, "moe_quant_f8", lambda x, q, s: parts.append((x.storage_offset() // 16, len(x), q.storage_offset() // 16,
                                                                              len(q), s.storage_offset(), len(s))))
    buffers = block._CodesF8((1 << 23) + 5, 16, "meta")
    for n in (1, 1 << 22, (1 << 22) + 1, (1 << 23) + 5):
        parts.clear()
        q, s = buffers.of(torch.empty(n, 16, dtype=BF, device="meta"))
        assert len(q) == len(s) == n
        at = 0
        for p in parts:
            assert p == (at, p[1]) * 3 and 1 <= p[1] <= 1 << 22
            at += p[1]
        assert at == n


# --------------------------------------------------------------- weights
def test_weight_blocks_of_tiny_values():
    """Scales that FP32 holds as subnormals: codes stay finite, values within half a code's step and half a scale's."""
    unit = 2.0 ** -149
    for top in (1, 2, 300, 448, 449, 628, 629, 700, 1000, 2000, 5000, 448 * 3 + 200, 448 * 1000):
        w = torch.full((130, 144), float(top), dtype=torch.float64) * unit
        w[:, ::3] *= -0.5
        c, s = block.f8_weight_blocks(w.float())
        assert torch.isfinite(c.float()).all() and torch.isfinite(s).all()
        v = c.double() * s.double().repeat_interleave(128, 0)[:130].repeat_interleave(128, 1)[:, :144]
        # half a step of e4m3 (of its smallest at least), and of the scale's own rounding up nothing: codes are of v / scale
        assert ((v - w.float().double()).abs() <= 2.0 ** -4 * w.abs() + 2.0 ** -10 * s.double().max()).all(), top
    w = torch.full((128, 128), 8.8e-43)
    assert torch.isfinite(block.f8_weight_blocks(w)[0].float()).all()
    w[0, 0], w[1, 1] = float("inf"), float("nan")
    assert not torch.isfinite(block.f8_weight_blocks(w)[1]).any()


# --------------------------------------------------------------- ids of another rank
def test_rows_of_another_ranks_experts_are_zeros_in_a_new_buffer(monkeypatch):
    """What no product writes is not left undefined: 0 times a NaN there would reach the combined output.  Buffers of the
    caller are left as they were, and MoeBlock, whose router names experts of this layer only, does not pay for zeros."""
    empty, zeros, filled = torch.empty, torch.zeros, []
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **k).fill_(float("nan")) if k.get("dtype") == BF else empty(*a, **k))
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: filled.append(a) or zeros(*a, **k))
    for name in ("moe_quant_f8", "moe_lists", "moe_grouped_f8", "moe_combine"):
        monkeypatch.setattr(m._lib, name, lambda *a, **k: None)
    ex, ids = _experts(), torch.full((3, 2), -1, dtype=I32)
    filled.clear()
    x = empty(3, 64, dtype=BF)
    out = ex.forward(x, ids)
    assert out.shape == (6, 64) and out.dtype == BF and (out == 0).all() and len(filled) == 1
    mine = torch.full((6, 64), 7.0, dtype=BF)
    assert ex.forward(x, ids, mine) is mine and (mine == 7).all() and len(filled) == 1
    router = types.SimpleNamespace(E=4, D=64, topk=2, forward=lambda x: (ids, empty(3, 2)))
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    block.MoeBlock(router, ex).forward(x)
    assert len(filled) == 1


def test_experts_refuse_an_output_of_too_few_rows(monkeypatch):
    """Routes behind its last row would be dropped without a word."""
    made = []
    for name in ("moe_quant_f8", "moe_lists", "moe_grouped_f8"):
        monkeypatch.setattr(m._lib, name, lambda *a, **k: made.append(a))
    ex, x, ids = _experts(), _z(3, 64, dtype=BF), _z(3, 2, dtype=I32)
    for bad in (_z(5, 64, dtype=BF), _z(6, 63, dtype=BF), _z(3, 2, 64, dtype=BF)):
        with pytest.raises(ValueError, match="out"):
            ex.forward(x, ids, bad)
    assert made == []
    for fine in (_z(6, 64, dtype=BF), _z(9, 64)):
        assert ex.forward(x, ids, fine) is fine


def test_grids_beyond_the_launch_limit_are_refused():
    """2^32 threads: an error of the arguments, not of the launch."""
    for M, K in ((1 << 22, 16384), (1 << 22, 131072), (1 << 19, 131072)):
        assert L.moe_quant_f8(FAKE, 0, K, M, K, FAKE, K, FAKE, K // 128, None) == EINVAL


@pytest.mark.parametrize("handle", [0, 7])
def test_raw_handle_of_the_default_stream(monkeypatch, handle):
    """0 names the default stream of the tensors' GPU (what the default stream's cuda_stream is); torch takes an external
    handle of 0 for none and hands out a stream of its own."""
    ex, layer = _experts(), object.__new__(MoeLayer)
    layer.E, layer.D, layer.B_max, layer.topk, layer.device = 4, 64, 8, 2, torch.device("cpu")
    s = _Streams(monkeypatch)
    default = types.SimpleNamespace(name="default")
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: default)
    monkeypatch.setattr(m._lib, "moe_combine", lambda *a, stream=None: s.calls.append(s.current if stream is None else stream))
    ran = s.side if handle else default
    ex.combine(_z(6, 64, dtype=BF), _z(3, 2), stream=handle)
    assert s.allocated == [ran] and s.calls == [ran] and s.recorded == [s.here]
    s.clear()
    layer.combine(_z(6, 64, dtype=BF), _z(3, 2), stream=handle)
    assert s.allocated == [ran] and s.recorded == [s.here]
