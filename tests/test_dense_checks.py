"""Refusals of the dense side's entry points: in the library (before any HIP call, with
pointers that are never dereferenced) and in the binding (on CPU tensors).  No GPU needed."""
import ctypes

import pytest
import torch

import moe_routed_expert_mx_amd as m

L, EINVAL, ENOSPACE = m._lib.lib, m._lib.MOE_EINVAL, m._lib.MOE_ENOSPACE
FAKE = ctypes.c_void_p(0x1000)
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def test_gate_sizes_and_refusals():
    assert m.moe_gate_packed_bytes(160, 3584, BF) == 160 * 3584 * 2
    assert m.moe_gate_packed_bytes(161, 512, F32) == 176 * 512 * 6
    for e, d, t in ((0, 512, BF), (1025, 512, BF), (8, 500, BF), (8, 0, BF), (8, 16896, BF), (8, 512, F16)):
        assert m.moe_gate_packed_bytes(e, d, t) == 0
    big = 1 << 30
    assert L.moe_gate_pack(None, 0, 16, 512, FAKE, big, None) == EINVAL
    assert L.moe_gate_pack(FAKE, 1, 16, 512, FAKE, big, None) == EINVAL
    assert L.moe_gate_pack(FAKE, 0, 16, 512, FAKE, 16 * 512 * 2 - 1, None) == ENOSPACE

    def gate(E=16, D=512, wtype=0, packed=0x1000, x=FAKE, ldx=512, B=1, out=FAKE, ldl=16):
        g = m.moe_gate_t(E, D, wtype, packed)
        return L.moe_gate(ctypes.byref(g), x, ldx, B, out, ldl, None)

    for bad in (dict(packed=0), dict(x=None), dict(out=None), dict(B=0), dict(B=-1), dict(B=(1 << 22) + 1),
                dict(ldx=511), dict(ldx=516), dict(ldl=15), dict(E=0), dict(D=100), dict(wtype=1),
                dict(x=ctypes.c_void_p(0x1008)), dict(packed=0x1002)):
        assert gate(**bad) == EINVAL, bad
    assert L.moe_gate(None, FAKE, 512, 1, FAKE, 16, None) == EINVAL


def test_route_refusals():
    def route(logits=FAKE, type=2, ldl=16, B=1, E=16, topk=4, ids=FAKE, w=FAKE, **o):
        opts = m.moe_route_opts_t(**o)
        return L.moe_route(logits, type, ldl, B, E, topk, ctypes.byref(opts), ids, w, None)

    for bad in (dict(logits=None), dict(ids=None), dict(w=None), dict(type=3), dict(type=-1), dict(ldl=15), dict(B=0),
                dict(B=(1 << 22) + 1), dict(E=0), dict(E=1025, ldl=1025), dict(topk=0), dict(topk=17),
                dict(E=128, ldl=128, topk=65), dict(score=2), dict(score=-1), dict(renorm=2),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(groups=-1), dict(groups=3, topk_groups=1),
                dict(groups=4), dict(groups=4, topk_groups=5), dict(topk_groups=1),
                dict(groups=8, topk_groups=1), dict(groups=4, topk_groups=2, group_score=2), dict(group_score=-1),
                dict(E=130, ldl=130, groups=65, topk_groups=65)):
        assert route(**bad) == EINVAL, bad


def test_quant_refusals():
    def quant(x=FAKE, type=0, ldx=8, M=1, K=8, q=FAKE, ldc=8, s=FAKE):
        return L.moe_quant_i8(x, type, ldx, M, K, q, ldc, s, None)

    for bad in (dict(x=None), dict(q=None), dict(s=None), dict(type=3), dict(ldx=7), dict(ldc=7), dict(M=0),
                dict(M=(1 << 22) + 1), dict(K=0), dict(K=131073, ldx=131073, ldc=131073)):
        assert quant(**bad) == EINVAL, bad


def test_linear_refusals():
    def linear(a=FAKE, lda=16, sa=FAKE, w=FAKE, ldw=16, sw=FAKE, M=1, N=8, K=16, out=FAKE, type=0, ldo=8, **o):
        opts = m.moe_linear_opts_t(**o)
        return L.moe_linear_i8(a, lda, sa, w, ldw, sw, M, N, K, ctypes.byref(opts), out, type, ldo, None)

    for bad in (dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(out=None), dict(type=3), dict(lda=15),
                dict(ldw=15), dict(lda=1 << 22), dict(ldw=1 << 22), dict(M=0), dict(N=0), dict(K=0),
                dict(K=131072, lda=131072, ldw=131072), dict(ldo=7), dict(act=2), dict(act=-1),
                dict(act=1, N=9, ldo=9), dict(act=1, ldo=3), dict(add_dev=0x1000, ldadd=7),
                dict(M=(1 << 22) + 1), dict(N=(1 << 20) + 1, ldo=1 << 21), dict(M=1 << 22, N=1 << 20, ldo=1 << 20)):
        assert linear(**bad) == EINVAL, bad


def _z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_checks_tensors():
    """Shapes, types, strides and devices are refused with ValueError; the last check is
    the device, so a call that is right but for it names the GPU."""
    x, lg, ids, w = _z(4, 512, dtype=BF), _z(4, 16), _z(4, 2, dtype=torch.int32), _z(4, 2)
    g = m.moe_gate_t(16, 512, 0, 0x1000)
    i8 = torch.int8
    a, sa, wt, sw, out = _z(4, 32, dtype=i8), _z(4), _z(8, 32, dtype=i8), _z(8), _z(4, 8, dtype=BF)
    right = [
        lambda: m.moe_gate_pack(_z(16, 512, dtype=BF), _z(16 * 512 * 2, dtype=torch.uint8)),
        lambda: m.moe_gate(g, x, lg),
        lambda: m.moe_route(lg, ids, w),
        lambda: m.moe_quant_i8(x, _z(4, 512, dtype=i8), _z(4)),
        lambda: m.moe_linear_i8(a, sa, wt, sw, out),
        lambda: m.moe_linear_i8(a, sa, wt, sw, out[:, :4], act="swiglu", bias=_z(8), add=_z(4, 4, dtype=BF)),
    ]
    for call in right:
        with pytest.raises(ValueError, match="must be on a GPU"):
            call()
    wrong = [
        lambda: m.moe_gate_pack(_z(512, 16, dtype=BF).t(), _z(16 * 512 * 2, dtype=torch.uint8)),
        lambda: m.moe_gate_pack(_z(16, 512, dtype=F16), _z(16 * 512 * 2, dtype=torch.uint8)),
        lambda: m.moe_gate(g, _z(4, 512), lg),
        lambda: m.moe_gate(g, _z(4, 1024, dtype=BF), lg),
        lambda: m.moe_gate(g, x, _z(4, 17)),
        lambda: m.moe_gate(g, x, _z(3, 16)),
        lambda: m.moe_gate(g, x, _z(4, 16, dtype=BF)),
        lambda: m.moe_gate(g, _z(512, 4, dtype=BF).t(), lg),
        lambda: m.moe_gate(g, _z(1, 512, dtype=BF).expand(4, 512), lg),
        lambda: m.moe_route(_z(4, 16, dtype=torch.float64), ids, w),
        lambda: m.moe_route(lg, ids.long(), w),
        lambda: m.moe_route(lg, ids[:3], w),
        lambda: m.moe_route(lg, ids, _z(4, 3)),
        lambda: m.moe_route(lg, ids, w.half()),
        lambda: m.moe_route(lg, _z(2, 4, dtype=torch.int32).t(), w),
        lambda: m.moe_route(lg, ids, w, bias=_z(15)),
        lambda: m.moe_route(lg, ids, w, bias=_z(16, dtype=BF)),
        lambda: m.moe_route(lg, ids, w, score="tanh"),
        lambda: m.moe_route(lg, ids, w, groups=4, topk_groups=2, group_score="mean"),
        lambda: m.moe_route(lg, ids, w, scale=0.0),
        lambda: m.moe_quant_i8(x, _z(4, 512, dtype=torch.uint8), _z(4)),
        lambda: m.moe_quant_i8(x, _z(4, 511, dtype=i8), _z(4)),
        lambda: m.moe_quant_i8(x, _z(4, 512, dtype=i8), _z(3)),
        lambda: m.moe_quant_i8(x, _z(4, 512, dtype=i8), _z(8)[::2]),
        lambda: m.moe_quant_i8(x[0], _z(4, 512, dtype=i8), _z(4)),
        lambda: m.moe_linear_i8(a, sa, wt[:, :31], sw, out),
        lambda: m.moe_linear_i8(a.float(), sa, wt, sw, out),
        lambda: m.moe_linear_i8(a, sa, wt, sw, out[:3]),
        lambda: m.moe_linear_i8(a, sa, wt, sw, out, act="swiglu"),
        lambda: m.moe_linear_i8(a, sa, wt, sw, out, act="gelu"),
        lambda: m.moe_linear_i8(a, sa, wt[:7], sw[:7], out[:, :3], act="swiglu"),
        lambda: m.moe_linear_i8(a, sa[:3], wt, sw, out),
        lambda: m.moe_linear_i8(a, sa, wt, sw.half(), out),
        lambda: m.moe_linear_i8(a, sa, wt, sw, out, bias=_z(7)),
        lambda: m.moe_linear_i8(a, sa, wt, sw, out, add=_z(4, 8)),
        lambda: m.moe_linear_i8(a, sa, wt, sw, out, add=_z(4, 7, dtype=BF)),
        lambda: m.moe_linear_i8(a, sa, wt, sw, out, add=_z(1, 8, dtype=BF).expand(4, 8)),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises(ValueError) as e:
            call()
        assert "must be on a GPU" not in str(e.value), i


def test_native_binding_declines():
    """The native binding enqueues nothing it is not sure of: tensors that are not on a GPU, of another type or
    shape, no tensors at all, the wrong number of arguments; the caller's own checks follow."""
    d, no = m._lib._dense, -100
    x, q, s = _z(4, 512, dtype=BF), _z(4, 512, dtype=torch.int8), _z(4)
    assert d.quant(x, q, s) == no
    assert d.quant(x, q, None) == no and d.quant(1, 2, 3) == no and d.quant(x, q) == no
    assert d.route(_z(4, 16), _z(4, 2, dtype=torch.int32), _z(4, 2), None, None, 0, 0, 0, True, 1.0) == no
    assert d.route(_z(4, 16), _z(4, 2, dtype=torch.int32), _z(4, 2), 0, None, 0, 0, 0, True, "1") == no
    assert d.linear(q, s, q, s, _z(4, 4), 0, None, None) == no
    assert d.gate(0x1000, 512, 16, x, _z(4, 16)) == no
    meta = torch.empty(4, 512, dtype=BF, device="meta")
    assert d.quant(meta, q, s) == no


def test_layer_objects_allocate_on_the_stream_they_run_on(monkeypatch):
    """Buffers of a call with a stream come from that stream's pool: one that is dropped at return, with the kernels still
    to run, must not be handed to work on another stream.  (Stand-ins for the library and the streams: no GPU needed.)"""
    import contextlib
    import types

    from moe_routed_expert_mx_amd import block

    here, side = types.SimpleNamespace(name="here"), types.SimpleNamespace(name="side", cuda_stream=7,
                                                                            device_index=None)
    state = types.SimpleNamespace(current=here, allocated=[], calls=[], recorded=[])

    @contextlib.contextmanager
    def entered(s):
        before, state.current = state.current, s
        yield
        state.current = before

    class Tensors(torch.Tensor):
        def record_stream(self, s):
            state.recorded.append(s)

    empty = torch.empty

    def recording(*a, **k):
        state.allocated.append(state.current)
        return empty(*a, **k).as_subclass(Tensors)

    def called(*a, stream=None, **k):
        state.calls.append(state.current if stream is None else stream)

    class Layer:
        E, D, topk = 16, 512, 2

        def forward(self, x, ids, *, stream=None, path="auto"):
            called(stream=stream)
            return torch.empty(len(ids) * 2, 512, dtype=BF)

        def combine(self, rows, weights, *, stream=None):
            called(stream=stream)
            return torch.empty(len(weights), 512, dtype=BF)

    fake = types.SimpleNamespace(moe_gate_packed_bytes=lambda *a: 64, moe_gate_pack=lambda w, p: p, moe_gate=called,
                                 moe_route=called, moe_quant_i8=called, moe_linear_i8=called)
    monkeypatch.setattr(block, "_lib", fake)
    monkeypatch.setattr(torch, "empty", recording)
    monkeypatch.setattr(torch.cuda, "stream", entered)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: state.current)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: side if h == 7 else None)
    router = block.Router(_z(16, 512, dtype=BF), topk=2, B_max=4, device="cpu")
    i8 = torch.int8
    shared = block.SharedExpertI8(_z(64, 512, dtype=i8), _z(64), _z(512, 32, dtype=i8), _z(512), B_max=4, device="cpu")
    x = _z(3, 512, dtype=BF)
    for stream in (side, 7):
        for obj, calls, made, returned in ((router, 2, 2, 2), (shared, 4, 1, 1),
                                           (block.MoeBlock(router, Layer(), shared), 8, 4, 1)):
            for record in (state.allocated, state.calls, state.recorded):
                record.clear()
            obj.forward(x, stream=stream)
            assert state.allocated == [side] * made
            assert len(state.calls) == calls and all(c in (side, 7) for c in state.calls)
            assert state.recorded.count(here) == returned and state.current is here
    with pytest.raises(ValueError, match="another GPU"):
        router.forward(x, stream=types.SimpleNamespace(cuda_stream=9, device_index=3))
    state.allocated.clear()
    router.forward(x)
    assert state.allocated == [here] * 2


def test_package_works_without_the_native_binding(tmp_path):
    """A tree with the HIP library alone imports, with a warning, and its calls go through ctypes."""
    import os
    import shutil
    import subprocess
    import sys
    shutil.copytree(m._lib.HERE, tmp_path / "moe_routed_expert_mx_amd",
                    ignore=shutil.ignore_patterns("_dense*", "__pycache__", "csrc", "*.tmp*"))
    code = """if True:
        import warnings
        with warnings.catch_warnings(record=True) as seen:
            warnings.simplefilter("always")
            import moe_routed_expert_mx_amd as m
        assert any("native binding" in str(w.message) for w in seen), seen
        import torch
        assert m.moe_plan_bytes(1, 512) > 0 and "site-packages" not in m.__file__
        x = torch.zeros(4, 32)
        try:
            m.moe_quant_i8(x, x.to(torch.int8), x[:, 0].contiguous())
        except ValueError as e:
            assert "must be on a GPU" in str(e)
            print("fine", m.__file__)
    """
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, env={**os.environ, "PYTHONPATH": str(tmp_path)},
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and f"fine {tmp_path}" in r.stdout, r.stderr


def test_build_goes_on_without_the_native_binding(tmp_path, monkeypatch, capsys):
    """... and leaves no binding of an older source behind."""
    import importlib.util
    import os
    spec = importlib.util.spec_from_file_location("builder", os.path.join(m._lib.HERE, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    stale = tmp_path / "_dense.so"
    stale.write_bytes(b"old")
    monkeypatch.setattr(b, "BINDING", str(stale))
    monkeypatch.setattr(b, "build_library", lambda verbose: "library")
    monkeypatch.setenv("CXX", str(tmp_path / "no-such-compiler"))
    assert b.build() == "library"
    assert not stale.exists() and "native binding not built" in capsys.readouterr().err


def test_shared_expert_takes_codes_only():
    """Weights that int8 does not hold are refused, not cut to it."""
    from moe_routed_expert_mx_amd.block import SharedExpertI8
    g = torch.Generator().manual_seed(0)
    w13, w2 = (torch.randint(-128, 128, s, generator=g) for s in ((64, 512), (512, 32)))

    def make(a, b):
        return SharedExpertI8(a, torch.ones(64), b, torch.ones(512), B_max=4, device="cpu")

    for t in (torch.int8, torch.int32, F32):
        e = make(w13.to(t), w2.to(t).numpy())
        assert e.w13.dtype == torch.int8 and torch.equal(e.w13.long(), w13) and torch.equal(e.w2.long(), w2)
    half = w13.abs().clamp_max(127).to(torch.uint8)
    assert torch.equal(make(half, w2).w13.long(), half.long())
    for bad in (w13 + 0.25, w13 * 1000, w13 * float("nan"), torch.full((64, 512), 128), w13.to(torch.int8).view(torch.uint8)):
        with pytest.raises(ValueError, match="int8"):
            make(bad, w2)
    with pytest.raises(ValueError, match="int8"):
        make(w13, w2 * 0.01)


def test_gate_weight_on_another_gpu():
    """The packed weight has to be where x and the logits are (here: on no GPU)."""
    import types
    g = m.moe_gate_t(16, 512, 0, 0x1000)
    with pytest.raises(ValueError, match="must be on a GPU"):
        m.moe_gate(g, _z(4, 512, dtype=BF), _z(4, 16))
    g.tensor = types.SimpleNamespace(get_device=lambda: 1)
    with pytest.raises(ValueError, match="must be on one GPU"):
        m.moe_gate(g, _z(4, 512, dtype=BF), _z(4, 16))


@pytest.mark.parametrize("scale", [0, -0.0, 1e-46, -7e-46, 1e39, float("inf"), float("nan")])
def test_route_scale_is_taken_in_fp32(scale):
    """A scale that FP32 holds as 0 is none the library could tell from its default, 1."""
    with pytest.raises(ValueError, match="scale"):
        m.moe_route(_z(4, 16), _z(4, 2, dtype=torch.int32), _z(4, 2), scale=scale)
    with pytest.raises(ValueError, match="must be on a GPU"):
        m.moe_route(_z(4, 16), _z(4, 2, dtype=torch.int32), _z(4, 2), scale=1e-45)


@pytest.mark.parametrize("status", [m._lib.MOE_EHIP, EINVAL])
def test_a_status_of_the_library_is_raised_not_retried(monkeypatch, status):
    """A call that the native binding made may be enqueued whatever its status: made again, moe_linear_i8 with add = out
    would add its product twice."""
    made = []
    for name in ("gate", "route", "quant", "linear"):
        monkeypatch.setattr(m._lib._dense, name, lambda *a: status)
    monkeypatch.setattr(m._lib, "_enqueue", lambda name, *a: made.append(name))
    x, q, s = _z(4, 512, dtype=BF), _z(4, 512, dtype=torch.int8), _z(4)
    out = _z(4, 4)
    for call in (lambda: m.moe_gate(m.moe_gate_t(16, 512, 0, 0x1000), x, _z(4, 16)),
                 lambda: m.moe_route(_z(4, 16), _z(4, 2, dtype=torch.int32), _z(4, 2)),
                 lambda: m.moe_quant_i8(x, q, s), lambda: m.moe_linear_i8(q, s, q, s, out, add=out)):
        with pytest.raises(m.MoeError) as e:
            call()
        assert e.value.status == status and made == []
