"""Refusals of the block-scaled FP8 operators: in the library (before any HIP call, with pointers that are never
dereferenced), in the bindings and in the layer's objects (on CPU tensors).  No GPU needed."""
import ctypes

import numpy as np
import pytest
import torch

import f8_ref as ref
import moe_routed_expert_mx_amd as m
from moe_routed_expert_mx_amd import block

L, EINVAL, ENOSPACE = m._lib.lib, m._lib.MOE_EINVAL, m._lib.MOE_ENOSPACE
FAKE, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)
BF, F16, F32, F8, I32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, torch.int32, torch.int8


def test_quant_refusals():
    def quant(x=FAKE, type=0, ldx=200, M=1, K=200, q=FAKE, ldc=200, s=FAKE, lds=2):
        return L.moe_quant_f8(x, type, ldx, M, K, q, ldc, s, lds, None)

    for bad in (dict(x=None), dict(q=None), dict(s=None), dict(type=3), dict(type=-1), dict(ldx=199), dict(ldc=199),
                dict(lds=1), dict(M=0), dict(M=(1 << 22) + 1), dict(K=0), dict(K=131073, ldx=131073, ldc=131073, lds=2000)):
        assert quant(**bad) == EINVAL, bad


def test_norm_refusals():
    def norm(x=FAKE, type=0, ldx=200, M=1, K=200, w=FAKE, wtype=2, **o):
        o = {"out_dev": 0x1000, "ldo": 200, **o}
        return L.moe_rms_norm(x, type, ldx, M, K, w, wtype, ctypes.byref(m.moe_norm_opts_t(**o)), None)

    codes = dict(codes=2, codes_dev=0x1000, ldc=200, scales_dev=0x1000, lds=2)
    for bad in (dict(x=None), dict(w=None), dict(type=3), dict(wtype=1), dict(type=2, wtype=0), dict(ldx=199), dict(M=0),
                dict(M=(1 << 22) + 1), dict(K=0), dict(K=16385, ldx=16385, ldo=16385), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(out_dev=None), dict(ldo=199), dict(residual_dev=0x1000, ldr=199),
                dict(total_dev=0x1000, ldt=100), dict(codes, codes=3), dict(codes, codes=-1), dict(codes, codes_dev=None),
                dict(codes, scales_dev=None), dict(codes, ldc=199), dict(codes, lds=1), dict(codes, codes=1, ldc=10)):
        assert norm(**bad) == EINVAL, bad
    assert L.moe_rms_norm(FAKE, 0, 200, 1, 200, FAKE, 2, None, None) == EINVAL      # no options: no output


LINEAR = dict(a=FAKE, lda=144, sa=FAKE, ldsa=2, w=FAKE, ldw=144, sw=FAKE, N=8, K=144, out=FAKE, type=0, ldo=8)
PRODUCT_BAD = (dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(out=None), dict(type=3), dict(type=-1),
               dict(lda=128), dict(ldw=128), dict(ldsa=1), dict(lda=152), dict(ldw=152), dict(a=ODD), dict(w=ODD), dict(K=136),
               dict(K=0), dict(K=8, lda=16, ldw=16), dict(K=65552, lda=65552, ldw=65552, ldsa=600), dict(lda=1 << 22),
               dict(ldw=1 << 22), dict(ldsa=1 << 22), dict(N=0), dict(N=(1 << 20) + 1, ldo=1 << 21), dict(ldo=7), dict(act=2),
               dict(act=-1), dict(act=1, N=9, ldo=9), dict(act=1, ldo=3))


def test_linear_refusals():
    def linear(M=1, **k):
        p = {**LINEAR, **k}
        opts = m.moe_linear_opts_t(**{n: v for n, v in p.items() if n not in LINEAR})
        return L.moe_linear_f8(p["a"], p["lda"], p["sa"], p["ldsa"], p["w"], p["ldw"], p["sw"], M, p["N"], p["K"],
                               ctypes.byref(opts), p["out"], p["type"], p["ldo"], None)

    for bad in (*PRODUCT_BAD, dict(M=0), dict(M=(1 << 22) + 1), dict(add_dev=0x1000, ldadd=7),
                dict(M=1 << 22, N=1 << 20, ldo=1 << 20)):
        assert linear(**bad) == EINVAL, bad


def test_grouped_refusals():
    def grouped(offsets=FAKE, R=4, E=2, rows=4, out_rows=4, ldwe=8 * 144, **k):
        p = {**LINEAR, **k}
        opts = m.moe_grouped_opts_t(**{n: v for n, v in p.items() if n not in LINEAR})
        return L.moe_grouped_f8(p["a"], p["lda"], p["sa"], p["ldsa"], rows, p["w"], p["ldw"], ldwe, p["sw"], offsets, R, E,
                                p["N"], p["K"], ctypes.byref(opts), p["out"], p["type"], p["ldo"], out_rows, None)

    pairs = dict(pairs_dev=0x1000)
    for bad in (*PRODUCT_BAD, dict(offsets=None), dict(R=0), dict(R=(1 << 26) + 1, rows=1 << 27, out_rows=1 << 27), dict(E=0),
                dict(E=1025), dict(rows=3), dict(out_rows=3), dict(rows=0, gather=2, **pairs), dict(gather=2), dict(scatter=1), pairs,
                dict(gather=-1, **pairs), dict(scatter=2, **pairs), dict(scatter=-1, **pairs), dict(ldwe=7 * 144),
                dict(ldwe=8 * 144 + 8), dict(scatter=1, rows=3, **pairs), dict(gather=2, out_rows=3, **pairs),
                dict(gather=2, rows=1 << 25, **pairs), dict(R=1 << 26, rows=1 << 26, out_rows=1 << 26, N=1 << 15, ldo=1 << 15,
                                                            ldwe=144 << 15), dict(scatter=1, out_rows=0, **pairs)):
        assert grouped(**bad) == EINVAL, bad


def test_lists_refusals_and_workspace():
    def lists(ids=FAKE, R=4, E=2, offsets=FAKE, pairs=FAKE, ws=FAKE, n=0):
        return L.moe_lists(ids, R, E, offsets, pairs, ws, n, None)

    for bad in (dict(ids=None), dict(offsets=None), dict(pairs=None), dict(R=0), dict(R=-1), dict(R=(1 << 26) + 1), dict(E=0),
                dict(E=1025), dict(R=10000, ws=None, n=1 << 20), dict(R=10000, ws=ctypes.c_void_p(0x1002), n=1 << 20)):
        assert lists(**bad) == EINVAL, bad
    need = m.moe_lists_ws_bytes(10000, 160)
    assert need > 0 and lists(R=10000, E=160, n=need - 1) == ENOSPACE
    assert m.moe_lists_ws_bytes(8192, 160) == 0 and m.moe_lists_ws_bytes(0, 160) == 0
    assert m.moe_lists_ws_bytes(1 << 20, 1025) == 0 and m.moe_lists_ws_bytes((1 << 26) + 1, 160) == 0
    assert 0 < m.moe_lists_ws_bytes(1 << 26, 1024) <= 256 * 1024 * 4


def _z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_checks_tensors():
    """Shapes, types, strides and devices are refused with ValueError; the last check is the device, so a call that is
    right but for it names the GPU."""
    x, q, s = _z(4, 272, dtype=BF), _z(4, 272, dtype=F8), _z(4, 3)
    w, n = _z(272), _z(4, 272, dtype=BF)
    wt, sw, out = _z(8, 272, dtype=F8), _z(1, 3), _z(4, 8, dtype=BF)
    ids, o, p = _z(4, 2, dtype=I32), _z(6, dtype=I32), _z(8, dtype=I32)
    we, se, rows = _z(5, 8, 272, dtype=F8), _z(5, 1, 3), _z(8, 8, dtype=BF)
    right = [
        lambda: m.moe_quant_f8(x, q, s),
        lambda: m.moe_quant_f8(_z(4, 600)[:, :272], _z(4, 300, dtype=F8)[:, :272], _z(4, 9)[:, :3]),
        lambda: m.moe_rms_norm(x, w, out=n),
        lambda: m.moe_rms_norm(x, _z(272, dtype=BF), residual=n, total=n, codes=q, scales=s, eps=0.0),
        lambda: m.moe_rms_norm(x, w, codes=_z(4, 272, dtype=I8), scales=_z(4)),
        lambda: m.moe_linear_f8(q, s, wt, sw, out, bias=_z(8), add=out),
        lambda: m.moe_linear_f8(q, s, wt, _z(2, 3), out[:, :4], act="swiglu"),
        lambda: m.moe_lists(ids, o, p),
        lambda: m.moe_grouped_f8(q, s, we, se, o, rows, pairs=p, gather=2, scatter=True),
        lambda: m.moe_grouped_f8(q, s, we, _z(5, 2, 3), o, rows[:4, :4], act="swiglu"),
    ]
    for i, call in enumerate(right):
        with pytest.raises(ValueError, match="must be on a GPU"):
            call()
    wrong = [
        lambda: m.moe_quant_f8(x.double(), q, s),
        lambda: m.moe_quant_f8(x, q.view(I8), s),
        lambda: m.moe_quant_f8(x, q, _z(4, 2)),
        lambda: m.moe_quant_f8(x, q, s.half()),
        lambda: m.moe_quant_f8(x, q, _z(4)),
        lambda: m.moe_quant_f8(x, q, _z(3, 4).t()),
        lambda: m.moe_quant_f8(x[0], q, s),
        lambda: m.moe_quant_f8(x, q[:3], s),
        lambda: m.moe_quant_f8(_z(1, 272, dtype=BF).expand(4, 272), q, s),
        lambda: m.moe_rms_norm(x, w),
        lambda: m.moe_rms_norm(x, w[:271], out=n),
        lambda: m.moe_rms_norm(x, w.half(), out=n),
        lambda: m.moe_rms_norm(x, _z(544)[::2], out=n),
        lambda: m.moe_rms_norm(x, w, out=n.float()),
        lambda: m.moe_rms_norm(x, w, out=n[:3]),
        lambda: m.moe_rms_norm(x, w, out=n, residual=n.half()),
        lambda: m.moe_rms_norm(x, w, out=n, residual=n[:, :271]),
        lambda: m.moe_rms_norm(x, w, out=n, total=_z(272, 4, dtype=BF).t()),
        lambda: m.moe_rms_norm(x, w, out=n, codes=q),
        lambda: m.moe_rms_norm(x, w, out=n, scales=s),
        lambda: m.moe_rms_norm(x, w, codes=q, scales=_z(4)),
        lambda: m.moe_rms_norm(x, w, codes=q.view(I8), scales=s),
        lambda: m.moe_rms_norm(x, w, codes=q.view(torch.uint8), scales=s),
        lambda: m.moe_rms_norm(x, w, out=n, eps=-1e-6),
        lambda: m.moe_rms_norm(x, w, out=n, eps=float("nan")),
        lambda: m.moe_rms_norm(x[0], w, out=n),
        lambda: m.moe_linear_f8(q, s, wt[:, :256], sw, out),
        lambda: m.moe_linear_f8(q.view(I8), s, wt, sw, out),
        lambda: m.moe_linear_f8(q, s, wt.view(I8), sw, out),
        lambda: m.moe_linear_f8(q, s[:, :2], wt, sw, out),
        lambda: m.moe_linear_f8(q, s, wt, sw[0], out),
        lambda: m.moe_linear_f8(q, s, wt, _z(3, 1).t(), out[:, :3]),
        lambda: m.moe_linear_f8(q, s, wt, _z(2, 3), out),
        lambda: m.moe_linear_f8(q, s, wt, sw, out[:, :4], act="swiglu"),
        lambda: m.moe_linear_f8(q, s, wt[:7], _z(2, 3), out[:, :3], act="swiglu"),
        lambda: m.moe_linear_f8(q, s, wt, sw, out, act="gelu"),
        lambda: m.moe_linear_f8(q, s, wt, sw, out.double()),
        lambda: m.moe_linear_f8(q, s, wt, sw, out, bias=_z(7)),
        lambda: m.moe_linear_f8(q, s, wt, sw, out, add=_z(4, 8)),
        lambda: m.moe_linear_f8(q, s, wt, sw, out, add=_z(1, 8, dtype=BF).expand(4, 8)),
        lambda: m.moe_linear_f8(q, s, wt, sw, out[0]),
        lambda: m.moe_lists(ids.long(), o, p),
        lambda: m.moe_lists(ids[0], o, p),
        lambda: m.moe_lists(_z(2, 4, dtype=I32).t(), o, p),
        lambda: m.moe_lists(ids, o[:1], p),
        lambda: m.moe_lists(ids, o.long(), p),
        lambda: m.moe_lists(ids, _z(12, dtype=I32)[::2], p),
        lambda: m.moe_lists(ids, o, p[:7]),
        lambda: m.moe_lists(ids, o, p, ws=_z(64, 2)[:, 0]),
        lambda: m.moe_grouped_f8(q, s, we[0], se, o, rows),
        lambda: m.moe_grouped_f8(q, s, we, se[:4], o, rows),
        lambda: m.moe_grouped_f8(q, s, we, se, o[:5], rows),
        lambda: m.moe_grouped_f8(q, s, we, se, o, rows, gather=2),
        lambda: m.moe_grouped_f8(q, s, we, se, o, rows, scatter=True),
        lambda: m.moe_grouped_f8(q, s, we, se, o, rows, pairs=p),
        lambda: m.moe_grouped_f8(q, s, we, se, o, rows, pairs=p.long(), gather=2),
        lambda: m.moe_grouped_f8(q, s, we, se, o, rows, pairs=p.view(4, 2), gather=2),
        lambda: m.moe_grouped_f8(q, s, we[:1].expand(5, 8, 272), se, o, rows),
        lambda: m.moe_grouped_f8(q, s, we, se, o, rows[:, :7]),
        lambda: m.moe_grouped_f8(q, s, we, se, o, rows, act="gelu"),
        lambda: m.moe_grouped_f8(q[:, :256], s[:, :2], we, se, o, rows),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises(ValueError) as e:
            call()
        assert "must be on a GPU" not in str(e.value), i


def test_native_binding_declines():
    """It enqueues nothing that it is not sure of; the caller's own checks follow."""
    d, no = m._lib._dense, -100
    x, q, s = _z(4, 256, dtype=BF), _z(4, 256, dtype=F8), _z(4, 2)
    assert d.quant_f8(x, q, s) == no and d.quant_f8(x, q, None) == no and d.quant_f8(x, q) == no
    assert d.norm(x, _z(256), x, None, None, None, None, 1e-6) == no
    assert d.norm(x, _z(256), x, None, None, q, None, "eps") == no
    assert d.linear_f8(q, s, q, _z(1, 2), _z(4, 4), 0, None, None) == no
    assert d.lists(_z(4, 2, dtype=I32), _z(3, dtype=I32), _z(8, dtype=I32), None) == no
    assert d.grouped_f8(q, s, _z(2, 4, 256, dtype=F8), _z(2, 1, 2), _z(3, dtype=I32), _z(4, 4), 0, None, 0, False) == no
    assert d.grouped_f8(1, 2, 3, 4, 5, 6, 7, 8, 9, 10) == no
    meta = torch.empty(4, 256, dtype=BF, device="meta")
    assert d.quant_f8(meta, q, s) == no


@pytest.mark.parametrize("status", [m._lib.MOE_EHIP, EINVAL])
def test_a_status_of_the_library_is_raised_not_retried(monkeypatch, status):
    made = []
    for name in ("quant_f8", "norm", "linear_f8", "lists", "grouped_f8"):
        monkeypatch.setattr(m._lib._dense, name, lambda *a: status)
    monkeypatch.setattr(m._lib, "_enqueue", lambda name, *a: made.append(name))
    x, q, s, o = _z(4, 256, dtype=BF), _z(4, 256, dtype=F8), _z(4, 2), _z(3, dtype=I32)
    for call in (lambda: m.moe_quant_f8(x, q, s), lambda: m.moe_rms_norm(x, _z(256), out=x),
                 lambda: m.moe_linear_f8(q, s, q, _z(1, 2), _z(4, 4)), lambda: m.moe_lists(o[:, None], o, o),
                 lambda: m.moe_grouped_f8(q, s, q[None], _z(1, 1, 2), o[:2], _z(4, 4))):
        with pytest.raises(m.MoeError) as e:
            call()
        assert e.value.status == status and made == []


def test_weight_blocks():
    """f8_weight_blocks: scales of 128 x 128, of each half by itself; values within half a step of e4m3."""
    g = torch.Generator().manual_seed(0)
    w = torch.randn(3, 2 * 144, 272, generator=g)
    w[1, 128:144] = 0.0
    for halves in (False, True):
        c, s = block.f8_weight_blocks(w, halves=halves)
        assert c.shape == w.shape and c.dtype == F8 and s.shape == (3, 4 if halves else 3, 3)
        rows = ref.row_blocks(288, halves)
        v = c.double().numpy() * np.repeat(s.double().numpy()[:, rows], 128, axis=2)[:, :, :272]
        top = np.repeat(s.double().numpy()[:, rows], 128, axis=2)[:, :, :272]
        assert np.all(np.abs(v - w.double().numpy()) <= 2.0 ** -4 * 1.001 * np.abs(w.numpy()) + 2.0 ** -10 * top)
        assert s[0, 0, 0] == w[0, :128, :128].abs().max() / 448
    assert block.f8_weight_blocks(w, halves=True)[1][0, 2, 0] == w[0, 144:272, :128].abs().max() / 448
    with pytest.raises(ValueError):
        block.f8_weight_blocks(w[:, :287], halves=True)


def test_objects_refuse_weights_that_do_not_fit():
    w13, s13 = block.f8_weight_blocks(torch.ones(4, 96, 64), halves=True)
    w2, s2 = block.f8_weight_blocks(torch.ones(4, 64, 48))
    cpu = dict(B_max=4, device="cpu")
    block.ExpertsF8(w13, s13, w2, s2, topk=2, **cpu)
    block.SharedExpertF8(w13[0], s13[0], w2[0], s2[0], **cpu)
    for bad in ((w13.float(), s13, w2, s2), (w13, s13[:, :1], w2, s2), (w13[:, :90], s13, w2, s2), (w13, s13, w2[:3], s2),
                (w13, s13, w2[0], s2), (w13, s13, w2, s2[..., None])):
        with pytest.raises(ValueError):
            block.ExpertsF8(*bad, topk=2, **cpu)
    c, s = block.f8_weight_blocks(torch.ones(4, 64, 40))
    with pytest.raises(ValueError, match="16"):
        block.ExpertsF8(w13, s13, c, s, topk=2, **cpu)
    for bad in ((w13[0].float(), s13[0], w2[0], s2[0]), (w13[0], s13[0], w2[0], s2[0].t()[:, :0]), (w13, s13, w2, s2)):
        with pytest.raises(ValueError):
            block.SharedExpertF8(*bad, **cpu)
    with pytest.raises(ValueError):
        block.Norm(torch.ones(2, 3), device="cpu")
    with pytest.raises(ValueError, match="topk"):
        block.MoeBlock(type("R", (), dict(E=4, D=64, topk=3)), block.ExpertsF8(w13, s13, w2, s2, topk=2, **cpu))


def test_reference_rounding():
    """The tests' own e4m3 rounding, by search in the table of its values, is the conversion's."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF).float()
    v = v[v.isfinite() & (v.abs() <= 448)]
    assert np.array_equal(ref.e4m3(v.double().numpy()), v.to(F8).double().numpy())
    c, s = ref.quant(np.array([[448.0, 1.0], [449.0, 1.0], [0.0, 0.0], [np.nan, 1.0]]))
    assert s[:3, 0].tolist() == [1.0, 2.0, 0.0] and np.isnan(s[3, 0]) and c[1].tolist() == [224.0, 0.5] and not c[2:].any()
