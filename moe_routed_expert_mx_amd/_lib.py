"""ctypes binding of libmoe_mx.so (include/moe_mx.h): argument marshalling only.

Every entry point keeps the C name.  Tensors are torch tensors on the GPU (PyTorch is
used for device memory and streams only); every step of the path runs in the HIP
library.  Errors from the library raise ``MoeError``.  There is no fallback: if the
library is not built, importing this module fails.
"""
from __future__ import annotations

import ctypes
import os
import struct
import warnings

# PyTorch first: the library runs on torch's streams and memory, so it must bind to the
# HIP runtime torch has loaded.  Loaded the other way round, the process holds two HIP
# runtimes and launches on torch's streams fail.
import torch  # noqa: F401

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_mx.so")

MOE_OK, MOE_EINVAL, MOE_ENOSPACE, MOE_EHIP, MOE_ELIMIT = 0, -1, -2, -3, -4


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} ({status})")
        self.status = status


class moe_weights_t(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("D", ctypes.c_int32), ("I", ctypes.c_int32),
                ("w13", ctypes.c_void_p), ("s13", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("s2", ctypes.c_void_p)]


class moe_run_opts_t(ctypes.Structure):
    _fields_ = [("hidden_rule", ctypes.c_int32), ("grid", ctypes.c_int32),
                ("col_tiles", ctypes.c_int32), ("ring", ctypes.c_int32), ("exchange", ctypes.c_int32),
                ("fc2_claims", ctypes.c_int32), ("reserved", ctypes.c_int32 * 2),
                ("hidden_codes_dev", ctypes.c_void_p), ("hidden_scales_dev", ctypes.c_void_p),
                ("plan_dev", ctypes.c_void_p), ("plan_bytes", ctypes.c_size_t), ("status_dev", ctypes.c_void_p),
                ("ahead", ctypes.c_void_p), ("ahead_rows", ctypes.c_int32)]


class moe_gate_t(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("D", ctypes.c_int32), ("wtype", ctypes.c_int32), ("packed", ctypes.c_void_p)]


class moe_route_opts_t(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("group_score", ctypes.c_int32), ("renorm", ctypes.c_int32), ("scale", ctypes.c_float),
                ("bias_dev", ctypes.c_void_p), ("reserved", ctypes.c_int32 * 2)]


class moe_linear_opts_t(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("exact", ctypes.c_int32), ("bias_dev", ctypes.c_void_p),
                ("add_dev", ctypes.c_void_p), ("ldadd", ctypes.c_int64)]


class moe_norm_opts_t(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_double), ("residual_dev", ctypes.c_void_p), ("ldr", ctypes.c_int64),
                ("total_dev", ctypes.c_void_p), ("ldt", ctypes.c_int64), ("out_dev", ctypes.c_void_p),
                ("ldo", ctypes.c_int64), ("codes", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("codes_dev", ctypes.c_void_p), ("ldc", ctypes.c_int64), ("scales_dev", ctypes.c_void_p),
                ("lds", ctypes.c_int64)]


class moe_grouped_opts_t(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("gather", ctypes.c_int32), ("scatter", ctypes.c_int32),
                ("exact", ctypes.c_int32), ("pairs_dev", ctypes.c_void_p)]


class moe_prefetch_row_t(ctypes.Structure):
    _fields_ = [("addr", ctypes.c_void_p), ("bytes", ctypes.c_uint64)]


def prefetch_rows(tensors_or_ranges):
    """A next-layer prefetch table (ctypes array of moe_prefetch_row_t, row count) from device
    tensors or (address, bytes) pairs."""
    rows = []
    for t in tensors_or_ranges:
        if isinstance(t, tuple):
            rows.append(moe_prefetch_row_t(t[0], t[1]))
        else:
            rows.append(moe_prefetch_row_t(t.data_ptr(), t.numel() * t.element_size()))
    return (moe_prefetch_row_t * max(len(rows), 1))(*rows), len(rows)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built: run `python moe_routed_expert_mx_amd/build.py` "
                          "(or __graft_entry__.build()) first")
    L = ctypes.CDLL(LIB_PATH)
    c, P = ctypes, ctypes.c_void_p
    sig = {
        "moe_status_string": (c.c_char_p, [c.c_int]),
        "moe_plan_bytes": (c.c_size_t, [c.c_int32, c.c_int32]),
        "moe_units_bytes": (c.c_size_t, [c.c_int32, c.c_int32, c.c_int32]),
        "moe_workspace_bytes": (c.c_size_t, [c.c_int32] * 5),
        "moe_packed_weight_bytes": (c.c_int, [c.c_int32] * 3 + [c.POINTER(c.c_size_t)] * 4),
        "moe_pack_weights": (c.c_int, [c.c_int32] * 3 + [P] * 9),
        "moe_workspace_init": (c.c_int, [P, c.c_size_t, P]),
        "moe_plan": (c.c_int, [P, c.c_int32, c.c_int32, P, c.c_size_t, P]),
        "moe_group": (c.c_int, [P, c.c_int32, c.c_int32, c.c_int32, P, c.c_size_t, P]),
        "moe_plan_group": (c.c_int, [P, P, c.c_int32, c.c_int32, c.c_int32, c.c_int32, P, c.c_size_t, P, c.c_size_t,
                                     P]),
        "moe_units_export": (c.c_int, [P, c.c_size_t, c.c_int32, c.c_int32, c.c_int32, P, P, P,
                                       c.c_int32, P]),
        "moe_experts_run": (c.c_int, [c.POINTER(moe_weights_t), c.POINTER(moe_run_opts_t), P, P, c.c_size_t,
                                      c.c_int32, c.c_int32, P, c.c_size_t, P, c.c_size_t, P]),
        "moe_decode_run": (c.c_int, [c.POINTER(moe_weights_t), c.POINTER(moe_run_opts_t), P, P, c.c_int32,
                                     c.c_int32, P, c.c_size_t, P, c.c_size_t, P]),
        "moe_decode_run_noalloc": (c.c_int, [c.POINTER(moe_weights_t), c.POINTER(moe_run_opts_t), P, P, c.c_int32,
                                             c.c_int32, P, c.c_size_t, P]),
        "moe_combine": (c.c_int, [P, c.c_size_t, P, c.c_int32, c.c_int32, c.c_int32, P, c.c_size_t, P]),
        "moe_gate_packed_bytes": (c.c_size_t, [c.c_int32] * 3),
        "moe_gate_pack": (c.c_int, [P, c.c_int32, c.c_int32, c.c_int32, P, c.c_size_t, P]),
        "moe_gate": (c.c_int, [c.POINTER(moe_gate_t), P, c.c_int64, c.c_int32, P, c.c_int64, P]),
        "moe_route": (c.c_int, [P, c.c_int32, c.c_int64, c.c_int32, c.c_int32, c.c_int32, P, P, P, P]),
        "moe_quant_i8": (c.c_int, [P, c.c_int32, c.c_int64, c.c_int32, c.c_int32, P, c.c_int64, P, P]),
        "moe_linear_i8": (c.c_int, [P, c.c_int64, P, P, c.c_int64, P, c.c_int32, c.c_int32, c.c_int32, P, P, c.c_int32,
                                    c.c_int64, P]),
        "moe_quant_f8": (c.c_int, [P, c.c_int32, c.c_int64, c.c_int32, c.c_int32, P, c.c_int64, P, c.c_int64, P]),
        "moe_rms_norm": (c.c_int, [P, c.c_int32, c.c_int64, c.c_int32, c.c_int32, P, c.c_int32, P, P]),
        "moe_linear_f8": (c.c_int, [P, c.c_int64, P, c.c_int64, P, c.c_int64, P, c.c_int32, c.c_int32, c.c_int32, P, P,
                                    c.c_int32, c.c_int64, P]),
        "moe_lists_ws_bytes": (c.c_size_t, [c.c_int64, c.c_int32]),
        "moe_lists": (c.c_int, [P, c.c_int64, c.c_int32, P, P, P, c.c_size_t, P]),
        "moe_grouped_f8": (c.c_int, [P, c.c_int64, P, c.c_int64, c.c_int64, P, c.c_int64, c.c_int64, P, P, c.c_int64,
                                     c.c_int32, c.c_int32, c.c_int32, P, P, c.c_int32, c.c_int64, c.c_int64, P]),
        "moe_work_split": (c.c_int, [c.c_int32] * 6 + [P, P]),
        "moe_grouped_runs": (c.c_int, [c.c_int32, P, c.c_int32, c.c_int32, c.c_int32, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    return L


lib = _load()
EXPORTED = ("moe_status_string", "moe_plan_bytes", "moe_units_bytes", "moe_workspace_bytes", "moe_packed_weight_bytes",
            "moe_pack_weights", "moe_workspace_init", "moe_plan", "moe_group", "moe_plan_group", "moe_units_export",
            "moe_experts_run", "moe_decode_run", "moe_decode_run_noalloc", "moe_combine", "moe_work_split",
            "moe_grouped_runs", "moe_gate_packed_bytes", "moe_gate_pack", "moe_gate", "moe_route", "moe_quant_i8",
            "moe_linear_i8", "moe_quant_f8", "moe_rms_norm", "moe_linear_f8", "moe_lists_ws_bytes", "moe_lists",
            "moe_grouped_f8")


def status_string(status: int) -> str:
    return lib.moe_status_string(status).decode()


def _check(fn: str, status: int):
    if status != MOE_OK:
        raise MoeError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _nbytes(t):
    return t.numel() * t.element_size()


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


# ------------------------------------------------------------------- entry points
def moe_plan_bytes(B: int, D: int) -> int:
    return lib.moe_plan_bytes(B, D)


def moe_units_bytes(B: int, topk: int, E: int) -> int:
    return lib.moe_units_bytes(B, topk, E)


def moe_workspace_bytes(E: int, D: int, I: int, B_max: int, topk: int) -> int:
    return lib.moe_workspace_bytes(E, D, I, B_max, topk)


def moe_packed_weight_bytes(E: int, D: int, I: int):
    out = [ctypes.c_size_t(0) for _ in range(4)]
    _check("moe_packed_weight_bytes", lib.moe_packed_weight_bytes(E, D, I, *[ctypes.byref(o) for o in out]))
    return tuple(o.value for o in out)


def moe_work_split(form: int, groups: int, D: int, I: int, grid: int, claims_ring: int = 0):
    """Host-side static split of an experts launch: (split [grid, 6], items [groups*I/32, 2])
    as numpy int32 arrays (no device call)."""
    import numpy as np
    split = np.zeros((grid, 6), np.int32)
    items = np.zeros((max(groups * (I // 32), 1), 2), np.int32)
    _check("moe_work_split", lib.moe_work_split(form, groups, D, I, grid, claims_ring, split.ctypes.data,
                                                items.ctypes.data))
    return split, items[:groups * (I // 32)]


def moe_grouped_runs(chunk_cols, D: int, I: int, grid: int):
    """Host-side FC2 runs of the grouped form's three-call launch: [grid, 2] int32
    {first tile, tiles} from the chunks' live column counts (no device call)."""
    import numpy as np
    cols = np.ascontiguousarray(chunk_cols, dtype=np.int32)
    runs = np.zeros((grid, 2), np.int32)
    _check("moe_grouped_runs", lib.moe_grouped_runs(len(cols), cols.ctypes.data if len(cols) else None, D, I, grid,
                                                    runs.ctypes.data))
    return runs


def moe_pack_weights(E, D, I, w13, s13, w2, s2, w13p, s13p, w2p, s2p, stream=None):
    _check("moe_pack_weights", lib.moe_pack_weights(E, D, I, *map(_ptr, (w13, s13, w2, s2, w13p, s13p, w2p, s2p)),
                                                    _stream(stream)))


def moe_workspace_init(ws, stream=None):
    _check("moe_workspace_init", lib.moe_workspace_init(_ptr(ws), _nbytes(ws), _stream(stream)))


def moe_plan(x, plan, stream=None):
    B, D = x.shape
    _check("moe_plan", lib.moe_plan(_ptr(x), B, D, _ptr(plan), _nbytes(plan), _stream(stream)))


def moe_group(ids, E: int, units, stream=None):
    B, K = ids.shape
    _check("moe_group", lib.moe_group(_ptr(ids), B, K, E, _ptr(units), _nbytes(units), _stream(stream)))


def moe_plan_group(x, ids, E: int, plan, units, stream=None):
    """moe_plan and moe_group in one launch."""
    B, D = x.shape
    K = ids.shape[1]
    _check("moe_plan_group", lib.moe_plan_group(_ptr(x), _ptr(ids), B, D, K, E, _ptr(plan), _nbytes(plan),
                                                _ptr(units), _nbytes(units), _stream(stream)))


def moe_units_export(units, B, topk, E, header, unit_expert, unit_rows, stream=None):
    _check("moe_units_export", lib.moe_units_export(_ptr(units), _nbytes(units), B, topk, E, _ptr(header),
                                                    _ptr(unit_expert), _ptr(unit_rows), unit_expert.numel(),
                                                    _stream(stream)))


def _opts(hidden_rule, grid, col_tiles, ring, hidden_codes, hidden_scales, plan=None, status=None, exchange=0,
          fc2_claims=0, ahead=None):
    """ahead: None or (ctypes array of moe_prefetch_row_t, rows), e.g. from prefetch_rows();
    the caller keeps the array alive until the call returns."""
    table, rows = ahead if ahead is not None else (None, 0)
    return moe_run_opts_t(hidden_rule, grid, col_tiles, ring, exchange, fc2_claims, (ctypes.c_int32 * 2)(0, 0),
                          _ptr(hidden_codes), _ptr(hidden_scales), _ptr(plan), 0 if plan is None else _nbytes(plan),
                          _ptr(status), None if table is None else ctypes.cast(table, ctypes.c_void_p), rows)


def moe_experts_run(weights: moe_weights_t, plan, units, B: int, topk: int, ws, out, *, hidden_rule=0, grid=0,
                    col_tiles=0, ring=0, hidden_codes=None, hidden_scales=None, stream=None):
    opts = _opts(hidden_rule, grid, col_tiles, ring, hidden_codes, hidden_scales)
    _check("moe_experts_run", lib.moe_experts_run(ctypes.byref(weights), ctypes.byref(opts), _ptr(plan),
                                                  _ptr(units), _nbytes(units), B, topk, _ptr(ws), _nbytes(ws),
                                                  _ptr(out), _nbytes(out), _stream(stream)))


def moe_decode_run(weights: moe_weights_t, x, ids, ws, out, *, hidden_rule=0, grid=0, ring=0, exchange=0,
                   fc2_claims=0, ahead=None, hidden_codes=None, hidden_scales=None, plan=None, status=None,
                   stream=None):
    """The whole step of a batch in one launch (B <= 8: the decode kernel; B > 8: the
    grouped kernel making its own plan and chunk table): x BF16 [B, D] (or uint16
    bits), ids int32 [B, topk] -> out BF16 [B*topk, D]; optional plan (u8, the moe_plan
    layout) and status (int32 [1]) outputs; exchange 0 (whole-K hidden blocks, the
    default), 1 (tagged partial sums) or 2 (finished split blocks); fc2_claims 1 turns
    on the FC2 tail claims of exchange 0; ahead (from prefetch_rows) names the next layer's
    weights for the whole-K kernel to read into the Infinity Cache."""
    B, K = ids.shape
    opts = _opts(hidden_rule, grid, 0, ring, hidden_codes, hidden_scales, plan, status, exchange, fc2_claims,
                 ahead)
    _check("moe_decode_run", lib.moe_decode_run(ctypes.byref(weights), ctypes.byref(opts), _ptr(x), _ptr(ids), B, K,
                                                _ptr(ws), _nbytes(ws), _ptr(out), _nbytes(out), _stream(stream)))


def moe_decode_run_noalloc(weights: moe_weights_t, x, ids, out, *, hidden_rule=0, grid=0, ring=0, fc2_claims=0,
                           ahead=None, hidden_codes=None, hidden_scales=None, plan=None, status=None, stream=None):
    """moe_decode_run with the library's fixed per-device scratch instead of a workspace
    (no allocation; the whole-K decode form only, MOE_ELIMIT beyond its limits)."""
    B, K = ids.shape
    opts = _opts(hidden_rule, grid, 0, ring, hidden_codes, hidden_scales, plan, status, 0, fc2_claims, ahead)
    _check("moe_decode_run_noalloc", lib.moe_decode_run_noalloc(ctypes.byref(weights), ctypes.byref(opts), _ptr(x),
                                                                _ptr(ids), B, K, _ptr(out), _nbytes(out),
                                                                _stream(stream)))


def moe_combine(rows, weights, out, stream=None):
    """rows: BF16 [B*topk, D] (or uint16 bits), weights: FP32 [B, topk], out: BF16 [B, D]."""
    B, K = weights.shape
    D = rows.shape[-1]
    _check("moe_combine", lib.moe_combine(_ptr(rows), _nbytes(rows), _ptr(weights), B, K, D, _ptr(out), _nbytes(out),
                                          _stream(stream)))


# --------------------------------------------------------------- dense side
# These entry points check their tensors (the library sees pointers only): types, shapes,
# unit stride within rows and one GPU for all of them raise ValueError.  They run on that
# GPU's current stream, whichever GPU is current.  A call takes some microseconds of host
# time, as long as the smallest kernels run, so the native binding (csrc/dense_binding.cpp)
# goes first: it enqueues what is plainly right, and leaves the rest to the code here.  Only what it
# did not take (_NOT_TAKEN) is tried here: another status is the library's own, and a call that it
# may have enqueued is not made a second time (the product of moe_linear_i8 would be added twice).
_MOE_TYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_BF16, _F32, _I32, _I8, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int8, torch.uint8
_ROUTE_OPTS = struct.Struct("@5ifP2i")   # moe_route_opts_t
_LINEAR_OPTS = struct.Struct("@2iPPq")   # moe_linear_opts_t
_NORM_OPTS = struct.Struct("@dPqPqPq2iPqPq")  # moe_norm_opts_t
_GROUPED_OPTS = struct.Struct("@4iP")    # moe_grouped_opts_t
assert _ROUTE_OPTS.size == ctypes.sizeof(moe_route_opts_t) and _LINEAR_OPTS.size == ctypes.sizeof(moe_linear_opts_t)
assert _NORM_OPTS.size == ctypes.sizeof(moe_norm_opts_t) and _GROUPED_OPTS.size == ctypes.sizeof(moe_grouped_opts_t)
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


_NOT_TAKEN = -100


class _NoBinding:
    """In the native binding's place where that is not built: takes no call, so that each goes through ctypes."""

    @staticmethod
    def gate(*args) -> int:
        return _NOT_TAKEN

    route = quant = linear = gate
    norm = quant_f8 = linear_f8 = lists = grouped_f8 = gate


def _load_binding():
    """The native binding, bound to the library.  It makes calls shorter, no more: without it (a build of the HIP
    library alone, or for another PyTorch) the package works, with a warning."""
    try:
        from . import _dense
    except ImportError as e:
        warnings.warn(f"the native binding is not built ({e}): calls of the dense side take 5 to 8 us instead of 3; "
                      "`python moe_routed_expert_mx_amd/build.py` builds it", RuntimeWarning, stacklevel=2)
        return _NoBinding
    addresses = [ctypes.cast(getattr(lib, f), ctypes.c_void_p).value
                 for f in ("moe_gate", "moe_route", "moe_quant_i8", "moe_linear_i8")]
    _dense.bind(*addresses, _current_stream, _current_device)
    _dense.bind_f8(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value
                     for f in ("moe_rms_norm", "moe_quant_f8", "moe_linear_f8", "moe_lists", "moe_grouped_f8")))
    return _dense


_dense = _load_binding()


def _refuse(what: str):
    raise ValueError(what)


def _rows(t, name: str, shape: tuple) -> int:
    """Row distance of a tensor [rows, columns] whose rows are contiguous."""
    if t.shape != shape:
        _refuse(f"{name}: expected {list(shape)}, got {list(t.shape)}")
    ld, inner = t.stride()
    rows, cols = shape
    if inner != 1 and cols != 1:
        _refuse(f"{name}: the elements of a row must be contiguous")
    if rows == 1:
        return cols
    if ld < cols:
        _refuse(f"{name}: rows overlap (stride {ld}, {cols} columns)")
    return ld


def _matrix(t, name: str) -> tuple:
    return t.shape if t.dim() == 2 else _refuse(f"{name}: expected two dimensions, got {t.dim()}")


def _vector(t, name: str, n: int) -> int:
    if t.dtype != _F32 or t.shape != (n,) or (n != 1 and t.stride(0) != 1):
        _refuse(f"{name}: expected contiguous FP32 [{n}]")
    return t.data_ptr()


def _enqueue(name: str, fn, stream, tensors: tuple, *args):
    """Run a library call, its stream appended, on the one GPU that holds the tensors."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != dev:
            _refuse("the tensors must be on one GPU")
    if dev < 0:
        _refuse("the tensors must be on a GPU")
    if stream is None:
        raw = _current_stream(dev)
    elif hasattr(stream, "cuda_stream"):
        raw = stream.cuda_stream
        if stream.device_index != dev:
            _refuse("the stream belongs to another GPU than the tensors")
    else:
        raw = int(stream)
    if _current_device() == dev:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status:
        raise MoeError(name, status)


def moe_gate_packed_bytes(E: int, D: int, wdtype=torch.bfloat16) -> int:
    """Bytes of a packed router weight [E, D] of wdtype (BF16 or FP32); 0 if not supported."""
    return lib.moe_gate_packed_bytes(E, D, _MOE_TYPE.get(wdtype, -1))


def moe_gate_pack(w, packed, stream=None) -> moe_gate_t:
    """Lay a router weight (BF16 or FP32 [E, D], contiguous) out into `packed` (uint8, moe_gate_packed_bytes)
    and return its handle for moe_gate, which keeps `packed` alive."""
    E, D = _matrix(w, "w")
    if w.dtype not in (_BF16, _F32) or not w.is_contiguous():
        _refuse("w: expected contiguous BF16 or FP32 [E, D]")
    if packed.dtype != _U8 or not packed.is_contiguous():
        _refuse("packed: expected contiguous uint8")
    _enqueue("moe_gate_pack", lib.moe_gate_pack, stream, (w, packed), w.data_ptr(), _MOE_TYPE[w.dtype], E, D,
             packed.data_ptr(), packed.numel())
    gate = moe_gate_t(E, D, _MOE_TYPE[w.dtype], packed.data_ptr())
    gate.tensor = packed
    return gate


def moe_gate(gate: moe_gate_t, x, logits, stream=None):
    """Router product: x BF16 [B, D] (rows may be strided) -> logits FP32 [B, E].  gate: from moe_gate_pack; of a
    moe_gate_t filled by hand, the caller sees to it that `packed` is on the GPU of x and stays alive."""
    packed = getattr(gate, "tensor", None)
    if stream is None:
        status = _dense.gate(ctypes.addressof(gate), gate.D, gate.E, x, logits, packed)
        if status != _NOT_TAKEN:
            return _check("moe_gate", status)
    B = _matrix(x, "x")[0]
    if x.dtype != _BF16 or logits.dtype != _F32:
        _refuse("x: expected BF16, logits: FP32")
    ldx, ldl = _rows(x, "x", (B, gate.D)), _rows(logits, "logits", (B, gate.E))
    tensors = (x, logits) if packed is None else (x, logits, packed)
    _enqueue("moe_gate", lib.moe_gate, stream, tensors, gate, x.data_ptr(), ldx, B, logits.data_ptr(), ldl)


_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": 0, "top2": 1}


def moe_route(logits, ids, weights, *, score: str = "softmax", bias=None, groups: int = 0, topk_groups: int = 0,
              group_score: str = "max", renorm: bool = True, scale: float = 1.0, stream=None):
    """Routing: logits [B, E] (FP32, BF16 or FP16) -> ids int32 [B, topk] and weights FP32 [B, topk], the experts of
    the largest choice (score + bias) first, as the expert calls and moe_combine take them.  score "softmax" or
    "sigmoid"; groups experts groups of which topk_groups stay, ranked by group_score "max" or "top2"; renorm
    divides a token's weights by their sum; scale multiplies them."""
    sc, gs = _SCORES.get(score), _GROUP_SCORES.get(group_score)
    if stream is None:
        status = _dense.route(logits, ids, weights, sc, bias, groups, topk_groups, gs, renorm, scale)
        if status != _NOT_TAKEN:
            return _check("moe_route", status)
    shape = _matrix(logits, "logits")
    B, E = shape
    kind = _MOE_TYPE.get(logits.dtype)
    if kind is None or sc is None or gs is None:
        _refuse(f"logits of {logits.dtype}, score {score!r} or group_score {group_score!r} not taken")
    ldl = _rows(logits, "logits", shape)
    out = ids.shape
    if len(out) != 2 or out[0] != B or ids.dtype != _I32 or not ids.is_contiguous():
        _refuse(f"ids: expected contiguous int32 [{B}, topk]")
    if weights.shape != out or weights.dtype != _F32 or not weights.is_contiguous():
        _refuse(f"weights: expected contiguous FP32 {list(out)}")
    if not 0.0 < abs(ctypes.c_float(scale).value) < float("inf"):  # (the library reads 0 as 1)
        _refuse(f"scale {scale!r}: expected a finite FP32 number other than 0")
    tensors, pb = (logits, ids, weights), 0
    if bias is not None:
        tensors, pb = (logits, ids, weights, bias), _vector(bias, "bias", E)
    _enqueue("moe_route", lib.moe_route, stream, tensors, logits.data_ptr(), kind, ldl, B, E, out[1],
             _ROUTE_OPTS.pack(sc, groups, topk_groups, gs, 1 if renorm else 0, scale, pb, 0, 0), ids.data_ptr(),
             weights.data_ptr())


def moe_quant_i8(x, codes, scales, stream=None):
    """Int8 quantization with one scale for each token: x [M, K] (FP32, BF16 or FP16) -> codes int8 [M, K], scales
    FP32 [M]; code * scale stands for x."""
    if stream is None:
        status = _dense.quant(x, codes, scales)
        if status != _NOT_TAKEN:
            return _check("moe_quant_i8", status)
    shape = _matrix(x, "x")
    kind = _MOE_TYPE.get(x.dtype)
    if kind is None or codes.dtype != _I8:
        _refuse(f"x of {x.dtype} or codes of {codes.dtype} not taken")
    ldx, ldc = _rows(x, "x", shape), _rows(codes, "codes", shape)
    M, K = shape
    _enqueue("moe_quant_i8", lib.moe_quant_i8, stream, (x, codes, scales), x.data_ptr(), kind, ldx, M, K,
             codes.data_ptr(), ldc, _vector(scales, "scales", M))


_ACTS = {"none": 0, "swiglu": 1}


def moe_linear_i8(a, a_scales, w, w_scales, out, *, act: str = "none", bias=None, add=None, stream=None):
    """Int8 product with scales for each token and channel: a int8 [M, K], w int8 [N, K] -> out [M, N] (FP32, BF16 or
    FP16), y = (a . w) * a_scales * w_scales + bias (FP32 [N]); act "swiglu": the first N/2 rows of w are the gate,
    the others up, and out is [M, N/2]; add (as out, may be out itself) is added last."""
    mode = _ACTS.get(act)
    if stream is None:
        status = _dense.linear(a, a_scales, w, w_scales, out, mode, bias, add)
        if status != _NOT_TAKEN:
            return _check("moe_linear_i8", status)
    shape, kind = _matrix(a, "a"), _MOE_TYPE.get(out.dtype)
    M, K = shape
    N = _matrix(w, "w")[0]
    if mode is None or kind is None or a.dtype != _I8 or w.dtype != _I8:
        _refuse(f"act {act!r}, a of {a.dtype}, w of {w.dtype} or out of {out.dtype} not taken")
    cols = N
    if mode:
        cols = N // 2
        if N % 2:
            _refuse("w: SwiGLU needs an even number of rows")
    lda, ldw, ldo = _rows(a, "a", shape), _rows(w, "w", (N, K)), _rows(out, "out", (M, cols))
    psa, psw = _vector(a_scales, "a_scales", M), _vector(w_scales, "w_scales", N)
    tensors, pb, pd, ldd = (a, a_scales, w, w_scales, out), 0, 0, 0
    if bias is not None:
        pb = _vector(bias, "bias", N)
        tensors += (bias,)
    if add is not None:
        if add.dtype != out.dtype:
            _refuse(f"add: expected {out.dtype}")
        ldd, pd = _rows(add, "add", (M, cols)), add.data_ptr()
        tensors += (add,)
    _enqueue("moe_linear_i8", lib.moe_linear_i8, stream, tensors, a.data_ptr(), lda, psa, w.data_ptr(), ldw, psw, M, N,
             K, _LINEAR_OPTS.pack(mode, 0, pb, pd, ldd), out.data_ptr(), kind, ldo)


# ------------------------------------------------------------ block-scaled FP8
# e4m3 codes are torch.float8_e4m3fn tensors, their scales FP32 with one column for each 128 of a row.
_F8 = torch.float8_e4m3fn


def _kb(K: int) -> int:
    return (K + 127) // 128


def _blocks_of(t, name: str, shape: tuple):
    """Scales of weight blocks: contiguous FP32."""
    if t.dtype != _F32 or t.shape != shape or not t.is_contiguous():
        _refuse(f"{name}: expected contiguous FP32 {list(shape)}")
    return t.data_ptr()


def _row_scales(t, name: str, shape: tuple) -> int:
    if t.dtype != _F32 or t.dim() != 2:
        _refuse(f"{name}: expected FP32 {list(shape)}")
    return _rows(t, name, shape)


def moe_quant_f8(x, codes, scales, stream=None):
    """Quantization into blocks of 128: x [M, K] (FP32, BF16 or FP16) -> codes float8_e4m3fn [M, K], scales FP32
    [M, ceil(K / 128)], powers of two."""
    if stream is None:
        status = _dense.quant_f8(x, codes, scales)
        if status != _NOT_TAKEN:
            return _check("moe_quant_f8", status)
    shape = _matrix(x, "x")
    kind = _MOE_TYPE.get(x.dtype)
    if kind is None or codes.dtype != _F8:
        _refuse(f"x of {x.dtype} or codes of {codes.dtype} not taken")
    M, K = shape
    ldx, ldc, lds = _rows(x, "x", shape), _rows(codes, "codes", shape), _row_scales(scales, "scales", (M, _kb(K)))
    _enqueue("moe_quant_f8", lib.moe_quant_f8, stream, (x, codes, scales), x.data_ptr(), kind, ldx, M, K,
             codes.data_ptr(), ldc, scales.data_ptr(), lds)


def moe_rms_norm(x, weight, *, out=None, residual=None, total=None, codes=None, scales=None, eps: float = 1e-6,
                 stream=None):
    """Root-mean-square norm of h = x + residual (h = x without one), x [M, K] (FP32, BF16 or FP16), weight [K] (FP32
    or as x).  Outputs, each optional: total [M, K], h itself (may be residual or x); out [M, K], the norm, as x (may
    be x or residual); codes of it in 8 bits, int8 with scales FP32 [M] as moe_quant_i8's, or float8_e4m3fn with
    scales FP32 [M, ceil(K / 128)] as moe_quant_f8's.  One of out and codes at least."""
    if stream is None:
        status = _dense.norm(x, weight, out, residual, total, codes, scales, eps)
        if status != _NOT_TAKEN:
            return _check("moe_rms_norm", status)
    shape = _matrix(x, "x")
    M, K = shape
    kind = _MOE_TYPE.get(x.dtype)
    if kind is None or weight.dtype not in (_F32, x.dtype) or weight.shape != (K,) or (K != 1 and weight.stride(0) != 1):
        _refuse(f"x of {x.dtype} not taken, or weight: expected contiguous FP32 or {x.dtype} [{K}]")
    tensors, at = [x, weight], []
    for t, name in ((residual, "residual"), (total, "total"), (out, "out")):
        if t is None:
            at += [0, 0]
            continue
        if t.dtype != x.dtype:
            _refuse(f"{name}: expected {x.dtype}")
        _matrix(t, name)
        at += [t.data_ptr(), _rows(t, name, shape)]
        tensors.append(t)
    form, pc, ldc, ps, lds = 0, 0, 0, 0, 0
    if codes is not None:
        form = 1 if codes.dtype == _I8 else 2 if codes.dtype == _F8 else _refuse(f"codes of {codes.dtype} not taken")
        if scales is None:
            _refuse("codes without scales")
        _matrix(codes, "codes")
        pc, ldc, ps = codes.data_ptr(), _rows(codes, "codes", shape), scales.data_ptr()
        lds = _row_scales(scales, "scales", (M, _kb(K))) if form == 2 else (_vector(scales, "scales", M), 0)[1]
        tensors += [codes, scales]
    elif scales is not None:
        _refuse("scales without codes")
    if out is None and codes is None:
        _refuse("neither out nor codes")
    if not 0.0 <= eps < float("inf"):
        _refuse(f"eps {eps!r}: expected a finite number, 0 or more")
    _enqueue("moe_rms_norm", lib.moe_rms_norm, stream, tuple(tensors), x.data_ptr(), kind, _rows(x, "x", shape), M, K,
             weight.data_ptr(), _MOE_TYPE[weight.dtype], _NORM_OPTS.pack(eps, *at, form, 0, pc, ldc, ps, lds))


def _f8_weight_blocks(N: int, K: int, mode: int) -> tuple:
    return (2 * ((N // 2 + 127) // 128) if mode else (N + 127) // 128, _kb(K))


def moe_linear_f8(a, a_scales, w, w_scales, out, *, act: str = "none", bias=None, add=None, exact: bool = False,
                  stream=None):
    """Product of block-scaled e4m3 matrices: a float8_e4m3fn [M, K] with scales FP32 [M, ceil(K / 128)], w
    float8_e4m3fn [N, K] with scales FP32 [ceil(N / 128), ceil(K / 128)] -> out [M, N] (FP32, BF16 or FP16), plus bias
    (FP32 [N]); act "swiglu": the first N/2 rows of w are the gate, the others up, each half with scale blocks of its
    own ([2 ceil(N/2 / 128), ..]), and out is [M, N/2]; add (as out, may be out itself) is added last.  K a multiple
    of 16, rows 16-byte aligned.  exact: the codes' products are added in FP32 as they are, as for FP32 outputs always;
    otherwise the FP8 matrix cores cut some 1.5e-5 of a sum off, in as little as half the time.  Ask for it where `out` is
    quantized again."""
    mode = _ACTS.get(act)
    if stream is None:
        status = _dense.linear_f8(a, a_scales, w, w_scales, out, mode, bias, add, exact)
        if status != _NOT_TAKEN:
            return _check("moe_linear_f8", status)
    shape, kind = _matrix(a, "a"), _MOE_TYPE.get(out.dtype)
    M, K = shape
    N = _matrix(w, "w")[0]
    if mode is None or kind is None or a.dtype != _F8 or w.dtype != _F8:
        _refuse(f"act {act!r}, a of {a.dtype}, w of {w.dtype} or out of {out.dtype} not taken")
    if mode and N % 2:
        _refuse("w: SwiGLU needs an even number of rows")
    cols = N // 2 if mode else N
    _matrix(out, "out")
    lda, ldw, ldo = _rows(a, "a", shape), _rows(w, "w", (N, K)), _rows(out, "out", (M, cols))
    ldsa = _row_scales(a_scales, "a_scales", (M, _kb(K)))
    psw = _blocks_of(w_scales, "w_scales", _f8_weight_blocks(N, K, mode))
    tensors, pb, pd, ldd = (a, a_scales, w, w_scales, out), 0, 0, 0
    if bias is not None:
        pb = _vector(bias, "bias", N)
        tensors += (bias,)
    if add is not None:
        if add.dtype != out.dtype:
            _refuse(f"add: expected {out.dtype}")
        _matrix(add, "add")
        ldd, pd = _rows(add, "add", (M, cols)), add.data_ptr()
        tensors += (add,)
    _enqueue("moe_linear_f8", lib.moe_linear_f8, stream, tensors, a.data_ptr(), lda, a_scales.data_ptr(), ldsa,
             w.data_ptr(), ldw, psw, M, N, K, _LINEAR_OPTS.pack(mode, 1 if exact else 0, pb, pd, ldd), out.data_ptr(), kind, ldo)


def moe_lists_ws_bytes(R: int, E: int) -> int:
    """Bytes of moe_lists' workspace for R = B * topk routes over E experts; 0: it needs none."""
    return lib.moe_lists_ws_bytes(R, E)


def _list_tensor(t, name: str, n: int) -> int:
    if t.dtype != _I32 or t.shape != (n,) or not t.is_contiguous():
        _refuse(f"{name}: expected contiguous int32 [{n}]")
    return t.data_ptr()


def moe_lists(ids, offsets, pairs, *, ws=None, stream=None):
    """Routes sorted by expert: ids int32 [B, topk] -> offsets int32 [E + 1], where each expert's routes begin, and
    pairs int32 [B * topk], the routes t * topk + s, ascending within an expert.  Ids outside [0, E) are left out;
    pairs behind offsets[E] are -1.  ws: uint8, moe_lists_ws_bytes(B * topk, E) of them (None where that is 0)."""
    if stream is None:
        status = _dense.lists(ids, offsets, pairs, ws)
        if status != _NOT_TAKEN:
            return _check("moe_lists", status)
    B, K = _matrix(ids, "ids")
    if ids.dtype != _I32 or not ids.is_contiguous():
        _refuse("ids: expected contiguous int32 [B, topk]")
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        _refuse("offsets: expected contiguous int32 [E + 1]")
    E = offsets.shape[0] - 1
    tensors, pw, nw = (ids, offsets, pairs), 0, 0
    po, pp = _list_tensor(offsets, "offsets", E + 1), _list_tensor(pairs, "pairs", B * K)
    if ws is not None and ws.numel():
        if not ws.is_contiguous():
            _refuse("ws: expected contiguous memory")
        pw, nw = ws.data_ptr(), _nbytes(ws)
        tensors += (ws,)
    _enqueue("moe_lists", lib.moe_lists, stream, tensors, ids.data_ptr(), B * K, E, po, pp, pw, nw)


def moe_grouped_f8(a, a_scales, w, w_scales, offsets, out, *, act: str = "none", pairs=None, gather: int = 0,
                   scatter: bool = False, exact: bool = False, stream=None):
    """Products grouped by expert: rows offsets[e] .. offsets[e + 1] - 1 with w[e], w float8_e4m3fn [E, N, K] with
    scales FP32 [E, blocks of rows, ceil(K / 128)], otherwise as moe_linear_f8.  Row i is a[i], or with gather = g
    a[pairs[i] / g] (g = topk: the tokens' rows); its result is out[i], or with scatter out[pairs[i]].  offsets and
    pairs from moe_lists.  Without pairs a and out have a row for each place of the lists."""
    mode = _ACTS.get(act)
    if stream is None:
        status = _dense.grouped_f8(a, a_scales, w, w_scales, offsets, out, mode, pairs, gather, scatter, exact)
        if status != _NOT_TAKEN:
            return _check("moe_grouped_f8", status)
    kind = _MOE_TYPE.get(out.dtype)
    if w.dim() != 3:
        _refuse(f"w: expected three dimensions, got {w.dim()}")
    E, N, K = w.shape
    shape, rows_out = _matrix(a, "a"), _matrix(out, "out")[0]
    if mode is None or kind is None or a.dtype != _F8 or w.dtype != _F8:
        _refuse(f"act {act!r}, a of {a.dtype}, w of {w.dtype} or out of {out.dtype} not taken")
    if mode and N % 2:
        _refuse("w: SwiGLU needs an even number of rows")
    lda, ldo = _rows(a, "a", (shape[0], K)), _rows(out, "out", (rows_out, N // 2 if mode else N))
    ldw = _rows(w[0], "w", (N, K))
    ldwe = w.stride(0) if E > 1 else (N - 1) * ldw + K + 15 & ~15
    if ldwe < (N - 1) * ldw + K:
        _refuse("w: experts overlap")
    ldsa = _row_scales(a_scales, "a_scales", (shape[0], _kb(K)))
    psw = _blocks_of(w_scales, "w_scales", (E, *_f8_weight_blocks(N, K, mode)))
    po = _list_tensor(offsets, "offsets", E + 1)
    tensors, pp, R = (a, a_scales, w, w_scales, offsets, out), 0, min(shape[0], rows_out)
    if gather or scatter:
        if pairs is None:
            _refuse("gather or scatter without pairs")
        R = pairs.numel()
        pp = _list_tensor(pairs, "pairs", R)
        tensors += (pairs,)
    elif pairs is not None:
        _refuse("pairs without gather or scatter")
    _enqueue("moe_grouped_f8", lib.moe_grouped_f8, stream, tensors, a.data_ptr(), lda, a_scales.data_ptr(), ldsa, shape[0],
             w.data_ptr(), ldw, ldwe, psw, po, R, E, N, K, _GROUPED_OPTS.pack(mode, gather, 1 if scatter else 0, 1 if exact else 0, pp),
             out.data_ptr(), kind, ldo, rows_out)
