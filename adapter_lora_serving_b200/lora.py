"""Thin Python binding of ``liblora_delta.so`` (the C ABI in ``include/lora_delta.h``).

Argument marshalling only: every function here has the C name, passes device
pointers, sizes and the stream straight through, and raises ``LoraError`` on a
non-OK status.  Tensors are ``torch`` tensors on the CUDA device (torch is used
for device memory and streams only); integers are accepted as raw device
pointers.  There is no fallback: if the library is missing, ``load()`` raises.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblora_delta.so")

LORA_OK = 0
LORA_ERR_INVALID = 1
LORA_ERR_UNSUPPORTED = 2
LORA_ERR_WORKSPACE = 3
LORA_ERR_CUDA = 4

LORA_FLAG_BAD_INDPTR = 1
LORA_FLAG_BAD_TOKEN = 2
LORA_FLAG_BAD_RANK = 4
LORA_FLAG_BAD_SLOT = 8
LORA_FLAG_BAD_PAIR = 16
LORA_FLAG_BAD_OFFSETS = 32
LORA_FLAG_TIMEOUT = 64
LORA_FLAG_BAD_EXPERT = 128
LORA_FLAG_BAD_ROW = 256
LORA_FLAG_NONFINITE = 512

LORA_REGIME_AUTO = 0
LORA_REGIME_BGMV = 1
LORA_REGIME_SGMV = 2
LORA_REGIME_BGMV_SPLIT = 3
LORA_REGIME_STREAM = 4

LORA_OP_SHRINK = 0
LORA_OP_EXPAND = 1
LORA_OP_APPLY_LINEAR = 2
LORA_OP_GATHER_SHRINK = 3
LORA_OP_APPLY_EMBEDDING = 4
LORA_OP_EXPERT_APPLY = 5

LORA_TYPE_BF16 = 0
LORA_TYPE_F16 = 1
LORA_TYPE_F32 = 2

LORA_SCORE_SOFTMAX = 0
LORA_SCORE_SIGMOID = 1

LORA_GROUP_MAX = 0
LORA_GROUP_TOP_PAIR = 1

LORA_ACT_NONE = 0
LORA_ACT_SILU_MUL = 1

LORA_ROUTE_MAX_EXPERTS = 1024
LORA_ROUTE_MAX_TOP_K = 32
LORA_ROUTE_MAX_GROUPS = 32

LORA_STATIC_SCRATCH_BYTES = 16 << 20

# (name, restype, argtypes) of every exported symbol.
_P = ctypes.c_void_p
_I = ctypes.c_int32
_Z = ctypes.c_size_t
_F = ctypes.c_float
_SIGS = [
    ("lora_shrink", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]),
    ("lora_expand", _I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _I, _I, _P, _P]),
    ("lora_apply_linear", _I,
     [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _I, _I, _P, _Z, _P, _P]),
    ("lora_apply_linear_noalloc", _I,
     [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _I, _I, _P, _P]),
    ("lora_apply_router", _I,
     [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _Z, _P, _P]),
    ("lora_gather_shrink", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P]),
    ("lora_apply_embedding", _I,
     [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _I, _I, _P, _P]),
    ("lora_expert_apply", _I,
     [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _I, _P, _Z, _P, _P]),
    ("lora_route_experts", _I,
     [_P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P]),
    ("lora_group_experts", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
    ("lora_mx_quantize", _I, [_P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    ("lora_mx_dequantize", _I, [_P, _P, _P, _I, _I, _I, _P]),
    ("lora_mx_linear", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    ("lora_mx_expert_linear", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P]),
    ("lora_combine_experts", _I, [_P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    ("lora_workspace_bytes", _Z, [_I, _I, _I, _I, _I, _I]),
    ("lora_resolve_regime", _I, [_I, _I, _I, _I, _I]),
    ("lora_plan_tile", _I, [_I, _I]),
    ("lora_plan_linear", _I, [_P, _P, _P, _I, _I, _I, _I, _P, _I, _P, _P, _P]),
    ("lora_plan_expert", _I, [_P, _P, _I, _I, _I, _I, _P, _I, _P, _P, _P]),
    ("lora_set_launch_overlap", _I, [_I]),
    ("lora_set_wait_limit_ns", ctypes.c_uint64, [ctypes.c_uint64]),
    ("lora_status_string", ctypes.c_char_p, [_I]),
    ("lora_last_error", ctypes.c_char_p, []),
    ("lora_version", ctypes.c_char_p, []),
]
EXPORTED = [s[0] for s in _SIGS]

_lib = None


class LoraError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{message} ({status})")
        self.status = status


def load(path: str | None = None):
    """Load the library once; raises if it is missing (there is no fallback)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with python -m adapter_lora_serving_b200.build")
    lib = ctypes.CDLL(p)
    for name, res, args in _SIGS:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _slices(out_slices):
    arr = (ctypes.c_int32 * len(out_slices))(*[int(v) for v in out_slices])
    return arr


def _check(status):
    if status != LORA_OK:
        lib = load()
        raise LoraError(lib.lora_status_string(status).decode(),
                        lib.lora_last_error().decode())


def lora_shrink(x, h, a, ranks, token_order, slot_indptr, T, in_features, slots, R,
                num_slices, regime=LORA_REGIME_AUTO, err_flags=None, stream=None):
    _check(load().lora_shrink(_ptr(x), _ptr(h), _ptr(a), _ptr(ranks), _ptr(token_order),
                              _ptr(slot_indptr), T, in_features, slots, R, num_slices, regime,
                              _ptr(err_flags), _stream(stream)))


def lora_expand(y, h, b, ranks, scalings, token_order, slot_indptr, T, slots, R, out_slices,
                regime=LORA_REGIME_AUTO, err_flags=None, stream=None):
    _check(load().lora_expand(_ptr(y), _ptr(h), _ptr(b), _ptr(ranks), _ptr(scalings),
                              _ptr(token_order), _ptr(slot_indptr), T, slots, R,
                              _slices(out_slices), len(out_slices), regime, _ptr(err_flags),
                              _stream(stream)))


def lora_apply_linear(x, y, a, b, ranks, scalings, token_order, slot_indptr, T, in_features,
                      slots, R, out_slices, regime=LORA_REGIME_AUTO, workspace=None,
                      workspace_bytes=0, err_flags=None, stream=None):
    _check(load().lora_apply_linear(_ptr(x), _ptr(y), _ptr(a), _ptr(b), _ptr(ranks),
                                    _ptr(scalings), _ptr(token_order), _ptr(slot_indptr), T,
                                    in_features, slots, R, _slices(out_slices), len(out_slices),
                                    regime, _ptr(workspace), workspace_bytes, _ptr(err_flags),
                                    _stream(stream)))


def lora_apply_linear_noalloc(x, y, a, b, ranks, scalings, token_order, slot_indptr, T,
                              in_features, slots, R, out_slices, regime=LORA_REGIME_AUTO,
                              err_flags=None, stream=None):
    """lora_apply_linear without a workspace, for callers that cannot allocate
    device memory: the library's fixed scratch array is used instead."""
    _check(load().lora_apply_linear_noalloc(_ptr(x), _ptr(y), _ptr(a), _ptr(b), _ptr(ranks),
                                            _ptr(scalings), _ptr(token_order),
                                            _ptr(slot_indptr), T, in_features, slots, R,
                                            _slices(out_slices), len(out_slices), regime,
                                            _ptr(err_flags), _stream(stream)))


def lora_apply_router(router_in, gate_logits, a, b, ranks, scalings, token_order, slot_indptr,
                      T, hidden, slots, R, num_experts, regime=LORA_REGIME_AUTO, workspace=None,
                      workspace_bytes=0, err_flags=None, stream=None):
    _check(load().lora_apply_router(_ptr(router_in), _ptr(gate_logits), _ptr(a), _ptr(b),
                                    _ptr(ranks), _ptr(scalings), _ptr(token_order),
                                    _ptr(slot_indptr), T, hidden, slots, R, num_experts, regime,
                                    _ptr(workspace), workspace_bytes, _ptr(err_flags),
                                    _stream(stream)))


def lora_gather_shrink(ids, h, a, ranks, token_order, slot_indptr, T, vocab, slots, R,
                       num_slices, err_flags=None, stream=None):
    _check(load().lora_gather_shrink(_ptr(ids), _ptr(h), _ptr(a), _ptr(ranks),
                                     _ptr(token_order), _ptr(slot_indptr), T, vocab, slots, R,
                                     num_slices, _ptr(err_flags), _stream(stream)))


def lora_apply_embedding(ids, y, a, b, ranks, scalings, token_order, slot_indptr, T, vocab,
                         slots, R, out_slices, regime=LORA_REGIME_AUTO, err_flags=None,
                         stream=None):
    _check(load().lora_apply_embedding(_ptr(ids), _ptr(y), _ptr(a), _ptr(b), _ptr(ranks),
                                       _ptr(scalings), _ptr(token_order), _ptr(slot_indptr), T,
                                       vocab, slots, R, _slices(out_slices), len(out_slices),
                                       regime, _ptr(err_flags), _stream(stream)))


def lora_expert_apply(x_sorted, y_sorted, a, b, pair_index, ranks, scalings, row_slot,
                      expert_offsets, rows_cap, in_features, num_experts, slots, num_pairs, R,
                      out_slices, workspace=None, workspace_bytes=0, err_flags=None,
                      stream=None):
    _check(load().lora_expert_apply(_ptr(x_sorted), _ptr(y_sorted), _ptr(a), _ptr(b),
                                    _ptr(pair_index), _ptr(ranks), _ptr(scalings),
                                    _ptr(row_slot), _ptr(expert_offsets), rows_cap, in_features,
                                    num_experts, slots, num_pairs, R, _slices(out_slices),
                                    len(out_slices), _ptr(workspace), workspace_bytes,
                                    _ptr(err_flags), _stream(stream)))


# The routed layer's entry points below look at the tensors they are given: a
# tensor's type, size, contiguity and device are checked (LORA_ERR_INVALID), its
# element type picks `type`, and the call runs on the tensors' device and that
# device's current stream.  Raw device pointers (ints) are passed unchecked, on
# the current device.  They are short (a call's host time is that of a small
# batch's kernel), so the checks are plain loops without closures or objects.

_torch = None      # the torch module and its element types, once a tensor is given
_dtypes = None
_kinds = None
_raw_stream = None
_current_device = None


def _import_torch():
    global _torch, _dtypes, _kinds, _raw_stream, _current_device
    import torch
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    # (a tensor on a CUDA device is there: no need to look whether CUDA is set up)
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _dtypes = {LORA_TYPE_BF16: torch.bfloat16, LORA_TYPE_F16: torch.float16,
               LORA_TYPE_F32: torch.float32, "int32": torch.int32, "uint8": torch.uint8}
    _kinds = {torch.bfloat16: LORA_TYPE_BF16, torch.float16: LORA_TYPE_F16,
              torch.float32: LORA_TYPE_F32}
    _torch = torch
    return torch


def _refuse(op, what):
    raise LoraError("LORA_ERR_INVALID", f"{op}: {what}")


def _pointers(op, tensors, kinds, least, names):
    """Device pointers of the tensors (None and ints as they are) and the index
    of their device (None: no tensor among them).  kinds: "int32", "uint8" or an
    LORA_TYPE_*; least: elements a tensor must have."""
    ptrs, dev = [], None
    dtypes = _dtypes
    for t, kind, n in zip(tensors, kinds, least):
        if t is None or t.__class__ is int:
            ptrs.append(t)
            continue
        if dtypes is None:
            _import_torch()
            dtypes = _dtypes
        d = t.get_device()
        if dev is None:
            dev = d
        if (t.dtype is not dtypes.get(kind) or d != dev or d < 0 or not t.is_contiguous()
                or t.numel() < n):
            _explain(op, names[len(ptrs)], t, dtypes.get(kind), dev, n)
        ptrs.append(t.data_ptr())
    return ptrs, dev


def _explain(op, name, t, dtype, dev, least):
    """Raises, saying what is wrong with a tensor."""
    if t.dtype is not dtype:
        _refuse(op, f"{name} has element type {t.dtype}")
    if t.get_device() < 0:
        _refuse(op, f"{name} is not on a CUDA device")
    if t.get_device() != dev:
        _refuse(op, f"{name} is on device {t.get_device()}, not on {dev}")
    if not t.is_contiguous():
        _refuse(op, f"{name} is not contiguous")
    _refuse(op, f"{name} has {t.numel()} elements, fewer than {least}")


def _call(fn, dev, stream, *args):
    """fn(*args, stream) on device `dev` (None: the current one) and `stream`
    (None: that device's current stream); raises on a non-OK status."""
    if stream is not None and stream.__class__ is not int:
        stream = stream.cuda_stream
    if dev is not None and dev != _current_device():
        with _torch.cuda.device(dev):
            _check(fn(*args, _torch.cuda.current_stream().cuda_stream if stream is None
                      else stream))
        return
    if stream is None:
        # the raw handle: torch.cuda.current_stream() builds an object around it,
        # which costs more than the rest of a call
        stream = _raw_stream(dev) if _raw_stream is not None and dev is not None else _stream(None)
    status = fn(*args, stream)
    if status != LORA_OK:
        _check(status)


def _type_of(op, name, t, given):
    """The LORA_TYPE_* of a tensor (`given` for raw pointers)."""
    if given is not None:
        return given
    if _torch is None:
        _import_torch()
    kind = _kinds.get(getattr(t, "dtype", None))
    if kind is None:
        _refuse(op, f"{name} has no element type of LORA_TYPE_*"
                    " (a raw pointer needs the `type` argument)")
    return kind


_ROUTE = ("logits", "bias", "topk_ids", "topk_weights", "err_flags")


def lora_route_experts(logits, bias, topk_ids, topk_weights, T, num_experts, top_k,
                       score=LORA_SCORE_SOFTMAX, num_groups=1, top_groups=1,
                       group_score=LORA_GROUP_MAX, renormalize=True, scale=1.0, type=None,
                       err_flags=None, stream=None):
    """Chosen experts and their weights from routing logits (after
    lora_apply_router)."""
    kind = _type_of("lora_route_experts", "logits", logits, type)
    n = T * top_k
    (lp, bp, ip, wp, fp), dev = _pointers(
        "lora_route_experts", (logits, bias, topk_ids, topk_weights, err_flags),
        (kind, LORA_TYPE_F32, "int32", LORA_TYPE_F32, "int32"),
        (T * num_experts, num_experts, n, n, 1), _ROUTE)
    _call((_lib or load()).lora_route_experts, dev, stream, lp, kind, bp, ip, wp, T, num_experts,
          top_k, score, num_groups, top_groups, group_score, 1 if renormalize else 0, scale, fp)


_GROUP = ("topk_ids", "token_slot", "expert_offsets", "row_token", "pair_row", "row_slot",
          "err_flags")


def lora_group_experts(topk_ids, token_slot, expert_offsets, row_token, pair_row, row_slot, T,
                       top_k, num_experts, err_flags=None, stream=None):
    """Sorts the (token, choice) pairs by expert: offsets, row <-> pair indices
    and the adapter slot of every sorted row."""
    n = T * top_k
    (ip, sp, op, tp, pp, rp, fp), dev = _pointers(
        "lora_group_experts",
        (topk_ids, token_slot, expert_offsets, row_token, pair_row, row_slot, err_flags),
        ("int32",) * 7, (n, T, num_experts + 1, n, n, n, 1), _GROUP)
    _call((_lib or load()).lora_group_experts, dev, stream, ip, sp, op, tp, pp, rp, T, top_k,
          num_experts, fp)


_QUANTIZE = ("x", "codes", "scales", "row_index", "row_count", "rows_out", "err_flags")


def lora_mx_quantize(x, codes, scales, rows, features, row_index=None, row_count=None,
                     rows_out=None, activation=LORA_ACT_NONE, x_rows=None, type=None,
                     err_flags=None, stream=None):
    """Rows of x (gathered by row_index, or after SwiGLU) as MXFP4 codes and
    scales.  x_rows: rows of x, by default those of the tensor (with a raw
    pointer: `rows`)."""
    kind = _type_of("lora_mx_quantize", "x", x, type)
    pitch = features * 2 if activation == LORA_ACT_SILU_MUL else features
    if x_rows is None:
        x_rows = rows if x is None or x.__class__ is int or pitch <= 0 else x.numel() // pitch
    n = rows * features
    (xp, cp, sp, ip, np, op, fp), dev = _pointers(
        "lora_mx_quantize", (x, codes, scales, row_index, row_count, rows_out, err_flags),
        (kind, "uint8", "uint8", "int32", "int32", kind, "int32"),
        (x_rows * pitch, n // 2, n // 32, rows, 1, n, 1), _QUANTIZE)
    _call((_lib or load()).lora_mx_quantize, dev, stream, xp, kind, ip, np, op, cp, sp, x_rows,
          rows, features, activation, fp)


_DEQUANTIZE = ("codes", "scales", "out")


def lora_mx_dequantize(codes, scales, out, rows, features, type=None, stream=None):
    """The values that MXFP4 codes and scales stand for."""
    kind = _type_of("lora_mx_dequantize", "out", out, type)
    n = rows * features
    (cp, sp, op), dev = _pointers("lora_mx_dequantize", (codes, scales, out),
                                  ("uint8", "uint8", kind), (n // 2, n // 32, n), _DEQUANTIZE)
    _call((_lib or load()).lora_mx_dequantize, dev, stream, cp, sp, op, kind, rows, features)


_LINEAR = ("x_codes", "x_scales", "w_codes", "w_scales", "y", "err_flags")


def lora_mx_linear(x_codes, x_scales, w_codes, w_scales, y, rows, in_features, out_features,
                   type=None, err_flags=None, stream=None):
    """y = x w^T of MXFP4 operands (a base projection)."""
    kind = _type_of("lora_mx_linear", "y", y, type)
    n, m = rows * in_features, out_features * in_features
    (xc, xs, wc, ws, yp, fp), dev = _pointers(
        "lora_mx_linear", (x_codes, x_scales, w_codes, w_scales, y, err_flags),
        ("uint8", "uint8", "uint8", "uint8", kind, "int32"),
        (n // 2, n // 32, m // 2, m // 32, rows * out_features, 1), _LINEAR)
    _call((_lib or load()).lora_mx_linear, dev, stream, xc, xs, wc, ws, yp, kind, rows,
          in_features, out_features, fp)


_EXPERT_LINEAR = ("x_codes", "x_scales", "w_codes", "w_scales", "expert_offsets", "y", "err_flags")


def lora_mx_expert_linear(x_codes, x_scales, w_codes, w_scales, expert_offsets, y, rows_cap,
                          in_features, out_features, num_experts, type=None, err_flags=None,
                          stream=None):
    """The experts' products over rows sorted by expert."""
    kind = _type_of("lora_mx_expert_linear", "y", y, type)
    n, m = rows_cap * in_features, num_experts * out_features * in_features
    (xc, xs, wc, ws, ep, yp, fp), dev = _pointers(
        "lora_mx_expert_linear",
        (x_codes, x_scales, w_codes, w_scales, expert_offsets, y, err_flags),
        ("uint8", "uint8", "uint8", "uint8", "int32", kind, "int32"),
        (n // 2, n // 32, m // 2, m // 32, num_experts + 1, rows_cap * out_features, 1),
        _EXPERT_LINEAR)
    _call((_lib or load()).lora_mx_expert_linear, dev, stream, xc, xs, wc, ws, ep, yp, kind,
          rows_cap, in_features, out_features, num_experts, fp)


_COMBINE = ("y_sorted", "pair_row", "topk_weights", "residual", "out", "err_flags")


def lora_combine_experts(y_sorted, pair_row, topk_weights, residual, out, T, top_k, rows_cap,
                         features, type=None, err_flags=None, stream=None):
    """Each token's expert rows weighted and added (onto a residual)."""
    kind = _type_of("lora_combine_experts", "out", out, type)
    n, m = T * top_k, T * features
    (yp, pp, wp, rp, op, fp), dev = _pointers(
        "lora_combine_experts", (y_sorted, pair_row, topk_weights, residual, out, err_flags),
        (kind, "int32", LORA_TYPE_F32, kind, kind, "int32"),
        (rows_cap * features, n, n, m, m, 1), _COMBINE)
    _call((_lib or load()).lora_combine_experts, dev, stream, yp, kind, pp, wp, rp, op, T, top_k,
          rows_cap, features, fp)


def lora_workspace_bytes(op, T, slots, R, num_slices, regime=LORA_REGIME_AUTO):
    return int(load().lora_workspace_bytes(op, T, slots, R, num_slices, regime))


def lora_resolve_regime(op, T, slots, R, num_slices):
    return int(load().lora_resolve_regime(op, T, slots, R, num_slices))


def lora_plan_tile(op, regime):
    return int(load().lora_plan_tile(op, regime))


def lora_plan_linear(slot_indptr, ranks, scalings, T, slots, R, tile, plan_out, plan_cap,
                     plan_count, err_flags=None, stream=None):
    _check(load().lora_plan_linear(_ptr(slot_indptr), _ptr(ranks), _ptr(scalings), T, slots, R,
                                   tile, _ptr(plan_out), plan_cap, _ptr(plan_count),
                                   _ptr(err_flags), _stream(stream)))


def lora_plan_expert(expert_offsets, pair_index, rows_cap, num_experts, slots, max_rows,
                     plan_out, plan_cap, plan_count, err_flags=None, stream=None):
    _check(load().lora_plan_expert(_ptr(expert_offsets), _ptr(pair_index), rows_cap,
                                   num_experts, slots, max_rows, _ptr(plan_out), plan_cap,
                                   _ptr(plan_count), _ptr(err_flags), _stream(stream)))


def lora_set_launch_overlap(enable):
    """Opt in or out of overlapping the fused few-tokens kernel's start with
    the preceding kernel in the stream; returns the previous setting."""
    return int(load().lora_set_launch_overlap(1 if enable else 0))


def lora_set_wait_limit_ns(ns):
    """Limit (ns) of the split kernel's bounded device waits; 0 = the default
    of one second.  Returns the previous setting."""
    return int(load().lora_set_wait_limit_ns(int(ns)))


def lora_version():
    return load().lora_version().decode()
