"""Thin ctypes binding of the C ABI in include/pw.h.

Argument marshalling only: every step of the layer runs in the CUDA library
``libpw_b200.so`` (built by ``any_precision_weight_pw_b200.build``).  PyTorch
supplies device memory, pinned host memory and streams.  There is no CPU or
PyTorch fallback: if the library is missing, loading raises.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import List, Optional, Sequence

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpw_b200.so")

PW_MAX_BITS = 8
STATUS = {0: "PW_OK", 1: "PW_ERR_INVALID_ARG", 2: "PW_ERR_CUDA", 3: "PW_ERR_OOM",
          4: "PW_ERR_TIMEOUT", 5: "PW_ERR_STATE", 6: "PW_ERR_UNSUPPORTED"}
EXPORTED = ["pw_moe_create", "pw_set_block_bits", "pw_moe_forward", "pw_destroy",
            "pw_moe_forward_host", "pw_linear", "pw_get_block_bits", "pw_get_routing",
            "pw_check_device_error", "pw_profile_enable", "pw_profile_read",
            "pw_forward_launches", "pw_plane_bytes", "pw_repack_planes", "pw_route_static",
            "pw_get_forward_bits", "pw_set_switch_lag", "pw_routing_stats", "pw_plan_release",
            "pw_enable_paging", "pw_resident_bytes", "pw_workspace_bytes", "pw_compact_pages",
            "pw_last_error", "pw_abi_version", "pw_route_geometry", "pw_add_rms_norm",
            "pw_token_logprobs", "pw_adapters", "pw_adapters_workspace_bytes", "pw_moe_forward_norm"]


class PwError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s: %s" % (STATUS.get(status, status), message))
        self.status = status


class Config(C.Structure):
    _fields_ = [("hidden", C.c_int32), ("ffn", C.c_int32), ("n_experts", C.c_int32),
                ("top_k", C.c_int32), ("shared_ffn", C.c_int32), ("n_max", C.c_int32),
                ("renorm_topk", C.c_int32), ("max_tokens", C.c_int32)]


class PlanBlock(C.Structure):
    _fields_ = [("bits", C.c_int32), ("min_bits", C.c_int32), ("plane_bytes", C.c_int64),
                ("rows", C.c_int32), ("mass", C.c_double), ("resid", C.c_double),
                ("sens", C.c_double * (PW_MAX_BITS + 1))]


class BlockDesc(C.Structure):
    _fields_ = [("d_planes", C.c_void_p), ("d_lut", C.c_void_p * 2), ("h_planes", C.c_void_p),
                ("h_lut", C.c_void_p * (PW_MAX_BITS + 1)), ("bits", C.c_int32)]


_lib = None


def lib():
    """Load libpw_b200.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libpw_b200.so is missing; build it with "
                               "any_precision_weight_pw_b200.build.build()")
        L = C.CDLL(LIB_PATH)
        P, i32 = C.c_void_p, C.c_int32
        L.pw_moe_create.argtypes = [C.POINTER(Config), C.POINTER(BlockDesc), i32, C.POINTER(P)]
        L.pw_set_block_bits.argtypes = [P, i32, i32, P]
        L.pw_moe_forward.argtypes = [P, P, i32, P, P, P, P]
        L.pw_destroy.argtypes = [P]
        L.pw_moe_forward_host.argtypes = [P, P, i32, P, P, P, P]
        L.pw_linear.argtypes = [P, P, i32, i32, i32, i32, P, i32, P, P]
        L.pw_get_block_bits.argtypes = [P, i32, C.POINTER(i32), C.POINTER(i32)]
        L.pw_get_forward_bits.argtypes = [P, C.POINTER(i32), i32]
        L.pw_set_switch_lag.argtypes = [P, i32]
        L.pw_routing_stats.argtypes = [P, P, P, i32, P]
        L.pw_enable_paging.argtypes = [P, P]
        L.pw_compact_pages.argtypes = [P, P]
        L.pw_workspace_bytes.argtypes = [C.POINTER(Config), C.POINTER(C.c_int64)]
        L.pw_resident_bytes.argtypes = [P, C.POINTER(C.c_int64), C.POINTER(C.c_int64)]
        L.pw_plan_release.argtypes = [C.POINTER(PlanBlock), i32, C.c_int64, C.POINTER(i32),
                                      C.POINTER(C.c_int64), C.POINTER(C.c_double),
                                      C.POINTER(i32)]
        L.pw_get_routing.argtypes = [P, P, P, P]
        L.pw_check_device_error.argtypes = [P]
        L.pw_profile_enable.argtypes = [P, i32]
        L.pw_profile_read.argtypes = [P, C.POINTER(C.c_float), i32, C.POINTER(i32)]
        L.pw_forward_launches.argtypes = [P, i32]
        L.pw_forward_launches.restype = i32
        L.pw_plane_bytes.argtypes = [i32, i32]
        L.pw_plane_bytes.restype = C.c_int64
        L.pw_repack_planes.argtypes = [P, P, i32, i32, i32, P]
        L.pw_route_static.argtypes = [P, P, P, i32, i32, i32, i32, i32, P, P, P]
        L.pw_route_geometry.argtypes = [i32, i32, i32, i32, C.POINTER(C.c_int64)]
        i64 = C.c_int64
        L.pw_add_rms_norm.argtypes = [P, i32, i64, P, i32, i64, P, i32, C.c_float, i32, i32, P,
                                      i64, P, i32, i64, P, i32, P]
        L.pw_token_logprobs.argtypes = [P, i32, i64, i32, i32, P, i32, P, P, P, P, P]
        L.pw_adapters.argtypes = [P, i64, P, P, P, P, P, i32, i32, i32, i32, i32, P, i64, P, i32,
                                  i64, P, i64, P]
        L.pw_adapters_workspace_bytes.argtypes = [i32, i32, i32]
        L.pw_adapters_workspace_bytes.restype = i64
        L.pw_moe_forward_norm.argtypes = [P, P, P, P, C.c_float, i32, P, P, P, P, P]
        L.pw_last_error.restype = C.c_char_p
        L.pw_abi_version.restype = i32
        for name in EXPORTED:
            if name not in ("pw_forward_launches", "pw_last_error", "pw_abi_version",
                            "pw_plane_bytes", "pw_adapters_workspace_bytes"):
                getattr(L, name).restype = C.c_int
        _lib = L
    return _lib


def check(status: int) -> None:
    if status != 0:
        raise PwError(status, lib().pw_last_error().decode())


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def plane_bytes(rows: int, cols: int) -> int:
    """Bytes of one plane page of a rows x cols block."""
    return int(lib().pw_plane_bytes(rows, cols))


def repack_planes(planes, cols: int, stream=None):
    """Row-major planes (int32 device tensor [n][rows][ceil(cols/32)], uint32
    bit patterns) -> the paged layout of an n-plane block (flat int32 device
    tensor of n * plane_bytes / 4 words)."""
    import torch
    n, rows, _ = planes.shape
    out = torch.empty(n * plane_bytes(rows, cols) // 4, dtype=torch.int32, device=planes.device)
    check(lib().pw_repack_planes(_ptr(planes), _ptr(out), rows, cols, n, _stream(stream)))
    return out


def linear(planes, lut, bits: int, x, rows: int, y=None, stream=None, adapters=None,
           adapter_ids=None):
    """y[t][o] = sum_i W_b[o][i] x[t][i] for one block.  planes: a block in
    the paged layout (repack_planes; its plane count follows from its size);
    lut: int16 [rows][2^bits] (fp16 bit patterns); x: bf16 [T][cols].
    Returns fp32 [T][rows].  With adapters (the keyword arguments of
    add_adapters: a, b and optionally scale, ranks) and adapter_ids, every
    token's low-rank adapter is added to y in place; the adapters, x and y
    (fp32, contiguous) are then checked before anything is enqueued."""
    import torch
    if adapters is not None:
        return _linear_with_adapters(planes, lut, bits, x, rows, y, stream, adapters, adapter_ids)
    if adapter_ids is not None:
        raise PwError(1, "adapter_ids: needs adapters")
    T, cols = x.shape
    n_max = planes.numel() * 4 // plane_bytes(rows, cols)
    if y is None:
        y = torch.empty((T, rows), dtype=torch.float32, device=x.device)
    check(lib().pw_linear(_ptr(planes), _ptr(lut), rows, cols, n_max, bits, _ptr(x), T, _ptr(y),
                          _stream(stream)))
    return y


def route_static(x, router_w, top_k: int, renorm_topk: int, router_bias=None, idx=None, w=None,
                 stream=None):
    """Routing alone through pw_route_static (no device allocation inside
    the library): x bf16 [T][H], router_w fp32 [E][H] -> (idx int32 [T][k],
    w fp32 [T][k]).  Pass idx / w to reuse output buffers."""
    import torch
    T, H = x.shape
    E = router_w.shape[0]
    if idx is None:
        idx = torch.empty((T, top_k), dtype=torch.int32, device=x.device)
    if w is None:
        w = torch.empty((T, top_k), dtype=torch.float32, device=x.device)
    check(lib().pw_route_static(_ptr(x), _ptr(router_w), _ptr(router_bias), T, H, E, top_k,
                                renorm_topk, _ptr(idx), _ptr(w), _stream(stream)))
    return idx, w


def route_geometry(T: int, E: int, H: int, top_k: int) -> dict:
    """The route kernel's launch geometry for a shape (host arithmetic)."""
    out = (C.c_int64 * 12)()
    check(lib().pw_route_geometry(T, E, H, top_k, out))
    keys = ("cb", "ce", "tb", "tbb", "eb", "kc", "n_clusters", "tt", "te", "sel_staged",
            "logits_off", "smem")
    return dict(zip(keys, list(out)))


def workspace_bytes(cfg: dict) -> int:
    """Device workspace bytes a layer with this config allocates."""
    c = Config(cfg["hidden"], cfg["ffn"], cfg["n_experts"], cfg["top_k"], cfg["shared_ffn"],
               cfg["n_max"], cfg["renorm_topk"], cfg["max_tokens"])
    out = C.c_int64()
    check(lib().pw_workspace_bytes(C.byref(c), C.byref(out)))
    return out.value


def plan_release(blocks, target_bytes: int):
    """Greedy release plan through pw_plan_release.  blocks: dicts with bits,
    min_bits, plane_bytes, rows, mass, resid, sens (sens[b] for b = 0..8).
    Returns {"bits", "released", "damage", "reached"}."""
    n = len(blocks)
    arr = (PlanBlock * max(n, 1))()
    for j, b in enumerate(blocks):
        arr[j].bits, arr[j].min_bits = int(b["bits"]), int(b["min_bits"])
        arr[j].plane_bytes, arr[j].rows = int(b["plane_bytes"]), int(b["rows"])
        arr[j].mass, arr[j].resid = float(b["mass"]), float(b.get("resid", 0.0))
        for k in range(PW_MAX_BITS + 1):
            arr[j].sens[k] = float(b["sens"][k]) if k < len(b["sens"]) else 0.0
    bits = (C.c_int32 * max(n, 1))()
    rel, dmg, reached = C.c_int64(), C.c_double(), C.c_int32()
    check(lib().pw_plan_release(arr, n, int(target_bytes), bits, C.byref(rel), C.byref(dmg),
                                C.byref(reached)))
    return {"bits": list(bits)[:n], "released": rel.value, "damage": dmg.value,
            "reached": bool(reached.value)}


# ---- around a projection ----------------------------------------------------
# These calls take views with a row stride, run on the tensors' device and
# check every tensor they are given; a refused argument raises
# PwError(PW_ERR_INVALID_ARG) before anything is enqueued.  They take a few
# microseconds on the GPU for a decode batch, so the host side is kept short:
# names are bound once, and tensors made here are not checked again.

_torch = None
_most = 0x7fffffff  # sizes are passed in 32 bits, which ctypes cuts without a word


def _bind() -> None:
    """Module names used on every call: torch, its types' pw_dtype_t codes
    (int16 / uint8 stand for bf16 / e4m3 bit patterns), the current stream."""
    global _torch, _types, _f32, _i32, _bf16, _bf16_like, _like, _dense
    global _current_device, _current_stream
    import torch
    _f32, _i32, _bf16, _bf16_like = (torch.float32, torch.int32, torch.bfloat16,
                                     (torch.bfloat16, torch.int16))
    _types = {_f32: 0, _bf16: 1, torch.int16: 1, torch.float16: 2, torch.float8_e4m3fn: 3,
              torch.uint8: 3}
    _like = torch.empty_like  # the shortest way to a new tensor
    # empty_like keeps the order of strides (rows that overlap one element
    # apart give columns one apart); outputs are rows one after the other
    _dense = torch.contiguous_format
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    # the handle alone: torch.cuda.current_stream() makes a Stream object, 3 us
    _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _torch = torch


def _refuse(message: str):
    raise PwError(1, message)


def _rows(t, name: str, shape, device: int, types) -> int:
    """Check a [rows][columns] tensor with contiguous rows; its row stride."""
    if shape[0] > _most or shape[1] > _most:
        _refuse("%s: shape %s, sizes are below 2^31" % (name, tuple(shape)))
    if t.shape != shape:
        _refuse("%s: shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.get_device() != device:
        _refuse("%s: on another device than the other tensors" % name)
    if _types.get(t.dtype) not in types:
        _refuse("%s: type %s" % (name, t.dtype))
    ld, unit = t.stride()
    if unit != 1 and shape[1] > 1:
        _refuse("%s: the columns of a row must be contiguous" % name)
    return ld


def _flat(t, name: str, shape, device: int, dtypes) -> int:
    """Check a contiguous tensor (None passes); its address."""
    if t is None:
        return 0
    if t.shape != shape:
        _refuse("%s: shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.get_device() != device:
        _refuse("%s: on another device than the other tensors" % name)
    if t.dtype not in dtypes:
        _refuse("%s: type %s" % (name, t.dtype))
    if not t.is_contiguous():
        _refuse("%s: must be contiguous" % name)
    return t.data_ptr()


def _elsewhere(fn, dev: int, stream, *args):
    """fn on `stream`, or on another device's current one.  On a stream,
    outputs are allocated there, and the tensors' memory is kept from reuse
    until the work on it is done."""
    if stream is None:
        with _torch.cuda.device(dev):
            return fn(*args)
    if stream.device.index != dev:
        _refuse("stream: on another device than the tensors")
    with _torch.cuda.stream(stream):
        out = fn(*args)
    for arg in args:
        for t in arg.values() if isinstance(arg, dict) else (arg,):
            if isinstance(t, _torch.Tensor):
                t.record_stream(stream)
    return out


def add_rms_norm(x, weight, eps: float, residual=None, residual_out=None, y=None, scales=None,
                 y_type=None, scale_group: int = 0, stream=None):
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight over each row.

    x [T][H] bf16 or fp32, residual [T][H] bf16 or fp32 (optional), weight
    [H] bf16 or fp32.  y_type torch.bfloat16 (default) or torch.float8_e4m3fn;
    the 8-bit output has fp32 scales per row (scale_group 0, [T][1]) or per 128
    columns (scale_group 128, [T][ceil(H / 128)]), y ~ scale * q.
    residual_out may be the residual itself.  Returns (y, scales or None,
    residual_out or None)."""
    if _torch is None:
        _bind()
    dev = x.get_device()
    if dev < 0 or x.dim() != 2:
        _refuse("x: a CUDA tensor [T][H] is needed")
    if stream is not None or dev != _current_device():
        return _elsewhere(add_rms_norm, dev, stream, x, weight, eps, residual, residual_out, y,
                          scales, y_type, scale_group)
    T, H = shape = x.shape
    x_ld = _rows(x, "x", shape, dev, (0, 1))
    if scale_group != 0 and scale_group != 128:
        _refuse("scale_group: 0 (a scale per row) or 128")
    w = _flat(weight, "weight", (H,), dev, (_bf16, _f32, _torch.int16))
    res = r_ld = r_out = ro_ld = r_code = 0
    if residual is not None:
        r_ld = _rows(residual, "residual", shape, dev, (0, 1))
        r_code, res = _types[residual.dtype], residual.data_ptr()
        if residual_out is None:
            residual_out, ro_ld = _like(residual, memory_format=_dense), H
        else:
            ro_ld = _rows(residual_out, "residual_out", shape, dev, (r_code,))
        r_out = residual_out.data_ptr()
    elif residual_out is not None:
        _refuse("residual_out: needs a residual")
    if y is None:
        y, y_ld = _like(x, dtype=y_type or _bf16, memory_format=_dense), H
    else:
        if y_type is not None and _types.get(y.dtype) != _types.get(y_type):
            _refuse("y: type %s, y_type %s" % (y.dtype, y_type))
        y_ld = _rows(y, "y", shape, dev, (1, 3))
    y_code = _types.get(y.dtype)
    s = 0
    if y_code == 3:
        want = (T, 1 if scale_group == 0 else -(-H // 128))
        if scales is None:
            scales = x.new_empty(want, dtype=_f32)
            s = scales.data_ptr()
        else:
            s = _flat(scales, "scales", want, dev, (_f32,))
    elif y_code != 1:
        _refuse("y: type %s" % y.dtype)
    elif scales is not None:
        _refuse("scales: only with an 8-bit y")
    status = (_lib or lib()).pw_add_rms_norm(x.data_ptr(), _types[x.dtype], x_ld, res, r_code, r_ld,
                                             w, _types[weight.dtype], eps, T, H, r_out, ro_ld,
                                             y.data_ptr(), y_code, y_ld, s, scale_group,
                                             _current_stream(dev))
    if status:
        check(status)
    return y, scales, residual_out


def token_logprobs(logits, tokens=None, n_top: int = 0, logprob=None, entropy=None, top_idx=None,
                   top_logprob=None, stream=None):
    """Log probabilities of tokens (int32 [T], -1 for none) under a softmax
    over each row of logits ([T][V] fp32, bf16 or fp16), the rows' entropy,
    and the n_top best alternatives (largest first, ties to the lower index).
    Returns (logprob fp32 [T] or None, entropy fp32 [T], top_idx int32
    [T][n_top] or None, top_logprob fp32 [T][n_top] or None)."""
    if _torch is None:
        _bind()
    dev = logits.get_device()
    if dev < 0 or logits.dim() != 2:
        _refuse("logits: a CUDA tensor [T][V] is needed")
    if stream is not None or dev != _current_device():
        return _elsewhere(token_logprobs, dev, stream, logits, tokens, n_top, logprob, entropy,
                          top_idx, top_logprob)
    T, V = shape = logits.shape
    ld = _rows(logits, "logits", shape, dev, (0, 1, 2))
    if n_top > 32:
        _refuse("n_top: at most 32")
    tok = lp = ti = tl = 0
    if tokens is not None:
        tok = _flat(tokens, "tokens", (T,), dev, (_i32,))
        if logprob is None:
            logprob = _like(tokens, dtype=_f32)
            lp = logprob.data_ptr()
        else:
            lp = _flat(logprob, "logprob", (T,), dev, (_f32,))
    elif logprob is not None:
        _refuse("logprob: needs tokens")
    if entropy is None:
        entropy = _like(logprob) if lp else logits.new_empty((T,), dtype=_f32)
        ent = entropy.data_ptr()
    else:
        ent = _flat(entropy, "entropy", (T,), dev, (_f32,))
    if n_top > 0:
        want = (T, n_top)
        if top_idx is None:
            top_idx = logits.new_empty(want, dtype=_i32)
            ti = top_idx.data_ptr()
        else:
            ti = _flat(top_idx, "top_idx", want, dev, (_i32,))
        if top_logprob is None:
            top_logprob = _like(top_idx, dtype=_f32)
            tl = top_logprob.data_ptr()
        else:
            tl = _flat(top_logprob, "top_logprob", want, dev, (_f32,))
    elif top_idx is not None or top_logprob is not None:
        _refuse("top_idx, top_logprob: need n_top > 0")
    status = (_lib or lib()).pw_token_logprobs(logits.data_ptr(), _types[logits.dtype], ld, T, V,
                                               tok, n_top, lp, ent, ti, tl, _current_stream(dev))
    if status:
        check(status)
    return logprob, entropy, top_idx, top_logprob


def add_adapters(x, a, b, ids, base=None, scale=None, ranks=None, y=None, y_type=None,
                 stream=None, _first=None):
    """y[t] = base[t] + scale[i] * B_i (A_i x[t]), i = ids[t]; base[t] alone
    where ids[t] is -1.

    x bf16 [T][cols]; a bf16 [n][max_rank][cols]; b bf16 [n][rows][max_rank];
    ids int32 [T]; scale fp32 [n] and ranks int32 [n] on the device
    (optional); base [T][rows] fp32 or bf16 (optional; may be y); y of base's
    type (y_type, default fp32, without a base).  Returns y."""
    if _torch is None:
        _bind()
    dev = x.get_device()
    if dev < 0 or x.dim() != 2 or a.dim() != 3 or b.dim() != 3 or ids is None:
        _refuse("CUDA tensors x [T][cols], a [n][max_rank][cols], b [n][rows][max_rank] and ids [T] "
                "are needed")
    if stream is not None or dev != _current_device():
        return _elsewhere(add_adapters, dev, stream, x, a, b, ids, base, scale, ranks, y, y_type)
    T, cols = shape = x.shape
    n, rows, r = b.shape
    x_ld = _rows(x, "x", shape, dev, (1,))
    if n > _most or r > _most or rows > _most:
        _refuse("b: shape %s, sizes are below 2^31" % (tuple(b.shape),))
    pa = _flat(a, "a", (n, r, cols), dev, _bf16_like)
    pb = _flat(b, "b", (n, rows, r), dev, _bf16_like)
    pi = _flat(ids, "ids", (T,), dev, (_i32,))
    pr = _flat(ranks, "ranks", (n,), dev, (_i32,))
    ps = _flat(scale, "scale", (n,), dev, (_f32,))
    shape, base_ld, pbase = (T, rows), 0, 0
    if base is not None:
        base_ld = _rows(base, "base", shape, dev, (0, 1))
        pbase = base.data_ptr()
    if y is None:
        y_ld = rows
        y = (_like(base, memory_format=_dense) if base is not None else
             x.new_empty(shape, dtype=y_type or _f32))
    else:
        y_ld = _rows(y, "y", shape, dev, (0, 1) if base is None else (_types[base.dtype],))
    y_code = _types.get(y.dtype)
    if y_type is not None and _types.get(y_type) != y_code:
        _refuse("y: type %s, y_type %s" % (y.dtype, y_type))
    L = _lib or lib()
    work, size = 0, L.pw_adapters_workspace_bytes(T, r, y_code or 0)
    if size:
        keep = x.new_empty((size,), dtype=_torch.uint8)
        work = keep.data_ptr()
    stream = _current_stream(dev)
    if _first is not None:
        # sizes out of range are refused for no tokens as for some
        check(L.pw_adapters(None, 0, None, None, None, None, None, n, r, 0, cols, rows, None, 0, None,
                            y_code, 0, None, 0, None))
        _first(stream)
    status = L.pw_adapters(x.data_ptr(), x_ld, pa, pb, pi, pr, ps, n, r, T, cols, rows, pbase,
                           base_ld, y.data_ptr(), -1 if y_code is None else y_code, y_ld, work, size,
                           stream)
    if status:
        check(status)
    return y


def _linear_with_adapters(planes, lut, bits, x, rows, y, stream, adapters, ids):
    """linear's two calls; the projection is enqueued (_first) once
    everything that the adapters could be refused for has been looked at."""
    if _torch is None:
        _bind()
    if not {"a", "b"} <= adapters.keys() <= {"a", "b", "scale", "ranks"}:
        _refuse("adapters: a and b, optionally scale and ranks, are taken")
    dev = x.get_device()
    if dev < 0 or x.dim() != 2:
        _refuse("x: a CUDA tensor [T][cols] is needed")
    if stream is not None or dev != _current_device():
        return _elsewhere(_linear_with_adapters, dev, stream, planes, lut, bits, x, rows, y, None,
                          adapters, ids)
    T, cols = x.shape
    px = _flat(x, "x", (T, cols), dev, _bf16_like)
    if y is None:
        y = x.new_empty((T, rows), dtype=_f32)
    py = _flat(y, "y", (T, rows), dev, (_f32,))
    n_max = planes.numel() * 4 // plane_bytes(rows, cols)
    return add_adapters(x, adapters["a"], adapters["b"], ids, y, adapters.get("scale"),
                        adapters.get("ranks"), y, _first=lambda stream: check(lib().pw_linear(
                            _ptr(planes), _ptr(lut), rows, cols, n_max, bits, px, T, py, stream)))


class MoELayer:
    """A layer over device-resident pages (torch tensors kept alive here)."""

    def __init__(self, cfg: dict, planes: Sequence, lut_slots: Sequence, bits: Sequence[int],
                 host_planes: Optional[Sequence] = None, host_luts: Optional[Sequence] = None):
        self.cfg = dict(cfg)
        self._keep: List = [planes, lut_slots, host_planes, host_luts]
        c = Config(cfg["hidden"], cfg["ffn"], cfg["n_experts"], cfg["top_k"], cfg["shared_ffn"],
                   cfg["n_max"], cfg["renorm_topk"], cfg["max_tokens"])
        n = len(planes)
        descs = (BlockDesc * n)()
        for j in range(n):
            d = descs[j]
            d.d_planes = _ptr(planes[j])
            d.d_lut[0] = _ptr(lut_slots[j][0])
            d.d_lut[1] = _ptr(lut_slots[j][1])
            d.h_planes = _ptr(host_planes[j]) if host_planes else None
            if host_luts:
                for b, t in host_luts[j].items():
                    d.h_lut[b] = _ptr(t)
            d.bits = int(bits[j])
        h = C.c_void_p()
        check(lib().pw_moe_create(C.byref(c), descs, n, C.byref(h)))
        self.h = h
        self.n_blocks = n
        self._device = planes[0].get_device()

    def forward(self, x, router_w, bias=None, y=None, stream=None):
        import torch
        T = x.shape[0]
        if y is None:
            y = torch.empty_like(x)
        check(lib().pw_moe_forward(self.h, _ptr(x), T, _ptr(router_w), _ptr(bias), _ptr(y),
                                   _stream(stream)))
        return y

    def forward_norm(self, x, norm_weight, eps: float, router_w, bias=None, residual=None,
                     residual_out=None, y=None, stream=None):
        """forward of x' = add_rms_norm(x, norm_weight, eps, residual): all
        bf16 (int16 bit patterns are taken too) and contiguous, on the layer's
        device; router_w fp32 [E][H], bias fp32 [E].  residual_out may be the
        residual.  Every tensor is checked as in the calls above; nothing is
        enqueued for a refused one.  Returns (y, residual_out or None)."""
        if _torch is None:
            _bind()
        H, E, dev = self.cfg["hidden"], self.cfg["n_experts"], self._device
        if x.dim() != 2:
            _refuse("x: [T][H] is needed")
        rows = (x.shape[0], H)
        for t, name, shape, types in (
                (x, "x", rows, _bf16_like), (residual, "residual", rows, _bf16_like),
                (norm_weight, "norm_weight", (H,), _bf16_like),
                (residual_out, "residual_out", rows, _bf16_like),
                (router_w, "router_w", (E, H), (_f32,)), (bias, "bias", (E,), (_f32,)),
                (y, "y", rows, _bf16_like)):
            _flat(t, name, shape, dev, types)
        if norm_weight is None or router_w is None:
            _refuse("norm_weight and router_w are needed")
        if residual is None and residual_out is not None:
            _refuse("residual_out: needs a residual")
        if stream is not None or dev != _current_device():
            return _elsewhere(self.forward_norm, dev, stream, x, norm_weight, eps, router_w, bias,
                              residual, residual_out, y)
        if y is None:
            y = _like(x)
        if residual is not None and residual_out is None:
            residual_out = _like(residual)
        check(lib().pw_moe_forward_norm(self.h, _ptr(x), _ptr(residual), _ptr(norm_weight), eps,
                                        rows[0], _ptr(router_w), _ptr(bias), _ptr(residual_out),
                                        _ptr(y), _current_stream(dev)))
        return y, residual_out

    def forward_host(self, x_host, router_w, bias=None, y_host=None, stream=None):
        """x_host: pinned CPU int16/bf16 tensor [T][H]; returns the host output."""
        import torch
        if y_host is None:
            y_host = torch.empty_like(x_host).pin_memory()
        check(lib().pw_moe_forward_host(self.h, _ptr(x_host), x_host.shape[0], _ptr(router_w),
                                        _ptr(bias), _ptr(y_host), _stream(stream)))
        return y_host

    def set_block_bits(self, block: int, bits: int, side_stream) -> None:
        check(lib().pw_set_block_bits(self.h, block, bits, side_stream.cuda_stream))

    def get_block_bits(self, block: int):
        """(bitwidth as of the last issued forward, pending width or 0)."""
        cur, pend = C.c_int32(), C.c_int32()
        check(lib().pw_get_block_bits(self.h, block, C.byref(cur), C.byref(pend)))
        return cur.value, pend.value

    def forward_bits(self) -> List[int]:
        """Bitwidth of every block in the most recently issued forward."""
        out = (C.c_int32 * self.n_blocks)()
        check(lib().pw_get_forward_bits(self.h, out, self.n_blocks))
        return list(out)

    def set_switch_lag(self, max_lag: int) -> None:
        check(lib().pw_set_switch_lag(self.h, max_lag))

    def routing(self, T: int, stream=None):
        import torch
        k = self.cfg["top_k"]
        idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
        w = torch.empty((T, k), dtype=torch.float32, device="cuda")
        check(lib().pw_get_routing(self.h, _ptr(idx), _ptr(w), _stream(stream)))
        return idx, w

    def enable_paging(self, stream=None) -> None:
        """Library-owned plane storage holding only each block's resident
        planes (the caller's plane buffers may be freed afterwards)."""
        check(lib().pw_enable_paging(self.h, _stream(stream)))

    def compact_pages(self, stream=None) -> None:
        """Pack the resident planes into one allocation (on the forward stream)."""
        check(lib().pw_compact_pages(self.h, _stream(stream)))

    def resident_bytes(self, trim: bool = False):
        """(plane bytes resident, pool bytes reserved after a trim or None)."""
        pb, pr = C.c_int64(), C.c_int64()
        check(lib().pw_resident_bytes(self.h, C.byref(pb), C.byref(pr) if trim else None))
        return pb.value, (pr.value if trim else None)

    def routing_stats(self, reset: bool = False, stream=None):
        """(counts uint64 [E], mass float64 [E]) accumulated over forwards."""
        E = self.cfg["n_experts"]
        counts = np.zeros(E, dtype=np.uint64)
        mass = np.zeros(E, dtype=np.float64)
        check(lib().pw_routing_stats(self.h, counts.ctypes.data, mass.ctypes.data,
                                     1 if reset else 0, _stream(stream)))
        return counts, mass

    def check_device_error(self) -> None:
        check(lib().pw_check_device_error(self.h))

    def profile(self, on: bool) -> None:
        check(lib().pw_profile_enable(self.h, 1 if on else 0))

    def profile_read(self):
        """(ms per launch slot summed since the last read, forwards summed)."""
        ms = (C.c_float * 4)()
        n = C.c_int32()
        check(lib().pw_profile_read(self.h, ms, 4, C.byref(n)))
        return list(ms), n.value

    def launches(self, T: int) -> int:
        return int(lib().pw_forward_launches(self.h, T))

    def close(self) -> None:
        if getattr(self, "h", None):
            check(lib().pw_destroy(self.h))
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def upload_synth_layer(layer, max_tokens: int, host_copies: bool = False,
                       device: str = "cuda", host_planes: bool = True) -> MoELayer:
    """Put a synth.Layer's pages on the device and create the library layer.
    With host_copies, pinned master copies of every LUT width, and of all
    planes unless host_planes is False, are kept for bitwidth switches."""
    import torch
    wl = layer.wl
    planes, slots, hp, hl = [], [], [], []
    for blk in range(wl.n_blocks):
        rows, cols = layer.shape(blk)
        pl = layer.planes(blk)
        paged = repack_planes(torch.from_numpy(pl.view(np.int32)).to(device), cols)
        planes.append(paged)
        s0 = torch.zeros(rows << wl.n_max, dtype=torch.int16, device=device)
        s1 = torch.zeros(rows << wl.n_max, dtype=torch.int16, device=device)
        lt = layer.lut(blk, layer.bits[blk])
        s0[: lt.size].copy_(torch.from_numpy(lt.reshape(-1).view(np.int16)))
        slots.append((s0, s1))
        if host_copies and host_planes:
            hp.append(paged.cpu().pin_memory())
        if host_copies:
            hl.append({b: torch.from_numpy(layer.lut(blk, b).reshape(-1).view(np.int16)).pin_memory()
                       for b in range(1, wl.n_max + 1)})
    cfg = dict(hidden=wl.hidden, ffn=wl.ffn, n_experts=wl.n_experts, top_k=wl.top_k,
               shared_ffn=wl.shared_ffn, n_max=wl.n_max, renorm_topk=wl.renorm_topk,
               max_tokens=max_tokens)
    return MoELayer(cfg, planes, slots, layer.bits, hp or None, hl or None)
