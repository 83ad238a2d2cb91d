"""Thin Python binding over libwqmoe.so.

Every function here only marshals arguments: torch tensors supply device
memory and the current HIP stream, numpy arrays supply host memory for the
offline packers.  All computation happens in the library's kernels (or, for
the packers, in its host code).  The names follow include/wqmoe.h.

stream: the raw handle of the HIP stream to run on (0: the default stream);
None is torch's current one.  Nothing waits: inputs have to be ready on that
stream, and a reader on another one waits for it.  Buffers that a call allocates
are of that stream's memory.
"""
from __future__ import annotations

import ctypes as C
from typing import NamedTuple, Optional, Tuple

import numpy as np

from . import _lib
from ._lib import (WQ_BF16, WQ_E4M3, WQ_F16, WQ_F32, WQ_GROUP_MAX, WQ_GROUP_TOP2, WQ_PACK_INTERLEAVE_GATE_UP,
                   WQ_SCORE_SIGMOID, WQ_SCORE_SOFTMAX, WQ_STAGE_DOWN, WQ_STAGE_GATE_UP, WQ_STAGE_RAW,
                   WqEpilogue, WqKvCache, WqMoeGemmDesc, check, load)

__all__ = [
    "moe_route", "moe_align", "moe_route_align", "moe_align_capacity", "moe_gemm_workspace_bytes", "moe_w4a16_gemm", "moe_w8a16_gemm",
    "moe_route_gate_up",
    "moe_w8a16_gemm_noalloc", "sparse24_w4a16_gemm", "sparse24_w8a16_gemm", "quantize_w8", "dense_gemm_workspace_bytes", "dense_epilogue_workspace_bytes", "dense_w4a16_gemm", "dense_w8a16_gemm",
    "pack_w4", "pack_w8", "pack_sparse24", "act_code", "moe_fp8_gemm_workspace_bytes", "moe_fp8_w8a8_gemm",
    "pack_fp8", "moe_route_grouped", "moe_route_grouped_align", "rms_norm", "RmsNormOut", "moe_fp8_codes_gemm",
    "Lora", "pack_lora", "dense_lora_gemm", "dense_lora_workspace_bytes",
    "KVCache", "kv_cache", "kv_cache_write", "kv_cache_read", "paged_attention", "paged_attention_workspace_bytes",
]


def _torch():
    import torch
    return torch


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream):
    """The HIP stream of a call: the one given, or torch's current one on the
    current device (its raw handle; a Stream object costs 2.5 us a call)."""
    if stream is not None:
        return stream
    c = _torch()._C
    return c._cuda_getCurrentRawStream(c._cuda_getDevice())


def act_code(dtype) -> int:
    torch = _torch()
    if dtype == torch.float16:
        return WQ_F16
    if dtype == torch.bfloat16:
        return WQ_BF16
    raise ValueError("activation dtype must be float16 or bfloat16, got %s" % dtype)


def _check(t, name: str, shape, dtypes, device=None, row_stride: bool = False):
    """A tensor argument has the shape, one of the types, and is contiguous
    (with row_stride: its last dimension is, and rows do not overlap)."""
    if t.shape == shape and t.dtype in dtypes and t.is_contiguous() and (device is None or t.device == device):
        return
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, the input on %s" % (name, t.device, device))
    if not t.is_contiguous():
        rows, n = (t.shape if t.dim() == 2 else (0, 0))
        if not row_stride or t.numel() and (t.stride(1) != 1 and n > 1 or t.stride(0) < n and rows > 1):
            raise ValueError("%s must be contiguous%s, got strides %s"
                             % (name, " in its rows" if row_stride else "", list(t.stride())))


def _holds(t, name: str, n: int, dtypes):
    """A tensor argument of any shape is contiguous, has one of the types and at
    least n values (its device the library checks)."""
    if t.numel() >= n and t.dtype in dtypes and t.is_contiguous():
        return
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    raise ValueError("%s must hold %d values, contiguous; got %s, strides %s" % (name, n, list(t.shape), list(t.stride())))


def _int32(**sizes):
    """Sizes go through C int arguments, which would take them modulo 2^32."""
    for name, v in sizes.items():
        if not -0x80000000 <= v <= 0x7fffffff:
            raise ValueError("%s = %d does not fit 32 bits" % (name, v))


def _row_stride(t) -> int:
    """The row stride of a [rows, n] tensor that _check has passed."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _alloc(stream, make, *args, **kw):
    """make(*args, **kw): a buffer that a call on `stream` allocates, out of that
    stream's memory.  A block of the current stream's may have been freed by a
    call whose kernel, on that stream, still uses it; here it is handed out in
    the order of the stream that the call's kernels run on."""
    if stream is None or stream == _stream(None):
        return make(*args, **kw)
    torch = _torch()
    # (ExternalStream makes a new stream of handle 0, the default stream's)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()):
        return make(*args, **kw)


def _keep_for(stream, *tensors):
    """Outputs allocated here for a call on another stream than the current one
    are not handed out again before the current stream, on which the caller
    reads them (once it waits for `stream`), is done with them."""
    if stream is None or stream == _stream(None):
        return
    here = _torch().cuda.current_stream()
    for t in tensors:
        if t is not None:
            t.record_stream(here)


def _np_ptr(a: Optional[np.ndarray]):
    return None if a is None else a.ctypes.data_as(C.c_void_p)


# ----------------------------------------------------------------------------
# hot path
# ----------------------------------------------------------------------------
def moe_route(logits, topk: int, renormalize: bool = True, topk_weights=None, topk_ids=None, stream=None):
    """logits [M, E] float32 (device) -> (topk_weights [M, topk] f32, topk_ids [M, topk] i32)."""
    torch = _torch()
    M, E = logits.shape
    new = []
    if topk_weights is None:
        topk_weights = _alloc(stream, torch.empty, (M, topk), dtype=torch.float32, device=logits.device)
        new.append(topk_weights)
    if topk_ids is None:
        topk_ids = _alloc(stream, torch.empty, (M, topk), dtype=torch.int32, device=logits.device)
        new.append(topk_ids)
    check(load().moe_route(_ptr(logits), M, E, topk, int(bool(renormalize)), _ptr(topk_weights), _ptr(topk_ids),
                           _stream(stream)), "moe_route")
    _keep_for(stream, *new)
    return topk_weights, topk_ids


def moe_route_align(logits, topk: int, renormalize: bool, block_size: int, topk_weights, topk_ids,
                    sorted_token_ids, expert_ids, num_tokens_post_padded, capacity: int, stream=None):
    """moe_route then moe_align in one call (one kernel for batches up to 16
    tokens); every output buffer is the caller's."""
    M, E = logits.shape
    check(load().moe_route_align(_ptr(logits), M, E, topk, int(bool(renormalize)), block_size, _ptr(topk_weights),
                                 _ptr(topk_ids), _ptr(sorted_token_ids), _ptr(expert_ids),
                                 _ptr(num_tokens_post_padded), capacity, _stream(stream)), "moe_route_align")
    return topk_weights, topk_ids, sorted_token_ids, expert_ids, num_tokens_post_padded


def moe_align_capacity(M: int, topk: int, E: int, block_size: int) -> int:
    return int(load().moe_align_capacity(M, topk, E, block_size))


def moe_align(topk_ids, E: int, block_size: int, capacity: Optional[int] = None, sorted_token_ids=None,
              expert_ids=None, num_tokens_post_padded=None, stream=None):
    """topk_ids [M, topk] i32 (device) -> (sorted_token_ids [cap], expert_ids [cap/BS], num_tokens_post_padded [1])."""
    torch = _torch()
    M, topk = topk_ids.shape
    cap = moe_align_capacity(M, topk, E, block_size) if capacity is None else capacity
    new = []

    def i32(n):
        new.append(_alloc(stream, torch.empty, n, dtype=torch.int32, device=topk_ids.device))
        return new[-1]

    if sorted_token_ids is None:
        sorted_token_ids = i32(max(cap, 1))
    if expert_ids is None:
        expert_ids = i32(max(cap // block_size, 1))
    if num_tokens_post_padded is None:
        num_tokens_post_padded = i32(1)
    check(load().moe_align(_ptr(topk_ids), M, topk, E, block_size, _ptr(sorted_token_ids), _ptr(expert_ids),
                           _ptr(num_tokens_post_padded), cap, _stream(stream)), "moe_align")
    _keep_for(stream, *new)
    return sorted_token_ids, expert_ids, num_tokens_post_padded


_SCORING = {"softmax": WQ_SCORE_SOFTMAX, "sigmoid": WQ_SCORE_SIGMOID}
_GROUP_SCORE = {"max": WQ_GROUP_MAX, "top2": WQ_GROUP_TOP2}


def _grouped_args(logits, topk, scoring, bias, n_group, topk_group, group_score, topk_weights, topk_ids, stream):
    torch = _torch()
    f32, dt = torch.float32, logits.dtype
    code = WQ_F32 if dt == f32 else WQ_BF16 if dt == torch.bfloat16 else WQ_F16
    if logits.dim() != 2:
        raise ValueError("logits must be [M, E], got %s" % list(logits.shape))
    M, E = logits.shape
    if topk < 1 or max(M, E, topk, abs(n_group), abs(topk_group)) > 0x7fffffff:
        raise ValueError("topk must be >= 1 and sizes fit 32 bits: M %d E %d topk %d n_group %d topk_group %d"
                         % (M, E, topk, n_group, topk_group))
    _check(logits, "logits", (M, E), (f32, torch.float16, torch.bfloat16))
    if scoring not in _SCORING or group_score not in _GROUP_SCORE:
        raise ValueError("scoring %r not in %s or group_score %r not in %s"
                         % (scoring, list(_SCORING), group_score, list(_GROUP_SCORE)))
    dev = logits.device
    if bias is not None:
        _check(bias, "bias", (E,), (f32,), dev)
    new = []
    if topk_weights is None:
        new.append(topk_weights := _alloc(stream, torch.empty, (M, topk), dtype=f32, device=dev))
    else:
        _check(topk_weights, "topk_weights", (M, topk), (f32,), dev)
    if topk_ids is None:
        new.append(topk_ids := _alloc(stream, torch.empty_like, topk_weights, dtype=torch.int32))
    else:
        _check(topk_ids, "topk_ids", (M, topk), (torch.int32,), dev)
    return M, E, code, topk_weights, topk_ids, new


def moe_route_grouped(logits, topk: int, scoring: str = "softmax", bias=None, n_group: int = 1, topk_group: int = 1,
                      group_score: str = "max", renormalize: bool = True, routed_scale: float = 1.0,
                      topk_weights=None, topk_ids=None, stream=None):
    """Router with softmax or sigmoid scores, a balancing bias (added for the
    choice only) and expert groups, of which the topk_group best (by their best
    expert, "max", or the sum of their two best scores, "top2") are open:
    logits [M, E] float32 / fp16 / bf16 (device) -> (topk_weights [M, topk]
    f32, topk_ids [M, topk] i32)."""
    M, E, dt, topk_weights, topk_ids, new = _grouped_args(logits, topk, scoring, bias, n_group, topk_group,
                                                          group_score, topk_weights, topk_ids, stream)
    check(load().moe_route_grouped(_ptr(logits), dt, M, E, topk, _SCORING[scoring], _ptr(bias), n_group, topk_group,
                                   _GROUP_SCORE[group_score], int(bool(renormalize)), routed_scale,
                                   _ptr(topk_weights), _ptr(topk_ids), _stream(stream)), "moe_route_grouped")
    _keep_for(stream, *new)
    return topk_weights, topk_ids


def moe_route_grouped_align(logits, topk: int, block_size: int, scoring: str = "softmax", bias=None, n_group: int = 1,
                            topk_group: int = 1, group_score: str = "max", renormalize: bool = True,
                            routed_scale: float = 1.0, topk_weights=None, topk_ids=None, sorted_token_ids=None,
                            expert_ids=None, num_tokens_post_padded=None, capacity: Optional[int] = None,
                            stream=None):
    """moe_route_grouped then moe_align in one call (one kernel for batches up
    to 16 tokens) -> (topk_weights, topk_ids, sorted_token_ids [capacity],
    expert_ids [capacity / block_size], num_tokens_post_padded [1]); buffers
    not given are allocated, for the least capacity unless one is given."""
    torch = _torch()
    M, E, dt, topk_weights, topk_ids, new = _grouped_args(logits, topk, scoring, bias, n_group, topk_group,
                                                          group_score, topk_weights, topk_ids, stream)
    _int32(block_size=block_size)
    if block_size < 1:
        raise ValueError("block_size must be >= 1, got %d" % block_size)
    cap = moe_align_capacity(M, topk, E, block_size) if capacity is None else capacity
    dev, i32, blocks = logits.device, torch.int32, cap // block_size
    if sorted_token_ids is None and expert_ids is None and num_tokens_post_padded is None:
        # one allocation for the three, each at a multiple of 16 bytes
        rows = -(-max(cap, 1) // 4) * 4
        new.append(_alloc(stream, torch.empty, rows + 4 + max(blocks, 1), dtype=i32, device=dev))
        arrays = torch.split_with_sizes(new[-1], (rows, 1, 3, max(blocks, 1)))
        arrays = [arrays[0], arrays[3], arrays[1]]
    else:
        arrays = [(sorted_token_ids, "sorted_token_ids", cap), (expert_ids, "expert_ids", blocks),
                  (num_tokens_post_padded, "num_tokens_post_padded", 1)]
        for k, (t, name, n) in enumerate(arrays):
            if t is None:
                t = _alloc(stream, torch.empty, max(n, 1), dtype=i32, device=dev)
                new.append(t)
            elif t.dim() != 1 or t.numel() < n:
                raise ValueError("%s must hold %d values, got %s" % (name, n, list(t.shape)))
            else:
                _check(t, name, t.shape, (i32,), dev)
            arrays[k] = t
    check(load().moe_route_grouped_align(_ptr(logits), dt, M, E, topk, _SCORING[scoring], _ptr(bias), n_group,
                                         topk_group, _GROUP_SCORE[group_score], int(bool(renormalize)), routed_scale,
                                         block_size, _ptr(topk_weights), _ptr(topk_ids), *map(_ptr, arrays), cap,
                                         _stream(stream)), "moe_route_grouped_align")
    _keep_for(stream, *new)
    return (topk_weights, topk_ids, *arrays)


class RmsNormOut(NamedTuple):
    out: object       # [rows, n] act dtype, or None
    residual: object  # [rows, n] act dtype, or None (no residual given)
    codes: object     # [rows, n] uint8 E4M3 codes, or None
    scales: object    # [rows] float32, or None (no row scales asked for)


def rms_norm(x, weight=None, eps: float = 1e-6, residual=None, quant: Optional[str] = None,
             scale: Optional[float] = None, want_out: bool = True, out=None, residual_out=None, codes=None,
             scales=None, stream=None) -> RmsNormOut:
    """Residual addition + RMS norm of x [rows, n] bf16/fp16 (device; rows may be
    strided): s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight.  out is
    y in x's type; with quant="row" codes are the E4M3 codes of y with one
    written scale per row, with quant="static" those of y / scale (the FP8
    layer's input in its two forms); residual is s in x's type.  Buffers not
    given are allocated; out and residual_out may be x or residual."""
    torch = _torch()
    dt = act_code(x.dtype)
    if x.dim() != 2:
        raise ValueError("x must be [rows, n], got %s" % list(x.shape))
    rows, n = x.shape
    if rows > 0x7fffffff or n > 0x7fffffff:
        raise ValueError("x is too large: %s" % list(x.shape))
    dev, same = x.device, (x.dtype,)
    shape = x.shape
    _check(x, "x", shape, same, row_stride=True)
    if weight is not None:
        _check(weight, "weight", (n,), same, dev)
    if quant is not None and quant not in ("row", "static"):
        raise ValueError("quant must be None, 'row' or 'static', got %r" % (quant,))
    if (quant == "static") != (scale is not None):
        raise ValueError("scale goes with quant='static'")
    if codes is not None and quant is None or scales is not None and quant != "row":
        raise ValueError("codes go with quant, scales with quant='row'")
    if out is not None and not want_out or residual_out is not None and residual is None:
        raise ValueError("out goes with want_out, residual_out with a residual")
    new = []

    def like_x(t, name):
        if t is None:
            t = _alloc(stream, torch.empty_like, x, memory_format=torch.contiguous_format)
            new.append(t)
        else:
            _check(t, name, shape, same, dev, row_stride=True)
        return t

    rs = ros = os_ = 0  # row strides of what there is
    if residual is not None:
        _check(residual, "residual", shape, same, dev, row_stride=True)
        residual_out = like_x(residual_out, "residual_out")
        rs, ros = _row_stride(residual), _row_stride(residual_out)
    if want_out:
        out = like_x(out, "out")
        os_ = _row_stride(out)
    if quant is not None:
        if codes is None:
            codes = _alloc(stream, torch.empty_like, x, dtype=torch.uint8, memory_format=torch.contiguous_format)
            new.append(codes)
        else:
            _check(codes, "codes", shape, (torch.uint8, torch.float8_e4m3fn), dev)
        if quant == "row":
            if scales is None:
                scales = _alloc(stream, torch.empty, rows, dtype=torch.float32, device=dev)
                new.append(scales)
            else:
                _check(scales, "scales", (rows,), (torch.float32,), dev)
    check(load().wq_rms_norm(x.data_ptr(), _row_stride(x), _ptr(residual), rs, _ptr(weight), rows, n, eps, dt,
                             _ptr(residual_out), ros, _ptr(out), os_, _ptr(codes), _ptr(scales),
                             0.0 if scale is None else scale, _stream(stream)), "wq_rms_norm")
    _keep_for(stream, *new)
    return RmsNormOut(out, residual_out, codes, scales)


def moe_gemm_workspace_bytes(stage: int, M: int, topk: int, E: int, n_out: int, k_in: int, capacity: int,
                             act_order: bool) -> int:
    return int(load().moe_gemm_workspace_bytes(stage, M, topk, E, n_out, k_in, capacity, int(bool(act_order))))


def _desc(stage: int, a, M: int, topk: int, E: int, n_out: int, k_in: int, w_packed, scales, group_size: int,
          k_perm, sorted_token_ids, expert_ids, num_tokens_post_padded, capacity: int, block_size: int, topk_weights,
          out, workspace, act_dtype: int):
    d = WqMoeGemmDesc()
    d.struct_size = C.sizeof(WqMoeGemmDesc)
    d.stage = stage
    d.act_dtype = act_dtype
    d.d_a = _ptr(a)
    d.M, d.topk, d.E, d.n_out, d.k_in = M, topk, E, n_out, k_in
    d.d_w_packed = _ptr(w_packed)
    d.d_scales = _ptr(scales)
    d.group_size = group_size
    d.d_k_perm = _ptr(k_perm)
    d.d_sorted_token_ids = _ptr(sorted_token_ids)
    d.d_expert_ids = _ptr(expert_ids)
    d.d_num_tokens_post_padded = _ptr(num_tokens_post_padded)
    d.capacity = capacity
    d.block_size = block_size
    d.d_topk_weights = _ptr(topk_weights)
    d.d_out = _ptr(out)
    d.d_workspace = _ptr(workspace)
    d.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return d


def _gemm(fn_name: str, stage: int, a, M: int, topk: int, E: int, n_out: int, k_in: int, w_packed, scales,
          group_size: int, k_perm, sorted_token_ids, expert_ids, num_tokens_post_padded, capacity: int,
          block_size: int, topk_weights, out, workspace, stream, act_dtype: int):
    d = _desc(stage, a, M, topk, E, n_out, k_in, w_packed, scales, group_size, k_perm, sorted_token_ids, expert_ids,
              num_tokens_post_padded, capacity, block_size, topk_weights, out, workspace, act_dtype)
    check(getattr(load(), fn_name)(C.byref(d), _stream(stream)), fn_name)
    return out


def moe_route_gate_up(wbits: int, logits, renormalize: bool, topk_weights, topk_ids, a, M, topk, E, n_out, k_in,
                      w_packed, scales, group_size, k_perm, sorted_token_ids, expert_ids, num_tokens_post_padded,
                      capacity, block_size, out, workspace=None, stream=None, act_dtype=WQ_BF16):
    """moe_route_align followed by the GATE_UP stage of moe_w{wbits}a16_gemm in
    one call (one kernel for the smallest batches); writes topk_weights,
    topk_ids, sorted_token_ids, expert_ids, num_tokens_post_padded and out."""
    d = _desc(WQ_STAGE_GATE_UP, a, M, topk, E, n_out, k_in, w_packed, scales, group_size, k_perm, sorted_token_ids,
              expert_ids, num_tokens_post_padded, capacity, block_size, None, out, workspace, act_dtype)
    check(load().moe_route_gate_up(_ptr(logits), int(bool(renormalize)), _ptr(topk_weights), _ptr(topk_ids),
                                   C.byref(d), wbits, _stream(stream)), "moe_route_gate_up")
    return out


def moe_w4a16_gemm(stage, a, M, topk, E, n_out, k_in, w_packed, scales, group_size, k_perm, sorted_token_ids,
                   expert_ids, num_tokens_post_padded, capacity, block_size, topk_weights, out, workspace=None,
                   stream=None, act_dtype=WQ_F16):
    return _gemm("moe_w4a16_gemm", stage, a, M, topk, E, n_out, k_in, w_packed, scales, group_size, k_perm,
                 sorted_token_ids, expert_ids, num_tokens_post_padded, capacity, block_size, topk_weights, out,
                 workspace, stream, act_dtype)


def moe_w8a16_gemm(stage, a, M, topk, E, n_out, k_in, w_packed, scales, sorted_token_ids, expert_ids,
                   num_tokens_post_padded, capacity, block_size, topk_weights, out, workspace=None, stream=None,
                   act_dtype=WQ_BF16):
    return _gemm("moe_w8a16_gemm", stage, a, M, topk, E, n_out, k_in, w_packed, scales, -1, None,
                 sorted_token_ids, expert_ids, num_tokens_post_padded, capacity, block_size, topk_weights, out,
                 workspace, stream, act_dtype)


def moe_w8a16_gemm_noalloc(stage, a, M, topk, E, n_out, k_in, w_packed, scales, sorted_token_ids, expert_ids,
                           num_tokens_post_padded, capacity, block_size, topk_weights, out, stream=None,
                           act_dtype=WQ_BF16):
    """moe_w8a16_gemm with the library's own scratch as the workspace (no
    workspace argument; nothing is allocated)."""
    return _gemm("moe_w8a16_gemm_noalloc", stage, a, M, topk, E, n_out, k_in, w_packed, scales, -1, None,
                 sorted_token_ids, expert_ids, num_tokens_post_padded, capacity, block_size, topk_weights, out,
                 None, stream, act_dtype)


def moe_fp8_gemm_workspace_bytes(stage: int, M: int, topk: int, E: int, n_out: int, k_in: int) -> int:
    return int(load().moe_fp8_gemm_workspace_bytes(stage, M, topk, E, n_out, k_in))


def moe_fp8_w8a8_gemm(stage, a, M, topk, E, n_out, k_in, w_packed, scales, sorted_token_ids, expert_ids,
                      num_tokens_post_padded, capacity, block_size, topk_weights, out, workspace, in_scale: float,
                      out_scale: float = 1.0, stream=None, act_dtype=WQ_BF16):
    """FP8 (E4M3) W8A8 grouped GEMM: GATE_UP (x in act dtype -> H codes), DOWN
    (H codes -> out in act dtype) or RAW (x -> fp32); in_scale / out_scale are
    the static activation scales (a1, a2 for GATE_UP; a2 for DOWN)."""
    d = WqMoeGemmDesc()
    d.struct_size = C.sizeof(WqMoeGemmDesc)
    d.stage = stage
    d.act_dtype = act_dtype
    d.d_a = _ptr(a)
    d.M, d.topk, d.E, d.n_out, d.k_in = M, topk, E, n_out, k_in
    d.d_w_packed = _ptr(w_packed)
    d.d_scales = _ptr(scales)
    d.group_size = -1
    d.d_k_perm = None
    d.d_sorted_token_ids = _ptr(sorted_token_ids)
    d.d_expert_ids = _ptr(expert_ids)
    d.d_num_tokens_post_padded = _ptr(num_tokens_post_padded)
    d.capacity = capacity
    d.block_size = block_size
    d.d_topk_weights = _ptr(topk_weights)
    d.d_out = _ptr(out)
    d.d_workspace = _ptr(workspace)
    d.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(load().moe_fp8_w8a8_gemm(C.byref(d), float(in_scale), float(out_scale), _stream(stream)),
          "moe_fp8_w8a8_gemm")
    return out


def moe_fp8_codes_gemm(stage, codes, row_scales, M, topk, E, n_out, k_in, w_packed, scales, sorted_token_ids,
                       expert_ids, num_tokens_post_padded, capacity, block_size, out, in_scale: float = 1.0,
                       out_scale: float = 1.0, stream=None):
    """The GATE_UP (-> H codes [capacity, n_out / 2]) or RAW (-> fp32 [M * topk,
    n_out]) stage of moe_fp8_w8a8_gemm on E4M3 codes [M, k_in] (rms_norm's),
    with row_scales [M] float32 or, for None, in_scale for every row.  w_packed
    (E * n_out * k_in codes), scales (E * n_out float32) and the routing arrays
    of moe_align are checked for their size and type."""
    torch = _torch()
    _int32(M=M, topk=topk, E=E, n_out=n_out, k_in=k_in, block_size=block_size)
    f8 = (torch.uint8, torch.float8_e4m3fn)
    _check(codes, "codes", (M, k_in), f8)
    if row_scales is not None:
        _check(row_scales, "row_scales", (M,), (torch.float32,), codes.device)
    if stage == WQ_STAGE_GATE_UP:
        _check(out, "out", (max(capacity, 1), n_out // 2), f8, codes.device)
    elif stage == WQ_STAGE_RAW:
        _check(out, "out", (M * topk, n_out), (torch.float32,), codes.device)
    i32 = (torch.int32,)
    _holds(w_packed, "w_packed", E * n_out * k_in, f8)
    _holds(scales, "scales", E * n_out, (torch.float32,))
    _holds(sorted_token_ids, "sorted_token_ids", capacity, i32)
    _holds(expert_ids, "expert_ids", capacity // block_size if block_size > 0 else 0, i32)
    _holds(num_tokens_post_padded, "num_tokens_post_padded", 1, i32)
    d = _desc(stage, codes, M, topk, E, n_out, k_in, w_packed, scales, -1, None, sorted_token_ids, expert_ids,
              num_tokens_post_padded, capacity, block_size, None, out, None, WQ_BF16)
    check(load().moe_fp8_codes_gemm(C.byref(d), _ptr(row_scales), in_scale, out_scale, _stream(stream)),
          "moe_fp8_codes_gemm")
    return out


def _sparse24(fn, x, vals, meta, scales, N, out, group_size, stream):
    torch = _torch()
    M, K = x.shape
    new = []
    if out is None:
        new.append(out := _alloc(stream, torch.empty, (M, N), dtype=torch.float16, device=x.device))
    check(fn(_ptr(x), M, K, N, _ptr(vals), _ptr(meta), _ptr(scales), group_size, _ptr(out), act_code(x.dtype),
             _stream(stream)), fn.__name__)
    _keep_for(stream, *new)
    return out


def sparse24_w4a16_gemm(x, vals, meta, scales, N: int, out=None, group_size: int = 128, stream=None):
    """x [M, K] fp16 (device) -> y [M, N] fp16, 4-bit kept codes."""
    return _sparse24(load().sparse24_w4a16_gemm, x, vals, meta, scales, N, out, group_size, stream)


def sparse24_w8a16_gemm(x, vals, meta, scales, N: int, out=None, group_size: int = 128, stream=None):
    """x [M, K] fp16 (device) -> y [M, N] fp16, 8-bit kept codes (packed with bits=8)."""
    return _sparse24(load().sparse24_w8a16_gemm, x, vals, meta, scales, N, out, group_size, stream)


def dense_gemm_workspace_bytes(M: int, K: int, N: int, act_order: bool = False) -> int:
    return int(load().dense_gemm_workspace_bytes(M, K, N, int(bool(act_order))))


class Lora(NamedTuple):
    """The adapters of a batch beside one projection: stacked weights of one
    rank (pack_lora pads lower ones) and every row's adapter (-1: none)."""
    adapter_ids: object  # [M] int32
    a: object            # [adapters, rank, K] act dtype
    b: object            # [adapters, N, rank] act dtype
    scales: object       # [adapters] float32, or None for ones


def pack_lora(adapters, act, device="cuda"):
    """Adapters [(A [r, K], B [N, r], scale), ...] of any ranks -> (a [L, R, K],
    b [L, N, R], scales [L] float32) on the device, R the largest rank rounded
    up to 8, lower ranks padded with zeros."""
    torch = _torch()
    act_code(act)
    if not adapters:
        raise ValueError("no adapters")
    K, N = adapters[0][0].shape[1], adapters[0][1].shape[0]
    for A, B, _ in adapters:
        if A.dim() != 2 or B.dim() != 2 or A.shape[1] != K or B.shape[0] != N or A.shape[0] != B.shape[1]:
            raise ValueError("adapters must be A [r, %d], B [%d, r], got %s, %s" % (K, N, list(A.shape), list(B.shape)))
    R = max(8, -(-max(A.shape[0] for A, _, _ in adapters) // 8) * 8)
    a = torch.zeros((len(adapters), R, K), dtype=act)
    b = torch.zeros((len(adapters), N, R), dtype=act)
    for i, (A, B, _) in enumerate(adapters):
        a[i, :A.shape[0]] = A.detach()
        b[i, :, :B.shape[1]] = B.detach()
    scales = torch.tensor([float(s) for _, _, s in adapters], dtype=torch.float32)
    return a.to(device), b.to(device), scales.to(device)


def dense_lora_workspace_bytes(M: int, K: int, N: int, R: int, adapters: int) -> int:
    return int(load().dense_lora_workspace_bytes(M, K, N, R, adapters))


def _lora_sizes(x, adapter_ids, a, b, scales, y):
    """Checks the arguments of dense_lora_gemm -> (M, K, N, R, adapters, workspace bytes)."""
    torch = _torch()
    act_code(x.dtype)
    if x.dim() != 2 or y.dim() != 2 or a.dim() != 3:
        raise ValueError("x must be [M, K], y [M, N], a [adapters, rank, K], got %s, %s, %s"
                         % (list(x.shape), list(y.shape), list(a.shape)))
    (M, K), N, (L, R, _) = x.shape, y.shape[1], a.shape
    _int32(M=M, K=K, N=N, rank=R, adapters=L)
    dev, same = x.device, (x.dtype,)
    _check(x, "x", (M, K), same, row_stride=True)
    _check(y, "y", (M, N), same, dev, row_stride=True)
    _check(a, "a", (L, R, K), same, dev)
    _check(b, "b", (L, N, R), same, dev)
    _check(adapter_ids, "adapter_ids", (M,), (torch.int32,), dev)
    if scales is not None:
        _check(scales, "scales", (L,), (torch.float32,), dev)
    nbytes = dense_lora_workspace_bytes(M, K, N, R, L)
    if M and not nbytes:
        raise ValueError("unsupported adapters: M %d K %d N %d rank %d (multiples of 8, rank at most 256, N * rank < 2^31)"
                         % (M, K, N, R))
    for t, name in ((x, "x"), (y, "y"), (adapter_ids, "adapter_ids"), (a, "a"), (b, "b"), (scales, "scales")):
        if M and t is not None and t.data_ptr() % 16:
            raise ValueError("%s is not 16-byte aligned" % name)
    return M, K, N, R, L, nbytes


def dense_lora_gemm(x, adapter_ids, a, b, scales, y, workspace=None, stream=None):
    """Adds the rows' own adapters to y in place: y[m] += scales[i] * (x[m] a[i]^T)
    b[i]^T with i = adapter_ids[m] (rows with an id outside [0, adapters) stay as
    they are).  x [M, K], y [M, N] bf16/fp16 (device; rows may be strided), a
    [adapters, rank, K] and b [adapters, N, rank] in their type, scales
    [adapters] float32 or None for ones.  Returns y."""
    sizes = _lora_sizes(x, adapter_ids, a, b, scales, y)
    if workspace is not None and (not workspace.is_contiguous() or workspace.device != x.device):
        raise ValueError("workspace must be contiguous on %s" % x.device)
    return _lora_call(sizes, x, adapter_ids, a, b, scales, y, workspace, stream)


def _lora_call(sizes, x, adapter_ids, a, b, scales, y, workspace, stream):
    """dense_lora_gemm of arguments that _lora_sizes has passed."""
    torch = _torch()
    M, K, N, R, L, nbytes = sizes
    if workspace is None:
        workspace = _alloc(stream, torch.empty, nbytes, dtype=torch.uint8, device=x.device)
    check(load().dense_lora_gemm(_ptr(x), _row_stride(x), M, K, N, R, L, _ptr(adapter_ids), _ptr(a), _ptr(b),
                                 _ptr(scales), _ptr(y), _row_stride(y), act_code(x.dtype), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)), "dense_lora_gemm")
    return y


_ACTIVATION = {None: _lib.WQ_ACT_NONE, "relu": _lib.WQ_ACT_RELU, "silu": _lib.WQ_ACT_SILU, "gelu": _lib.WQ_ACT_GELU,
               "gelu_tanh": _lib.WQ_ACT_GELU_TANH}


def dense_epilogue_workspace_bytes(wbits: int, M: int, K: int, N: int, act_order: bool = False) -> int:
    _int32(M=M, K=K, N=N)
    return int(load().dense_epilogue_workspace_bytes(wbits, M, K, N, int(bool(act_order))))


def _dense_epilogue(wbits, x, N, w_packed, scales, group_size, k_perm, out, workspace, stream, lora, bias, activation,
                    residual):
    """The dense call that has a bias, an activation or a residual."""
    torch = _torch()
    if x.dim() != 2:
        raise ValueError("x must be [M, K], got %s" % list(x.shape))
    (M, K), dt, dev = x.shape, x.dtype, x.device
    act = act_code(dt)
    _int32(M=M, K=K, N=N)
    same = (dt,)
    _check(x, "x", (M, K), same)
    if activation not in _ACTIVATION:
        raise ValueError("activation must be one of %s, got %r" % (list(_ACTIVATION), activation))
    if lora is not None and activation is not None:
        raise ValueError("an activation beside adapters: they are added to the output, not before it")
    # (uint8, int8: the packers' bytes; 16-bit scales in the activation type or as its bits)
    _holds(w_packed, "w_packed", N * K * wbits // 8, (torch.uint8, torch.int8))
    _holds(scales, "scales", N * (K // 128 if group_size == 128 else 1), (dt, torch.int16, torch.uint16))
    if k_perm is not None:
        _holds(k_perm, "k_perm", K, (torch.int32,))
    e = WqEpilogue(C.sizeof(WqEpilogue), None, None, 0, _ACTIVATION[activation])
    if bias is not None:
        _check(bias, "bias", (N,), same, dev)
        e.d_bias = bias.data_ptr()
    if residual is not None:
        _check(residual, "residual", (M, N), same, dev, row_stride=True)
        e.d_residual, e.residual_stride = residual.data_ptr(), _row_stride(residual)
    new = []
    if out is None:
        out = _new(stream, new, (M, N), dt, dev)
    else:
        _check(out, "out", (M, N), same, dev)
    sizes = None if lora is None else _lora_sizes(x, *lora, out)  # before anything is launched
    L = load()
    if workspace is None:
        nb = L.dense_epilogue_workspace_bytes(wbits, M, K, N, int(k_perm is not None))
        if nb:
            workspace = _new(stream, [], nb, torch.uint8, dev)
    elif not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError("workspace must be contiguous on %s" % dev)
    tail = (C.byref(e), out.data_ptr(), act, _ptr(workspace),
            0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream))
    if wbits == 4:
        check(L.dense_w4a16_epilogue_gemm(x.data_ptr(), M, K, N, _ptr(w_packed), _ptr(scales), group_size, _ptr(k_perm),
                                          *tail), "dense_w4a16_epilogue_gemm")
    else:
        check(L.dense_w8a16_epilogue_gemm(x.data_ptr(), M, K, N, _ptr(w_packed), _ptr(scales), *tail),
              "dense_w8a16_epilogue_gemm")
    if lora is not None:
        _lora_call(sizes, x, *lora, out, None, stream)
    _keep_for(stream, *new)
    return out


def _dense(fn, x, N, w_packed, scales, extra, out, workspace, stream, act_order, lora):
    torch = _torch()
    M, K = x.shape
    new = []
    if out is None:
        new.append(out := _alloc(stream, torch.empty, (M, N), dtype=x.dtype, device=x.device))
    if lora is not None:  # before anything is launched
        if not (x.is_contiguous() and out.is_contiguous()):
            raise ValueError("x and out must be contiguous")
        if out.shape != (M, N):
            raise ValueError("out must be %s, got %s" % ([M, N], list(out.shape)))
        sizes = _lora_sizes(x, *lora, out)
    if workspace is None:
        nb = dense_gemm_workspace_bytes(M, K, N, act_order)
        workspace = _alloc(stream, torch.empty, max(nb, 1), dtype=torch.uint8, device=x.device)
    check(fn(_ptr(x), M, K, N, _ptr(w_packed), _ptr(scales), *extra, _ptr(out), act_code(x.dtype), _ptr(workspace),
             workspace.numel(), _stream(stream)), fn.__name__)
    if lora is not None:
        _lora_call(sizes, x, *lora, out, None, stream)
    _keep_for(stream, *new)
    return out


def dense_w4a16_gemm(x, N: int, w_packed, scales, group_size: int = 128, k_perm=None, out=None, workspace=None,
                     stream=None, lora: Optional[Lora] = None, bias=None, activation: Optional[str] = None,
                     residual=None):
    """Dense int4 linear: x [M, K] fp16 (device) -> y [M, N] fp16, weights
    packed by pack_w4 with E = 1; lora: the rows' adapters, added to y.  With a
    bias [N], an activation ("relu", "silu", "gelu", "gelu_tanh") or a residual
    [M, N] (rows may be strided; may be out): y = activation(x W^T + bias) +
    residual in float32, then rounded (workspace: dense_epilogue_workspace_bytes).
    Large batches take each weight, code times scale, rounded to fp16."""
    if bias is not None or activation is not None or residual is not None:
        return _dense_epilogue(4, x, N, w_packed, scales, group_size, k_perm, out, workspace, stream, lora, bias,
                               activation, residual)
    return _dense(load().dense_w4a16_gemm, x, N, w_packed, scales, (group_size, _ptr(k_perm)), out, workspace,
                  stream, k_perm is not None, lora)


def dense_w8a16_gemm(x, N: int, w_packed, scales, out=None, workspace=None, stream=None,
                     lora: Optional[Lora] = None, bias=None, activation: Optional[str] = None, residual=None):
    """Dense int8 linear: x [M, K] bf16/fp16 (device) -> y [M, N], weights
    packed by pack_w8 with E = 1; lora: the rows' adapters, added to y; bias,
    activation and residual as for dense_w4a16_gemm."""
    if bias is not None or activation is not None or residual is not None:
        return _dense_epilogue(8, x, N, w_packed, scales, -1, None, out, workspace, stream, lora, bias, activation,
                               residual)
    return _dense(load().dense_w8a16_gemm, x, N, w_packed, scales, (), out, workspace, stream, False, lora)


# ----------------------------------------------------------------------------
# paged key-value cache and attention over it
# ----------------------------------------------------------------------------
class KVCache(NamedTuple):
    """A paged key-value cache [pages, kv_heads, page_size, head_dim]: 16-bit
    values, or E4M3 codes with a scale a row (tensors) or one for all (numbers)."""
    k: object               # act dtype, or uint8 / float8_e4m3fn codes
    v: object
    k_scale: object = None  # of codes: float32 [pages, kv_heads, page_size], or a number
    v_scale: object = None


def kv_cache(pages: int, kv_heads: int, page_size: int, head_dim: int, act, quant: Optional[str] = None,
             k_scale: Optional[float] = None, v_scale: Optional[float] = None, device="cuda") -> KVCache:
    """An empty cache: of the act dtype, or of E4M3 codes with a scale a row
    (quant="row") or the calibrated k_scale and v_scale (quant="static")."""
    torch = _torch()
    act_code(act)
    if quant not in (None, "row", "static"):
        raise ValueError("quant must be None, 'row' or 'static', got %r" % (quant,))
    if (quant == "static") != (k_scale is not None) or (quant == "static") != (v_scale is not None):
        raise ValueError("k_scale and v_scale go with quant='static'")
    shape = (pages, kv_heads, page_size, head_dim)
    k, v = (torch.empty(shape, dtype=torch.uint8 if quant else act, device=device) for _ in range(2))
    if quant == "row":
        k_scale, v_scale = (torch.empty(shape[:3], dtype=torch.float32, device=device) for _ in range(2))
    c = KVCache(k, v, k_scale, v_scale)
    _kv_desc(c, act)
    return c


def _kv_desc(c: KVCache, act, device=None) -> WqKvCache:
    """Checks a cache for a call with activations of type act -> its descriptor."""
    torch = _torch()
    k, v, ks, vs = c
    shape, dt = k.shape, k.dtype
    if len(shape) != 4:
        raise ValueError("the cache must be [pages, kv_heads, page_size, head_dim], got %s" % list(shape))
    codes = dt != act
    if codes and dt not in (torch.uint8, torch.float8_e4m3fn):
        raise TypeError("the cache must be %s or E4M3 codes, got %s" % (act, dt))
    dev = k.device if device is None else device
    if not (v.shape == shape and v.dtype == dt and k.device == dev and v.device == dev and k.is_contiguous()
            and v.is_contiguous()):
        _check(k, "cache k", shape, (dt,), dev)
        _check(v, "cache v", shape, (dt,), dev)
    P, H, S, D = shape
    if P > 0x7fffffff or H > 0x7fffffff or S > 0x7fffffff or D > 0x7fffffff:
        _int32(pages=P, kv_heads=H, page_size=S, head_dim=D)
    if codes:
        if ks is None or vs is None:
            raise ValueError("a cache of codes has k_scale and v_scale")
        if isinstance(ks, torch.Tensor) != isinstance(vs, torch.Tensor):
            raise TypeError("k_scale and v_scale are both tensors or both numbers")
        if isinstance(ks, torch.Tensor):
            _check(ks, "cache k_scale", shape[:3], (torch.float32,), dev)
            _check(vs, "cache v_scale", shape[:3], (torch.float32,), dev)
            return WqKvCache(_KV_SIZE, k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), 0.0, 0.0, WQ_E4M3, P,
                             H, S, D)
        return WqKvCache(_KV_SIZE, k.data_ptr(), v.data_ptr(), None, None, ks, vs, WQ_E4M3, P, H, S, D)
    if ks is not None or vs is not None:
        raise ValueError("a cache of 16-bit values has no scales")
    return WqKvCache(_KV_SIZE, k.data_ptr(), v.data_ptr(), None, None, 0.0, 0.0, act_code(act), P, H, S, D)


_KV_SIZE = C.sizeof(WqKvCache)


def _head_rows(t, name: str, T: int, H: int, D: int, act, device) -> int:
    """A [T, H, D] argument whose heads lie next to each other (rows may be
    strided) -> its row stride in elements."""
    if t.shape != (T, H, D):
        raise ValueError("%s must be %s, got %s" % (name, [T, H, D], list(t.shape)))
    if t.dtype != act:
        raise TypeError("%s must be %s, got %s" % (name, act, t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
    s0, s1, s2 = t.stride()
    if T <= 1:
        s0 = H * D
    if (s2 != 1 and D > 1 or s1 != D and H > 1 or s0 < H * D) and t.numel():
        raise ValueError("%s must be contiguous in its rows, got strides %s" % (name, list(t.stride())))
    return s0


def _new(stream, new, shape, dtype, device):
    """A buffer that the call allocates, noted in `new`."""
    if stream is None:
        t = _torch().empty(shape, dtype=dtype, device=device)
    else:
        t = _alloc(stream, _torch().empty, shape, dtype=dtype, device=device)
    new.append(t)
    return t


def kv_cache_write(k, v, cache: KVCache, slots, stream=None) -> KVCache:
    """The rows of new tokens into the cache, quantised where it holds codes: k, v
    [T, kv_heads, head_dim] bf16/fp16 (device; rows may be strided), slots [T]
    int64 (page * page_size + position; outside the cache, as -1 of a padding
    token: not written).  The slots of a call differ.  Returns the cache."""
    dt, dev = k.dtype, k.device
    act = act_code(dt)
    d = _kv_desc(cache, dt, dev)
    if k.dim() != 3:
        raise ValueError("k must be [T, kv_heads, head_dim], got %s" % list(k.shape))
    T, H, D = k.shape[0], d.kv_heads, d.head_dim
    _int32(T=T)
    ks, vs = _head_rows(k, "k", T, H, D, dt, dev), _head_rows(v, "v", T, H, D, dt, dev)
    _check(slots, "slots", (T,), (_torch().int64,), dev)
    check(load().wq_kv_cache_write(C.byref(d), k.data_ptr(), ks, v.data_ptr(), vs, slots.data_ptr(), T, act,
                                   _stream(stream)), "wq_kv_cache_write")
    return cache


def kv_cache_read(cache: KVCache, slots, act, k=None, v=None, stream=None):
    """The rows of slots [T] int64 back -> (k, v) [T, kv_heads, head_dim] of type
    act (rows of given buffers may be strided); zeros where a slot is outside
    the cache."""
    dev = cache.k.device
    code = act_code(act)
    d = _kv_desc(cache, act, dev)
    if slots.dim() != 1:
        raise ValueError("slots must be [T], got %s" % list(slots.shape))
    T, H, D = slots.shape[0], d.kv_heads, d.head_dim
    _check(slots, "slots", (T,), (_torch().int64,), dev)
    _int32(T=T)
    new = []
    ks = vs = H * D
    if k is None:
        k = _new(stream, new, (T, H, D), act, dev)
    else:
        ks = _head_rows(k, "k", T, H, D, act, dev)
    if v is None:
        v = _new(stream, new, (T, H, D), act, dev)
    else:
        vs = _head_rows(v, "v", T, H, D, act, dev)
    check(load().wq_kv_cache_read(C.byref(d), slots.data_ptr(), T, k.data_ptr(), ks, v.data_ptr(), vs, code,
                                  _stream(stream)), "wq_kv_cache_read")
    _keep_for(stream, *new)
    return k, v


def paged_attention_workspace_bytes(B: int, heads: int, kv_heads: int, head_dim: int, page_size: int,
                                    table_width: int, window: int = 0) -> int:
    _int32(B=B, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page_size=page_size, table_width=table_width,
           window=window)
    return int(load().wq_paged_attention_workspace_bytes(B, heads, kv_heads, head_dim, page_size, table_width, window))


def paged_attention(q, cache: KVCache, block_table, lengths, scale: Optional[float] = None, window: int = 0,
                    out=None, want_lse: bool = False, lse=None, workspace=None, stream=None):
    """Attention of one new token a sequence over its tokens in the cache: q [B,
    heads, head_dim] bf16/fp16 (device; rows may be strided), block_table [B,
    width] int32 (the page of each page_size tokens), lengths [B] int32 (0: no
    tokens, zeros out), heads a multiple of the cache's; scale: head_dim ** -0.5
    unless given; window: the last so many tokens only.  -> out like q, with
    want_lse (out, lse [B, heads] float32), the logarithm of each row's sum."""
    torch = _torch()
    dt, dev = q.dtype, q.device
    act = act_code(dt)
    d = _kv_desc(cache, dt, dev)
    if q.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q must be [B, heads, head_dim], block_table [B, width], got %s, %s"
                         % (list(q.shape), list(block_table.shape)))
    B, heads, D = q.shape
    width = block_table.shape[1]
    if D != d.head_dim or heads % d.kv_heads:
        raise ValueError("q must be [B, a multiple of %d heads, %d], got %s" % (d.kv_heads, d.head_dim, list(q.shape)))
    _int32(B=B, heads=heads, width=width, window=window)
    qs = _head_rows(q, "q", B, heads, D, dt, dev)
    i32 = (torch.int32,)
    _check(block_table, "block_table", (B, width), i32, dev)
    _check(lengths, "lengths", (B,), i32, dev)
    if lse is not None and not want_lse:
        raise ValueError("lse goes with want_lse")
    new = []
    if out is None:
        out, os_ = _new(stream, new, (B, heads, D), dt, dev), heads * D
    else:
        os_ = _head_rows(out, "out", B, heads, D, dt, dev)
    if want_lse:
        if lse is None:
            lse = _new(stream, new, (B, heads), torch.float32, dev)
        else:
            _check(lse, "lse", (B, heads), (torch.float32,), dev)
    L = load()
    if workspace is None:
        nb = L.wq_paged_attention_workspace_bytes(B, heads, d.kv_heads, D, d.page_size, width, window)
        if nb:
            workspace = _new(stream, [], nb, torch.uint8, dev)
    else:
        if not workspace.is_contiguous() or workspace.device != dev:
            raise ValueError("workspace must be contiguous on %s" % dev)
        nb = workspace.numel() * workspace.element_size()
    check(L.wq_paged_attention(C.byref(d), q.data_ptr(), qs, B, heads, block_table.data_ptr(), width,
                               lengths.data_ptr(), D ** -0.5 if scale is None else scale, window, out.data_ptr(), os_,
                               _ptr(lse), act, _ptr(workspace), nb, _stream(stream)), "wq_paged_attention")
    if stream is not None:
        _keep_for(stream, *new)
    return (out, lse) if want_lse else out


def quantize_w8(w, q=None, scales=None, stream=None):
    """ExpertsInt8 load-time quantization on the device: w [..., k] bf16/fp16
    (the 16-bit checkpoint; leading dims = experts x output columns) ->
    (q int8 [..., k], scales [...] in w's dtype), one scale per row."""
    torch = _torch()
    if w.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("quantize_w8 takes bf16 or fp16 weights, got %s" % w.dtype)
    w = _alloc(stream, w.contiguous)  # (a copy runs on the stream, before the kernel)
    k = w.shape[-1]
    rows = w.numel() // k if k else 0
    new = []
    if q is None:
        new.append(q := _alloc(stream, torch.empty, w.shape, dtype=torch.int8, device=w.device))
    if scales is None:
        new.append(scales := _alloc(stream, torch.empty, w.shape[:-1], dtype=w.dtype, device=w.device))
    check(load().wq_quantize_w8(_ptr(w), rows, k, act_code(w.dtype), _ptr(q), _ptr(scales), _stream(stream)),
          "wq_quantize_w8")
    _keep_for(stream, *new)
    return q, scales


# ----------------------------------------------------------------------------
# offline packers (host numpy in / out)
# ----------------------------------------------------------------------------
def pack_w4(q: np.ndarray, scales_bits: np.ndarray, group_size: int, g_idx: Optional[np.ndarray] = None,
            row_perm: Optional[np.ndarray] = None, interleave_gate_up: bool = False
            ) -> Tuple[np.ndarray, np.ndarray, Optional[np.ndarray]]:
    """q int8 [E, n_out, k_in], scales uint16 [E, G, n_out] -> (packed uint8, scales uint16, k_perm or None)."""
    q = np.ascontiguousarray(q, dtype=np.int8)
    E, n_out, k_in = q.shape
    s = np.ascontiguousarray(scales_bits, dtype=np.uint16)
    L = load()
    nbytes = int(L.wq_pack_w4_bytes(E, n_out, k_in))
    if nbytes == 0:
        raise ValueError("unsupported int4 shape %s" % (q.shape,))
    packed = np.empty(nbytes, np.uint8)
    sp = np.empty_like(s)
    gi = None if g_idx is None else np.ascontiguousarray(g_idx, dtype=np.int32)
    rp = None if row_perm is None else np.ascontiguousarray(row_perm, dtype=np.int32)
    kp = np.empty((E, k_in), np.int32) if gi is not None else None
    flags = WQ_PACK_INTERLEAVE_GATE_UP if interleave_gate_up else 0
    check(L.wq_pack_w4(E, n_out, k_in, _np_ptr(q), _np_ptr(s), group_size, _np_ptr(gi), _np_ptr(rp), flags,
                       _np_ptr(packed), _np_ptr(sp), _np_ptr(kp)), "wq_pack_w4")
    return packed, sp, kp


def pack_w8(q: np.ndarray, scales_bits: np.ndarray, row_perm: Optional[np.ndarray] = None,
            interleave_gate_up: bool = False) -> Tuple[np.ndarray, np.ndarray]:
    """q int8 [E, n_out, k_in], scales uint16 [E, 1, n_out] -> (packed uint8, scales uint16)."""
    q = np.ascontiguousarray(q, dtype=np.int8)
    E, n_out, k_in = q.shape
    s = np.ascontiguousarray(scales_bits, dtype=np.uint16)
    L = load()
    nbytes = int(L.wq_pack_w8_bytes(E, n_out, k_in))
    if nbytes == 0:
        raise ValueError("unsupported int8 shape %s" % (q.shape,))
    packed = np.empty(nbytes, np.uint8)
    sp = np.empty_like(s)
    rp = None if row_perm is None else np.ascontiguousarray(row_perm, dtype=np.int32)
    flags = WQ_PACK_INTERLEAVE_GATE_UP if interleave_gate_up else 0
    check(L.wq_pack_w8(E, n_out, k_in, _np_ptr(q), _np_ptr(s), _np_ptr(rp), flags, _np_ptr(packed), _np_ptr(sp)),
          "wq_pack_w8")
    return packed, sp


def pack_fp8(codes: np.ndarray, scales: np.ndarray, row_perm: Optional[np.ndarray] = None,
             interleave_gate_up: bool = False) -> Tuple[np.ndarray, np.ndarray]:
    """E4M3 codes uint8 [E, n_out, k_in], scales float32 [E, n_out] -> (packed uint8, scales float32)."""
    c = np.ascontiguousarray(codes, dtype=np.uint8)
    E, n_out, k_in = c.shape
    s = np.ascontiguousarray(scales, dtype=np.float32).reshape(E, n_out)
    L = load()
    nbytes = int(L.wq_pack_fp8_bytes(E, n_out, k_in))
    if nbytes == 0:
        raise ValueError("unsupported FP8 shape %s" % (c.shape,))
    packed = np.empty(nbytes, np.uint8)
    sp = np.empty_like(s)
    rp = None if row_perm is None else np.ascontiguousarray(row_perm, dtype=np.int32)
    flags = WQ_PACK_INTERLEAVE_GATE_UP if interleave_gate_up else 0
    check(L.wq_pack_fp8(E, n_out, k_in, _np_ptr(c), _np_ptr(s), _np_ptr(rp), flags, _np_ptr(packed), _np_ptr(sp)),
          "wq_pack_fp8")
    return packed, sp


def pack_sparse24(vals: np.ndarray, idx: np.ndarray, scales_bits: np.ndarray, group_size: int = 128, bits: int = 4):
    """vals int8 [N, K/2], idx uint8 [N, K/2], scales uint16 [K/128, N] (group
    128) or [1, N] (group -1) -> (vals, meta, scales) packed for 4- or 8-bit
    kept codes."""
    vals = np.ascontiguousarray(vals, dtype=np.int8)
    idx = np.ascontiguousarray(idx, dtype=np.uint8)
    s = np.ascontiguousarray(scales_bits, dtype=np.uint16)
    N, Kh = vals.shape
    K = 2 * Kh
    L = load()
    vb = int(L.wq_pack_sparse24_vals_bytes(N, K, bits))
    mb = int(L.wq_pack_sparse24_meta_bytes(N, K))
    if vb == 0 or mb == 0:
        raise ValueError("unsupported 2:4 shape N=%d K=%d" % (N, K))
    vp = np.empty(vb, np.uint8)
    mp = np.empty(mb, np.uint8)
    sp = np.empty_like(s)
    G = 1 if group_size == -1 else K // 128
    if s.shape != (G, N):
        raise ValueError("scales must be [%d, %d] for group_size %d, got %s" % (G, N, group_size, s.shape))
    check(L.wq_pack_sparse24(N, K, bits, group_size, _np_ptr(vals), _np_ptr(idx), _np_ptr(s), _np_ptr(vp),
                             _np_ptr(mp), _np_ptr(sp)), "wq_pack_sparse24")
    return vp, mp, sp


_ = (WQ_STAGE_GATE_UP, WQ_STAGE_DOWN, WQ_STAGE_RAW, WQ_F16, WQ_BF16, _lib)
