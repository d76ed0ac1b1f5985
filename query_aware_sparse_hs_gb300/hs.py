"""ctypes binding of ``libhs.so`` (the C ABI declared in ``include/hs.h``).

Argument marshalling only: tensors become device pointers and sizes, the call
goes to the CUDA library, a non-OK status raises :class:`HSError`.  Every step
of the computation runs in the library's kernels; there is no fallback.  The
library is built by ``python -m query_aware_sparse_hs_gb300.build`` (or
``__graft_entry__.build()``); importing this module without it fails loudly.
"""

from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_float, c_int32, c_int64, c_size_t, c_uint32, c_ulonglong, c_void_p

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libhs.so")

HS_OK, HS_ERR_INVALID_ARG, HS_ERR_UNSUPPORTED, HS_ERR_CUDA = 0, 1, 2, 3
HS_ERR_OUT_OF_RANGE, HS_ERR_CAPACITY, HS_ERR_TIMEOUT, HS_ERR_WORKSPACE = 4, 5, 6, 7
HS_ERR_SCRATCH_LIMIT = 8
HS_NOALLOC_SCRATCH_BYTES = 8 * 1024 * 1024
HS_ATTN_EARLY_SUMMARIES = 1
HS_ATTN_RANGES = 2
HS_ATTN_NO_RANGES = 4
HS_EBIT_PAGE_RANGE, HS_EBIT_CAPACITY, HS_EBIT_TIMEOUT, HS_EBIT_BLOCK_RANGE = 0x1, 0x2, 0x4, 0x8
HS_EBIT_POSITION = 0x10
KV_DTYPES = {"f32": 0, "bf16": 1, "fp8": 2, "fp8_block": 3, "int4": 4}
ALGO = {"auto": 0, "simt": 1, "tcgen05": 2}


class HSError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {hs_status_string(status)} (status {status})")


class AttnShape(ctypes.Structure):
    _fields_ = [("num_q_heads", c_int32), ("num_kv_heads", c_int32), ("head_dim", c_int32),
                ("block_size", c_int32), ("kv_dtype", c_int32)]


class PagedKV(ctypes.Structure):
    _fields_ = [("k_pages", c_void_p), ("v_pages", c_void_p), ("k_scales", c_void_p),
                ("v_scales", c_void_p), ("page_table", c_void_p), ("seq_lens", c_void_p),
                ("batch", c_int32), ("max_blocks", c_int32), ("num_pages", c_int64)]


class SelectParams(ctypes.Structure):
    _fields_ = [("sink_tokens", c_int32), ("window_tokens", c_int32), ("k_scored", c_int32),
                ("capacity", c_int32), ("history_weight", c_float), ("score_history", c_void_p)]


class AppendParams(ctypes.Structure):
    _fields_ = [("new_offsets", c_void_p), ("positions", c_void_p), ("cos_sin", c_void_p),
                ("table_rows", c_int32), ("rotary_dim", c_int32), ("interleaved", c_int32)]
    _requests = _rows = _device = None  # what append_params knows of its tensors; of addresses nothing is known


class AttnParams(ctypes.Structure):
    _fields_ = [("scale", c_float), ("out_is_fp32", c_int32), ("blocks_per_split", c_int32),
                ("algo", c_int32), ("max_ctas", c_int32), ("split_counters", c_void_p),
                ("wait_limit_ns", c_uint32), ("flags", c_uint32)]


class HotBuffer(ctypes.Structure):
    _fields_ = [("page_table", c_void_p), ("slot_owner", c_void_p), ("last_used", c_void_p),
                ("k_slots", c_void_p), ("v_slots", c_void_p), ("k_slot_scales", c_void_p),
                ("v_slot_scales", c_void_p), ("host_k", c_void_p), ("host_v", c_void_p),
                ("host_k_scales", c_void_p), ("host_v_scales", c_void_p), ("batch", c_int32),
                ("max_blocks", c_int32), ("slots_per_stream", c_int32)]


class EvictParams(ctypes.Structure):
    _fields_ = [("budget", c_int32), ("sink_tokens", c_int32), ("recent_tokens", c_int32)]


class SwapStats(ctypes.Structure):
    _fields_ = [("hits", c_ulonglong), ("misses", c_ulonglong), ("evictions", c_ulonglong),
                ("bytes_in", c_ulonglong)]


SYMBOLS = {
    "hs_status_string": (ctypes.c_char_p, [c_int32]),
    "hs_version": (c_int32, []),
    "hs_workspace_bytes": (c_size_t, [POINTER(AttnShape), c_int32, c_int32, POINTER(AttnParams)]),
    "hs_attn_geometry": (c_int32, [POINTER(AttnShape), c_int32, c_int32, POINTER(AttnParams),
                                   POINTER(c_int32), POINTER(c_int32)]),
    "hs_select_workspace_bytes": (c_size_t, [POINTER(AttnShape), c_int32, c_int32]),
    "hs_build_block_summaries": (c_int32, [POINTER(AttnShape), POINTER(PagedKV), c_int32, c_void_p,
                                           c_void_p, c_void_p]),
    "hs_append_token": (c_int32, [POINTER(AttnShape), POINTER(PagedKV), c_void_p, c_void_p, c_void_p,
                                  c_void_p, c_void_p]),
    "hs_append_tokens": (c_int32, [POINTER(AttnShape), POINTER(PagedKV), POINTER(AppendParams), c_int64,
                                   c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64,
                                   c_void_p, c_void_p, c_void_p]),
    "hs_score_select_topk": (c_int32, [POINTER(AttnShape), POINTER(PagedKV), c_void_p, c_void_p,
                                       c_void_p, POINTER(SelectParams), c_void_p, c_void_p, c_void_p,
                                       c_void_p, c_size_t, c_void_p]),
    "hs_sparse_paged_decode_attn": (c_int32, [POINTER(AttnShape), POINTER(PagedKV), c_void_p, c_void_p,
                                              c_void_p, c_int32, POINTER(AttnParams), c_void_p, c_void_p,
                                              c_void_p, c_size_t, c_void_p]),
    "hs_score_select_attend_workspace_bytes": (c_size_t, [POINTER(AttnShape), c_int32, c_int32, c_int32,
                                                          POINTER(AttnParams)]),
    "hs_score_select_attend_fused": (c_int32, [POINTER(AttnShape), c_int32, c_int32, c_int32,
                                               POINTER(AttnParams)]),
    "hs_score_select_attend": (c_int32, [POINTER(AttnShape), POINTER(PagedKV), c_void_p, c_void_p, c_void_p,
                                         POINTER(SelectParams), c_void_p, c_void_p, c_void_p, POINTER(AttnParams),
                                         c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "hs_decode_step": (c_int32, [POINTER(AttnShape), POINTER(PagedKV), c_void_p, c_void_p, c_void_p, c_void_p,
                                 c_void_p, POINTER(SelectParams), c_void_p, c_void_p, c_void_p, POINTER(AttnParams),
                                 c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "hs_decode_step_reuse": (c_int32, [POINTER(AttnShape), POINTER(PagedKV), c_void_p, c_void_p, c_void_p,
                                       c_void_p, c_void_p, c_void_p, c_void_p, c_int32, POINTER(AttnParams),
                                       c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "hs_sparse_paged_decode_attn_noalloc": (c_int32, [POINTER(AttnShape), POINTER(PagedKV), c_void_p,
                                                      c_void_p, c_void_p, c_int32, POINTER(AttnParams),
                                                      c_void_p, c_void_p, c_void_p]),
    "hs_swapin_misses": (c_int32, [POINTER(AttnShape), POINTER(HotBuffer), c_void_p, c_void_p, c_int32,
                                   c_int32, c_void_p, c_void_p]),
    "hs_swapin_plan": (c_int32, [POINTER(AttnShape), POINTER(HotBuffer), c_void_p, c_void_p, c_int32, c_int32,
                                 c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "hs_score_select_swapin_plan": (c_int32, [POINTER(AttnShape), POINTER(PagedKV), c_void_p, c_void_p, c_void_p,
                                              POINTER(SelectParams), c_void_p, c_void_p, c_void_p, c_void_p,
                                              c_size_t, POINTER(HotBuffer), c_int32, c_void_p, c_void_p, c_void_p,
                                              c_void_p, c_void_p, c_void_p]),
    "hs_swapin_copy": (c_int32, [POINTER(AttnShape), POINTER(HotBuffer), c_void_p, c_void_p, c_int32, c_int32,
                                 c_void_p, c_void_p]),
    "hs_swapin_copy_attend": (c_int32, [POINTER(AttnShape), POINTER(HotBuffer), c_void_p, c_void_p, c_void_p,
                                        c_void_p, c_int32, c_float, c_int32, c_void_p, c_void_p, c_void_p,
                                        c_void_p]),
    "hs_merge_attn_partials": (c_int32, [POINTER(AttnShape), c_int32, c_int32, c_void_p, c_void_p, c_void_p,
                                         c_int32, c_void_p, c_void_p]),
    "hs_quantize_e4m3_g32": (c_int32, [c_void_p, c_int32, c_int64, c_int32, c_void_p, c_void_p,
                                       c_void_p]),
    "hs_quantize_int4_g32": (c_int32, [c_void_p, c_int32, c_int64, c_int32, c_void_p, c_void_p, c_void_p]),
    "hs_dequantize_int4_g32": (c_int32, [c_void_p, c_void_p, c_int64, c_int32, c_void_p, c_int32, c_void_p]),
    "hs_accumulate_attn_weights": (c_int32, [POINTER(AttnShape), POINTER(PagedKV), c_void_p, c_void_p, c_void_p,
                                             c_void_p, c_int32, c_float, c_void_p, c_void_p]),
    "hs_evict_tokens": (c_int32, [POINTER(AttnShape), POINTER(PagedKV), POINTER(PagedKV), POINTER(EvictParams),
                                  c_void_p, c_void_p, c_void_p, c_void_p]),
    "hs_get_device_error": (c_int32, [c_void_p, POINTER(c_uint32)]),
    "hs_get_device_error_detail": (c_int32, [c_void_p, POINTER(c_uint32), POINTER(c_uint32)]),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m query_aware_sparse_hs_gb300.build`")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SYMBOLS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def library():
    return _lib


def hs_status_string(status: int) -> str:
    return _lib.hs_status_string(int(status)).decode()


def hs_version() -> int:
    return int(_lib.hs_version())


def _check(status: int, where: str):
    if status != HS_OK:
        raise HSError(status, where)


def _ptr(t) -> int | None:
    if t is None or isinstance(t, int):  # None, or an address already
        return t
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return t.data_ptr()


# The short ways, several microseconds a call shorter; a torch without them (or without CUDA) has the public ones.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream) -> int | None:
    if stream is None:
        if torch.cuda.is_initialized():  # the current device's current stream, without building a Stream object
            return _raw_stream(_current_device())
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def attn_shape(num_q_heads, num_kv_heads, head_dim, block_size, kv_dtype) -> AttnShape:
    return AttnShape(num_q_heads, num_kv_heads, head_dim, block_size,
                     KV_DTYPES[kv_dtype] if isinstance(kv_dtype, str) else int(kv_dtype))


def paged_kv(k_pages, v_pages, page_table, seq_lens, k_scales=None, v_scales=None) -> PagedKV:
    """Describe a paged cache: pages [num_pages][B][D] (4-bit: [num_pages][B][D/2] bytes), page_table
    [batch][Hkv][max_blocks], scales as hs.h lays them out (4-bit: [num_pages][B][2][D/32] bf16)."""
    kv = PagedKV(_ptr(k_pages), _ptr(v_pages), _ptr(k_scales), _ptr(v_scales), _ptr(page_table),
                 _ptr(seq_lens), int(page_table.shape[0]), int(page_table.shape[-1]),
                 int(k_pages.shape[0]))
    kv._keep = (k_pages, v_pages, page_table, seq_lens, k_scales, v_scales)
    return kv


def select_params(sink_tokens, window_tokens, k_scored, capacity, history_weight=0.0,
                  score_history=None) -> SelectParams:
    p = SelectParams(sink_tokens, window_tokens, k_scored, capacity, float(history_weight), _ptr(score_history))
    p._keep = score_history
    return p


def attn_params(scale, out_is_fp32=False, blocks_per_split=0, algo="auto", max_ctas=0,
                split_counters=None, wait_limit_ns=0, early_summaries=False, ranges=None) -> AttnParams:
    """wait_limit_ns: bound of the tensor-core kernels' waits (0 = 2 s).
    early_summaries: HS_ATTN_EARLY_SUMMARIES (smin/smax are not written by the
    kernel launched just before the call on its stream).  ranges: True =
    HS_ATTN_RANGES, False = HS_ATTN_NO_RANGES, None = the library's choice."""
    flags = (HS_ATTN_EARLY_SUMMARIES if early_summaries else 0) | \
        {None: 0, True: HS_ATTN_RANGES, False: HS_ATTN_NO_RANGES}[ranges]
    p = AttnParams(float(scale), 1 if out_is_fp32 else 0, int(blocks_per_split),
                   ALGO[algo] if isinstance(algo, str) else int(algo), int(max_ctas), _ptr(split_counters),
                   int(wait_limit_ns), flags)
    p._keep = split_counters
    return p


def hs_workspace_bytes(shape: AttnShape, batch: int, capacity: int, params: AttnParams) -> int:
    return int(_lib.hs_workspace_bytes(ctypes.byref(shape), batch, capacity, ctypes.byref(params)))


def hs_attn_geometry(shape: AttnShape, batch: int, capacity: int, params: AttnParams):
    """(splits, chunks_per_cta) of the tensor-core attention; chunks_per_cta 0 = equal splits."""
    sp, per = c_int32(0), c_int32(0)
    if _lib.hs_attn_geometry(ctypes.byref(shape), batch, capacity, ctypes.byref(params), ctypes.byref(sp),
                             ctypes.byref(per)) != 0:
        raise HSError(HS_ERR_INVALID_ARG, "hs_attn_geometry")
    return sp.value, per.value


def hs_select_workspace_bytes(shape: AttnShape, batch: int, max_blocks: int) -> int:
    return int(_lib.hs_select_workspace_bytes(ctypes.byref(shape), batch, max_blocks))


def hs_build_block_summaries(shape, kv, first_block, smin, smax, stream=None):
    _check(_lib.hs_build_block_summaries(ctypes.byref(shape), ctypes.byref(kv), int(first_block),
                                         _ptr(smin), _ptr(smax), _stream(stream)),
           "hs_build_block_summaries")


def hs_append_token(shape, kv, new_k, new_v, smin, smax, stream=None):
    _check(_lib.hs_append_token(ctypes.byref(shape), ctypes.byref(kv), _ptr(new_k), _ptr(new_v), _ptr(smin),
                                _ptr(smax), _stream(stream)),
           "hs_append_token")


def append_params(cos_sin=None, interleaved=False, new_offsets=None, positions=None, rotary_dim=None) -> AppendParams:
    """What hs_append_tokens is told besides the rows.  cos_sin: [positions][rotary_dim] f32, the cosines of a
    position's rotary_dim/2 angles, then their sines (None: no rotation).  interleaved: pairs (2i, 2i+1) instead of
    (i, i + rotary_dim/2).  new_offsets: [batch + 1] int32, the rows of each request (None: one row each).
    positions: [rows] int32 (None: each row's position in the cache)."""
    if rotary_dim is None:
        rotary_dim = int(cos_sin.shape[1]) if cos_sin is not None else 0
    elif cos_sin is not None and cos_sin.shape[1] != rotary_dim:
        raise ValueError("cos_sin must be [positions][rotary_dim]")
    for t, dt in ((cos_sin, torch.float32), (new_offsets, torch.int32), (positions, torch.int32)):
        if t is not None and t.dtype != dt:
            raise ValueError(f"expected {dt}, got {t.dtype}")
    devices = {t.get_device() for t in (cos_sin, new_offsets, positions) if t is not None}
    if len(devices) > 1:
        raise ValueError("cos_sin, new_offsets and positions must be on one device")
    p = AppendParams(_ptr(new_offsets), _ptr(positions), _ptr(cos_sin),
                     0 if cos_sin is None else int(cos_sin.shape[0]), int(rotary_dim), 1 if interleaved else 0)
    p._keep = (cos_sin, new_offsets, positions)
    p._requests = None if new_offsets is None else new_offsets.numel() - 1
    p._rows = None if positions is None else positions.numel()
    p._device = devices.pop() if devices else None
    return p


_append_tokens, _byref = _lib.hs_append_tokens, ctypes.byref
_BF16, _F32 = torch.bfloat16, torch.float32
_NEW_ROWS = "{} must be [{}][{}][{}] of {} with contiguous rows, on the current device"


def _new_rows(t, rows, heads, dim, dtype, device, what):
    """Address and row stride of a [rows][heads][dim] tensor whose rows are contiguous."""
    n, h, d = t.shape
    s, sh, sd = t.stride()
    if (n != rows or h != heads or d != dim or sd != 1 or (sh != dim and heads != 1) or t.dtype is not dtype
            or t.get_device() != device):
        raise ValueError(_NEW_ROWS.format(what, rows, heads, dim, dtype))
    return t.data_ptr(), s if n > 1 else heads * dim


def hs_append_tokens(shape, kv, params, new_k, new_v, q=None, q_out=None, smin=None, smax=None, stream=None):
    """Any number of new tokens per request into the paged cache, K and Q rotated on the way (see hs.h).  new_k,
    new_v [rows][Hkv][D], q, q_out [rows][Hq][D]; the rows may be strided views (of a fused projection)."""
    dim, hkv = shape.head_dim, shape.num_kv_heads
    rows = new_k.shape[0]
    dtype = _BF16 if shape.kv_dtype else _F32
    device = _current_device() if new_k.is_cuda else -2
    kp, ks = _new_rows(new_k, rows, hkv, dim, dtype, device, "new_k")
    vp, vs = _new_rows(new_v, rows, hkv, dim, dtype, device, "new_v")
    if q is not None and q_out is not None:
        hq = shape.num_q_heads
        qp, qs = _new_rows(q, rows, hq, dim, dtype, device, "q")
        op, os_ = _new_rows(q_out, rows, hq, dim, dtype, device, "q_out")
    elif q is None and q_out is None:
        qp = op = None
        qs = os_ = 0
    else:
        raise ValueError("q and q_out are given together")
    if params._requests is not None and params._requests != kv.batch:
        raise ValueError("new_offsets must have batch + 1 entries")
    if params._rows is not None and params._rows < rows:
        raise ValueError("positions must have an entry for every row")
    if params._device is not None and params._device != device:
        raise ValueError("cos_sin, new_offsets and positions must be on the current device")
    st = _append_tokens(_byref(shape), _byref(kv), _byref(params), rows, qp, qs, op, os_, kp, ks, vp, vs, _ptr(smin),
                        _ptr(smax), _raw_stream(device) if stream is None else _stream(stream))
    if st:
        raise HSError(st, "hs_append_tokens")


def hs_score_select_topk(shape, kv, q, smin, smax, params, sel, sel_count, scores=None,
                         workspace=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.hs_score_select_topk(ctypes.byref(shape), ctypes.byref(kv), _ptr(q), _ptr(smin),
                                     _ptr(smax), ctypes.byref(params), _ptr(sel), _ptr(sel_count),
                                     _ptr(scores), _ptr(workspace), ws_bytes, _stream(stream)),
           "hs_score_select_topk")


def hs_sparse_paged_decode_attn(shape, kv, q, sel, sel_count, capacity, params, out, lse=None,
                                workspace=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.hs_sparse_paged_decode_attn(ctypes.byref(shape), ctypes.byref(kv), _ptr(q), _ptr(sel),
                                            _ptr(sel_count), int(capacity), ctypes.byref(params),
                                            _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
                                            _stream(stream)),
           "hs_sparse_paged_decode_attn")


def hs_score_select_attend_workspace_bytes(shape: AttnShape, batch: int, max_blocks: int, capacity: int,
                                           params: AttnParams) -> int:
    return int(_lib.hs_score_select_attend_workspace_bytes(ctypes.byref(shape), batch, max_blocks, capacity,
                                                           ctypes.byref(params)))


def hs_score_select_attend_fused(shape: AttnShape, batch: int, max_blocks: int, capacity: int,
                                 params: AttnParams) -> int:
    """1: the combined call is one launch for this geometry on the current device; 0: separate launches."""
    return int(_lib.hs_score_select_attend_fused(ctypes.byref(shape), batch, max_blocks, capacity,
                                                 ctypes.byref(params)))


def hs_decode_step(shape, kv, q, new_k, new_v, smin, smax, sel_params, sel, sel_count, scores, attn_params, out,
                   lse=None, workspace=None, stream=None):
    """Append of the newest token, selection and attention of one decode step
    in one call (one launch where the library can fuse them)."""
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.hs_decode_step(ctypes.byref(shape), ctypes.byref(kv), _ptr(q), _ptr(new_k), _ptr(new_v), _ptr(smin),
                               _ptr(smax), ctypes.byref(sel_params), _ptr(sel), _ptr(sel_count), _ptr(scores),
                               ctypes.byref(attn_params), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
                               _stream(stream)),
           "hs_decode_step")


def hs_decode_step_reuse(shape, kv, q, new_k, new_v, smin, smax, sel, sel_count, capacity, attn_params, out,
                         lse=None, workspace=None, stream=None):
    """Append of the newest token and attention over another layer's selection
    (sel / sel_count, read only) in one call (one launch where the library can
    fuse them)."""
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.hs_decode_step_reuse(ctypes.byref(shape), ctypes.byref(kv), _ptr(q), _ptr(new_k), _ptr(new_v),
                                     _ptr(smin), _ptr(smax), _ptr(sel), _ptr(sel_count), int(capacity),
                                     ctypes.byref(attn_params), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
                                     _stream(stream)),
           "hs_decode_step_reuse")


def hs_score_select_attend(shape, kv, q, smin, smax, sel_params, sel, sel_count, scores, attn_params, out,
                           lse=None, workspace=None, stream=None):
    """Selection and attention of one decode step in one call (one launch where
    the library can fuse them)."""
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.hs_score_select_attend(ctypes.byref(shape), ctypes.byref(kv), _ptr(q), _ptr(smin), _ptr(smax),
                                       ctypes.byref(sel_params), _ptr(sel), _ptr(sel_count), _ptr(scores),
                                       ctypes.byref(attn_params), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
                                       _stream(stream)),
           "hs_score_select_attend")


def hs_sparse_paged_decode_attn_noalloc(shape, kv, q, sel, sel_count, capacity, params, out, lse=None,
                                        stream=None):
    """hs_sparse_paged_decode_attn without a workspace argument, for callers that
    cannot allocate device memory: the library's own fixed scratch array
    (HS_NOALLOC_SCRATCH_BYTES per GPU) holds the split partials."""
    _check(_lib.hs_sparse_paged_decode_attn_noalloc(ctypes.byref(shape), ctypes.byref(kv), _ptr(q), _ptr(sel),
                                                    _ptr(sel_count), int(capacity), ctypes.byref(params),
                                                    _ptr(out), _ptr(lse), _stream(stream)),
           "hs_sparse_paged_decode_attn_noalloc")


def hot_buffer(page_table, slot_owner, last_used, k_slots, v_slots, host_k, host_v,
               slots_per_stream, k_slot_scales=None, v_slot_scales=None, host_k_scales=None,
               host_v_scales=None) -> HotBuffer:
    hb = HotBuffer(_ptr(page_table), _ptr(slot_owner), _ptr(last_used), _ptr(k_slots), _ptr(v_slots),
                   _ptr(k_slot_scales), _ptr(v_slot_scales), _ptr(host_k), _ptr(host_v),
                   _ptr(host_k_scales), _ptr(host_v_scales), int(page_table.shape[0]),
                   int(page_table.shape[-1]), int(slots_per_stream))
    hb._keep = (page_table, slot_owner, last_used, k_slots, v_slots, host_k, host_v, k_slot_scales,
                v_slot_scales, host_k_scales, host_v_scales)
    return hb


def hs_swapin_misses(shape, hb, sel, sel_count, capacity, step, stats=None, stream=None):
    _check(_lib.hs_swapin_misses(ctypes.byref(shape), ctypes.byref(hb), _ptr(sel), _ptr(sel_count),
                                 int(capacity), int(step), _ptr(stats), _stream(stream)),
           "hs_swapin_misses")


def hs_swapin_plan(shape, hb, sel, sel_count, capacity, step, hit_sel, hit_count, miss_sel, miss_count,
                   stats=None, stream=None):
    _check(_lib.hs_swapin_plan(ctypes.byref(shape), ctypes.byref(hb), _ptr(sel), _ptr(sel_count), int(capacity),
                               int(step), _ptr(hit_sel), _ptr(hit_count), _ptr(miss_sel), _ptr(miss_count),
                               _ptr(stats), _stream(stream)),
           "hs_swapin_plan")


def hs_score_select_swapin_plan(shape, kv, q, smin, smax, params, sel, sel_count, hb, step, hit_sel, hit_count,
                                miss_sel, miss_count, scores=None, workspace=None, stats=None, stream=None):
    """hs_score_select_topk then hs_swapin_plan, each stream's plan in the selection's launch where it fits."""
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.hs_score_select_swapin_plan(ctypes.byref(shape), ctypes.byref(kv), _ptr(q), _ptr(smin), _ptr(smax),
                                            ctypes.byref(params), _ptr(sel), _ptr(sel_count), _ptr(scores),
                                            _ptr(workspace), ws_bytes, ctypes.byref(hb), int(step), _ptr(hit_sel),
                                            _ptr(hit_count), _ptr(miss_sel), _ptr(miss_count), _ptr(stats),
                                            _stream(stream)),
           "hs_score_select_swapin_plan")


def hs_swapin_copy(shape, hb, miss_sel, miss_count, capacity, max_ctas=0, stats=None, stream=None):
    _check(_lib.hs_swapin_copy(ctypes.byref(shape), ctypes.byref(hb), _ptr(miss_sel), _ptr(miss_count),
                               int(capacity), int(max_ctas), _ptr(stats), _stream(stream)),
           "hs_swapin_copy")


def hs_swapin_copy_attend(shape, hb, seq_lens, q, miss_sel, miss_count, capacity, scale, out, lse, max_ctas=0,
                          stats=None, stream=None):
    _check(_lib.hs_swapin_copy_attend(ctypes.byref(shape), ctypes.byref(hb), _ptr(seq_lens), _ptr(q), _ptr(miss_sel),
                                      _ptr(miss_count), int(capacity), float(scale), int(max_ctas), _ptr(out),
                                      _ptr(lse), _ptr(stats), _stream(stream)),
           "hs_swapin_copy_attend")


def hs_merge_attn_partials(shape, outs, lses, out, lse=None, stream=None):
    """outs [parts][batch][Hq][D] f32, lses [parts][batch][Hq] f32 -> out (bf16 or f32), lse."""
    parts, batch = outs.shape[0], outs.shape[1]
    _check(_lib.hs_merge_attn_partials(ctypes.byref(shape), int(batch), int(parts), _ptr(outs), _ptr(lses),
                                       _ptr(out), 1 if out.dtype == torch.float32 else 0, _ptr(lse),
                                       _stream(stream)),
           "hs_merge_attn_partials")


def hs_quantize_e4m3_g32(src, codes, scales, stream=None):
    """src [rows][D] f32 or bf16 -> codes [rows][D] uint8, scales [rows][D/32] f32."""
    D = src.shape[-1]
    rows = src.numel() // D
    _check(_lib.hs_quantize_e4m3_g32(_ptr(src), 1 if src.dtype == torch.float32 else 0, rows, D,
                                     _ptr(codes), _ptr(scales), _stream(stream)),
           "hs_quantize_e4m3_g32")


_U8, _I32 = torch.uint8, torch.int32
_quantize_int4, _dequantize_int4 = _lib.hs_quantize_int4_g32, _lib.hs_dequantize_int4_g32
_accumulate, _evict = _lib.hs_accumulate_attn_weights, _lib.hs_evict_tokens


def _here(what, *tensors):
    """The current device, which contiguous CUDA tensors (None: not given) must be on."""
    device = _current_device() if tensors[0].is_cuda else -2
    for t in tensors:
        if t is not None and (t.get_device() != device or not t.is_contiguous()):
            raise ValueError(f"{what}: tensors must be contiguous and on the current CUDA device")
    return device


def _int4_rows(values, codes, scales, what):
    """Rows, head_dim, whether f32, and device of [rows][D] values, [rows][D/2] codes and [rows][2][D/32] scales
    (leading dimensions alike)."""
    d, n, dtype = values.shape[-1], values.numel(), values.dtype
    if (codes.numel() * 2 != n or scales.numel() * 16 != n or codes.shape[-1] * 2 != d or codes.dtype is not _U8
            or scales.dtype is not _BF16 or (dtype is not _BF16 and dtype is not _F32)):
        raise ValueError(f"{what}: [rows][D] values of f32 or bf16 go with [rows][D/2] uint8 codes and [rows][2][D/32] "
                         "bf16 scales")
    return n // d if d else 0, d, 0 if dtype is _BF16 else 1, _here(what, values, codes, scales)


def hs_quantize_int4_g32(src, codes, scales, stream=None):
    """src [rows][D] f32 or bf16 -> codes [rows][D/2] uint8, scales [rows][2][D/32] bf16 (scales, then centres)."""
    rows, d, f32, device = _int4_rows(src, codes, scales, "hs_quantize_int4_g32")
    st = _quantize_int4(src.data_ptr(), f32, rows, d, codes.data_ptr(), scales.data_ptr(),
                        _raw_stream(device) if stream is None else _stream(stream))
    if st:
        raise HSError(st, "hs_quantize_int4_g32")


def hs_dequantize_int4_g32(codes, scales, out, stream=None):
    """codes [rows][D/2] uint8, scales [rows][2][D/32] bf16 -> out [rows][D] f32 or bf16 (pages as they are: any
    leading dimensions)."""
    rows, d, f32, device = _int4_rows(out, codes, scales, "hs_dequantize_int4_g32")
    st = _dequantize_int4(codes.data_ptr(), scales.data_ptr(), rows, d, out.data_ptr(), f32,
                          _raw_stream(device) if stream is None else _stream(stream))
    if st:
        raise HSError(st, "hs_dequantize_int4_g32")


def hs_accumulate_attn_weights(shape, kv, q, lse, sel, sel_count, capacity, scale, weights, stream=None):
    """weights [batch][Hkv][max_blocks * B] f32 += the group's softmax weights of every token of the selected blocks,
    lse [batch][Hq] f32 as the attention over the same selection left it."""
    heads, pairs = kv.batch * shape.num_q_heads, kv.batch * shape.num_kv_heads
    if (lse.dtype is not _F32 or weights.dtype is not _F32 or sel.dtype is not _I32 or sel_count.dtype is not _I32
            or q.dtype is not (_BF16 if shape.kv_dtype else _F32) or q.numel() != heads * shape.head_dim
            or lse.numel() != heads or sel.numel() != pairs * capacity or sel_count.numel() != pairs
            or weights.numel() != pairs * kv.max_blocks * shape.block_size):
        raise ValueError("hs_accumulate_attn_weights: q [batch][Hq][D], lse [batch][Hq] f32, sel [batch][Hkv][capacity] "
                         "and sel_count [batch][Hkv] int32, weights [batch][Hkv][max_blocks * B] f32")
    device = _here("hs_accumulate_attn_weights", q, lse, sel, sel_count, weights)
    st = _accumulate(_byref(shape), _byref(kv), q.data_ptr(), lse.data_ptr(), sel.data_ptr(), sel_count.data_ptr(),
                     int(capacity), float(scale), weights.data_ptr(),
                     _raw_stream(device) if stream is None else _stream(stream))
    if st:
        raise HSError(st, "hs_accumulate_attn_weights")


def evict_params(budget, sink_tokens=0, recent_tokens=0) -> EvictParams:
    """Tokens that hs_evict_tokens keeps of each (request, kv head), the first sink_tokens and the last recent_tokens
    among them."""
    return EvictParams(int(budget), int(sink_tokens), int(recent_tokens))


def hs_evict_tokens(shape, kv, dst, params, weights, dst_weights, kept, stream=None):
    """The heaviest tokens of every (request, kv head) gathered into the pages of ``dst`` (a paged_kv whose seq_lens is
    written).  weights [batch][Hkv][max_blocks * B] f32, dst_weights the same for dst (or None), kept
    [batch][Hkv][budget] int32."""
    pairs, block = kv.batch * shape.num_kv_heads, shape.block_size
    if weights.dtype is not _F32 or weights.numel() != pairs * kv.max_blocks * block:
        raise ValueError("hs_evict_tokens: weights must be f32 [batch][Hkv][max_blocks * B]")
    if dst_weights is not None and (dst_weights.dtype is not _F32 or dst_weights.numel() != pairs * dst.max_blocks * block):
        raise ValueError("hs_evict_tokens: dst_weights must be f32 [batch][Hkv][max_blocks of dst * B]")
    if kept.dtype is not _I32 or kept.numel() != pairs * params.budget:
        raise ValueError("hs_evict_tokens: kept must be int32 [batch][Hkv][budget]")
    device = _here("hs_evict_tokens", weights, kept, dst_weights)
    st = _evict(_byref(shape), _byref(kv), _byref(dst), _byref(params), weights.data_ptr(),
                None if dst_weights is None else dst_weights.data_ptr(), kept.data_ptr(),
                _raw_stream(device) if stream is None else _stream(stream))
    if st:
        raise HSError(st, "hs_evict_tokens")


def hs_get_device_error(stream=None) -> tuple[int, int]:
    """Synchronise, read and clear the device error word: (status, bits)."""
    bits = c_uint32(0)
    st = _lib.hs_get_device_error(_stream(stream), ctypes.byref(bits))
    return int(st), int(bits.value)


TIMEOUT_KERNELS = {1: "tensor-core attention", 2: "single-launch step", 3: "e4m3 attention",
                   4: "tensor-core bound scoring"}


def hs_get_device_error_detail(stream=None) -> tuple[int, int, dict | None]:
    """(status, bits, where) - where describes the first bounded wait that ran
    out since the last read (None if none): kernel, CTA, barrier address,
    parity, warp."""
    bits = c_uint32(0)
    rec = (c_uint32 * 11)()
    st = _lib.hs_get_device_error_detail(_stream(stream), ctypes.byref(bits), rec)
    where = None
    if rec[0]:
        w = rec[2]
        names = ("issued", "mma_s", "mma_o", "softmax0", "softmax1", "producer_item", "softmax_item", "item_chunks")
        where = {"kernel": TIMEOUT_KERNELS.get(rec[0], rec[0]), "cta": int(rec[1]), "barrier": w & 0x3FFFF,
                 "parity": (w >> 18) & 1, "warp": (w >> 19) & 31,
                 "progress": {n: int(ctypes.c_int32(rec[3 + i]).value) for i, n in enumerate(names)}}
    return int(st), int(bits.value), where
