"""Thin ctypes binding of libps.so (include/ps.h).

Argument marshalling only: every function takes torch tensors (device memory allocated by
PyTorch), passes their data pointers, sizes and the current CUDA stream to the C entry
point of the same name, and raises PsError on a negative status.  All computation runs in
the library's CUDA kernels; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import math
import os
import re
from ctypes import POINTER, c_char_p, c_double, c_float, c_int32, c_int64, c_size_t, c_void_p
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libps.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "ps.h")

PS_OK = 0
PS_ERR_INVALID_ARG = -1
PS_ERR_UNSUPPORTED = -2
PS_ERR_WORKSPACE = -3
PS_ERR_CUDA = -4

PS_DEV_BAD_POS = 1
PS_DEV_POS_RANGE = 2
PS_DEV_TIMEOUT = 4

PS_TILE_FULL = 1
PS_TILE_PARTIAL = 2

PS_ROPE_HALF = 0
PS_ROPE_INTERLEAVED = 1
PS_ROPE_SCALE_NONE = 0
PS_ROPE_SCALE_LINEAR = 1
PS_ROPE_SCALE_BY_PARTS = 2
PS_ROPE_SCALE_YARN = 3
PS_TYPE_BF16 = 0
PS_TYPE_FP32 = 1


class PsError(RuntimeError):
    def __init__(self, code: int, func: str, msg: str):
        super().__init__(f"{func} failed with status {code}: {msg}")
        self.code = code


class PsParams(ctypes.Structure):
    _fields_ = [
        ("n_q_heads", c_int32),
        ("n_kv_heads", c_int32),
        ("head_dim", c_int32),
        ("l_prefix", c_int32),
        ("window", c_int32),
        ("reserved", c_int32),
        ("rope_theta", c_double),
        ("softmax_scale", c_float),
        ("reserved2", c_int32),
    ]


class PsKVCache(ctypes.Structure):
    _fields_ = [
        ("k_prefix", c_void_p),
        ("v_prefix", c_void_p),
        ("k_ring", c_void_p),
        ("v_ring", c_void_p),
        ("batch", c_int64),
    ]
    held = None  # make_cache's tensors; None: addresses alone
    fits = None  # the geometry they were last compared with


class PsRope(ctypes.Structure):
    _fields_ = [
        ("layout", c_int32),
        ("rotary_dim", c_int32),
        ("attn_factor", c_float),
        ("reserved", c_int32),
        ("inv_freq", c_double * 64),
    ]


class PsRopeScaling(ctypes.Structure):
    _fields_ = [
        ("kind", c_int32),
        ("reserved", c_int32),
        ("factor", c_double),
        ("low", c_double),
        ("high", c_double),
        ("original_len", c_double),
    ]


class PsQkNorm(ctypes.Structure):
    _fields_ = [
        ("q_weight", c_void_p),
        ("k_weight", c_void_p),
        ("weight_type", c_int32),
        ("eps", c_float),
    ]
    device = None  # of make_norm's weights; None: not known


class PsKVCacheQ4(ctypes.Structure):
    _fields_ = [
        ("k_prefix", c_void_p),
        ("v_prefix", c_void_p),
        ("s_prefix", c_void_p),
        ("k_ring", c_void_p),
        ("v_ring", c_void_p),
        ("s_ring", c_void_p),
        ("batch", c_int64),
        ("block_table", c_void_p),
        ("n_blocks", c_int64),
        ("table_stride", c_int32),
        ("reserved", c_int32),
    ]
    device = None  # of make_cache_q4's tensors; None: not known
    rows = None    # their (prefix, ring) rows; None: addresses alone
    fits = None    # the geometry they were last compared with


_lib = None

_SIGS = {
    "ps_kv_append_rope": (c_int32, [POINTER(PsParams), POINTER(PsKVCache), c_void_p, c_void_p,
                                    c_void_p, c_void_p, c_int32, c_void_p, c_void_p]),
    "ps_decode_workspace_bytes": (c_size_t, [POINTER(PsParams), c_int64]),
    "ps_decode_attn": (c_int32, [POINTER(PsParams), POINTER(PsKVCache), c_void_p, c_void_p,
                                 c_void_p, c_void_p, c_void_p, c_size_t, c_void_p, c_void_p]),
    "ps_decode_attn_noalloc": (c_int32, [POINTER(PsParams), POINTER(PsKVCache), c_void_p,
                                         c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "ps_full_attn_workspace_bytes": (c_size_t, [POINTER(PsParams), c_int64, c_int64]),
    "ps_full_attn_ref": (c_int32, [POINTER(PsParams), c_void_p, c_void_p, c_int64, c_void_p,
                                   c_void_p, c_int64, c_void_p, c_void_p, c_void_p, c_size_t,
                                   c_void_p, c_void_p]),
    "ps_prefill_tile_geometry": (c_int32, [POINTER(c_int32), POINTER(c_int32)]),
    "ps_prefill_plan_tiles": (c_int64, [POINTER(PsParams), c_int64]),
    "ps_prefill_workspace_bytes": (c_size_t, [POINTER(PsParams), c_int64, c_int64]),
    "ps_masked_prefill_attn": (c_int32, [POINTER(PsParams), c_void_p, c_void_p, c_void_p, c_int64,
                                         c_int64, c_void_p, c_void_p, c_void_p, c_int64,
                                         POINTER(c_int64), c_void_p, c_size_t, c_void_p,
                                         c_void_p]),
    "ps_kv_append_rope_paged": (c_int32, [POINTER(PsParams), c_void_p, c_void_p, c_int64,
                                          c_void_p, c_int32, c_int64, c_void_p, c_void_p,
                                          c_void_p, c_void_p, c_int32, c_void_p, c_void_p]),
    "ps_decode_attn_paged": (c_int32, [POINTER(PsParams), c_void_p, c_void_p, c_int64, c_void_p,
                                       c_int32, c_int64, c_void_p, c_void_p, c_void_p, c_void_p,
                                       c_void_p, c_size_t, c_void_p, c_void_p]),
    "ps_decode_step": (c_int32, [POINTER(PsParams), POINTER(PsKVCache), c_void_p, c_void_p,
                                 c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                 c_void_p, c_void_p]),
    "ps_decode_attn_reset_pe": (c_int32, [POINTER(PsParams), POINTER(PsKVCache), c_void_p,
                                          c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                          c_void_p, c_void_p]),
    "ps_kv_pin": (c_int32, [POINTER(PsParams), POINTER(PsKVCache), c_int32, c_void_p, c_void_p,
                            c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "ps_decode_pinned_workspace_bytes": (c_size_t, [POINTER(PsParams), c_int64, c_int32]),
    "ps_decode_attn_pinned": (c_int32, [POINTER(PsParams), POINTER(PsKVCache), c_int32,
                                        c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                        c_void_p, c_void_p, c_size_t, c_void_p, c_void_p]),
    "ps_decode_shared_prefix_workspace_bytes": (c_size_t, [POINTER(PsParams), c_int64,
                                                           c_int64]),
    "ps_decode_attn_shared_prefix": (c_int32, [POINTER(PsParams), POINTER(PsKVCache), c_int64,
                                               c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                               c_size_t, c_void_p, c_void_p]),
    "ps_prefill_bwd_workspace_bytes": (c_size_t, [POINTER(PsParams), c_int64, c_int64]),
    "ps_masked_prefill_attn_bwd": (c_int32, [POINTER(PsParams), c_void_p, c_void_p, c_void_p,
                                             c_void_p, c_void_p, c_void_p, c_int64, c_int64,
                                             c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                             c_void_p, c_void_p]),
    "ps_decode_visible_ranges": (c_int32, [POINTER(PsParams), c_void_p, c_int64, c_void_p,
                                           c_void_p]),
    "ps_rope_init": (c_int32, [POINTER(PsRope), POINTER(PsParams), c_int32, c_int32,
                               POINTER(PsRopeScaling), c_float]),
    "ps_qk_norm_rope": (c_int32, [POINTER(PsParams), POINTER(PsRope), POINTER(PsQkNorm), c_void_p,
                                  c_int64, c_void_p, c_int64, c_void_p, c_int64, c_void_p,
                                  c_void_p, c_void_p, c_void_p]),
    "ps_qk_norm_rope_bwd_workspace_bytes": (c_size_t, [POINTER(PsParams), c_int64]),
    "ps_qk_norm_rope_bwd": (c_int32, [POINTER(PsParams), POINTER(PsRope), POINTER(PsQkNorm),
                                      c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64,
                                      c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_int64,
                                      c_void_p, c_void_p, c_void_p, c_size_t, c_void_p,
                                      c_void_p]),
    "ps_kv_append_norm_rope": (c_int32, [POINTER(PsParams), POINTER(PsRope), POINTER(PsQkNorm),
                                         POINTER(PsKVCache), c_void_p, c_int64, c_void_p, c_int64,
                                         c_void_p, c_int64, c_void_p, c_void_p, c_int32, c_void_p,
                                         c_void_p]),
    "ps_kv_append_norm_rope_paged": (c_int32, [POINTER(PsParams), POINTER(PsRope),
                                               POINTER(PsQkNorm), c_void_p, c_void_p, c_int64,
                                               c_void_p, c_int32, c_int64, c_void_p, c_int64,
                                               c_void_p, c_int64, c_void_p, c_int64, c_void_p,
                                               c_void_p, c_int32, c_void_p, c_void_p]),
    "ps_kv_append_norm_rope_q4": (c_int32, [POINTER(PsParams), POINTER(PsRope),
                                            POINTER(PsQkNorm), POINTER(PsKVCacheQ4), c_void_p,
                                            c_int64, c_void_p, c_int64, c_void_p, c_int64,
                                            c_void_p, c_void_p, c_int32, c_void_p, c_void_p]),
    "ps_kv_read_q4": (c_int32, [POINTER(PsParams), POINTER(PsKVCacheQ4), c_void_p, c_int32,
                                c_void_p, c_void_p, c_void_p, c_void_p]),
    "ps_decode_q4_workspace_bytes": (c_size_t, [POINTER(PsParams), c_int64]),
    "ps_decode_attn_q4": (c_int32, [POINTER(PsParams), POINTER(PsKVCacheQ4), c_void_p, c_void_p,
                                    c_void_p, c_void_p, c_void_p, c_size_t, c_void_p, c_void_p]),
    "ps_check_wait_timeout": (c_int32, [c_void_p, c_void_p]),
    "ps_last_error": (c_char_p, []),
    "ps_version": (c_char_p, []),
}


def header_functions() -> list:
    """Names of the functions include/ps.h declares."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:int|int64_t|size_t|const char\*)\s+(ps_\w+)\s*\(",
                                 text, flags=re.M)))


def load():
    """Load libps.so (raises loudly if it is missing: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing; build it with `python -m prefix_sliding_window_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def last_error() -> str:
    return load().ps_last_error().decode()


def _check(rc: int, func: str):
    if rc != PS_OK:
        raise PsError(rc, func, last_error())


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_params(n_q_heads, n_kv_heads, head_dim=128, l_prefix=0, window=1, rope_theta=1.0e6,
                softmax_scale=0.0) -> PsParams:
    return PsParams(int(n_q_heads), int(n_kv_heads), int(head_dim), int(l_prefix), int(window), 0,
                    float(rope_theta), float(softmax_scale), 0)


def make_cache(k_prefix, v_prefix, k_ring, v_ring, batch: int) -> PsKVCache:
    cache = PsKVCache(_ptr(k_prefix), _ptr(v_prefix), _ptr(k_ring), _ptr(v_ring), int(batch))
    cache.held = (k_prefix, v_prefix, k_ring, v_ring)  # the struct keeps only addresses
    return cache


_ROPE_LAYOUTS = {"half": PS_ROPE_HALF, "interleaved": PS_ROPE_INTERLEAVED}
_ROPE_SCALINGS = {"none": PS_ROPE_SCALE_NONE, "linear": PS_ROPE_SCALE_LINEAR,
                  "by_parts": PS_ROPE_SCALE_BY_PARTS, "yarn": PS_ROPE_SCALE_YARN}


def make_rope(params: PsParams, layout="half", rotary_dim: int = 128, scaling="none", factor=1.0,
              low=1.0, high=32.0, original_len=32768.0, attn_factor=1.0) -> PsRope:
    """The rotary plan of a model (ps_rope_init); make it once and keep it."""
    rope = PsRope()
    sc = PsRopeScaling(_ROPE_SCALINGS[scaling], 0, float(factor), float(low), float(high),
                       float(original_len))
    rc = load().ps_rope_init(ctypes.byref(rope), ctypes.byref(params), _ROPE_LAYOUTS[layout],
                             int(rotary_dim), ctypes.byref(sc), float(attn_factor))
    _check(rc, "ps_rope_init")
    return rope


def make_norm(q_weight=None, k_weight=None, eps: float = 1e-6) -> PsQkNorm:
    """Head norm of queries and keys: weights [128] on the GPU, both bf16 or both fp32 (None:
    that side is not normalised)."""
    import torch
    types = {torch.bfloat16: PS_TYPE_BF16, torch.float32: PS_TYPE_FP32}
    given = [w for w in (q_weight, k_weight) if w is not None]
    for w in given:
        if not w.is_cuda or w.dtype not in types or w.shape != (128,) or not w.is_contiguous():
            raise ValueError("norm weights are contiguous [128] CUDA tensors, bf16 or fp32")
        if w.dtype != given[0].dtype or w.device != given[0].device:
            raise ValueError("both norm weights have one type and one device")
    norm = PsQkNorm(_ptr(q_weight), _ptr(k_weight),
                    types[given[0].dtype] if given else PS_TYPE_BF16, float(eps))
    norm.held = given  # the struct keeps only addresses
    norm.device = given[0].get_device() if given else None
    return norm


def make_cache_q4(prefix, ring, batch: int, block_table=None) -> PsKVCacheQ4:
    """View of a 4-bit store.  prefix and ring: (k, v, record) tensors or None; paged: prefix
    holds the pools, ring is None and block_table [batch, stride] int32 is given."""
    import torch
    held = [t for part in (prefix, ring) if part is not None for t in part]
    if block_table is not None:
        held.append(block_table)
    for t in held:
        if t.get_device() != held[0].get_device():
            raise ValueError("the parts of a 4-bit store are on one device")
    for part in (prefix, ring):
        for t, dtype, width in zip(part or (), (torch.uint8, torch.uint8, torch.bfloat16),
                                   (64, 64, 8)):
            if not t.is_cuda or t.dtype != dtype or t.shape[-1] != width or \
                    t.shape[:-1] != part[0].shape[:-1] or not t.is_contiguous():
                raise ValueError("a 4-bit store part is contiguous uint8 [..., 64] k and v and "
                                 "bf16 [..., 8] records on the GPU")
    n_blocks = stride = 0
    if block_table is not None:
        if not block_table.is_cuda or block_table.dtype != torch.int32 or \
                block_table.dim() != 2 or not block_table.is_contiguous() or \
                block_table.shape[0] < batch or prefix is None:
            raise ValueError("block_table is a contiguous int32 [batch, stride] CUDA tensor "
                             "beside the pools")
        n_blocks, stride = int(prefix[0].shape[0]), int(block_table.shape[1])
    ptrs = [_ptr(t) if t is not None and t.numel() else None
            for part in (prefix, ring) for t in (part or (None,) * 3)]
    cache = PsKVCacheQ4(*ptrs, int(batch), _ptr(block_table), n_blocks, stride, 0)
    cache.held = held  # the struct keeps only addresses
    cache.device = held[0].get_device() if held else None
    # what _store_q4_fits compares with a call's geometry
    cache.rows = tuple(tuple(part[0].shape[:-1]) if part is not None and part[0].numel() else None
                       for part in (prefix, ring))
    cache.table_rows = None if block_table is None else int(block_table.shape[0])
    return cache


def _store_q4_fits(params: PsParams, cache: PsKVCacheQ4) -> None:
    """Refuses a 4-bit store (of make_cache_q4) whose tensors are not those of the call's geometry:
    the kernels index by that alone."""
    geometry = hkv, lp, w, batch = (params.n_kv_heads, params.l_prefix, params.window, cache.batch)
    if cache.fits == geometry or cache.rows is None:
        return
    prefix, ring = cache.rows

    def holds(shape, rows):  # [batch, Hkv, rows], or rows in other dims if there are enough
        if len(shape) == 3:
            return shape[0] >= batch and shape[1:] == (hkv, rows)
        return math.prod(shape) >= batch * hkv * rows
    if cache.table_rows is not None:
        ok = cache.table_rows >= batch and (prefix is None or prefix[1:] == (hkv, 64)
                                            or len(prefix) != 3
                                            and math.prod(prefix[1:]) >= hkv * 64)
    else:
        ok = (prefix is None or lp == 0 or holds(prefix, lp)) and (ring is None or holds(ring, w))
    if not ok:
        raise ValueError(f"a 4-bit store of prefix rows {prefix} and ring rows {ring} ([batch, "
                         f"Hkv, rows], pools [blocks, Hkv, 64]) does not hold batch {batch}, Hkv "
                         f"{hkv}, l_prefix {lp}, window {w}")
    cache.fits = geometry


def _store_fits(params: PsParams, cache: PsKVCache, device: int) -> None:
    """The same for a bf16 store of make_cache."""
    hkv, lp, w, batch, _ = geometry = (params.n_kv_heads, params.l_prefix, params.window,
                                       cache.batch, device)
    if cache.fits == geometry or cache.held is None:
        return
    for t, rows in zip(cache.held, (lp, lp, w, w)):
        if t is not None and rows and t.numel():
            shape = tuple(t.shape)
            if t.dtype is not _torch().bfloat16 or t.get_device() != device or \
                    not t.is_contiguous() or t.numel() < batch * hkv * rows * 128 or \
                    (len(shape) == 4 and shape[1:] != (hkv, rows, 128)):
                raise ValueError(f"a store part of batch {batch} is contiguous bf16 [batch, {hkv}, "
                                 f"{rows}, 128] on cuda:{device}, got {t.dtype} {shape} on "
                                 f"{t.device}")
    cache.fits = geometry


# ---------------------------------------------------------------- entry points
def ps_kv_append_rope(params: PsParams, cache: PsKVCache, k_new, v_new, q_inout, pos0, T: int,
                      dev_status=None, stream=None) -> None:
    rc = load().ps_kv_append_rope(ctypes.byref(params), ctypes.byref(cache), _ptr(k_new),
                                  _ptr(v_new), _ptr(q_inout), _ptr(pos0), int(T),
                                  _ptr(dev_status), _stream(stream))
    _check(rc, "ps_kv_append_rope")


def ps_decode_workspace_bytes(params: PsParams, batch: int) -> int:
    return int(load().ps_decode_workspace_bytes(ctypes.byref(params), int(batch)))


def ps_decode_attn(params: PsParams, cache: PsKVCache, q, pos, out, lse=None, workspace=None,
                   dev_status=None, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().ps_decode_attn(ctypes.byref(params), ctypes.byref(cache), _ptr(q), _ptr(pos),
                               _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes, _ptr(dev_status),
                               _stream(stream))
    _check(rc, "ps_decode_attn")


def ps_kv_append_rope_paged(params: PsParams, k_pool, v_pool, block_table, batch: int, k_new,
                            v_new, q_inout, pos0, T: int, dev_status=None, stream=None) -> None:
    """Append into a paged store: pools [n_blocks, Hkv, 64, D], block_table [batch, stride]."""
    rc = load().ps_kv_append_rope_paged(ctypes.byref(params), _ptr(k_pool), _ptr(v_pool),
                                        int(k_pool.shape[0]), _ptr(block_table),
                                        int(block_table.shape[1]), int(batch), _ptr(k_new),
                                        _ptr(v_new), _ptr(q_inout), _ptr(pos0), int(T),
                                        _ptr(dev_status), _stream(stream))
    _check(rc, "ps_kv_append_rope_paged")


def ps_decode_attn_paged(params: PsParams, k_pool, v_pool, block_table, batch: int, q, pos, out,
                         lse=None, workspace=None, dev_status=None, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().ps_decode_attn_paged(ctypes.byref(params), _ptr(k_pool), _ptr(v_pool),
                                     int(k_pool.shape[0]), _ptr(block_table),
                                     int(block_table.shape[1]), int(batch), _ptr(q), _ptr(pos),
                                     _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
                                     _ptr(dev_status), _stream(stream))
    _check(rc, "ps_decode_attn_paged")


def ps_decode_step(params: PsParams, cache: PsKVCache, k_new, v_new, q_inout, pos, out,
                   lse=None, workspace=None, dev_status=None, stream=None) -> None:
    """Append one token per sequence at pos (q rotated in place), then decode at pos."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().ps_decode_step(ctypes.byref(params), ctypes.byref(cache), _ptr(k_new),
                               _ptr(v_new), _ptr(q_inout), _ptr(pos), _ptr(out), _ptr(lse),
                               _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(stream))
    _check(rc, "ps_decode_step")


def ps_decode_attn_reset_pe(params: PsParams, cache: PsKVCache, q, pos, out, lse=None,
                            workspace=None, dev_status=None, stream=None) -> None:
    """Decode under Reset PE from a Continue-PE cache (prefix rows see the query at its
    Reset-PE id)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().ps_decode_attn_reset_pe(ctypes.byref(params), ctypes.byref(cache), _ptr(q),
                                        _ptr(pos), _ptr(out), _ptr(lse), _ptr(workspace),
                                        ws_bytes, _ptr(dev_status), _stream(stream))
    _check(rc, "ps_decode_attn_reset_pe")


def ps_kv_pin(params: PsParams, cache: PsKVCache, prefix_capacity: int, pin_count, pin_pos, t0,
              t1, pos, dev_status=None, stream=None) -> None:
    """Promote tokens [t0[b], t1[b]) (still in the window) into the pinned prefix."""
    rc = load().ps_kv_pin(ctypes.byref(params), ctypes.byref(cache), int(prefix_capacity),
                          _ptr(pin_count), _ptr(pin_pos), _ptr(t0), _ptr(t1), _ptr(pos),
                          _ptr(dev_status), _stream(stream))
    _check(rc, "ps_kv_pin")


def ps_decode_pinned_workspace_bytes(params: PsParams, batch: int, prefix_capacity: int) -> int:
    return int(load().ps_decode_pinned_workspace_bytes(ctypes.byref(params), int(batch),
                                                       int(prefix_capacity)))


def ps_decode_attn_pinned(params: PsParams, cache: PsKVCache, prefix_capacity: int, pin_count,
                          pin_pos, q, pos, out, lse=None, workspace=None, dev_status=None,
                          stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().ps_decode_attn_pinned(ctypes.byref(params), ctypes.byref(cache),
                                      int(prefix_capacity), _ptr(pin_count), _ptr(pin_pos),
                                      _ptr(q), _ptr(pos), _ptr(out), _ptr(lse), _ptr(workspace),
                                      ws_bytes, _ptr(dev_status), _stream(stream))
    _check(rc, "ps_decode_attn_pinned")


def ps_decode_attn_noalloc(params: PsParams, cache: PsKVCache, q, pos, out, lse=None,
                           dev_status=None, stream=None) -> None:
    """ps_decode_attn whose split-K scratch is the library's built-in device array."""
    rc = load().ps_decode_attn_noalloc(ctypes.byref(params), ctypes.byref(cache), _ptr(q),
                                       _ptr(pos), _ptr(out), _ptr(lse), _ptr(dev_status),
                                       _stream(stream))
    _check(rc, "ps_decode_attn_noalloc")


def ps_decode_shared_prefix_workspace_bytes(params: PsParams, batch: int, group_size: int) -> int:
    return int(load().ps_decode_shared_prefix_workspace_bytes(ctypes.byref(params), int(batch),
                                                              int(group_size)))


def ps_decode_attn_shared_prefix(params: PsParams, cache: PsKVCache, group_size: int, q, pos,
                                 out, lse=None, workspace=None, dev_status=None,
                                 stream=None) -> None:
    """Decode where sequences [j*group_size, (j+1)*group_size) share prefix j of
    cache.k_prefix / v_prefix ([batch / group_size, Hkv, l_prefix, D])."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().ps_decode_attn_shared_prefix(ctypes.byref(params), ctypes.byref(cache),
                                             int(group_size), _ptr(q), _ptr(pos), _ptr(out),
                                             _ptr(lse), _ptr(workspace), ws_bytes,
                                             _ptr(dev_status), _stream(stream))
    _check(rc, "ps_decode_attn_shared_prefix")


def ps_full_attn_workspace_bytes(params: PsParams, batch: int, lmax: int) -> int:
    return int(load().ps_full_attn_workspace_bytes(ctypes.byref(params), int(batch), int(lmax)))


def ps_full_attn_ref(params: PsParams, k_full, v_full, lmax: int, q, pos, batch: int, out,
                     lse=None, workspace=None, dev_status=None, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().ps_full_attn_ref(ctypes.byref(params), _ptr(k_full), _ptr(v_full), int(lmax),
                                 _ptr(q), _ptr(pos), int(batch), _ptr(out), _ptr(lse),
                                 _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(stream))
    _check(rc, "ps_full_attn_ref")


def ps_prefill_tile_geometry():
    bq, bk = c_int32(0), c_int32(0)
    _check(load().ps_prefill_tile_geometry(ctypes.byref(bq), ctypes.byref(bk)),
           "ps_prefill_tile_geometry")
    return bq.value, bk.value


def ps_prefill_plan_tiles(params: PsParams, seq: int) -> int:
    n = int(load().ps_prefill_plan_tiles(ctypes.byref(params), int(seq)))
    if n < 0:
        raise PsError(n, "ps_prefill_plan_tiles", last_error())
    return n


def ps_prefill_workspace_bytes(params: PsParams, batch: int, seq: int) -> int:
    return int(load().ps_prefill_workspace_bytes(ctypes.byref(params), int(batch), int(seq)))


def ps_masked_prefill_attn(params: PsParams, q, k, v, batch: int, seq: int, out, lse=None,
                           tile_plan=None, workspace=None, dev_status=None, stream=None) -> int:
    """Returns the number of plan rows (tiles per (batch, head))."""
    n_tiles = c_int64(-1)
    cap = 0 if tile_plan is None else tile_plan.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().ps_masked_prefill_attn(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), int(batch),
                                       int(seq), _ptr(out), _ptr(lse), _ptr(tile_plan), int(cap),
                                       ctypes.byref(n_tiles), _ptr(workspace), ws_bytes,
                                       _ptr(dev_status), _stream(stream))
    _check(rc, "ps_masked_prefill_attn")
    return n_tiles.value


def ps_prefill_bwd_workspace_bytes(params: PsParams, batch: int, seq: int) -> int:
    return int(load().ps_prefill_bwd_workspace_bytes(ctypes.byref(params), int(batch), int(seq)))


def ps_masked_prefill_attn_bwd(params: PsParams, q, k, v, out, dout, lse, batch: int, seq: int,
                               dq, dk, dv, workspace=None, dev_status=None, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().ps_masked_prefill_attn_bwd(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v),
                                           _ptr(out), _ptr(dout), _ptr(lse), int(batch), int(seq),
                                           _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), ws_bytes,
                                           _ptr(dev_status), _stream(stream))
    _check(rc, "ps_masked_prefill_attn_bwd")


def _tensor(name: str, t, dtype, device: int, numel: int):
    """A contiguous tensor of the library's type and of at least numel elements on CUDA device
    `device`."""
    if t.dtype is not dtype or t.get_device() != device or t.numel() < numel or \
            not t.is_contiguous():
        raise ValueError(f"{name}: contiguous {dtype} of >= {numel} elements on cuda:{device} "
                         f"expected, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _pair(name: str, given, out) -> None:
    """Both of them are tensors, or both None: one alone would be left unwritten or unread."""
    if (given is None) != (out is None):
        raise ValueError(f"{name} go together")


def _heads(name: str, t, tokens: int, heads: int, device: int):
    """Rows of heads: [tokens, heads, 128] (or leading dims that flatten to tokens) with heads
    contiguous in a token.  Returns the address and the stride between tokens."""
    sh, st = t.shape, t.stride()
    if len(sh) == 3 and st[2] == 1 and st[1] == 128 and sh[2] == 128 and sh[1] == heads and \
            sh[0] == tokens > 1 and t.dtype is _torch_module.bfloat16 and \
            t.get_device() == device:
        return t.data_ptr(), st[0]  # the usual case, decided in few steps
    ok = (t.dtype is _torch().bfloat16 and t.get_device() == device and len(sh) >= 3
          and sh[-1] == 128 and sh[-2] == heads and st[-1] == 1 and (st[-2] == 128 or heads == 1))
    n, stride = 1, heads * 128
    if ok:
        for size, step in zip(sh[-3::-1], st[-3::-1]):  # leading dims: evenly spaced tokens
            if size != 1:
                if n == 1:
                    stride = step
                ok = ok and step == n * stride
                n *= size
        ok = ok and n == tokens
    if not ok:
        raise ValueError(f"{name}: bf16 [{tokens}, {heads}, 128] with contiguous heads on "
                         f"cuda:{device} expected, got {t.dtype} {tuple(sh)} strides {st} on "
                         f"{t.device}")
    return t.data_ptr(), stride


_torch_module = None
_current_device = _current_stream = None  # (device index), (device index -> handle)


def _torch():
    """torch, and the runtime's own calls for the current device and stream where torch offers
    them: the public ones build objects, which takes longer than a launch."""
    global _torch_module, _current_device, _current_stream
    if _torch_module is None:
        import torch
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda _: _stream(None))
        _torch_module = torch
    return _torch_module


def _device_of(pos, norm=None, cache=None) -> int:
    """The device index of a call: the current device, where everything it is given lives."""
    if _torch_module is None:
        _torch()
    dev = pos.get_device()
    if dev < 0 or dev != _current_device():
        raise ValueError(f"positions are on {pos.device}, the current device is "
                         f"cuda:{_torch().cuda.current_device()}")
    if norm is not None and norm.device != dev and norm.device is not None:
        raise ValueError(f"weights on cuda:{norm.device}, positions on cuda:{dev}")
    if cache is not None and cache.device != dev and cache.device is not None:
        raise ValueError(f"cache on cuda:{cache.device}, positions on cuda:{dev}")
    return dev


def _stream_on(stream, device: int):
    """The stream's handle; None: the current stream of the device."""
    return _current_stream(device) if stream is None else _stream(stream)


def _workspace(ws, device: int):
    if ws is None:
        return None, 0
    if ws.get_device() != device or not ws.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on cuda:{device} expected, got one on "
                         f"{ws.device}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _status_ptr(t, device: int):
    return None if t is None else _tensor("dev_status", t, _torch_module.int32, device, 1)


def ps_qk_norm_rope(params: PsParams, rope: PsRope, norm, q, k, pos, q_out, k_out,
                    dev_status=None, stream=None) -> None:
    """Head norm (norm None: none) and rotation of q [N, Hq, 128] and k [N, Hkv, 128] (views of
    packed rows allowed; either None with its output) at pos [N]."""
    torch = _torch()
    _pair("q and q_out", q, q_out)
    _pair("k and k_out", k, k_out)
    dev = _device_of(pos, norm)
    n = pos.numel()
    hq, hkv = params.n_q_heads, params.n_kv_heads
    qp = kp = qo = ko = None
    qs = ks = 0
    if q is not None:
        qp, qs = _heads("q", q, n, hq, dev)
        qo = _tensor("q_out", q_out, torch.bfloat16, dev, n * hq * 128)
    if k is not None:
        kp, ks = _heads("k", k, n, hkv, dev)
        ko = _tensor("k_out", k_out, torch.bfloat16, dev, n * hkv * 128)
    rc = load().ps_qk_norm_rope(params, rope, norm, qp, qs, kp, ks,
                                _tensor("pos", pos, torch.int64, dev, n), n, qo, ko,
                                _status_ptr(dev_status, dev), _stream_on(stream, dev))
    _check(rc, "ps_qk_norm_rope")


def ps_qk_norm_rope_bwd_workspace_bytes(params: PsParams, n_tokens: int) -> int:
    return int(load().ps_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(params), int(n_tokens)))


def ps_qk_norm_rope_bwd(params: PsParams, rope: PsRope, norm, q, k, pos, dq_out, dk_out, dq, dk,
                        dq_weight=None, dk_weight=None, workspace=None, dev_status=None,
                        stream=None) -> None:
    """Gradients of ps_qk_norm_rope: dq, dk (views of packed rows allowed) and, where given, the
    weights' (fp32 [128])."""
    torch = _torch()
    _pair("dq_out and dq", dq_out, dq)
    _pair("dk_out and dk", dk_out, dk)
    dev = _device_of(pos, norm)
    n = pos.numel()
    hq, hkv = params.n_q_heads, params.n_kv_heads
    qp = kp = gq = gk = dqp = dkp = None
    qs = ks = dqs = dks = 0
    if q is not None:
        qp, qs = _heads("q", q, n, hq, dev)
    if k is not None:
        kp, ks = _heads("k", k, n, hkv, dev)
    if dq_out is not None:
        gq = _tensor("dq_out", dq_out, torch.bfloat16, dev, n * hq * 128)
        dqp, dqs = _heads("dq", dq, n, hq, dev)
    if dk_out is not None:
        gk = _tensor("dk_out", dk_out, torch.bfloat16, dev, n * hkv * 128)
        dkp, dks = _heads("dk", dk, n, hkv, dev)
    dwq = None if dq_weight is None else _tensor("dq_weight", dq_weight, torch.float32, dev, 128)
    dwk = None if dk_weight is None else _tensor("dk_weight", dk_weight, torch.float32, dev, 128)
    ws, ws_bytes = _workspace(workspace, dev)
    rc = load().ps_qk_norm_rope_bwd(params, rope, norm, qp, qs, kp, ks,
                                    _tensor("pos", pos, torch.int64, dev, n), n, gq, gk, dqp, dqs,
                                    dkp, dks, dwq, dwk, ws, ws_bytes,
                                    _status_ptr(dev_status, dev), _stream_on(stream, dev))
    _check(rc, "ps_qk_norm_rope_bwd")


def _append_rows(params, batch, k_new, v_new, q, q_out, pos0, T, dev):
    torch = _torch()
    _pair("q and q_out", q, q_out)
    n = int(batch) * int(T)
    kp, ks = _heads("k_new", k_new, n, params.n_kv_heads, dev)
    vp, vs = _heads("v_new", v_new, n, params.n_kv_heads, dev)
    qp = qo = None
    qs = 0
    if q is not None:
        qp, qs = _heads("q", q, n, params.n_q_heads, dev)
        qo = _tensor("q_out", q_out, torch.bfloat16, dev, n * params.n_q_heads * 128)
    return kp, ks, vp, vs, qp, qs, qo, _tensor("pos0", pos0, torch.int64, dev, batch), int(T)


def ps_kv_append_norm_rope(params: PsParams, rope: PsRope, norm, cache: PsKVCache, k_new, v_new,
                           q, q_out, pos0, T: int, dev_status=None, stream=None) -> None:
    """ps_kv_append_rope with a head norm and any rotary plan; q (or None) goes to q_out."""
    dev = _device_of(pos0, norm)
    _store_fits(params, cache, dev)
    rc = load().ps_kv_append_norm_rope(params, rope, norm, cache,
                                       *_append_rows(params, cache.batch, k_new, v_new, q, q_out,
                                                     pos0, T, dev),
                                       _status_ptr(dev_status, dev), _stream_on(stream, dev))
    _check(rc, "ps_kv_append_norm_rope")


def ps_kv_append_norm_rope_paged(params: PsParams, rope: PsRope, norm, k_pool, v_pool,
                                 block_table, batch: int, k_new, v_new, q, q_out, pos0, T: int,
                                 dev_status=None, stream=None) -> None:
    """The same into a paged store: pools [n_blocks, Hkv, 64, 128], block_table [batch, stride]."""
    torch = _torch()
    dev = _device_of(pos0, norm)
    blocks = int(k_pool.shape[0])
    rows = blocks * params.n_kv_heads * 64 * 128
    rc = load().ps_kv_append_norm_rope_paged(
        params, rope, norm, _tensor("k_pool", k_pool, torch.bfloat16, dev, rows),
        _tensor("v_pool", v_pool, torch.bfloat16, dev, rows), blocks,
        _tensor("block_table", block_table, torch.int32, dev, batch * block_table.shape[1]),
        int(block_table.shape[1]), int(batch),
        *_append_rows(params, batch, k_new, v_new, q, q_out, pos0, T, dev),
        _status_ptr(dev_status, dev), _stream_on(stream, dev))
    _check(rc, "ps_kv_append_norm_rope_paged")


def ps_kv_append_norm_rope_q4(params: PsParams, rope: PsRope, norm, cache: PsKVCacheQ4, k_new,
                              v_new, q, q_out, pos0, T: int, dev_status=None,
                              stream=None) -> None:
    """The same into a 4-bit store (make_cache_q4)."""
    dev = _device_of(pos0, norm, cache)
    _store_q4_fits(params, cache)
    rc = load().ps_kv_append_norm_rope_q4(params, rope, norm, cache,
                                          *_append_rows(params, cache.batch, k_new, v_new, q,
                                                        q_out, pos0, T, dev),
                                          _status_ptr(dev_status, dev), _stream_on(stream, dev))
    _check(rc, "ps_kv_append_norm_rope_q4")


def ps_kv_read_q4(params: PsParams, cache: PsKVCacheQ4, pos0, T: int, k_out, v_out,
                  dev_status=None, stream=None) -> None:
    """Rows of positions [pos0, pos0 + T) of a 4-bit store as bf16 [batch, T, Hkv, 128]."""
    torch = _torch()
    dev = _device_of(pos0, None, cache)
    _store_q4_fits(params, cache)
    n = cache.batch * int(T) * params.n_kv_heads * 128
    out = [None if t is None else _tensor(name, t, torch.bfloat16, dev, n)
           for name, t in (("k_out", k_out), ("v_out", v_out))]
    rc = load().ps_kv_read_q4(params, cache, _tensor("pos0", pos0, torch.int64, dev, cache.batch),
                              int(T), *out, _status_ptr(dev_status, dev), _stream_on(stream, dev))
    _check(rc, "ps_kv_read_q4")


def ps_decode_q4_workspace_bytes(params: PsParams, batch: int) -> int:
    return int(load().ps_decode_q4_workspace_bytes(ctypes.byref(params), int(batch)))


def ps_decode_attn_q4(params: PsParams, cache: PsKVCacheQ4, q, pos, out, lse=None, workspace=None,
                      dev_status=None, stream=None) -> None:
    """ps_decode_attn over a 4-bit store."""
    torch = _torch()
    dev = _device_of(pos, None, cache)
    _store_q4_fits(params, cache)
    rows = cache.batch * params.n_q_heads
    ws, ws_bytes = _workspace(workspace, dev)
    rc = load().ps_decode_attn_q4(
        params, cache, _tensor("q", q, torch.bfloat16, dev, rows * 128),
        _tensor("pos", pos, torch.int64, dev, cache.batch),
        _tensor("out", out, torch.bfloat16, dev, rows * 128),
        None if lse is None else _tensor("lse", lse, torch.float32, dev, rows), ws, ws_bytes,
        _status_ptr(dev_status, dev), _stream_on(stream, dev))
    _check(rc, "ps_decode_attn_q4")


def ps_decode_visible_ranges(params: PsParams, pos, batch: int, ranges_out, stream=None) -> None:
    rc = load().ps_decode_visible_ranges(ctypes.byref(params), _ptr(pos), int(batch),
                                         _ptr(ranges_out), _stream(stream))
    _check(rc, "ps_decode_visible_ranges")


def ps_check_wait_timeout(dev_status, stream=None) -> None:
    rc = load().ps_check_wait_timeout(_ptr(dev_status), _stream(stream))
    _check(rc, "ps_check_wait_timeout")


def ps_version() -> str:
    return load().ps_version().decode()
