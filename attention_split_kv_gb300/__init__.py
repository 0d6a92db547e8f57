"""Python binding of libattn (C ABI in include/attn.h).

Argument marshalling only: every step of the attention path runs in the CUDA
kernels of ``libattn.so``.  There is no fallback: importing works without the
library (so sizes can be planned on a machine without a GPU), but every call
that needs it raises ``AttnLibraryMissing`` if ``libattn.so`` was not built.

Functions keep the C names; pointer arguments accept torch tensors (their
``data_ptr()``), plain integers (device addresses) or None (NULL).
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

__all__ = [
    "ATTN_OK", "ATTN_EINVAL", "ATTN_EUNSUPPORTED", "ATTN_ECUDA", "ATTN_EBOUNDS", "ATTN_ETIMEOUT",
    "ATTN_KV_F16", "ATTN_KV_INT8", "ATTN_F16", "ATTN_F32", "AttnError", "AttnLibraryMissing",
    "lib_path", "load", "build", "exported_symbols",
    "attn_version", "attn_last_error", "attn_decode_workspace_size", "attn_decode",
    "attn_decode_ring", "attn_decode_ex", "attn_decode_tiered", "attn_decode_tiered_workspace_size",
    "attn_decode_noalloc", "attn_prefill", "attn_prefill_paged", "attn_decode_validate", "attn_device_status",
    "attn_testing_set_waits", "attn_prefill_paged_ex", "attn_prefill_paged_workspace_size", "attn_append",
    "attn_kv_read", "decode", "decode_tiered", "prefill", "prefill_paged", "append", "kv_read",
    "attn_latent_append", "attn_latent_read", "attn_latent_workspace_size", "attn_latent_attend",
    "attn_latent_prefill", "latent_append", "latent_read", "latent_attend", "latent_prefill",
]

ATTN_OK, ATTN_EINVAL, ATTN_EUNSUPPORTED, ATTN_ECUDA, ATTN_EBOUNDS, ATTN_ETIMEOUT = range(6)
ATTN_KV_F16, ATTN_KV_INT8 = 0, 1
ATTN_F16, ATTN_F32 = 0, 1
_STATUS = {0: "ATTN_OK", 1: "ATTN_EINVAL", 2: "ATTN_EUNSUPPORTED", 3: "ATTN_ECUDA", 4: "ATTN_EBOUNDS",
           5: "ATTN_ETIMEOUT"}

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libattn.so")
_lib = None

# every entry point include/attn.h declares
exported_symbols = ("attn_version", "attn_last_error", "attn_decode_workspace_size", "attn_decode",
                    "attn_decode_ring", "attn_decode_ex", "attn_decode_tiered", "attn_decode_tiered_workspace_size",
                    "attn_decode_noalloc", "attn_prefill", "attn_prefill_paged", "attn_decode_validate",
                    "attn_device_status", "attn_testing_set_waits", "attn_prefill_paged_ex",
                    "attn_prefill_paged_workspace_size", "attn_append", "attn_kv_read", "attn_latent_append",
                    "attn_latent_read", "attn_latent_workspace_size", "attn_latent_attend", "attn_latent_prefill",
                    "attn_latent_append_from", "attn_latent_read_from", "attn_latent_attend_from",
                    "attn_latent_prefill_from")


class AttnLibraryMissing(RuntimeError):
    pass


class AttnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s: %s" % (_STATUS.get(status, str(status)), message))
        self.status = status


def lib_path() -> str:
    return _LIB_PATH


def build(force: bool = False, verbose: bool = False) -> str:
    from . import _build
    return _build.build(force=force, verbose=verbose)


def load():
    """Load libattn.so (raises AttnLibraryMissing if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise AttnLibraryMissing("libattn.so is not built (run attention_split_kv_gb300.build())")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.attn_version.restype = ctypes.c_char_p
    lib.attn_last_error.restype = ctypes.c_char_p
    lib.attn_decode_workspace_size.argtypes = [I, I, I, I, I, I]
    lib.attn_decode_workspace_size.restype = SZ
    lib.attn_decode.argtypes = [P, P, P, P, P, I, I, I, I, P, P, I, I, I, I, I, I, F, F, I, P, P, P, SZ, P]
    lib.attn_decode.restype = I
    lib.attn_decode_ring.argtypes = [P, P, P, P, I, P, P, I, I, I, I, I, I, F, F, I, P, P, P, SZ, P]
    lib.attn_decode_ring.restype = I
    lib.attn_decode_tiered_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.attn_decode_tiered_workspace_size.restype = SZ
    lib.attn_decode_tiered.argtypes = [P, I, P, P, P, P, I, P, P, I, I, I, I, P, P, P, P, I, I, I, I, I, I, F, F,
                                       I, P, I, P, P, SZ, P]
    lib.attn_decode_ex.argtypes = [P, I, P, P, P, P, I, I, I, I, I, P, P, I, I, I, I, I, I, F, F, I, P, I, P, P, SZ,
                                   P]
    lib.attn_decode_ex.restype = I
    lib.attn_decode_tiered.restype = I
    lib.attn_decode_noalloc.argtypes = [P, P, P, P, P, I, I, I, I, P, P, I, I, I, I, I, I, F, F, I, P, P, P]
    lib.attn_decode_noalloc.restype = I
    lib.attn_prefill.argtypes = [P, P, P, I, I, I, I, I, I, F, F, P, P, P]
    lib.attn_prefill.restype = I
    lib.attn_prefill_paged.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, F, F, P, P, P]
    lib.attn_prefill_paged.restype = I
    LL = ctypes.c_longlong
    lib.attn_prefill_paged_workspace_size.argtypes = [I, I, I, I, I, I]
    lib.attn_prefill_paged_workspace_size.restype = SZ
    lib.attn_prefill_paged_ex.argtypes = [P, P, P, P, P, P, I, I, I, P, P, I, I, I, I, I, I, I, I, F, F, P, P, P, SZ,
                                          P]
    lib.attn_prefill_paged_ex.restype = I
    lib.attn_append.argtypes = [P, P, P, I, LL, LL, LL, P, P, F, F, P, P, I, I, I, P, P, P, P, P, I, I, I, I, I, P, P,
                                I, I, I, I, I, I, P, I, P]
    lib.attn_append.restype = I
    lib.attn_kv_read.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P, P, I, I, I, I, I, P, P, I, P]
    lib.attn_kv_read.restype = I
    lib.attn_latent_append.argtypes = [P, P, P, I, LL, LL, LL, LL, P, F, F, P, P, I, I, P, P, P, P, I, I, I, I, I, I,
                                       I, I, I, P, LL, LL, P]
    lib.attn_latent_append.restype = I
    lib.attn_latent_read.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, P, P, I, P]
    lib.attn_latent_read.restype = I
    lib.attn_latent_attend.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, F, P, P, P, SZ, P]
    lib.attn_latent_attend.restype = I
    for f in (lib.attn_latent_append_from, lib.attn_latent_read_from, lib.attn_latent_attend_from,
              lib.attn_latent_prefill_from):
        f.argtypes = [ctypes.c_char_p]   # (the bytes of an argument struct)
        f.restype = I
    lib.attn_latent_workspace_size.argtypes = [I, I, I, I]
    lib.attn_latent_workspace_size.restype = SZ
    lib.attn_latent_prefill.argtypes = [P, P, P, P, LL, LL, LL, LL, LL, LL, P, P, I, I, I, I, I, I, I, I, F, P, P, P]
    lib.attn_latent_prefill.restype = I
    lib.attn_decode_validate.argtypes = [P, P, I, I, I, I, I, ctypes.POINTER(ctypes.c_int), P]
    lib.attn_decode_validate.restype = I
    lib.attn_device_status.argtypes = [P]
    lib.attn_device_status.restype = I
    lib.attn_testing_set_waits.argtypes = [ctypes.c_ulonglong, I]
    lib.attn_testing_set_waits.restype = I
    _lib = lib
    return lib


def _ptr(x) -> Optional[int]:
    if x is None or isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s) -> Optional[int]:
    if s is None:
        import torch
        raw, device = (getattr(torch._C, name, None) for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
        if raw and device and torch.cuda.is_initialized():
            return raw(device())   # without a Stream object, which takes 2.8 us
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _empty(shape, dtype, device, stream, scratch=False):
    """torch.empty for a call on ``stream``.  Memory that torch hands out belongs to its
    current stream: what that stream freed may still be in use there, and what a call drops
    may be handed out again at once.  So with another stream the memory is that stream's
    own, and what the caller gets back (not ``scratch``) is kept for the current one too."""
    import torch
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if _stream(stream) == current.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream), device=device)
    with torch.cuda.stream(stream):
        x = torch.empty(shape, dtype=dtype, device=device)
    if not scratch:
        x.record_stream(current)
    return x


def _check(status: int):
    if status != ATTN_OK:
        raise AttnError(status, load().attn_last_error().decode())


def attn_version() -> str:
    return load().attn_version().decode()


def attn_last_error() -> str:
    return load().attn_last_error().decode()


def attn_decode_workspace_size(batch, n_heads, n_kv_heads, head_dim, max_kv, split_keys=0) -> int:
    return int(load().attn_decode_workspace_size(batch, n_heads, n_kv_heads, head_dim, max_kv, split_keys))


def attn_decode(q, k_cache, v_cache, kv_len, page_table, page_size, max_pages_per_seq, n_pages, max_kv,
                k_scales, v_scales, kv_dtype, batch, n_heads, n_kv_heads, head_dim, window, softcap, scale,
                split_keys, out, lse_out, workspace, workspace_bytes, stream=None) -> None:
    _check(load().attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kv_len), _ptr(page_table),
                              int(page_size), int(max_pages_per_seq), int(n_pages), int(max_kv),
                              _ptr(k_scales), _ptr(v_scales), int(kv_dtype), int(batch), int(n_heads),
                              int(n_kv_heads), int(head_dim), int(window), float(softcap), float(scale),
                              int(split_keys), _ptr(out), _ptr(lse_out), _ptr(workspace),
                              int(workspace_bytes), _stream(stream)))


def attn_decode_ring(q, k_ring, v_ring, seq_len, ring_size, k_scales, v_scales, kv_dtype, batch, n_heads,
                     n_kv_heads, head_dim, window, softcap, scale, split_keys, out, lse_out, workspace,
                     workspace_bytes, stream=None) -> None:
    _check(load().attn_decode_ring(_ptr(q), _ptr(k_ring), _ptr(v_ring), _ptr(seq_len), int(ring_size),
                                   _ptr(k_scales), _ptr(v_scales), int(kv_dtype), int(batch), int(n_heads),
                                   int(n_kv_heads), int(head_dim), int(window), float(softcap), float(scale),
                                   int(split_keys), _ptr(out), _ptr(lse_out), _ptr(workspace),
                                   int(workspace_bytes), _stream(stream)))


def attn_decode_tiered_workspace_size(batch, n_heads, n_kv_heads, head_dim, cold_max_kv, hot_ring,
                                      split_keys=0) -> int:
    return int(load().attn_decode_tiered_workspace_size(batch, n_heads, n_kv_heads, head_dim, cold_max_kv,
                                                        hot_ring, split_keys))


def attn_decode_ex(q, q_dtype, k_cache, v_cache, kv_len, page_table, page_size, max_pages_per_seq, n_pages, max_kv,
                   ring_size, k_scales, v_scales, kv_dtype, batch, n_heads, n_kv_heads, head_dim, window, softcap,
                   scale, split_keys, out, out_dtype, lse_out, workspace, workspace_bytes, stream=None) -> None:
    _check(load().attn_decode_ex(_ptr(q), int(q_dtype), _ptr(k_cache), _ptr(v_cache), _ptr(kv_len), _ptr(page_table),
                                 int(page_size), int(max_pages_per_seq), int(n_pages), int(max_kv), int(ring_size),
                                 _ptr(k_scales), _ptr(v_scales), int(kv_dtype), int(batch), int(n_heads),
                                 int(n_kv_heads), int(head_dim), int(window), float(softcap), float(scale),
                                 int(split_keys), _ptr(out), int(out_dtype), _ptr(lse_out), _ptr(workspace),
                                 int(workspace_bytes), _stream(stream)))


def _dtype_of(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return ATTN_F32
    if t.dtype == torch.float16:
        return ATTN_F16
    raise AttnError(ATTN_EINVAL, "q and out must be float16 or float32, not %s" % t.dtype)


def attn_decode_tiered(q, q_dtype, cold_k, cold_v, cold_k_scales, cold_v_scales, cold_dtype, cold_len,
                       cold_page_table, cold_page_size, cold_max_pages_per_seq, cold_n_pages, cold_max_kv, hot_k,
                       hot_v, hot_len, hot_start, hot_ring, batch, n_heads, n_kv_heads, head_dim, window, softcap,
                       scale, split_keys, out, out_dtype, lse_out, workspace, workspace_bytes, stream=None) -> None:
    _check(load().attn_decode_tiered(_ptr(q), int(q_dtype), _ptr(cold_k), _ptr(cold_v), _ptr(cold_k_scales),
                                     _ptr(cold_v_scales),
                                     int(cold_dtype), _ptr(cold_len), _ptr(cold_page_table), int(cold_page_size),
                                     int(cold_max_pages_per_seq), int(cold_n_pages), int(cold_max_kv), _ptr(hot_k),
                                     _ptr(hot_v), _ptr(hot_len), _ptr(hot_start), int(hot_ring), int(batch),
                                     int(n_heads), int(n_kv_heads), int(head_dim), int(window), float(softcap),
                                     float(scale), int(split_keys), _ptr(out), int(out_dtype), _ptr(lse_out),
                                     _ptr(workspace), int(workspace_bytes), _stream(stream)))


def decode_tiered(case, out=None, lse_out=None, workspace=None, split_keys: int = 0, stream=None, out_f32=False):
    """attn_decode_tiered on a TieredCase-like object (tensors already on the GPU);
    q f16 or f32 as the case holds it, out f16 (or f32 with ``out_f32``)."""
    import torch
    dev = case.q.device
    B, Hq, Hkv, D = case.batch, case.n_heads, case.n_kv_heads, case.head_dim
    if out is None:
        out = _empty((B, Hq, D), torch.float32 if out_f32 else torch.float16, dev, stream)
    ws_bytes = attn_decode_tiered_workspace_size(B, Hq, Hkv, D, case.cap, case.hot_ring, split_keys)
    if ws_bytes == 0:
        raise AttnError(ATTN_EINVAL, "invalid sizes for the tiered decode workspace")
    if workspace is None:
        workspace = _empty(ws_bytes, torch.uint8, dev, stream, scratch=True)
    attn_decode_tiered(case.q, _dtype_of(case.q), case.k, case.v, case.k_scales, case.v_scales,
                       ATTN_KV_INT8 if case.int8 else ATTN_KV_F16, case.kv_len, case.page_table, case.page_size,
                       case.max_pages, case.n_pages, case.cap, case.hot_k, case.hot_v, case.hot_len,
                       case.hot_start, case.hot_ring, B, Hq, Hkv, D, case.window, case.softcap, case.scale,
                       split_keys, out, _dtype_of(out), lse_out, workspace, workspace.numel(), stream)
    return out


def attn_decode_noalloc(q, k_cache, v_cache, kv_len, page_table, page_size, max_pages_per_seq, n_pages,
                        max_kv, k_scales, v_scales, kv_dtype, batch, n_heads, n_kv_heads, head_dim, window,
                        softcap, scale, split_keys, out, lse_out, stream=None) -> None:
    """attn_decode without a caller workspace: the library's fixed 16 MiB
    device scratch array is used instead (for callers that cannot allocate)."""
    _check(load().attn_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kv_len), _ptr(page_table),
                                      int(page_size), int(max_pages_per_seq), int(n_pages), int(max_kv),
                                      _ptr(k_scales), _ptr(v_scales), int(kv_dtype), int(batch), int(n_heads),
                                      int(n_kv_heads), int(head_dim), int(window), float(softcap), float(scale),
                                      int(split_keys), _ptr(out), _ptr(lse_out), _stream(stream)))


def attn_prefill(q, k, v, seq_len, n_heads, n_kv_heads, head_dim, causal, window, softcap, scale,
                 out, lse_out=None, stream=None) -> None:
    _check(load().attn_prefill(_ptr(q), _ptr(k), _ptr(v), int(seq_len), int(n_heads), int(n_kv_heads),
                               int(head_dim), int(bool(causal)), int(window), float(softcap), float(scale),
                               _ptr(out), _ptr(lse_out), _stream(stream)))


def attn_decode_validate(kv_len, page_table, batch, page_size, max_pages_per_seq, n_pages, max_kv,
                         stream=None):
    """Returns (status, first bad sequence or -1); never raises on EBOUNDS/EINVAL."""
    bad = ctypes.c_int(-1)
    st = load().attn_decode_validate(_ptr(kv_len), _ptr(page_table), int(batch), int(page_size),
                                     int(max_pages_per_seq), int(n_pages), int(max_kv), ctypes.byref(bad),
                                     _stream(stream))
    if st == ATTN_ECUDA:
        _check(st)
    return st, bad.value


def attn_device_status(stream=None) -> int:
    return int(load().attn_device_status(_stream(stream)))


# ---------------------------------------------------------------- conveniences
def attn_testing_set_waits(wait_limit_ns: int, stall_first_tile: int) -> int:
    """Testing hook: pipeline-wait time limit (0 = the default) and the first-tile stall."""
    return load().attn_testing_set_waits(int(wait_limit_ns), int(stall_first_tile))


def decode(case, out=None, lse_out=None, workspace=None, split_keys: int = 0, max_kv: Optional[int] = None,
           stream=None, out_f32=False):
    """attn_decode on a DecodeCase-like object (tensors already on the GPU);
    attn_decode_ring when the case holds a ring cache (``case.ring > 0``).

    Allocates ``out`` (and the workspace) with torch when not given.
    """
    import torch
    dev = case.q.device
    B, Hq, Hkv, D = case.batch, case.n_heads, case.n_kv_heads, case.head_dim
    ring = int(getattr(case, "ring", 0) or 0)
    if max_kv is None:
        max_kv = ring if ring else case.cap
    if out is None:
        out = _empty((B, Hq, D), torch.float32 if out_f32 else torch.float16, dev, stream)
    ws_bytes = attn_decode_workspace_size(B, Hq, Hkv, D, max_kv, split_keys)
    if ws_bytes == 0:
        raise AttnError(ATTN_EINVAL, "invalid sizes for the decode workspace")
    if workspace is None:
        workspace = _empty(ws_bytes, torch.uint8, dev, stream, scratch=True)
    qt, ot = _dtype_of(case.q), _dtype_of(out)
    if qt != ATTN_F16 or ot != ATTN_F16:
        attn_decode_ex(case.q, qt, case.k, case.v, case.kv_len, case.page_table, case.page_size, case.max_pages,
                       case.n_pages, max_kv, ring, case.k_scales, case.v_scales,
                       ATTN_KV_INT8 if case.int8 else ATTN_KV_F16, B, Hq, Hkv, D, case.window, case.softcap,
                       case.scale, split_keys, out, ot, lse_out, workspace, workspace.numel(), stream)
        return out
    if ring:
        attn_decode_ring(case.q, case.k, case.v, case.kv_len, ring, case.k_scales, case.v_scales,
                         ATTN_KV_INT8 if case.int8 else ATTN_KV_F16, B, Hq, Hkv, D, case.window, case.softcap,
                         case.scale, split_keys, out, lse_out, workspace, workspace.numel(), stream)
        return out
    attn_decode(case.q, case.k, case.v, case.kv_len, case.page_table, case.page_size, case.max_pages,
                case.n_pages, max_kv, case.k_scales, case.v_scales,
                ATTN_KV_INT8 if case.int8 else ATTN_KV_F16, B, Hq, Hkv, D, case.window, case.softcap,
                case.scale, split_keys, out, lse_out, workspace, workspace.numel(), stream)
    return out


def prefill(case, out=None, lse_out=None, stream=None):
    """attn_prefill on a PrefillCase-like object (tensors already on the GPU)."""
    if out is None:
        out = _empty(case.q.shape, case.q.dtype, case.q.device, stream)
    attn_prefill(case.q, case.k, case.v, case.seq_len, case.n_heads, case.n_kv_heads, case.head_dim,
                 case.causal, case.window, case.softcap, case.scale, out, lse_out, stream)
    return out


def attn_prefill_paged(q, k_cache, v_cache, q_start, kv_len, page_table, page_size, max_pages, n_pages, batch,
                       total_q, max_q, n_heads, n_kv_heads, head_dim, window, softcap, scale, out, lse_out,
                       stream=None) -> None:
    _check(load().attn_prefill_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(q_start), _ptr(kv_len),
                                     _ptr(page_table), int(page_size), int(max_pages), int(n_pages), int(batch),
                                     int(total_q), int(max_q), int(n_heads), int(n_kv_heads), int(head_dim),
                                     int(window), float(softcap), float(scale), _ptr(out), _ptr(lse_out),
                                     _stream(stream)))


def attn_prefill_paged_workspace_size(batch, max_q, n_heads, n_kv_heads, head_dim, kv_dtype) -> int:
    return int(load().attn_prefill_paged_workspace_size(batch, max_q, n_heads, n_kv_heads, head_dim, kv_dtype))


def attn_prefill_paged_ex(q, k_cache, v_cache, q_start, kv_len, page_table, page_size, max_pages, n_pages, k_scales,
                          v_scales, kv_dtype, batch, total_q, max_q, n_heads, n_kv_heads, head_dim, window, softcap,
                          scale, out, lse_out, workspace, workspace_bytes, stream=None) -> None:
    _check(load().attn_prefill_paged_ex(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(q_start), _ptr(kv_len),
                                        _ptr(page_table), int(page_size), int(max_pages), int(n_pages),
                                        _ptr(k_scales), _ptr(v_scales), int(kv_dtype), int(batch), int(total_q),
                                        int(max_q), int(n_heads), int(n_kv_heads), int(head_dim), int(window),
                                        float(softcap), float(scale), _ptr(out), _ptr(lse_out), _ptr(workspace),
                                        int(workspace_bytes), _stream(stream)))


def attn_append(q, k, v, in_dtype, q_stride, k_stride, v_stride, q_norm, k_norm, norm_eps, norm_offset, rope_cos,
                rope_sin, rope_positions, rope_dim, rope_interleaved, q_start, kv_len, k_cache, v_cache, page_table,
                page_size, max_pages, n_pages, max_kv, ring_size, k_scales, v_scales, kv_dtype, batch, total_q,
                n_heads, n_kv_heads, head_dim, q_out, q_out_dtype, stream=None) -> None:
    _check(load().attn_append(_ptr(q), _ptr(k), _ptr(v), int(in_dtype), int(q_stride), int(k_stride), int(v_stride),
                              _ptr(q_norm), _ptr(k_norm), float(norm_eps), float(norm_offset), _ptr(rope_cos),
                              _ptr(rope_sin), int(rope_positions), int(rope_dim), int(bool(rope_interleaved)),
                              _ptr(q_start), _ptr(kv_len), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
                              int(page_size), int(max_pages), int(n_pages), int(max_kv), int(ring_size),
                              _ptr(k_scales), _ptr(v_scales), int(kv_dtype), int(batch), int(total_q), int(n_heads),
                              int(n_kv_heads), int(head_dim), _ptr(q_out), int(q_out_dtype), _stream(stream)))


def attn_kv_read(k_cache, v_cache, kv_len, first, out_start, page_table, page_size, max_pages, n_pages, max_kv,
                 ring_size, k_scales, v_scales, kv_dtype, batch, total, n_kv_heads, head_dim, k_out, v_out, out_dtype,
                 stream=None) -> None:
    _check(load().attn_kv_read(_ptr(k_cache), _ptr(v_cache), _ptr(kv_len), _ptr(first), _ptr(out_start),
                               _ptr(page_table), int(page_size), int(max_pages), int(n_pages), int(max_kv),
                               int(ring_size), _ptr(k_scales), _ptr(v_scales), int(kv_dtype), int(batch), int(total),
                               int(n_kv_heads), int(head_dim), _ptr(k_out), _ptr(v_out), int(out_dtype),
                               _stream(stream)))


def prefill_paged(case, out=None, lse_out=None, stream=None, workspace=None):
    """attn_prefill_paged on a ChunkCase-like object (tensors already on the GPU);
    attn_prefill_paged_ex over int8 pages when its cache holds int8 codes."""
    import torch
    if out is None:
        out = _empty(case.q.shape, case.q.dtype, case.q.device, stream)
    if case.total_q == 0 or case.max_q == 0:   # (empty tensors have no address to pass on)
        return out
    if case.k.dtype == torch.int8:
        _cache_args(case)
        _lengths(case, None, q_start=case.q_start)
        rows = case.total_q * case.n_heads
        for what, x, dtype, n in (("q", case.q, torch.float16, rows * case.head_dim),
                                  ("out", out, torch.float16, rows * case.head_dim),
                                  ("lse_out", lse_out, torch.float32, rows)):
            if x is not None:
                _dense(what, x, dtype, case.k, least=n)
        if workspace is None:
            size = attn_prefill_paged_workspace_size(case.batch, case.max_q, case.n_heads, case.n_kv_heads,
                                                     case.head_dim, ATTN_KV_INT8)
            if size == 0:
                raise AttnError(ATTN_EINVAL, "invalid sizes for the chunked prefill workspace")
            workspace = _empty(size, torch.uint8, case.q.device, stream, scratch=True)
        attn_prefill_paged_ex(case.q, case.k, case.v, case.q_start, case.kv_len, case.page_table, case.page_size,
                              case.max_pages, int(case.k.shape[0]), case.k_scales, case.v_scales, ATTN_KV_INT8,
                              case.batch, case.total_q, case.max_q, case.n_heads, case.n_kv_heads, case.head_dim,
                              case.window, case.softcap, case.scale, out, lse_out, workspace, workspace.numel(),
                              stream)
        return out
    attn_prefill_paged(case.q, case.k, case.v, case.q_start, case.kv_len, case.page_table, case.page_size,
                       case.max_pages, int(case.k.shape[0]), case.batch, case.total_q, case.max_q, case.n_heads,
                       case.n_kv_heads, case.head_dim, case.window, case.softcap, case.scale, out, lse_out, stream)
    return out


def _need(ok, message, *values):
    if not ok:
        raise AttnError(ATTN_EINVAL, message % values)


def _dense(what, x, dtype, like, shape=None, least=0):
    """A contiguous tensor of dtype beside the cache ``like``, of the given shape or with at least
    ``least`` elements: the kernels address all of them from their first element."""
    _need(x.dtype == dtype and x.is_contiguous(), "%s must be a contiguous %s tensor", what, dtype)
    _need(x.device == like.device, "%s must be on the cache's device", what)
    if shape is not None:
        _need(tuple(x.shape) == shape, "%s must have the shape %s, not %s", what, shape, tuple(x.shape))
    _need(x.numel() >= least, "%s must have at least %d elements", what, least)


def _cache_args(case):
    """page_size, max_pages, n_pages, max_kv and ring_size of a DecodeCase- or ChunkCase-like
    cache, whose tensors agree with its sizes."""
    import torch
    k, B, ring = case.k, int(case.batch), int(getattr(case, "ring", 0) or 0)
    _need(k.dim() == 4 and k.dtype in (torch.float16, torch.int8),
          "the cache must be a float16 or int8 tensor [B or pages, tokens, Hkv, D]")
    slots, rows, Hkv, D = k.shape
    _need((Hkv, D) == (case.n_kv_heads, case.head_dim),
          "the cache's heads must be n_kv_heads of head_dim, not %d of %d", Hkv, D)
    _dense("k", k, k.dtype, k)
    _dense("v", case.v, k.dtype, k, (slots, rows, Hkv, D))
    if k.dtype == torch.int8:
        for what in ("k_scales", "v_scales"):
            x = getattr(case, what)
            _need(x is not None, "an int8 cache needs %s", what)
            _dense(what, x, torch.float16, k, (slots, Hkv, rows))
    if case.page_table is not None:
        _need(int(case.page_size) == rows, "page_size must be the pages' tokens (%d)", rows)
        _dense("page_table", case.page_table, torch.int32, k, least=B * int(case.max_pages))
        _need(case.page_table.shape[-1] == int(case.max_pages), "page_table must have max_pages columns")
        return rows, int(case.max_pages), slots, 0, 0
    _need(slots >= B, "the cache must hold a slot for each of %d sequences", B)
    _need(ring in (0, rows), "ring must be the cache's tokens (%d)", rows)
    return 0, 0, 0, 0 if ring else rows, ring


def _lengths(case, kv_len, **others):
    """The per-sequence lengths and starts of a call; returns kv_len (default: the case's)."""
    import torch
    kv_len = case.kv_len if kv_len is None else kv_len
    _dense("kv_len", kv_len, torch.int32, case.k, least=case.batch)
    for what, x in others.items():
        if x is not None:
            _dense(what, x, torch.int32, case.k, least=case.batch + (what != "first"))
    return kv_len


def append(case, q, k, v, q_start, kv_len=None, q_norm=None, k_norm=None, norm_eps=1e-6, norm_offset=0.0,
           rope_cos=None, rope_sin=None, rope_interleaved=False, q_out=None, stream=None):
    """attn_append of packed token rows (q [T, Hq, D] or None; k, v [T, Hkv, D], f16
    or f32, the heads of a token together) to the cache that a DecodeCase- or
    ChunkCase-like object holds; ``kv_len`` (default: the case's) counts each
    sequence's tokens with the new ones.  Returns q_out (f16 unless given; it may be q
    where q is contiguous and of its type)."""
    import torch
    P, max_pages, n_pages, max_kv, ring = _cache_args(case)
    int8 = case.k.dtype == torch.int8
    D = case.k.shape[3]
    _need(k.dim() == 3 and k.shape[1:] == case.k.shape[2:], "k must be [T, Hkv, D] rows of the cache's heads")
    _need(v.shape == k.shape, "v must have k's shape")
    _need(q is None or (q.dim() == 3 and q.shape[0] == k.shape[0] and q.shape[2] == D),
          "q must be [T, Hq, D] with k's T and D")

    def stride(x):
        if x is None:
            return 0
        if x.dtype != k.dtype or x.stride(2) != 1 or x.stride(1) != D:
            raise AttnError(ATTN_EINVAL, "q, k and v rows must have one type and their heads side by side")
        _need(x.device == case.k.device, "q, k and v must be on the cache's device")
        return x.stride(0) if x.shape[0] > 1 else x.shape[1] * D

    kv_len = _lengths(case, kv_len, q_start=q_start)
    for what, x in (("q_norm", q_norm), ("k_norm", k_norm)):
        if x is not None:
            _dense(what, x, torch.float32, case.k, (D,))
    _need((rope_cos is None) == (rope_sin is None), "rope_cos and rope_sin go together")
    if rope_cos is not None:
        _need(rope_cos.dim() == 2, "rope_cos must be [positions, rope_dim / 2]")
        _dense("rope_cos", rope_cos, torch.float32, case.k)
        _dense("rope_sin", rope_sin, torch.float32, case.k, tuple(rope_cos.shape))
    if q is not None and q_out is not None:
        _dense("q_out", q_out, q_out.dtype, case.k, tuple(q.shape))
    if q is not None and q_out is None:
        q_out = _empty(q.shape, torch.float16, q.device, stream)
    if k.shape[0] == 0:
        return q_out
    rows = 0 if rope_cos is None else rope_cos.shape[0]
    rot = 0 if rope_cos is None else 2 * rope_cos.shape[1]
    attn_append(q, k, v, _dtype_of(k), stride(q), stride(k), stride(v), q_norm, k_norm, norm_eps, norm_offset,
                rope_cos, rope_sin, rows, rot, rope_interleaved, q_start, kv_len,
                case.k, case.v, case.page_table, P, max_pages, n_pages, max_kv, ring,
                case.k_scales if int8 else None, case.v_scales if int8 else None,
                ATTN_KV_INT8 if int8 else ATTN_KV_F16, case.batch, k.shape[0], 0 if q is None else q.shape[1],
                k.shape[1], k.shape[2], q_out, ATTN_F16 if q_out is None else _dtype_of(q_out), stream)
    return q_out


def kv_read(case, out_start, total, first=None, kv_len=None, out_f32=False, stream=None):
    """attn_kv_read of a DecodeCase- or ChunkCase-like object's cache: (k, v) rows
    [total, Hkv, D], f16 or f32; rows past out_start[B] are not written."""
    import torch
    P, max_pages, n_pages, max_kv, ring = _cache_args(case)
    int8 = case.k.dtype == torch.int8
    kv_len = _lengths(case, kv_len, out_start=out_start, first=first)
    shape = (total, case.n_kv_heads, case.head_dim)
    dt = torch.float32 if out_f32 else torch.float16
    k, v = (_empty(shape, dt, case.k.device, stream) for _ in range(2))
    if total == 0:
        return k, v
    attn_kv_read(case.k, case.v, kv_len, first, out_start, case.page_table, P,
                 max_pages, n_pages, max_kv, ring, case.k_scales if int8 else None, case.v_scales if int8 else None,
                 ATTN_KV_INT8 if int8 else ATTN_KV_F16, case.batch, total, case.n_kv_heads, case.head_dim, k, v,
                 _dtype_of(k), stream)
    return k, v


# ---------------------------------------------------------------- latent attention
# The calls' argument structs, packed in one step: each argument on its own costs a ctypes call 0.15 us and as
# much again in Python (32 of them: 13 us a call, packed 3.6).
_LATENT_APPEND_ARGS = struct.Struct("@3Pi4qP2f2P2i4P9iP2qP")
_LATENT_READ_ARGS = struct.Struct("@5P8i2PiP")
_LATENT_ATTEND_ARGS = struct.Struct("@5P10if3PNP")
_LATENT_PREFILL_ARGS = struct.Struct("@4P6q2P8if3P")


def _addr(x) -> int:
    if x is None:
        return 0
    return x if isinstance(x, int) else x.data_ptr()


def _packed(layout, *args) -> bytes:
    try:
        return layout.pack(*args)
    except (struct.error, OverflowError) as e:
        raise AttnError(ATTN_EINVAL, "an argument that its type does not hold (%s)" % e) from None


def attn_latent_append(c, k_rope, q_rope, in_dtype, c_stride, k_rope_stride, q_stride, q_head_stride, c_norm, norm_eps,
                       norm_offset, rope_cos, rope_sin, rope_positions, rope_interleaved, q_start, kv_len, cache,
                       page_table, page_size, max_pages, n_pages, max_kv, batch, total_q, n_heads, latent_dim,
                       rope_dim, q_out, q_out_stride, q_out_head_stride, stream=None) -> None:
    _check(load().attn_latent_append_from(_packed(
        _LATENT_APPEND_ARGS, _addr(c), _addr(k_rope), _addr(q_rope), in_dtype, c_stride, k_rope_stride, q_stride,
        q_head_stride, _addr(c_norm), norm_eps, norm_offset, _addr(rope_cos), _addr(rope_sin), rope_positions,
        bool(rope_interleaved), _addr(q_start), _addr(kv_len), _addr(cache), _addr(page_table), page_size, max_pages,
        n_pages, max_kv, batch, total_q, n_heads, latent_dim, rope_dim, _addr(q_out), q_out_stride, q_out_head_stride,
        _stream(stream) or 0)))


def attn_latent_read(cache, kv_len, first, out_start, page_table, page_size, max_pages, n_pages, max_kv, batch, total,
                     latent_dim, rope_dim, c_out, k_rope_out, out_dtype, stream=None) -> None:
    _check(load().attn_latent_read_from(_packed(
        _LATENT_READ_ARGS, _addr(cache), _addr(kv_len), _addr(first), _addr(out_start), _addr(page_table), page_size,
        max_pages, n_pages, max_kv, batch, total, latent_dim, rope_dim, _addr(c_out), _addr(k_rope_out), out_dtype,
        _stream(stream) or 0)))


def attn_latent_workspace_size(batch, max_q, n_heads, latent_dim) -> int:
    return int(load().attn_latent_workspace_size(int(batch), int(max_q), int(n_heads), int(latent_dim)))


def attn_latent_attend(q, cache, q_start, kv_len, page_table, page_size, max_pages, n_pages, max_kv, batch, total_q,
                       max_q, n_heads, latent_dim, rope_dim, scale, out, lse_out, workspace, workspace_bytes,
                       stream=None) -> None:
    _check(load().attn_latent_attend_from(_packed(
        _LATENT_ATTEND_ARGS, _addr(q), _addr(cache), _addr(q_start), _addr(kv_len), _addr(page_table), page_size,
        max_pages, n_pages, max_kv, batch, total_q, max_q, n_heads, latent_dim, rope_dim, scale, _addr(out),
        _addr(lse_out), _addr(workspace), workspace_bytes, _stream(stream) or 0)))


def attn_latent_prefill(q, k, v, k_rope, q_stride, k_stride, k_head_stride, v_stride, v_head_stride, k_rope_stride,
                        q_start, kv_start, batch, total_q, total_kv, max_q, n_heads, head_dim, rope_dim, causal, scale,
                        out, lse_out=None, stream=None) -> None:
    _check(load().attn_latent_prefill_from(_packed(
        _LATENT_PREFILL_ARGS, _addr(q), _addr(k), _addr(v), _addr(k_rope), q_stride, k_stride, k_head_stride, v_stride,
        v_head_stride, k_rope_stride, _addr(q_start), _addr(kv_start), batch, total_q, total_kv, max_q, n_heads,
        head_dim, rope_dim, bool(causal), scale, _addr(out), _addr(lse_out), _stream(stream) or 0)))


_ROPE = 64   # values of the rotated part of a latent cache's rows


def _latent_args(case):
    """page_size, max_pages, n_pages, max_kv and R of a LatentCase-like cache, whose tensors
    agree with its sizes."""
    import torch
    x = case.cache
    _need(x.dim() == 3 and x.dtype == torch.float16, "the cache must be a float16 tensor [B or pages, tokens, R + 64]")
    slots, rows, width = x.shape
    _dense("cache", x, torch.float16, x)
    if case.page_table is not None:
        _need(int(case.page_size) == rows, "page_size must be the pages' tokens (%d)", rows)
        _dense("page_table", case.page_table, torch.int32, x, least=int(case.batch) * int(case.max_pages))
        _need(case.page_table.shape[-1] == int(case.max_pages), "page_table must have max_pages columns")
        return rows, int(case.max_pages), slots, 0, width - _ROPE
    _need(slots >= int(case.batch), "the cache must hold a slot for each of %d sequences", int(case.batch))
    return 0, 0, 0, rows, width - _ROPE


def _latent_lengths(case, kv_len, **others):
    import torch
    kv_len = case.kv_len if kv_len is None else kv_len
    _dense("kv_len", kv_len, torch.int32, case.cache, least=case.batch)
    for what, x in others.items():
        if x is not None:
            _dense(what, x, torch.int32, case.cache, least=case.batch + (what != "first"))
    return kv_len


def _rows(what, x, width, like, dtype=None):
    """Token rows (2-D) or heads of token rows (3-D) of ``width`` values, neighbours in memory;
    returns their strides."""
    _need(x.shape[-1] == width and x.stride(-1) == 1, "%s must have rows of %d neighbouring values", what, width)
    _need(dtype is None or x.dtype == dtype, "%s must be %s", what, dtype)
    _need(x.device == like.device, "%s must be on the cache's device", what)
    head = 0
    if x.dim() == 3:
        head = x.stride(1) if x.shape[1] > 1 else width   # (one head's stride is not used)
    least = width if x.dim() == 2 else (x.shape[1] - 1) * head + width
    if x.shape[0] > 1:
        return x.stride(0), head
    return -(-least // 8) * 8, head   # (a single row's stride is not used)


def latent_append(case, c, k_rope, q_start, kv_len=None, q_rope=None, c_norm=None, norm_eps=1e-6, norm_offset=0.0,
                  rope_cos=None, rope_sin=None, rope_interleaved=True, q_out=None, stream=None):
    """attn_latent_append of token rows (c [T, R], k_rope [T, 64], q_rope [T, Hq, 64] or None,
    f16 or f32; slices of wider rows are fine) to the cache that a LatentCase-like object
    holds; ``kv_len`` (default: the case's) counts each sequence's tokens with the new ones.
    Returns q_out (f16, packed unless given)."""
    import torch
    P, max_pages, n_pages, max_kv, R = _latent_args(case)
    x = case.cache
    _need(c.dim() == 2 and k_rope.dim() == 2 and k_rope.shape[0] == c.shape[0], "c and k_rope must be [T, R] and [T, 64]")
    T, dt = c.shape[0], c.dtype
    c_stride, _ = _rows("c", c, R, x)
    k_stride, _ = _rows("k_rope", k_rope, _ROPE, x, dt)
    kv_len = _latent_lengths(case, kv_len, q_start=q_start)
    if c_norm is not None:
        _dense("c_norm", c_norm, torch.float32, x, (R,))
    _need((rope_cos is None) == (rope_sin is None), "rope_cos and rope_sin go together")
    if rope_cos is not None:
        _need(rope_cos.dim() == 2 and rope_cos.shape[1] == _ROPE // 2, "rope_cos must be [positions, 32]")
        _dense("rope_cos", rope_cos, torch.float32, x)
        _dense("rope_sin", rope_sin, torch.float32, x, tuple(rope_cos.shape))
    q_strides = out_strides = (0, 0)
    H = 0
    if q_rope is not None:
        _need(q_rope.dim() == 3 and q_rope.shape[0] == T, "q_rope must be [T, Hq, 64] with c's T")
        H = q_rope.shape[1]
        q_strides = _rows("q_rope", q_rope, _ROPE, x, dt)
        if q_out is None:
            q_out = _empty(q_rope.shape, torch.float16, q_rope.device, stream)
        _need(q_out.shape == q_rope.shape, "q_out must have q_rope's shape")
        out_strides = _rows("q_out", q_out, _ROPE, x, torch.float16)
    if T == 0:
        return q_out
    attn_latent_append(c, k_rope, q_rope, _dtype_of(c), c_stride, k_stride, *q_strides, c_norm, norm_eps, norm_offset,
                       rope_cos, rope_sin, 0 if rope_cos is None else rope_cos.shape[0], rope_interleaved, q_start,
                       kv_len, x, case.page_table, P, max_pages, n_pages, max_kv, case.batch, T, H, R, _ROPE,
                       None if q_rope is None else q_out, *out_strides, stream)
    return q_out


def latent_read(case, out_start, total, first=None, kv_len=None, out_f32=False, stream=None):
    """attn_latent_read of a LatentCase-like object's cache: (c [total, R], k_rope [total, 64]),
    f16 or f32; rows past out_start[B] are not written."""
    import torch
    P, max_pages, n_pages, max_kv, R = _latent_args(case)
    kv_len = _latent_lengths(case, kv_len, out_start=out_start, first=first)
    dt = torch.float32 if out_f32 else torch.float16
    c, k = (_empty((total, n), dt, case.cache.device, stream) for n in (R, _ROPE))
    if total:
        attn_latent_read(case.cache, kv_len, first, out_start, case.page_table, P, max_pages, n_pages, max_kv,
                         case.batch, total, R, _ROPE, c, k, _dtype_of(c), stream)
    return c, k


def latent_attend(case, q, q_start, max_q, kv_len=None, out=None, lse_out=None, workspace=None, stream=None):
    """attn_latent_attend of q [T, Hq, R + 64] (f16, packed) over a LatentCase-like object's cache
    with its ``scale``; ``max_q`` bounds the sequences' new tokens.  Returns out [T, Hq, R]."""
    import torch
    P, max_pages, n_pages, max_kv, R = _latent_args(case)
    x = case.cache
    _need(q.dim() == 3 and q.shape[2] == R + _ROPE, "q must be [T, Hq, %d]", R + _ROPE)
    T, H = q.shape[:2]
    _dense("q", q, torch.float16, x)
    kv_len = _latent_lengths(case, kv_len, q_start=q_start)
    if out is None:
        out = _empty((T, H, R), torch.float16, q.device, stream)
    _dense("out", out, torch.float16, x, (T, H, R))
    if lse_out is not None:
        _dense("lse_out", lse_out, torch.float32, x, least=T * H)
    if T == 0 or max_q == 0:
        return out
    if workspace is None:
        size = attn_latent_workspace_size(case.batch, max_q, H, R)
        if size == 0:
            raise AttnError(ATTN_EINVAL, "invalid sizes for the latent attention workspace")
        workspace = _empty(size, torch.uint8, q.device, stream, scratch=True)
    attn_latent_attend(q, x, q_start, kv_len, case.page_table, P, max_pages, n_pages, max_kv, case.batch, T, max_q, H,
                       R, _ROPE, case.scale, out, lse_out, workspace, workspace.numel(), stream)
    return out


def latent_prefill(q, k, v, k_rope, q_start, kv_start, max_q, scale, causal=True, out=None, lse_out=None, stream=None):
    """attn_latent_prefill of packed q [Tq, Hq, 192], k and v [Tk, Hq, 128] (slices of wider rows
    are fine) and k_rope [Tk, 64], all f16; ``max_q`` bounds the sequences' queries.  Returns
    out [Tq, Hq, 128]."""
    import torch
    HD = 128
    _need(q.dim() == 3 and k.dim() == 3 and v.shape == k.shape and k.shape[1] == q.shape[1] and k_rope.dim() == 2
          and k_rope.shape[0] == k.shape[0], "q, k, v and k_rope must be [Tq, Hq, 192], [Tk, Hq, 128] twice and [Tk, 64]")
    T, H = q.shape[:2]
    q_stride, q_head = _rows("q", q, HD + _ROPE, q, torch.float16)
    _need(q_head == HD + _ROPE, "q's heads must lie side by side")
    k_strides, v_strides = (_rows(what, t, HD, q, torch.float16) for what, t in (("k", k), ("v", v)))
    r_stride, _ = _rows("k_rope", k_rope, _ROPE, q, torch.float16)
    B = q_start.numel() - 1
    _need(B > 0, "q_start must have an element more than there are sequences")
    _dense("q_start", q_start, torch.int32, q)
    _dense("kv_start", kv_start, torch.int32, q, tuple(q_start.shape))
    if out is None:
        out = _empty((T, H, HD), torch.float16, q.device, stream)
    _dense("out", out, torch.float16, q, (T, H, HD))
    if lse_out is not None:
        _dense("lse_out", lse_out, torch.float32, q, least=T * H)
    if T == 0 or max_q == 0:
        return out
    attn_latent_prefill(q, k, v, k_rope, q_stride, *k_strides, *v_strides, r_stride, q_start, kv_start, B, T,
                        k.shape[0], max_q, H, HD, _ROPE, causal, scale, out, lse_out, stream)
    return out
