"""paged_kv_cache_82_gb300 -- Python binding of libpa (paged-KV attention on
GB300).

Thin ctypes marshalling over the C ABI declared in ``include/pa.h``: the
functions here have the same names and the same semantics; they only turn
torch tensors into pointers, sizes and the current CUDA stream.  Every step of
the computation runs in the CUDA kernels of ``libpa.so``; there is no other
implementation.  If the library is missing or no CUDA device is present the
calls raise; nothing falls back.

    pa_reshape_and_cache  -- write this step's K/V into their cache slots
    pa_copy_blocks        -- block-granular copy-on-write
    pa_attention          -- unified decode + chunked-prefill paged attention
    pa_attention_workspace_size, pa_get_device_error
    pa_build_step         -- a step's metadata on the GPU, from request lengths
    pa_norm_rope_and_cache -- q/k norm per head, position rotation, K/V write
    pa_summarise_blocks, pa_select_blocks, pa_attention_selected -- attention
                             over the blocks that a cheap score selects
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import metadata  # noqa: F401  (host step metadata builder)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa.so")

PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_CUDA, PA_ERR_DEVICE = \
    range(5)
PA_F32, PA_F16, PA_BF16, PA_FP8_E4M3, PA_INT4, PA_NVFP4 = range(6)
PA_DEV_ERR_SLOT, PA_DEV_ERR_BLOCK_ID, PA_DEV_ERR_METADATA, \
    PA_DEV_ERR_TIMEOUT, PA_DEV_ERR_NO_BLOCKS = 0x1, 0x2, 0x4, 0x8, 0x10
BLOCK_SIZE = 16

EXPORTED = ("pa_status_string", "pa_reshape_and_cache", "pa_copy_blocks",
            "pa_attention_workspace_size", "pa_attention",
            "pa_get_device_error", "pa_set_profile_events",
            "pa_launch_count", "pa_attention_noalloc",
            "pa_set_debug_bounds", "pa_attention_window",
            "pa_attention_window_workspace_size", "pa_set_wait_limit_ns",
            "pa_test_skip_copy", "pa_attention_cascade",
            "pa_attention_cascade_workspace_size", "pa_build_step",
            "pa_norm_rope_and_cache", "pa_summarise_blocks",
            "pa_select_blocks_workspace_size", "pa_select_blocks",
            "pa_attention_selected_workspace_size", "pa_attention_selected")

_DT = {"f32": PA_F32, "f16": PA_F16, "bf16": PA_BF16, "e4m3": PA_FP8_E4M3,
       "int4": PA_INT4, "nvfp4": PA_NVFP4}
_ELEM_BYTES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}


def page_bytes_4bit(cache_dtype: str, head_dim: int) -> int:
    """PA_PAGE_BYTES of pa.h: bytes of one (block, KV head) page of a 4-bit
    cache (int4: codes + 16 fp32 scales; nvfp4: codes + E4M3 block scales)."""
    return 8 * head_dim + (64 if cache_dtype == "int4" else head_dim)


def bounds_bytes(head_dim: int) -> int:
    """PA_BOUNDS_BYTES of pa.h: bytes of one (block, KV head) record of key
    bounds; a bounds tensor is uint8 [num_blocks, Hkv, bounds_bytes(D)]."""
    return 2 * head_dim + 16


def _cache_geometry(cache: torch.Tensor, cache_dtype: Optional[str],
                    head_dim: Optional[int] = None):
    """(num_blocks, kv_heads, block_size, head_dim) of a cache tensor:
    [NB, Hkv, 16, D] elements, or [NB, Hkv, page_bytes] uint8 for the 4-bit
    formats (head_dim from the page size when not given)."""
    if cache_dtype in ("int4", "nvfp4"):
        if cache.dim() != 3 or cache.dtype != torch.uint8:
            raise ValueError("a 4-bit cache is a uint8 [NB, Hkv, page_bytes] "
                             "tensor")
        NB, H, pb = cache.shape
        D = (pb - 64) // 8 if cache_dtype == "int4" else pb // 9
        if head_dim is not None and head_dim != D:
            raise ValueError("head_dim does not match the cache's pages")
        if page_bytes_4bit(cache_dtype, D) != pb:
            raise ValueError("page size matches no head_dim")
        return NB, H, BLOCK_SIZE, D
    if cache.dim() != 4:
        raise ValueError("the caches must be [NB, Hkv, 16, D]")
    if cache_dtype is not None and cache.element_size() != _ELEM_BYTES[cache_dtype]:
        raise ValueError(f"a cache of {cache.dtype} holds no {cache_dtype} elements")
    return tuple(cache.shape)


_lib = None


class PaError(RuntimeError):
    def __init__(self, status: int, what: str, flags: int = 0):
        self.status = status
        self.flags = flags
        name = _load().pa_status_string(status).decode() if _lib else str(status)
        super().__init__(f"{what}: {name}" + (f" (flags 0x{flags:x})"
                                              if flags else ""))


def load_library(path: str = LIB_PATH):
    """Load libpa.so (built in-tree by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    P, i64, i32, f32, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                            ctypes.c_float, ctypes.c_size_t)
    lib.pa_status_string.argtypes = [i32]
    lib.pa_status_string.restype = ctypes.c_char_p
    lib.pa_reshape_and_cache.argtypes = [P, P, i32, i64, i64, i64, P, P, i32,
                                         i64, i32, i32, i32, P, f32, f32, P]
    lib.pa_reshape_and_cache.restype = i32
    lib.pa_copy_blocks.argtypes = [P, P, i32, i64, i32, i32, i32, P, i64, P]
    lib.pa_copy_blocks.restype = i32
    lib.pa_attention_workspace_size.argtypes = [i64, i32, i32, i32, i32, i32,
                                                i32, ctypes.POINTER(sz)]
    lib.pa_attention_workspace_size.restype = i32
    lib.pa_attention.argtypes = [P, i32, P, P, i32, i64, i32, i32, i32, i32, P,
                                 i32, P, P, i32, i64, i32, i32, f32, f32, f32,
                                 P, P, sz, P]
    lib.pa_attention.restype = i32
    lib.pa_get_device_error.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
    lib.pa_get_device_error.restype = i32
    lib.pa_set_profile_events.argtypes = [P, P]
    lib.pa_set_profile_events.restype = i32
    lib.pa_launch_count.argtypes = [ctypes.POINTER(ctypes.c_uint64)]
    lib.pa_launch_count.restype = i32
    lib.pa_attention_window.argtypes = [P, i32, P, P, i32, i64, i32, i32, i32,
                                        i32, P, i32, P, P, i32, i64, i32, i32,
                                        f32, f32, f32, i32, P, P, sz, P]
    lib.pa_attention_window.restype = i32
    lib.pa_attention_window_workspace_size.argtypes = [
        i64, i32, i32, i32, i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.pa_attention_window_workspace_size.restype = i32
    lib.pa_attention_cascade.argtypes = [P, i32, P, P, i32, i64, i32, i32, i32,
                                         i32, P, i32, P, P, i32, i64, i32, i32,
                                         f32, f32, f32, i32, P, P, sz, P]
    lib.pa_attention_cascade.restype = i32
    lib.pa_attention_cascade_workspace_size.argtypes = [
        i64, i32, i32, i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.pa_attention_cascade_workspace_size.restype = i32
    lib.pa_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.pa_set_wait_limit_ns.restype = i32
    lib.pa_test_skip_copy.argtypes = [i64]
    lib.pa_test_skip_copy.restype = i32
    lib.pa_set_debug_bounds.argtypes = [i32]
    lib.pa_set_debug_bounds.restype = i32
    lib.pa_attention_noalloc.argtypes = [P, i32, P, P, i32, i64, i32, i32, i32,
                                         i32, P, i32, P, P, i32, i64, i32, i32,
                                         f32, f32, f32, P, P]
    lib.pa_attention_noalloc.restype = i32
    lib.pa_build_step.argtypes = [P, P, i32, P, i32, P, i64, P, P, i64, i32,
                                  i64, P, P, P, P, P]
    lib.pa_build_step.restype = i32
    lib.pa_norm_rope_and_cache.argtypes = [
        P, P, P, i32, i64, i64, i64, i64, P, P, i32, f32, P, i64, i32, i32, P,
        P, P, P, i32, i64, i32, i32, i32, i32, P, f32, f32, P]
    lib.pa_norm_rope_and_cache.restype = i32
    lib.pa_summarise_blocks.argtypes = [P, i32, i64, i32, i32, i32, P, i32, P,
                                        P, i32, i64, i32, i32, P, P]
    lib.pa_summarise_blocks.restype = i32
    lib.pa_select_blocks_workspace_size.argtypes = [i64, i32, i32,
                                                    ctypes.POINTER(sz)]
    lib.pa_select_blocks_workspace_size.restype = i32
    lib.pa_select_blocks.argtypes = [P, i32, P, i64, i32, i32, i32, i32, P, i32,
                                     P, P, i32, i64, i32, i32, i32, i32, i32, P,
                                     P, P, sz, P]
    lib.pa_select_blocks.restype = i32
    lib.pa_attention_selected_workspace_size.argtypes = [
        i64, i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.pa_attention_selected_workspace_size.restype = i32
    lib.pa_attention_selected.argtypes = [
        P, i32, P, P, i32, i64, i32, i32, i32, i32, P, i32, P, P, i32, i64, i32,
        i32, P, P, i32, f32, f32, f32, P, P, sz, P]
    lib.pa_attention_selected.restype = i32
    _lib = lib
    return lib


def _load():
    return _lib if _lib is not None else load_library()


_TYPE_CODES = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16,
               torch.uint8: PA_FP8_E4M3}
if hasattr(torch, "float8_e4m3fn"):
    _TYPE_CODES[torch.float8_e4m3fn] = PA_FP8_E4M3


def _dtype_code(t: torch.Tensor, override: Optional[str] = None) -> int:
    if override is not None:
        return _DT[override]
    code = _TYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported tensor dtype {t.dtype}")
    return code


def _dev(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.data_ptr()


# the current stream's handle without a Stream object around it: 0.1 us instead
# of 2.9 us of every call on the Arm host
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _new(shape, dtype, device, stream, returned: bool = True) -> torch.Tensor:
    """A tensor that a call on `stream` allocates, from that stream's memory, so
    that neither what the memory held before nor what is put there after the
    tensor's release meets the call's kernels.  One that is returned is known to
    the current stream too, where the caller will use it."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    current = torch.cuda.current_stream()
    if stream.cuda_stream == current.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(current)
    return t


def _check(status: int, what: str) -> None:
    if status != PA_OK:
        raise PaError(status, what)


def _step_shapes(q, k_cache, v_cache, block_tables, seq_lens,
                 query_start_loc, out, cache_dtype=None):
    """Check the tensors of one attention step the way the C ABI reads them
    (contiguous, int32 metadata, consistent sizes) and return (T, Hq, D, NB,
    Hkv, block_size, B).  Runs before any pointer is taken, so a strided q or
    an int64 length array is refused instead of being read as raw bytes."""
    if q.dim() != 3 or v_cache.shape != k_cache.shape:
        raise ValueError("q must be [T, Hq, D] and both caches alike")
    T, Hq, D = q.shape
    NB, Hkv, bs, Dc = _cache_geometry(k_cache, cache_dtype)
    if Dc != D:
        raise ValueError("head_dim of q and of the caches differ")
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    for t, n in ((block_tables, "block_tables"), (seq_lens, "seq_lens"),
                 (query_start_loc, "query_start_loc")):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous int32 tensor")
    B = seq_lens.numel()
    if (query_start_loc.numel() != B + 1 or block_tables.dim() != 2
            or block_tables.shape[0] != B):
        raise ValueError("inconsistent number of sequences")
    if out is not None and (out.shape != q.shape or out.dtype != q.dtype
                            or not out.is_contiguous()):
        raise ValueError("out must be a contiguous tensor like q")
    return T, Hq, D, NB, Hkv, bs, B


def pa_reshape_and_cache(key: torch.Tensor, value: torch.Tensor,
                         k_cache: torch.Tensor, v_cache: torch.Tensor,
                         slot_mapping: torch.Tensor, k_scale: float = 1.0,
                         v_scale: float = 1.0, cache_dtype: Optional[str] = None,
                         stream=None) -> None:
    """key/value [T, Hkv, D] (row stride may exceed Hkv*D), caches
    [NB, Hkv, 16, D], slot_mapping int64 [T]."""
    T, Hkv, D = key.shape
    if value.shape != key.shape or key.stride(2) != 1 or key.stride(1) != D \
            or value.stride(2) != 1 or value.stride(1) != D:
        raise ValueError("key/value must be [T, Hkv, D] with contiguous rows")
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != T:
        raise ValueError("slot_mapping must be int64 [num_tokens]")
    NB, Hc, bs, Dc = _cache_geometry(k_cache, cache_dtype, D)
    if (Hc, Dc) != (Hkv, D) or v_cache.shape != k_cache.shape:
        raise ValueError("cache shape does not match key/value")
    lib = _load()
    st = lib.pa_reshape_and_cache(
        _dev(key, "key"), _dev(value, "value"), _dtype_code(key), T,
        key.stride(0), value.stride(0), _dev(k_cache, "k_cache"),
        _dev(v_cache, "v_cache"), _dtype_code(k_cache, cache_dtype), NB, bs,
        Hkv, D, _dev(slot_mapping, "slot_mapping"), float(k_scale),
        float(v_scale), _stream(stream))
    _check(st, "pa_reshape_and_cache")


def pa_copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor,
                   block_mapping: torch.Tensor,
                   cache_dtype: Optional[str] = None, stream=None) -> None:
    """block_mapping int64 [P, 2] of (src, dst) pairs."""
    if block_mapping.dtype != torch.int64 or not block_mapping.is_contiguous():
        raise ValueError("block_mapping must be a contiguous int64 [P, 2]")
    NB, Hkv, bs, D = _cache_geometry(k_cache, cache_dtype)
    lib = _load()
    st = lib.pa_copy_blocks(_dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
                            _dtype_code(k_cache, cache_dtype), NB, bs, Hkv, D,
                            _dev(block_mapping, "block_mapping"),
                            block_mapping.numel() // 2, _stream(stream))
    _check(st, "pa_copy_blocks")


def pa_attention_workspace_size(num_tokens: int, num_q_heads: int,
                                num_kv_heads: int, head_dim: int,
                                num_seqs: int, max_query_len: int,
                                max_seq_len: int) -> int:
    out = ctypes.c_size_t(0)
    st = _load().pa_attention_workspace_size(num_tokens, num_q_heads,
                                             num_kv_heads, head_dim, num_seqs,
                                             max_query_len, max_seq_len,
                                             ctypes.byref(out))
    _check(st, "pa_attention_workspace_size")
    return int(out.value)


def pa_attention(q: torch.Tensor, k_cache: torch.Tensor,
                 v_cache: torch.Tensor, block_tables: torch.Tensor,
                 seq_lens: torch.Tensor, query_start_loc: torch.Tensor,
                 max_query_len: int, max_seq_len: int, scale: float,
                 k_scale: float = 1.0, v_scale: float = 1.0,
                 out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None,
                 cache_dtype: Optional[str] = None, stream=None) -> torch.Tensor:
    """q [T, Hq, D]; caches [NB, Hkv, 16, D]; block_tables int32 [B, M];
    seq_lens int32 [B]; query_start_loc int32 [B+1].  Returns out [T, Hq, D]
    (allocated if not given; the workspace too)."""
    T, Hq, D, NB, Hkv, bs, B = _step_shapes(q, k_cache, v_cache, block_tables,
                                            seq_lens, query_start_loc, out,
                                            cache_dtype)
    if out is None:
        out = _new(q.shape, q.dtype, q.device, stream)
    if workspace is None:
        nbytes = pa_attention_workspace_size(T, Hq, Hkv, D, B, max_query_len,
                                             max_seq_len)
        workspace = _new(max(nbytes, 1), torch.uint8, q.device, stream, False)
    lib = _load()
    st = lib.pa_attention(
        _dev(q, "q"), _dtype_code(q), _dev(k_cache, "k_cache"),
        _dev(v_cache, "v_cache"), _dtype_code(k_cache, cache_dtype), NB, bs, Hq,
        Hkv, D, _dev(block_tables, "block_tables"), block_tables.shape[1],
        _dev(seq_lens, "seq_lens"), _dev(query_start_loc, "query_start_loc"),
        B, T, int(max_query_len), int(max_seq_len), float(scale),
        float(k_scale), float(v_scale), _dev(out, "out"),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream))
    _check(st, "pa_attention")
    return out


def pa_attention_window_workspace_size(num_tokens: int, num_q_heads: int,
                                       num_kv_heads: int, head_dim: int,
                                       num_seqs: int, max_query_len: int,
                                       max_seq_len: int,
                                       sliding_window: int) -> int:
    out = ctypes.c_size_t(0)
    st = _load().pa_attention_window_workspace_size(
        num_tokens, num_q_heads, num_kv_heads, head_dim, num_seqs,
        max_query_len, max_seq_len, sliding_window, ctypes.byref(out))
    _check(st, "pa_attention_window_workspace_size")
    return int(out.value)


def pa_attention_window(q: torch.Tensor, k_cache: torch.Tensor,
                        v_cache: torch.Tensor, block_tables: torch.Tensor,
                        seq_lens: torch.Tensor, query_start_loc: torch.Tensor,
                        max_query_len: int, max_seq_len: int, scale: float,
                        sliding_window: int, k_scale: float = 1.0,
                        v_scale: float = 1.0,
                        out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None,
                        cache_dtype: Optional[str] = None,
                        stream=None) -> torch.Tensor:
    """pa_attention with a sliding window of `sliding_window` keys (each
    query sees its own key and the window - 1 keys before it; 0: none)."""
    T, Hq, D, NB, Hkv, bs, B = _step_shapes(q, k_cache, v_cache, block_tables,
                                            seq_lens, query_start_loc, out,
                                            cache_dtype)
    if out is None:
        out = _new(q.shape, q.dtype, q.device, stream)
    if workspace is None:
        nbytes = pa_attention_window_workspace_size(
            T, Hq, Hkv, D, B, max_query_len, max_seq_len, sliding_window)
        workspace = _new(max(nbytes, 1), torch.uint8, q.device, stream, False)
    st = _load().pa_attention_window(
        _dev(q, "q"), _dtype_code(q), _dev(k_cache, "k_cache"),
        _dev(v_cache, "v_cache"), _dtype_code(k_cache, cache_dtype), NB, bs, Hq,
        Hkv, D, _dev(block_tables, "block_tables"), block_tables.shape[1],
        _dev(seq_lens, "seq_lens"), _dev(query_start_loc, "query_start_loc"),
        B, T, int(max_query_len), int(max_seq_len), float(scale),
        float(k_scale), float(v_scale), int(sliding_window), _dev(out, "out"),
        _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "pa_attention_window")
    return out


def pa_attention_cascade_workspace_size(num_tokens: int, num_q_heads: int,
                                        num_kv_heads: int, head_dim: int,
                                        num_seqs: int, max_query_len: int,
                                        max_seq_len: int) -> int:
    out = ctypes.c_size_t(0)
    st = _load().pa_attention_cascade_workspace_size(
        num_tokens, num_q_heads, num_kv_heads, head_dim, num_seqs,
        max_query_len, max_seq_len, ctypes.byref(out))
    _check(st, "pa_attention_cascade_workspace_size")
    return int(out.value)


def pa_attention_cascade(q: torch.Tensor, k_cache: torch.Tensor,
                         v_cache: torch.Tensor, block_tables: torch.Tensor,
                         seq_lens: torch.Tensor, query_start_loc: torch.Tensor,
                         max_query_len: int, max_seq_len: int, scale: float,
                         common_prefix_blocks: int, k_scale: float = 1.0,
                         v_scale: float = 1.0,
                         out: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None,
                         cache_dtype: Optional[str] = None,
                         stream=None) -> torch.Tensor:
    """pa_attention for a step whose requests all begin with the same
    `common_prefix_blocks` block ids (the shared prefix is read once per KV
    head and merged with each request's own part)."""
    T, Hq, D, NB, Hkv, bs, B = _step_shapes(q, k_cache, v_cache, block_tables,
                                            seq_lens, query_start_loc, out,
                                            cache_dtype)
    if out is None:
        out = _new(q.shape, q.dtype, q.device, stream)
    if workspace is None:
        nbytes = pa_attention_cascade_workspace_size(
            T, Hq, Hkv, D, B, max_query_len, max_seq_len)
        workspace = _new(max(nbytes, 1), torch.uint8, q.device, stream, False)
    st = _load().pa_attention_cascade(
        _dev(q, "q"), _dtype_code(q), _dev(k_cache, "k_cache"),
        _dev(v_cache, "v_cache"), _dtype_code(k_cache, cache_dtype), NB, bs, Hq,
        Hkv, D, _dev(block_tables, "block_tables"), block_tables.shape[1],
        _dev(seq_lens, "seq_lens"), _dev(query_start_loc, "query_start_loc"),
        B, T, int(max_query_len), int(max_seq_len), float(scale),
        float(k_scale), float(v_scale), int(common_prefix_blocks),
        _dev(out, "out"), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "pa_attention_cascade")
    return out


def pa_get_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error flags."""
    flags = ctypes.c_uint32(0)
    st = _load().pa_get_device_error(_stream(stream), ctypes.byref(flags))
    if st not in (PA_OK, PA_ERR_DEVICE):
        raise PaError(st, "pa_get_device_error")
    return int(flags.value)


def pa_set_profile_events(start: Optional[torch.cuda.Event],
                          stop: Optional[torch.cuda.Event]) -> None:
    """Record `start` / `stop` around the attention kernels of every later
    pa_attention call of this thread (measurement hook); None, None turns it
    off."""
    def handle(ev):
        if ev is None:
            return None
        ev.record()  # make sure the event object exists on the device
        return ev.cuda_event
    _check(_load().pa_set_profile_events(handle(start), handle(stop)),
           "pa_set_profile_events")


def pa_set_debug_bounds(enable: bool) -> None:
    """The device-side index checks are always on: True is accepted, False
    raises (PA_ERR_UNSUPPORTED)."""
    _check(_load().pa_set_debug_bounds(1 if enable else 0),
           "pa_set_debug_bounds")


def pa_set_wait_limit_ns(ns: int) -> None:
    """Longest one pipeline wait in the kernels may last (0: the default
    2 s); a wait that runs out is reported as PA_DEV_ERR_TIMEOUT."""
    _check(_load().pa_set_wait_limit_ns(int(ns)), "pa_set_wait_limit_ns")


def pa_test_skip_copy(stage: int) -> None:
    """Testing hook: CTA 0 of the pipelined kernels leaves out the copy of
    pipeline stage `stage` (-1: off), so that the waits on it run out."""
    _check(_load().pa_test_skip_copy(int(stage)), "pa_test_skip_copy")


def pa_launch_count() -> int:
    """Kernels the library has launched from this thread so far."""
    n = ctypes.c_uint64(0)
    _check(_load().pa_launch_count(ctypes.byref(n)), "pa_launch_count")
    return int(n.value)


def pa_attention_noalloc(q: torch.Tensor, k_cache: torch.Tensor,
                         v_cache: torch.Tensor, block_tables: torch.Tensor,
                         seq_lens: torch.Tensor, query_start_loc: torch.Tensor,
                         max_query_len: int, max_seq_len: int, scale: float,
                         k_scale: float = 1.0, v_scale: float = 1.0,
                         out: Optional[torch.Tensor] = None,
                         cache_dtype: Optional[str] = None,
                         stream=None) -> torch.Tensor:
    """pa_attention with the library's fixed device scratch instead of a
    workspace, for callers that cannot allocate device memory per step (the
    output tensor is still the caller's)."""
    if out is None:
        raise ValueError("pa_attention_noalloc needs a caller-provided out")
    T, Hq, D, NB, Hkv, bs, B = _step_shapes(q, k_cache, v_cache, block_tables,
                                            seq_lens, query_start_loc, out,
                                            cache_dtype)
    st = _load().pa_attention_noalloc(_dev(q, "q"), _dtype_code(q), _dev(k_cache, "k_cache"),
           _dev(v_cache, "v_cache"), _dtype_code(k_cache, cache_dtype), NB, bs,
           Hq, Hkv, D, _dev(block_tables, "block_tables"),
           block_tables.shape[1], _dev(seq_lens, "seq_lens"),
           _dev(query_start_loc, "query_start_loc"), B, T, int(max_query_len),
           int(max_seq_len), float(scale), float(k_scale), float(v_scale),
           _dev(out, "out"), _stream(stream))
    _check(st, "pa_attention_noalloc")
    return out


def _plain(*specs) -> None:
    """Check contiguous tensors of a call, (name, tensor, dtype or None: any,
    elements or None: any) each, None tensors left out: types, sizes, and that
    all are on the current CUDA device, where the library launches."""
    dev, off = -2, None
    for name, t, dtype, n in specs:
        if t is None:
            continue
        if (dtype is not None and t.dtype is not dtype) \
                or (n is not None and t.numel() != n) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype or ''} tensor"
                             + (f" of {n} elements" if n is not None else ""))
        d = t.get_device()
        if d != dev:
            if off is None and (d < 0 or dev != -2 or d != torch.cuda.current_device()):
                off = name, d
            dev = d
    if off is not None:
        raise ValueError(f"{off[0]} must be a CUDA tensor" if off[1] < 0 else
                         f"{off[0]} must be on the current CUDA device")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


_I32, _I64, _U8 = torch.int32, torch.int64, torch.uint8


def pa_build_step(query_lens: torch.Tensor, computed_lens: torch.Tensor,
                  block_tables: torch.Tensor, free_blocks: torch.Tensor,
                  free_count: torch.Tensor, num_blocks: int, num_tokens: int,
                  seq_lens: Optional[torch.Tensor] = None,
                  query_start_loc: Optional[torch.Tensor] = None,
                  positions: Optional[torch.Tensor] = None,
                  slot_mapping: Optional[torch.Tensor] = None,
                  free_count_out: Optional[torch.Tensor] = None, stream=None):
    """query_lens, computed_lens int32 [B]; block_tables int32 [B, M] (extended
    in place); free_blocks int32 [F], a stack of free ids; free_count int32
    [1].  Returns (seq_lens int32 [B], query_start_loc int32 [B+1], positions
    int32 [num_tokens], slot_mapping int64 [num_tokens], free_count_out int32
    [1]), allocated where not given; seq_lens may be computed_lens and
    free_count_out may be free_count (updated in place)."""
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [B, M]")
    B, M = block_tables.shape
    T = int(num_tokens)
    dev = block_tables.device
    if seq_lens is None:
        seq_lens = _new(B, _I32, dev, stream)
    if query_start_loc is None:
        query_start_loc = _new(B + 1, _I32, dev, stream)
    if positions is None:
        positions = _new(T, _I32, dev, stream)
    if slot_mapping is None:
        slot_mapping = _new(T, _I64, dev, stream)
    if free_count_out is None:
        free_count_out = _new(1, _I32, dev, stream)
    _plain(("query_lens", query_lens, _I32, B),
           ("computed_lens", computed_lens, _I32, B),
           ("block_tables", block_tables, _I32, None),
           ("free_blocks", free_blocks, _I32, None),
           ("free_count", free_count, _I32, 1), ("seq_lens", seq_lens, _I32, B),
           ("query_start_loc", query_start_loc, _I32, B + 1),
           ("positions", positions, _I32, T),
           ("slot_mapping", slot_mapping, _I64, T),
           ("free_count_out", free_count_out, _I32, 1))
    st = _load().pa_build_step(
        query_lens.data_ptr(), computed_lens.data_ptr(), B,
        block_tables.data_ptr(), M, free_blocks.data_ptr(), free_blocks.numel(),
        free_count.data_ptr(), free_count_out.data_ptr(), int(num_blocks),
        BLOCK_SIZE, T, seq_lens.data_ptr(), query_start_loc.data_ptr(),
        positions.data_ptr(), slot_mapping.data_ptr(), _stream(stream))
    _check(st, "pa_build_step")
    return seq_lens, query_start_loc, positions, slot_mapping, free_count_out


def pa_norm_rope_and_cache(q: torch.Tensor, key: torch.Tensor,
                           value: torch.Tensor, k_cache: torch.Tensor,
                           v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                           positions: Optional[torch.Tensor] = None,
                           cos_sin: Optional[torch.Tensor] = None,
                           q_weight: Optional[torch.Tensor] = None,
                           k_weight: Optional[torch.Tensor] = None,
                           eps: float = 1e-6, interleaved: bool = False,
                           k_scale: float = 1.0, v_scale: float = 1.0,
                           q_out: Optional[torch.Tensor] = None,
                           cache_dtype: Optional[str] = None,
                           stream=None) -> torch.Tensor:
    """q [T, Hq, D], key/value [T, Hkv, D] (rows may be slices of one QKV row);
    positions int32 [T] and cos_sin fp32 [max_position, rotary_dim] (cosines,
    then sines; None: no rotation); q_weight / k_weight [D] (None: no norm).
    Writes the caches and returns q_out [T, Hq, D] (q itself if given as such
    and contiguous)."""
    qs, ks, dtype = q.shape, key.shape, q.dtype
    if len(qs) != 3 or len(ks) != 3 or value.shape != ks or qs[0] != ks[0] \
            or qs[2] != ks[2]:
        raise ValueError("q must be [T, Hq, D] and key/value [T, Hkv, D]")
    T, Hq, D = qs
    Hkv = ks[1]
    if key.dtype is not dtype or value.dtype is not dtype:
        raise ValueError("q, key and value must be of one type")
    rows = []
    for t, h, n in ((q, Hq, "q"), (key, Hkv, "key"), (value, Hkv, "value")):
        row, head, one = t.stride()
        if one != 1 or (h > 1 and head != D):
            raise ValueError(f"{n} must have contiguous rows")
        # (a single token's row is contiguous whatever its stride)
        rows.append(row if T > 1 else h * D)
    NB, Hc, bs, Dc = _cache_geometry(k_cache, cache_dtype, D)
    if Hc != Hkv or Dc != D or v_cache.shape != k_cache.shape \
            or v_cache.dtype is not k_cache.dtype:
        raise ValueError("cache shape does not match key/value")
    span = rot = 0
    if cos_sin is not None:
        if len(cos_sin.shape) != 2:
            raise ValueError("cos_sin must be [max_position, rotary_dim]")
        span, rot = cos_sin.shape
        if positions is None:
            raise ValueError("a rotation needs positions")
    weight = q_weight if q_weight is not None else k_weight
    wdt = None if weight is None else weight.dtype
    if q_out is None:
        q_out = _new((T, Hq, D), dtype, q.device, stream)
    elif q_out.shape != qs:
        raise ValueError("q_out must be a tensor like q")
    _plain(("slot_mapping", slot_mapping, _I64, T),
           ("positions", positions, _I32, T if rot else None),
           ("cos_sin", cos_sin, torch.float32, None),
           ("q_weight", q_weight, wdt, D), ("k_weight", k_weight, wdt, D),
           ("q_out", q_out, dtype, None), ("k_cache", k_cache, None, None),
           ("v_cache", v_cache, None, None))
    dev = q_out.get_device()
    if q.get_device() != dev or key.get_device() != dev or value.get_device() != dev:
        raise ValueError("q, key and value must be on the current CUDA device")
    st = _load().pa_norm_rope_and_cache(
        q.data_ptr(), key.data_ptr(), value.data_ptr(), _dtype_code(q), T,
        *rows, _ptr(q_weight), _ptr(k_weight),
        PA_F32 if weight is None else _dtype_code(weight), float(eps), _ptr(cos_sin),
        span, rot, 1 if interleaved else 0, _ptr(positions), q_out.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), _dtype_code(k_cache, cache_dtype),
        NB, bs, Hq, Hkv, D, slot_mapping.data_ptr(), float(k_scale),
        float(v_scale), _stream(stream))
    _check(st, "pa_norm_rope_and_cache")
    return q_out


def _bounds_shape(bounds: torch.Tensor, NB, Hkv: int, D: int) -> int:
    shape = bounds.shape
    if len(shape) != 3 or shape[1] != Hkv or shape[2] != 2 * D + 16 \
            or (NB is not None and shape[0] != NB):
        raise ValueError("bounds must be a uint8 [num_blocks, Hkv, bounds_bytes(D)] "
                         "tensor")
    return shape[0]


def _step_tables(block_tables, seq_lens, query_start_loc):
    """(sequences, block-table entries of each)."""
    B, shape = seq_lens.numel(), block_tables.shape
    if len(shape) != 2 or shape[0] != B or query_start_loc.numel() != B + 1:
        raise ValueError("inconsistent number of sequences")
    return shape


def pa_summarise_blocks(k_cache: torch.Tensor, bounds: torch.Tensor,
                        block_tables: torch.Tensor, seq_lens: torch.Tensor,
                        query_start_loc: torch.Tensor, num_tokens: int,
                        max_query_len: int, max_seq_len: int,
                        cache_dtype: Optional[str] = None, stream=None) -> None:
    """Key bounds of the blocks this step's tokens were written to, into bounds
    (uint8 [num_blocks, Hkv, bounds_bytes(D)])."""
    NB, Hkv, bs, D = _cache_geometry(k_cache, cache_dtype)
    _bounds_shape(bounds, NB, Hkv, D)
    B, M = _step_tables(block_tables, seq_lens, query_start_loc)
    _plain(("k_cache", k_cache, None, None), ("bounds", bounds, _U8, None),
           ("block_tables", block_tables, _I32, None),
           ("seq_lens", seq_lens, _I32, B),
           ("query_start_loc", query_start_loc, _I32, None))
    st = _load().pa_summarise_blocks(
        k_cache.data_ptr(), _dtype_code(k_cache, cache_dtype), NB, bs, Hkv, D,
        block_tables.data_ptr(), M, seq_lens.data_ptr(),
        query_start_loc.data_ptr(), B, int(num_tokens), int(max_query_len),
        int(max_seq_len), bounds.data_ptr(), _stream(stream))
    _check(st, "pa_summarise_blocks")


def pa_select_blocks_workspace_size(num_tokens: int, num_kv_heads: int,
                                    max_seq_len: int) -> int:
    out = ctypes.c_size_t(0)
    st = _load().pa_select_blocks_workspace_size(num_tokens, num_kv_heads,
                                                 max_seq_len, ctypes.byref(out))
    _check(st, "pa_select_blocks_workspace_size")
    return int(out.value)


def pa_select_blocks(q: torch.Tensor, bounds: torch.Tensor,
                     block_tables: torch.Tensor, seq_lens: torch.Tensor,
                     query_start_loc: torch.Tensor, max_query_len: int,
                     max_seq_len: int, max_selected: int, keep_first: int = 1,
                     keep_last: int = 1,
                     selected: Optional[torch.Tensor] = None,
                     num_selected: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """q [T, Hq, D]; bounds as pa_summarise_blocks leaves them.  Returns
    (selected int32 [T, Hkv, max_selected], num_selected int32 [T, Hkv])."""
    shape, records = q.shape, bounds.shape
    if len(shape) != 3 or len(records) != 3:
        raise ValueError("q must be [T, Hq, D] and bounds [num_blocks, Hkv, bytes]")
    T, Hq, D = shape
    Hkv, K = records[1], int(max_selected)
    NB = _bounds_shape(bounds, None, Hkv, D)
    B, M = _step_tables(block_tables, seq_lens, query_start_loc)
    if selected is None:
        selected = _new((T, Hkv, K), _I32, q.device, stream)
    if num_selected is None:
        num_selected = _new((T, Hkv), _I32, q.device, stream)
    if workspace is None:
        n = pa_select_blocks_workspace_size(T, Hkv, int(max_seq_len))
        workspace = _new(max(n, 1), _U8, q.device, stream, False)
    _plain(("q", q, None, None), ("bounds", bounds, _U8, None),
           ("block_tables", block_tables, _I32, None),
           ("seq_lens", seq_lens, _I32, B),
           ("query_start_loc", query_start_loc, _I32, B + 1),
           ("selected", selected, _I32, T * Hkv * K),
           ("num_selected", num_selected, _I32, T * Hkv),
           ("workspace", workspace, None, None))
    st = _load().pa_select_blocks(
        q.data_ptr(), _dtype_code(q), bounds.data_ptr(), NB, BLOCK_SIZE, Hq, Hkv,
        D, block_tables.data_ptr(), M, seq_lens.data_ptr(),
        query_start_loc.data_ptr(), B, T, int(max_query_len), int(max_seq_len), K,
        int(keep_first), int(keep_last), selected.data_ptr(),
        num_selected.data_ptr(), workspace.data_ptr(),
        workspace.nbytes, _stream(stream))
    _check(st, "pa_select_blocks")
    return selected, num_selected


def pa_attention_selected_workspace_size(num_tokens: int, num_q_heads: int,
                                         num_kv_heads: int, head_dim: int,
                                         max_selected: int) -> int:
    out = ctypes.c_size_t(0)
    st = _load().pa_attention_selected_workspace_size(
        num_tokens, num_q_heads, num_kv_heads, head_dim, max_selected,
        ctypes.byref(out))
    _check(st, "pa_attention_selected_workspace_size")
    return int(out.value)


def pa_attention_selected(q: torch.Tensor, k_cache: torch.Tensor,
                          v_cache: torch.Tensor, block_tables: torch.Tensor,
                          seq_lens: torch.Tensor, query_start_loc: torch.Tensor,
                          max_query_len: int, max_seq_len: int, scale: float,
                          selected: torch.Tensor, num_selected: torch.Tensor,
                          k_scale: float = 1.0, v_scale: float = 1.0,
                          out: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None,
                          cache_dtype: Optional[str] = None,
                          stream=None) -> torch.Tensor:
    """pa_attention over the listed blocks only: selected int32 [T, Hkv, K] in
    ascending order per row, num_selected int32 [T, Hkv]."""
    shape, lists = q.shape, selected.shape
    if len(shape) != 3 or v_cache.shape != k_cache.shape \
            or v_cache.dtype is not k_cache.dtype:
        raise ValueError("q must be [T, Hq, D] and both caches alike")
    T, Hq, D = shape
    NB, Hkv, bs, Dc = _cache_geometry(k_cache, cache_dtype)
    if Dc != D:
        raise ValueError("head_dim of q and of the caches differ")
    B, M = _step_tables(block_tables, seq_lens, query_start_loc)
    if len(lists) != 3 or lists[0] != T or lists[1] != Hkv:
        raise ValueError("selected must be [T, Hkv, K]")
    K = lists[2]
    if out is None:
        out = _new(q.shape, q.dtype, q.device, stream)
    if workspace is None:
        n = pa_attention_selected_workspace_size(T, Hq, Hkv, D, K)
        workspace = _new(max(n, 1), _U8, q.device, stream, False)
    _plain(("q", q, None, None), ("k_cache", k_cache, None, None),
           ("v_cache", v_cache, None, None),
           ("block_tables", block_tables, _I32, None),
           ("seq_lens", seq_lens, _I32, B),
           ("query_start_loc", query_start_loc, _I32, B + 1),
           ("selected", selected, _I32, None),
           ("num_selected", num_selected, _I32, T * Hkv),
           ("out", out, q.dtype, T * Hq * D), ("workspace", workspace, None, None))
    st = _load().pa_attention_selected(
        q.data_ptr(), _dtype_code(q), k_cache.data_ptr(), v_cache.data_ptr(),
        _dtype_code(k_cache, cache_dtype), NB, bs, Hq, Hkv, D,
        block_tables.data_ptr(), M, seq_lens.data_ptr(),
        query_start_loc.data_ptr(), B, T, int(max_query_len), int(max_seq_len),
        selected.data_ptr(), num_selected.data_ptr(), K, float(scale),
        float(k_scale), float(v_scale), out.data_ptr(), workspace.data_ptr(),
        workspace.nbytes, _stream(stream))
    _check(st, "pa_attention_selected")
    return out
