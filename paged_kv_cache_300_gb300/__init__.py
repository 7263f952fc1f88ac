"""Paged-attention forward for GB300: thin Python binding of libpa300.so.

Each function marshals torch tensors into the C ABI declared in
``include/pa.h`` (device pointers, sizes, the current CUDA stream) and
raises on a non-zero status.  All computation happens in the library's
CUDA kernels; there is no Python or CPU fallback: if the library is not
built, or no GPU is present, calls raise.

    pa_decode        decode step: in-place append + attention, one query per
                     sequence, through block_table
    pa_decode_contiguous  the same step over a contiguous cache (no table):
                     the twin that measures what paging costs
    pa_cache_update  scatter a packed varlen chunk into the paged pool
                     (optionally gather prefix + chunk into packed k/v)
    pa_varlen        packed variable-length attention (bf16: tcgen05)
    pa_varlen_paged  the same, reading keys through block_table from the pool
    pa_block_tables  a step's block tables, slot map, cumulative lengths and the
                     lengths for its decode, built on the GPU from the requests'
                     lengths
    pa_cache_update_q4  quantise a chunk into the 4-bit pool, by slot map
    pa_cache_gather_q4  read whole sequences of the 4-bit pool back
    pa_decode_q4     the decode step over the 4-bit pool
    pa_reset_workspaces  zero the kept workspaces after a call that gave up
    pa_rotary        queries and keys turned by their positions, on one axis or several
    pa_cache_append_rotary  the same and the append to the paged cache in one pass, with
                     the bounds of each block's keys
    pa_select_blocks  the blocks each query attends to, chosen by those bounds
    pa_sparse        attention over the selected blocks of the paged cache
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

__all__ = [
    "PAError", "library_path", "load", "pa_decode", "pa_decode_static_scratch",
    "pa_decode_contiguous", "pa_decode_contiguous_workspace_size",
    "pa_cache_update", "pa_varlen", "pa_varlen_paged",
    "pa_decode_workspace_size", "pa_status_string", "pa_version", "DEVERR_BAD_BLOCK",
    "DEVERR_OVERFLOW", "DEVERR_BAD_CU", "DEVERR_TIMEOUT", "DEVERR_NO_SPACE", "pa_block_tables",
    "pa_q4_block_bytes", "pa_q4_pool", "pa_cache_update_q4", "pa_cache_gather_q4", "pa_decode_q4",
    "pa_decode_q4_workspace_size", "PA_LEFT_OUT", "pa_reset_workspaces", "pa_rotary",
    "pa_cache_append_rotary", "pa_select_blocks", "pa_sparse",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_lib", "libpa300.so")

PA_F32, PA_BF16 = 0, 1
DEVERR_BAD_BLOCK, DEVERR_OVERFLOW, DEVERR_BAD_CU, DEVERR_TIMEOUT = 1, 2, 4, 8
DEVERR_NO_SPACE = 16
PA_LEFT_OUT = -2**31  # as a length: the sequence takes no part in the pa_decode_q4 call

_lock = threading.Lock()
_lib = None
_workspaces: dict = {}
_q4_workspaces: dict = {}


class PAError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: status {status} ({pa_status_string(status)})")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load libpa300.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build the CUDA library first "
                "(python -m paged_kv_cache_300_gb300._build)")
        lib = ctypes.CDLL(_LIB_PATH)
        p, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.pa_decode_workspace_size.argtypes = [i] * 5 + [i]
        lib.pa_decode_workspace_size.restype = sz
        lib.pa_decode.argtypes = [p] * 8 + [i] * 7 + [i, f, p, sz, p, p]
        lib.pa_decode.restype = i
        lib.pa_decode_static_scratch.argtypes = [p] * 8 + [i] * 7 + [f, p, p]
        lib.pa_decode_static_scratch.restype = i
        lib.pa_decode_contiguous_workspace_size.argtypes = [i] * 4
        lib.pa_decode_contiguous_workspace_size.restype = sz
        lib.pa_decode_contiguous.argtypes = [p] * 7 + [i] * 5 + [f, p, sz, p, p]
        lib.pa_decode_contiguous.restype = i
        lib.pa_cache_update.argtypes = [p] * 10 + [i] * 8 + [i, p, p]
        lib.pa_cache_update.restype = i
        lib.pa_varlen.argtypes = [p] * 5 + [i] * 3 + [p] + [i] * 6 + [i, f, p, p]
        lib.pa_varlen.restype = i
        lib.pa_varlen_paged.argtypes = [p] * 6 + [i] * 3 + [p] + [i] * 8 + [i, f, p, p]
        lib.pa_varlen_paged.restype = i
        lib.pa_q4_block_bytes.argtypes = [i] * 3
        lib.pa_q4_block_bytes.restype = sz
        lib.pa_cache_update_q4.argtypes = [p] * 4 + [i] * 6 + [p, p]
        lib.pa_cache_update_q4.restype = i
        lib.pa_cache_gather_q4.argtypes = [p] * 5 + [i] * 8 + [p, p]
        lib.pa_cache_gather_q4.restype = i
        lib.pa_decode_q4_workspace_size.argtypes = [i] * 6
        lib.pa_decode_q4_workspace_size.restype = sz
        lib.pa_decode_q4.argtypes = [p] * 9 + [i] * 8 + [f, p, sz, p, p]
        lib.pa_decode_q4.restype = i
        lib.pa_block_tables.argtypes = [p] * 10 + [i] * 5 + [p, p]
        lib.pa_block_tables.restype = i
        lib.pa_block_tables_decode.argtypes = [p] * 11 + [i] * 5 + [p, p]
        lib.pa_block_tables_decode.restype = i
        n = ctypes.c_longlong
        lib.pa_rotary.argtypes = [p] * 6 + [i] * 7 + [p, i] + [n] * 4 + [i, p, p]
        lib.pa_rotary.restype = i
        lib.pa_cache_append_rotary.argtypes = [p] * 10 + [i] * 7 + [p, i] + [n] * 4 + [i] * 3 + [p, p]
        lib.pa_cache_append_rotary.restype = i
        lib.pa_select_blocks.argtypes = [p] * 6 + [i] * 12 + [p, p]
        lib.pa_select_blocks.restype = i
        lib.pa_sparse.argtypes = [p] * 8 + [i] * 10 + [f, p, p]
        lib.pa_sparse.restype = i
        lib.pa_status_string.argtypes = [i]
        lib.pa_status_string.restype = ctypes.c_char_p
        lib.pa_version.argtypes = []
        lib.pa_version.restype = i
        _lib = lib
        return lib


def pa_status_string(status: int) -> str:
    return load().pa_status_string(int(status)).decode()


def pa_version() -> int:
    return int(load().pa_version())


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return PA_BF16
    if t.dtype == torch.float32:
        return PA_F32
    raise TypeError(f"element tensors must be bfloat16 or float32, got {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check_dev(*ts):
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("all tensors must live on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("all tensors must be on the same device")
    return dev


def _check_host_or_dev(dev, *ts):
    """Per-step tensors of pa_decode: on `dev`, or page-locked host memory
    (which the kernel reads and writes in place over NVLink-C2C)."""
    for t in ts:
        if t is None:
            continue
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
        if t.is_cuda:
            if t.device != dev:
                raise ValueError("all tensors must be on the same device")
        elif not t.is_pinned():
            raise ValueError("host tensors must be page-locked (pin_memory())")


def _i32(t, name):
    if t is not None and t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _call(name, rc):
    if rc != 0:
        raise PAError(name, rc)


def pa_decode_workspace_size(batch, num_heads, num_kv_heads, head_dim, block_size,
                             dtype=torch.bfloat16) -> int:
    dt = PA_BF16 if dtype == torch.bfloat16 else PA_F32
    return int(load().pa_decode_workspace_size(batch, num_heads, num_kv_heads, head_dim,
                                               block_size, dt))


def _workspace(dev, nbytes):
    if nbytes == 0:
        return None
    key = (dev.index, torch.cuda.current_stream(dev).cuda_stream)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)  # zero on first use
        _workspaces[key] = ws
    return ws


def pa_reset_workspaces():
    """Zero the workspaces kept for calls of pa_decode, pa_decode_contiguous and
    pa_decode_q4 that were given none (in place: captured calls may use them).
    Needed after such a call has set DEVERR_TIMEOUT: counters of the sequences
    that were given up may be left in its workspace, and later calls would join
    those sequences' parts too early or not at all.  Call it when no such call
    is running; it waits for the GPU.  (A caller's own workspace is zeroed by the
    caller; a captured pa_decode_q4 clears its counters in the graph.)"""
    for kept in (_workspaces, _q4_workspaces):
        for ws in list(kept.values()):
            ws.zero_()
            if ws.is_cuda:
                torch.cuda.synchronize(ws.device)


def pa_decode(q, k_cache, v_cache, block_table, cache_seqlens, k_new, v_new, out=None,
              softmax_scale: float = 0.0, workspace=None, dev_err=None, stream=None):
    """Decode step (see include/pa.h).  q [B, Hq, D]; k_cache/v_cache
    [NB, bs, Hkv, D] (the new token is written in place); block_table
    [B, MB] int32; cache_seqlens [B] int32; k_new/v_new [B, Hkv, D].
    Returns out [B, Hq, D].  q, block_table, cache_seqlens, k_new, v_new
    and out may be pinned host tensors (read and written in place; `out`
    defaults to a pinned host tensor then); the pools, workspace and
    dev_err live on the GPU.  Without a workspace the call uses one that is
    kept for the device and stream; after DEVERR_TIMEOUT it has to be zeroed
    with pa_reset_workspaces()."""
    dev = _check_dev(k_cache, v_cache, workspace, dev_err)
    _check_host_or_dev(dev, q, block_table, cache_seqlens, k_new, v_new, out)
    _i32(block_table, "block_table")
    _i32(cache_seqlens, "cache_seqlens")
    _i32(dev_err, "dev_err")
    dt = _dtype(q)
    for t in (k_cache, v_cache, k_new, v_new):
        if t.dtype != q.dtype:
            raise TypeError("q, k_cache, v_cache, k_new, v_new must share a dtype")
    b, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    if d2 != d or v_cache.shape != k_cache.shape or k_new.shape != (b, hkv, d) or \
            v_new.shape != (b, hkv, d) or block_table.shape[0] != b or cache_seqlens.shape != (b,):
        raise ValueError("inconsistent shapes")
    mb = block_table.shape[1]
    if out is None:
        out = torch.empty_like(q, pin_memory=not q.is_cuda)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must match q")
    lib = load()
    if workspace is None:
        workspace = _workspace(dev, int(lib.pa_decode_workspace_size(b, hq, hkv, d, bs, dt)))
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.pa_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                       _ptr(cache_seqlens), _ptr(k_new), _ptr(v_new), _ptr(out), b, hq, hkv, d,
                       nb, bs, mb, dt, float(softmax_scale), _ptr(workspace), wbytes,
                       _ptr(dev_err), _stream(stream))
    _call("pa_decode", rc)
    return out


def pa_decode_static_scratch(q, k_cache, v_cache, block_table, cache_seqlens, k_new, v_new,
                             out=None, softmax_scale: float = 0.0, dev_err=None, stream=None):
    """pa_decode (bf16) with the library's built-in 16 MiB scratch instead
    of a workspace: for callers that cannot allocate device memory at call
    time.  Calls that may overlap on the GPU must be serialised."""
    _check_dev(q, k_cache, v_cache, block_table, cache_seqlens, k_new, v_new, out, dev_err)
    _i32(block_table, "block_table")
    _i32(cache_seqlens, "cache_seqlens")
    _i32(dev_err, "dev_err")
    if q.dtype != torch.bfloat16:
        raise TypeError("pa_decode_static_scratch takes bfloat16 tensors")
    b, hq, d = q.shape
    nb, bs, hkv, _ = k_cache.shape
    if out is None:
        out = torch.empty_like(q)
    rc = load().pa_decode_static_scratch(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                         _ptr(cache_seqlens), _ptr(k_new), _ptr(v_new), _ptr(out),
                                         b, hq, hkv, d, nb, bs, block_table.shape[1],
                                         float(softmax_scale), _ptr(dev_err), _stream(stream))
    _call("pa_decode_static_scratch", rc)
    return out


def pa_decode_contiguous_workspace_size(batch, num_heads, num_kv_heads, head_dim) -> int:
    return int(load().pa_decode_contiguous_workspace_size(batch, num_heads, num_kv_heads,
                                                          head_dim))


def pa_decode_contiguous(q, k_cache, v_cache, cache_seqlens, k_new, v_new, out=None,
                         softmax_scale: float = 0.0, workspace=None, dev_err=None, stream=None):
    """Decode step over a contiguous cache (see include/pa.h): q [B, Hq, D];
    k_cache/v_cache [B, max_seqlen, Hkv, D] (the new token is written in
    place at [b, cache_seqlens[b]]); k_new/v_new [B, Hkv, D].  bf16 only.
    Returns out [B, Hq, D]."""
    dev = _check_dev(q, k_cache, v_cache, cache_seqlens, k_new, v_new, out, workspace, dev_err)
    _i32(cache_seqlens, "cache_seqlens")
    _i32(dev_err, "dev_err")
    if q.dtype != torch.bfloat16:
        raise TypeError("pa_decode_contiguous takes bfloat16 tensors")
    for t in (k_cache, v_cache, k_new, v_new):
        if t.dtype != q.dtype:
            raise TypeError("q, k_cache, v_cache, k_new, v_new must share a dtype")
    b, hq, d = q.shape
    b2, lmax, hkv, d2 = k_cache.shape
    if b2 != b or d2 != d or v_cache.shape != k_cache.shape or k_new.shape != (b, hkv, d) or \
            v_new.shape != (b, hkv, d) or cache_seqlens.shape != (b,):
        raise ValueError("inconsistent shapes")
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must match q")
    lib = load()
    if workspace is None:
        workspace = _workspace(dev, int(lib.pa_decode_contiguous_workspace_size(b, hq, hkv, d)))
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.pa_decode_contiguous(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cache_seqlens),
                                  _ptr(k_new), _ptr(v_new), _ptr(out), b, hq, hkv, d, lmax,
                                  float(softmax_scale), _ptr(workspace), wbytes, _ptr(dev_err),
                                  _stream(stream))
    _call("pa_decode_contiguous", rc)
    return out


def pa_cache_update(k_chunk, v_chunk, cu_seq_lens_q, cache_seqlens, block_table, k_cache,
                    v_cache, k_full=None, v_full=None, cu_seq_lens_k=None, dev_err=None,
                    stream=None):
    """Scatter the packed chunk [Tq, Hkv, D] into the pool at positions
    cache_seqlens[b] + i; with k_full/v_full/cu_seq_lens_k also gather each
    request's prefix + chunk into the packed [Tk, Hkv, D] tensors."""
    _check_dev(k_chunk, v_chunk, cu_seq_lens_q, cache_seqlens, block_table, k_cache, v_cache,
               k_full, v_full, cu_seq_lens_k, dev_err)
    for t, n in ((cu_seq_lens_q, "cu_seq_lens_q"), (cache_seqlens, "cache_seqlens"),
                 (block_table, "block_table"), (cu_seq_lens_k, "cu_seq_lens_k"),
                 (dev_err, "dev_err")):
        _i32(t, n)
    dt = _dtype(k_cache)
    nb, bs, hkv, d = k_cache.shape
    b = cache_seqlens.shape[0]
    tq = k_chunk.shape[0]
    tk = 0 if k_full is None else k_full.shape[0]
    rc = load().pa_cache_update(_ptr(k_chunk), _ptr(v_chunk), _ptr(cu_seq_lens_q),
                                _ptr(cache_seqlens), _ptr(block_table), _ptr(k_cache),
                                _ptr(v_cache), _ptr(k_full), _ptr(v_full), _ptr(cu_seq_lens_k),
                                b, tq, tk, hkv, d, nb, bs, block_table.shape[1], dt,
                                _ptr(dev_err), _stream(stream))
    _call("pa_cache_update", rc)
    return k_full, v_full


def pa_varlen(q, k, v, cu_seq_lens_q, cu_seq_lens_k, max_length_q: int, max_length_k: int,
              causal: bool, out=None, softmax_scale: float = 0.0, dev_err=None, stream=None):
    """Varlen attention: q [Tq, Hq, D], k/v [Tk, Hkv, D] -> out [Tq, Hq, D]."""
    _check_dev(q, k, v, cu_seq_lens_q, cu_seq_lens_k, out, dev_err)
    _i32(cu_seq_lens_q, "cu_seq_lens_q")
    _i32(cu_seq_lens_k, "cu_seq_lens_k")
    dt = _dtype(q)
    tq, hq, d = q.shape
    tk, hkv, _ = k.shape
    if out is None:
        out = torch.empty_like(q)
    rc = load().pa_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seq_lens_q), _ptr(cu_seq_lens_k),
                          int(max_length_q), int(max_length_k), int(bool(causal)), _ptr(out),
                          cu_seq_lens_q.shape[0] - 1, tq, tk, hq, hkv, d, dt,
                          float(softmax_scale), _ptr(dev_err), _stream(stream))
    _call("pa_varlen", rc)
    return out


def pa_varlen_paged(q, k_cache, v_cache, block_table, cu_seq_lens_q, seqlens_k,
                    max_length_q: int, max_length_k: int, causal: bool, out=None,
                    softmax_scale: float = 0.0, dev_err=None, stream=None):
    """Varlen attention with keys read through block_table: q [Tq, Hq, D];
    k_cache/v_cache [NB, bs, Hkv, D]; block_table [B, MB]; seqlens_k [B]
    (keys of each request in the pool).  Returns out [Tq, Hq, D]."""
    _check_dev(q, k_cache, v_cache, block_table, cu_seq_lens_q, seqlens_k, out, dev_err)
    for t, n in ((block_table, "block_table"), (cu_seq_lens_q, "cu_seq_lens_q"),
                 (seqlens_k, "seqlens_k"), (dev_err, "dev_err")):
        _i32(t, n)
    dt = _dtype(q)
    tq, hq, d = q.shape
    nb, bs, hkv, _ = k_cache.shape
    if out is None:
        out = torch.empty_like(q)
    rc = load().pa_varlen_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                _ptr(cu_seq_lens_q), _ptr(seqlens_k), int(max_length_q),
                                int(max_length_k), int(bool(causal)), _ptr(out),
                                cu_seq_lens_q.shape[0] - 1, tq, hq, hkv, d, nb, bs,
                                block_table.shape[1], dt, float(softmax_scale), _ptr(dev_err),
                                _stream(stream))
    _call("pa_varlen_paged", rc)
    return out


# ------------------------------------------------------------------ 4-bit pool
# A step of a small model is a few microseconds on the GPU, so the checks below
# touch each tensor as few times as they can.  They pass or fail as a whole;
# _refuse then says which tensor it was.
def _fits(index, dtype, *ts):
    """Every tensor given is of `dtype`, contiguous and on device `index`."""
    for t in ts:
        if t is not None and (t.dtype is not dtype or t.get_device() != index
                              or not t.is_contiguous()):
            return False
    return True


def _refuse(index, dtype, **ts):
    for name, t in ts.items():
        if t is None:
            continue
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}")
        if t.get_device() != index:
            raise ValueError("all tensors must be on the same CUDA device")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    raise ValueError("inconsistent shapes")


def _q4_geometry(kv_cache, num_kv_heads, head_dim):
    """(device index, number of blocks, block size) of a 4-bit pool
    [num_blocks, num_kv_heads, block_size * (head_dim + 8)]."""
    if not kv_cache.is_cuda:
        raise ValueError("all tensors must live on a CUDA device")
    if kv_cache.dtype is not torch.uint8 or kv_cache.dim() != 3 or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be a contiguous uint8 tensor "
                         "[num_blocks, num_kv_heads, block_size * (head_dim + 8)]")
    nb, h, record = kv_cache.shape
    if h != num_kv_heads or record % (head_dim + 8) != 0:
        raise ValueError("kv_cache does not fit the number of kv heads or the head_dim")
    return kv_cache.get_device(), nb, record // (head_dim + 8)


# The current stream's handle; torch.cuda.current_stream() makes an object for
# it first, which takes longer (3 us) than the launch.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(name, index, stream, *args):
    """Call the library with the tensors' device current, on `stream` (default:
    that device's current stream)."""
    fn = getattr(_lib or load(), name)
    handle = _current_raw_stream(index) if stream is None else stream.cuda_stream
    if _current_device() == index:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, handle)
    if rc != 0:
        raise PAError(name, rc)


def _addr(t):
    return None if t is None else t.data_ptr()


def _empty(stream, shape, dtype, device):
    """An output the caller gave no tensor for, in memory of the stream that
    writes it: memory that the current stream has given back may still be in use
    there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _too_large():
    raise ValueError("a size passes 2^31 - 1")  # ctypes would cut it to 32 bits


def pa_q4_block_bytes(num_kv_heads, head_dim, block_size) -> int:
    """Bytes of one block of the 4-bit pool; 0 for sizes it does not have."""
    return int(load().pa_q4_block_bytes(num_kv_heads, head_dim, block_size))


def pa_q4_pool(num_blocks, num_kv_heads, head_dim, block_size, device="cuda"):
    """A zeroed 4-bit pool: uint8 [num_blocks, num_kv_heads,
    block_size * (head_dim + 8)] (layout in include/pa.h)."""
    nbytes = pa_q4_block_bytes(num_kv_heads, head_dim, block_size)
    if nbytes == 0:
        raise ValueError("the 4-bit pool has head_dim 64 or 128 and block_size 16 or 32")
    return torch.zeros(num_blocks, num_kv_heads, nbytes // num_kv_heads, dtype=torch.uint8,
                       device=device)


def pa_cache_update_q4(k_chunk, v_chunk, slot_map, kv_cache, dev_err=None, stream=None):
    """Quantise the rows of k_chunk, v_chunk [T, Hkv, D] (bfloat16 or float32)
    into the slots slot_map [T] int32 of the 4-bit pool; a negative slot skips
    its row."""
    shape = k_chunk.shape
    t, hkv, d = shape
    if t > 0x7FFFFFFF:
        _too_large()
    dt = _dtype(k_chunk)
    index, nb, bs = _q4_geometry(kv_cache, hkv, d)
    if v_chunk.shape != shape or not _fits(index, k_chunk.dtype, k_chunk, v_chunk):
        _refuse(index, k_chunk.dtype, k_chunk=k_chunk, v_chunk=v_chunk)
    if slot_map.shape != (t,) or not _fits(index, torch.int32, slot_map, dev_err):
        _refuse(index, torch.int32, slot_map=slot_map, dev_err=dev_err)
    _launch("pa_cache_update_q4", index, stream, k_chunk.data_ptr(), v_chunk.data_ptr(),
            slot_map.data_ptr(), kv_cache.data_ptr(), t, hkv, d, nb, bs, dt, _addr(dev_err))


def pa_cache_gather_q4(kv_cache, block_table, cu_seq_lens_k, k_full, v_full, dev_err=None,
                       stream=None):
    """Read positions 0.. of every request back from the 4-bit pool into the
    packed k_full, v_full [Tk, Hkv, D] (bfloat16 or float32), request r's rows
    being [cu_seq_lens_k[r], cu_seq_lens_k[r+1]).  Returns (k_full, v_full)."""
    shape = k_full.shape
    tk, hkv, d = shape
    dt = _dtype(k_full)
    index, nb, bs = _q4_geometry(kv_cache, hkv, d)
    b, mb = block_table.shape
    if tk | b | mb > 0x7FFFFFFF:
        _too_large()
    if v_full.shape != shape or not _fits(index, k_full.dtype, k_full, v_full):
        _refuse(index, k_full.dtype, k_full=k_full, v_full=v_full)
    if cu_seq_lens_k.shape != (b + 1,) or \
            not _fits(index, torch.int32, block_table, cu_seq_lens_k, dev_err):
        _refuse(index, torch.int32, block_table=block_table, cu_seq_lens_k=cu_seq_lens_k,
                dev_err=dev_err)
    _launch("pa_cache_gather_q4", index, stream, kv_cache.data_ptr(), block_table.data_ptr(),
            cu_seq_lens_k.data_ptr(), k_full.data_ptr(), v_full.data_ptr(), b, tk, hkv, d, nb, bs,
            mb, dt, _addr(dev_err))
    return k_full, v_full


def pa_decode_q4_workspace_size(batch, num_heads, num_kv_heads, head_dim, block_size,
                                dtype=torch.bfloat16) -> int:
    """Bytes of workspace pa_decode_q4 needs on the current device."""
    dt = PA_BF16 if dtype == torch.bfloat16 else PA_F32
    return int(load().pa_decode_q4_workspace_size(batch, num_heads, num_kv_heads, head_dim,
                                                  block_size, dt))


_q4_sizes: dict = {}


def _q4_workspace(index, stream, sizes):
    """Workspace of a pa_decode_q4 call that was given none.  Eager calls
    share one per (device, stream), zeroed when it is made.  A call that is
    being captured gets its own from the graph's memory, with its counters
    (one int32 per sequence and kv head, at its start) cleared inside the
    graph: two graphs may replay at the same time."""
    key = (index,) + sizes
    nbytes = _q4_sizes.get(key)
    if nbytes is None:
        with torch.cuda.device(index):
            nbytes = int(load().pa_decode_q4_workspace_size(*sizes))
        _q4_sizes[key] = nbytes
    if nbytes == 0:
        return None  # sizes the call refuses, or an empty batch
    if stream is None and torch.cuda.current_device() == index:
        return _q4_stream_workspace(index, nbytes, 4 * sizes[0] * sizes[2])
    with torch.cuda.device(index), torch.cuda.stream(stream):  # None: the device's current stream
        return _q4_stream_workspace(index, nbytes, 4 * sizes[0] * sizes[2])


def _q4_stream_workspace(index, nbytes, counter_bytes):
    """_q4_workspace on the current stream of device `index`, the current one."""
    if torch.cuda.is_current_stream_capturing():
        ws = torch.empty(nbytes, dtype=torch.uint8, device=f"cuda:{index}")
        ws[:counter_bytes].zero_()
        return ws
    handle = _current_raw_stream(index)
    ws = _q4_workspaces.get((index, handle))
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=f"cuda:{index}")
        _q4_workspaces[(index, handle)] = ws
    return ws


def pa_decode_q4(q, kv_cache, block_table, cache_seqlens, k_new, v_new, out=None,
                 softmax_scale: float = 0.0, k_stored=None, v_stored=None, workspace=None,
                 dev_err=None, stream=None):
    """Decode step over the 4-bit pool (see include/pa.h): k_new, v_new
    [B, Hkv, D] are quantised in place at position cache_seqlens[b] and
    q [B, Hq, D] attends over positions 0..cache_seqlens[b].  bfloat16 or
    float32.  A sequence whose length is PA_LEFT_OUT takes no part (its rows of
    out are zeros).  k_stored, v_stored, when given, receive the new token as the
    pool now holds it.  Without a workspace the call uses one that is kept for
    the device and stream; after DEVERR_TIMEOUT it has to be zeroed with
    pa_reset_workspaces().  Returns out [B, Hq, D]."""
    shape, rows = q.shape, k_new.shape
    b, hq, d = shape
    hkv = rows[1]
    dtype = q.dtype
    dt = _dtype(q)
    index, nb, bs = _q4_geometry(kv_cache, hkv, d)
    if out is None:
        out = _empty(stream, shape, dtype, q.device)
    if out.shape != shape or rows != (b, hkv, d) or v_new.shape != rows or \
            (k_stored is not None and k_stored.shape != rows) or \
            (v_stored is not None and v_stored.shape != rows):
        raise ValueError("inconsistent shapes")
    if not _fits(index, dtype, q, out, k_new, v_new, k_stored, v_stored):
        _refuse(index, dtype, q=q, out=out, k_new=k_new, v_new=v_new, k_stored=k_stored,
                v_stored=v_stored)
    tb, mb = block_table.shape
    if b | mb > 0x7FFFFFFF:
        _too_large()
    if tb != b or cache_seqlens.shape != (b,) or \
            not _fits(index, torch.int32, block_table, cache_seqlens, dev_err):
        _refuse(index, torch.int32, block_table=block_table, cache_seqlens=cache_seqlens,
                dev_err=dev_err)
    if workspace is None:
        workspace = _q4_workspace(index, stream, (b, hq, hkv, d, bs, dt))
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the same device")
    wptr, wbytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    _launch("pa_decode_q4", index, stream, q.data_ptr(), kv_cache.data_ptr(),
            block_table.data_ptr(), cache_seqlens.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
            out.data_ptr(), _addr(k_stored), _addr(v_stored), b, hq, hkv, d, nb, bs, mb, dt,
            softmax_scale, wptr, wbytes, _addr(dev_err))
    return out


# ------------------------------------------------------------------ block tables
def pa_block_tables(cache_seqlens, new_lens, block_table, free_blocks, num_free, slot_map,
                    block_size, cu_seq_lens_q=None, cu_seq_lens_k=None, seqlens_k=None,
                    num_free_out=None, dev_err=None, stream=None, decode_lens=None):
    """One step's block tables from the requests' lengths (see include/pa.h).
    cache_seqlens, new_lens [B]; block_table [B, MB] and free_blocks
    [num_blocks] are updated in place; slot_map [any length] is filled, -1
    behind the last token.  All int32.  num_free [1] is advanced in place
    unless num_free_out is given.  decode_lens [B], when given, receives the
    lengths for a pa_decode_q4 call over the whole batch: those before the step
    where one token is new, PA_LEFT_OUT elsewhere.  Returns (cu_seq_lens_q, cu_seq_lens_k,
    seqlens_k)."""
    if not block_table.is_cuda:
        raise ValueError("all tensors must live on a CUDA device")
    b, mb = block_table.shape
    index = block_table.get_device()
    if cu_seq_lens_q is None:
        cu_seq_lens_q = _empty(stream, b + 1, torch.int32, block_table.device)
    if cu_seq_lens_k is None:
        cu_seq_lens_k = _empty(stream, b + 1, torch.int32, block_table.device)
    if seqlens_k is None:
        seqlens_k = _empty(stream, b, torch.int32, block_table.device)
    if num_free_out is None:
        num_free_out = num_free
    if not _fits(index, torch.int32, cache_seqlens, new_lens, block_table, free_blocks, num_free,
                 slot_map, cu_seq_lens_q, cu_seq_lens_k, seqlens_k, num_free_out, decode_lens,
                 dev_err):
        _refuse(index, torch.int32, cache_seqlens=cache_seqlens, new_lens=new_lens,
                block_table=block_table, free_blocks=free_blocks, num_free=num_free,
                slot_map=slot_map, cu_seq_lens_q=cu_seq_lens_q, cu_seq_lens_k=cu_seq_lens_k,
                seqlens_k=seqlens_k, num_free_out=num_free_out, decode_lens=decode_lens,
                dev_err=dev_err)
    if cache_seqlens.shape != (b,) or new_lens.shape != (b,) or seqlens_k.shape != (b,) or \
            cu_seq_lens_q.shape != (b + 1,) or cu_seq_lens_k.shape != (b + 1,) or \
            free_blocks.dim() != 1 or slot_map.dim() != 1 or num_free.numel() != 1 or \
            num_free_out.numel() != 1 or (decode_lens is not None and decode_lens.shape != (b,)):
        raise ValueError("inconsistent shapes")
    slots, blocks = slot_map.numel(), free_blocks.numel()
    if b | slots | blocks | mb | block_size > 0x7FFFFFFF:
        _too_large()
    _launch("pa_block_tables_decode", index, stream, cache_seqlens.data_ptr(), new_lens.data_ptr(),
            block_table.data_ptr(), free_blocks.data_ptr(), num_free.data_ptr(),
            slot_map.data_ptr(), cu_seq_lens_q.data_ptr(), cu_seq_lens_k.data_ptr(),
            seqlens_k.data_ptr(), num_free_out.data_ptr(), _addr(decode_lens), b, slots, blocks,
            block_size, mb, _addr(dev_err))
    return cu_seq_lens_q, cu_seq_lens_k, seqlens_k


# ------------------------------------------------------------------ rotary positions
@functools.lru_cache(maxsize=64)
def _pair_axes(axes):
    """The host array of a tuple of axes, one of each pair."""
    if not axes or min(axes) < 0 or max(axes) > 255:
        raise ValueError("pair_axis holds an axis from 0 for each pair")
    return (ctypes.c_uint8 * len(axes))(*axes)


_DTYPES = {torch.bfloat16: PA_BF16, torch.float32: PA_F32}


def _token_rows(index, dtype, name, t, tokens, head_dim):
    """(heads, address, elements from token to token) of rows [T, H, D] whose
    tokens may stand apart (a part of a projection's output); (0, None, 0) for None."""
    if t is None:
        return 0, None, 0
    n, heads, d = t.shape
    if n == tokens and d == head_dim and t.dtype is dtype and t.get_device() == index:
        if t.is_contiguous():
            return heads, t.data_ptr(), heads * d
        step, row, one = t.stride()
        if one == 1 and (row == d or heads <= 1):
            return heads, t.data_ptr(), step
        raise ValueError(f"{name}: the rows of a token must be dense")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.get_device() != index:
        raise ValueError("all tensors must be on the same CUDA device")
    raise ValueError("inconsistent shapes")


def _rotary_table(index, positions, cos_sin, pair_axis, tokens):
    """(positions, cos_sin, rotary_dim, rows of the table, axes, host array of the
    pairs' axes), checked."""
    if positions is None or cos_sin is None:
        raise ValueError("positions and cos_sin are needed")
    rows, rot = cos_sin.shape
    shape = positions.shape
    if len(shape) == 1:
        axes, n = 1, shape[0]
    else:
        axes, n = shape
    if n != tokens or positions.dtype is not torch.int32 or positions.get_device() != index or \
            not positions.is_contiguous():
        _refuse(index, torch.int32, positions=positions)
    if cos_sin.dtype is not torch.float32 or cos_sin.get_device() != index or \
            not cos_sin.is_contiguous():
        _refuse(index, torch.float32, cos_sin=cos_sin)
    if rows | axes > 0x7FFFFFFF:
        _too_large()
    host = None
    if pair_axis is not None:
        host = _pair_axes(tuple(pair_axis))
        if len(host) != rot // 2:
            raise ValueError("pair_axis must have an axis for each of the rotary_dim / 2 pairs")
    return positions.data_ptr(), cos_sin.data_ptr(), rot, rows, axes, host


def pa_rotary(q, k, positions, cos_sin, q_out=None, k_out=None, interleaved: bool = False,
              pair_axis=None, dev_err=None, stream=None):
    """Turn queries q [T, Hq, D] and keys k [T, Hkv, D] (one of them may be None) by
    their positions (see include/pa.h).  bfloat16 or float32; the tokens of a tensor
    may stand apart (slices of one projection's output).  positions [T], or
    [axes, T] with pair_axis, a sequence of the axis of each pair; cos_sin float32
    [max_position, rotary_dim], cosines in the first half of a row.  interleaved: pairs
    are neighbouring dims instead of split halves.  q_out, k_out may be q, k
    themselves.  Returns (q_out, k_out)."""
    some = k if q is None else q
    if some is None:
        raise ValueError("q or k is needed")
    tokens, _, d = some.shape
    index, dtype = some.get_device(), some.dtype
    if index < 0:
        raise ValueError("all tensors must live on a CUDA device")
    if _current_device() != index:
        with torch.cuda.device(index):
            return pa_rotary(q, k, positions, cos_sin, q_out, k_out, interleaved, pair_axis, dev_err,
                             stream)
    dt = _DTYPES.get(dtype)
    if dt is None:
        dt = _dtype(some)
    if tokens > 0x7FFFFFFF:
        _too_large()
    if q_out is None and q is not None:
        q_out = _empty(stream, q.shape, dtype, q.device)
    if k_out is None and k is not None:
        k_out = _empty(stream, k.shape, dtype, k.device)
    hq, qp, qs = _token_rows(index, dtype, "q", q, tokens, d)
    hk, kp, ks = _token_rows(index, dtype, "k", k, tokens, d)
    ho, qo, qos = _token_rows(index, dtype, "q_out", q_out, tokens, d)
    hko, ko, kos = _token_rows(index, dtype, "k_out", k_out, tokens, d)
    if ho != hq or hko != hk:
        raise ValueError("inconsistent shapes")
    pos, table, rot, rows, axes, host = _rotary_table(index, positions, cos_sin, pair_axis, tokens)
    if dev_err is not None and not _fits(index, torch.int32, dev_err):
        _refuse(index, torch.int32, dev_err=dev_err)
    rc = (_lib or load()).pa_rotary(
        qp, kp, pos, table, qo, ko, tokens, hq, hk, d, rot, rows, axes, host, interleaved, qs, ks, qos,
        kos, dt, None if dev_err is None else dev_err.data_ptr(),
        _current_raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        raise PAError("pa_rotary", rc)
    return q_out, k_out


def pa_cache_append_rotary(q, k, v, slot_map, k_cache, v_cache, positions=None, cos_sin=None,
                           q_out=None, bounds=None, interleaved: bool = False, pair_axis=None,
                           dev_err=None, stream=None):
    """Turn a step's q [T, Hq, D] (or None) and k [T, Hkv, D] by their positions and put
    k, v into the slots slot_map [T] of k_cache, v_cache [NB, bs, Hkv, D] (see
    include/pa.h); a negative slot skips its row.  positions, cos_sin, interleaved and
    pair_axis as pa_rotary; without them k is put as it is.  bounds [NB, Hkv, 2, D], when
    given, keeps the least and the largest key of each block for pa_select_blocks.
    Returns q_out."""
    shape = k_cache.shape
    nb, bs, hkv, d = shape
    index, dtype, tokens = k_cache.get_device(), k_cache.dtype, k.shape[0]
    if index < 0:
        raise ValueError("all tensors must live on a CUDA device")
    if _current_device() != index:
        with torch.cuda.device(index):
            return pa_cache_append_rotary(q, k, v, slot_map, k_cache, v_cache, positions, cos_sin, q_out,
                                          bounds, interleaved, pair_axis, dev_err, stream)
    dt = _DTYPES.get(dtype)
    if dt is None:
        dt = _dtype(k_cache)
    if tokens | nb | bs > 0x7FFFFFFF:
        _too_large()
    if v_cache.shape != shape or (bounds is not None and bounds.shape != (nb, hkv, 2, d)) or \
            not _fits(index, dtype, k_cache, v_cache, bounds):
        _refuse(index, dtype, k_cache=k_cache, v_cache=v_cache, bounds=bounds)
    if slot_map.shape != (tokens,) or not _fits(index, torch.int32, slot_map, dev_err):
        _refuse(index, torch.int32, slot_map=slot_map, dev_err=dev_err)
    if q_out is None and q is not None:
        q_out = _empty(stream, q.shape, dtype, q.device)
    hq, qp, qs = _token_rows(index, dtype, "q", q, tokens, d)
    hk, kp, ks = _token_rows(index, dtype, "k", k, tokens, d)
    hv, vp, vs = _token_rows(index, dtype, "v", v, tokens, d)
    ho, qo, qos = _token_rows(index, dtype, "q_out", q_out, tokens, d)
    if hk != hkv or hv != hkv or ho != hq:
        raise ValueError("inconsistent shapes")
    if positions is None and cos_sin is None:
        if pair_axis is not None or interleaved:
            raise ValueError("pairs to turn need positions and cos_sin")
        pos = table = host = None
        rot = rows = axes = 0
    else:
        pos, table, rot, rows, axes, host = _rotary_table(index, positions, cos_sin, pair_axis, tokens)
    rc = (_lib or load()).pa_cache_append_rotary(
        qp, kp, vp, slot_map.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        None if bounds is None else bounds.data_ptr(), pos, table, qo, tokens, hq, hkv, d, rot, rows, axes,
        host, interleaved, qs, ks, vs, qos, nb, bs, dt, None if dev_err is None else dev_err.data_ptr(),
        _current_raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        raise PAError("pa_cache_append_rotary", rc)
    return q_out


# ------------------------------------------------------------------ block-sparse attention
def _query_rows(index, tokens, block_table, seqlens_k, cu_seq_lens_q, dev_err, selected):
    """Checks of the index tensors that both calls take; (batch, table's width)."""
    b, mb = block_table.shape
    if b | mb | tokens > 0x7FFFFFFF:
        _too_large()
    if seqlens_k.shape != (b,) or \
            (tokens != b if cu_seq_lens_q is None else cu_seq_lens_q.shape != (b + 1,)) or \
            not _fits(index, torch.int32, block_table, seqlens_k, cu_seq_lens_q, dev_err, selected):
        _refuse(index, torch.int32, block_table=block_table, seqlens_k=seqlens_k,
                cu_seq_lens_q=cu_seq_lens_q, dev_err=dev_err, selected=selected)
    return b, mb


def pa_select_blocks(q, bounds, block_table, seqlens_k, top_k: int, block_size: int,
                     first_blocks: int = 1, last_blocks: int = 1, cu_seq_lens_q=None, selected=None,
                     dev_err=None, stream=None):
    """The blocks each query and kv head attends to (see include/pa.h): q [Tq, Hq, D]
    (turned already), bounds [NB, Hkv, 2, D] of the blocks' keys, block_table [B, MB],
    seqlens_k [B] with the new tokens; cu_seq_lens_q [B + 1] locates the requests'
    queries (None: one of each).  Returns selected [Tq, Hkv, top_k] int32: logical blocks,
    ascending, the first first_blocks and last last_blocks visible ones always among
    them, -1 behind the last.  A table no wider than the longest request is fastest."""
    tq, hq, d = q.shape
    index, dtype = q.get_device(), q.dtype
    if index < 0:
        raise ValueError("all tensors must live on a CUDA device")
    dt = _DTYPES.get(dtype)
    if dt is None:
        dt = _dtype(q)
    if _current_device() != index:
        with torch.cuda.device(index):
            return pa_select_blocks(q, bounds, block_table, seqlens_k, top_k, block_size, first_blocks,
                                    last_blocks, cu_seq_lens_q, selected, dev_err, stream)
    nb, hkv, two, d2 = bounds.shape
    if two != 2 or d2 != d or not _fits(index, dtype, q, bounds):
        _refuse(index, dtype, q=q, bounds=bounds)
    if nb | top_k | block_size | first_blocks | last_blocks > 0x7FFFFFFF:
        _too_large()
    if selected is None:
        selected = _empty(stream, (tq, hkv, top_k), torch.int32, q.device)
    elif selected.shape != (tq, hkv, top_k):
        raise ValueError("selected must be [Tq, Hkv, top_k]")
    b, mb = _query_rows(index, tq, block_table, seqlens_k, cu_seq_lens_q, dev_err, selected)
    rc = (_lib or load()).pa_select_blocks(
        q.data_ptr(), bounds.data_ptr(), block_table.data_ptr(), seqlens_k.data_ptr(),
        None if cu_seq_lens_q is None else cu_seq_lens_q.data_ptr(), selected.data_ptr(), b, tq, hq, hkv, d,
        nb, block_size, mb, top_k, first_blocks, last_blocks, dt,
        None if dev_err is None else dev_err.data_ptr(),
        _current_raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        raise PAError("pa_select_blocks", rc)
    return selected


def pa_sparse(q, k_cache, v_cache, block_table, seqlens_k, selected, cu_seq_lens_q=None, out=None,
              softmax_scale: float = 0.0, dev_err=None, stream=None):
    """Attention of each query over its selected blocks (see include/pa.h): q [Tq, Hq, D];
    k_cache, v_cache [NB, bs, Hkv, D], the new tokens written already; selected
    [Tq, Hkv, top_k] int32 logical blocks (negative: none); block_table, seqlens_k and
    cu_seq_lens_q as pa_select_blocks.  bfloat16 or float32.  Returns out [Tq, Hq, D]."""
    shape, pool = q.shape, k_cache.shape
    tq, hq, d = shape
    index, dtype = q.get_device(), q.dtype
    if index < 0:
        raise ValueError("all tensors must live on a CUDA device")
    dt = _DTYPES.get(dtype)
    if dt is None:
        dt = _dtype(q)
    if _current_device() != index:
        with torch.cuda.device(index):
            return pa_sparse(q, k_cache, v_cache, block_table, seqlens_k, selected, cu_seq_lens_q, out,
                             softmax_scale, dev_err, stream)
    nb, bs, hkv, d2 = pool
    if out is None:
        out = _empty(stream, shape, dtype, q.device)
    elif out.shape != shape:
        raise ValueError("inconsistent shapes")
    if d2 != d or v_cache.shape != pool or not _fits(index, dtype, q, k_cache, v_cache, out):
        _refuse(index, dtype, q=q, k_cache=k_cache, v_cache=v_cache, out=out)
    rows, heads, top_k = selected.shape
    if rows != tq or heads != hkv:
        raise ValueError("selected must be [Tq, Hkv, top_k]")
    if nb | bs | top_k > 0x7FFFFFFF:
        _too_large()
    b, mb = _query_rows(index, tq, block_table, seqlens_k, cu_seq_lens_q, dev_err, selected)
    rc = (_lib or load()).pa_sparse(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), seqlens_k.data_ptr(),
        None if cu_seq_lens_q is None else cu_seq_lens_q.data_ptr(), selected.data_ptr(), out.data_ptr(), b,
        tq, hq, hkv, d, nb, bs, mb, top_k, dt, softmax_scale,
        None if dev_err is None else dev_err.data_ptr(),
        _current_raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        raise PAError("pa_sparse", rc)
    return out
