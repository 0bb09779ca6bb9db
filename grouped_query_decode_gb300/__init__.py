"""GB300 (sm_103a) grouped-query decode attention.

A thin ctypes binding over the C ABI of libgqa_decode.so (include/gqa_decode.h):
the functions here only check and marshal arguments -- every step of the
computation runs in the library's CUDA kernels. There is no CPU fallback: if
the library cannot be built or loaded, every call raises.

    out, lse = torch.empty(...), torch.empty(...)
    gqa_decode(q, k_cache, v_cache, seq_lens, scale, out, lse)

q [B, sq, H, D], k_cache / v_cache [B, G, Tmax, D] and out are bfloat16 CUDA
tensors; seq_lens [B] is int32 on the same device; lse [B, sq, H] float32 or
None. Calls are enqueued on the current torch CUDA stream (or `stream`).
"""
from __future__ import annotations

import ctypes
import functools
import math
import threading
import weakref

from . import build as _build

GQA_OK = 0
GQA_ERR_INVALID_ARG = -1
GQA_ERR_HEAD_RATIO = -2
GQA_ERR_UNSUPPORTED = -3
GQA_ERR_MISALIGNED = -4
GQA_ERR_WORKSPACE = -5
GQA_ERR_CUDA = -6
GQA_ERR_DEVICE_TIMEOUT = -7

LIB_PATH = _build.LIB_PATH
_lib = None
_lock = threading.Lock()


class GQADecodeError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        msg = strerror(status) if _lib is not None else str(status)
        if status == GQA_ERR_CUDA and _lib is not None:
            msg += f" (cudaError {gqa_decode_last_cuda_error()})"
        super().__init__(f"{what}: {msg}" if what else msg)


class PagePoolT(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_bytes", ctypes.c_size_t),
                ("layer_bytes", ctypes.c_size_t), ("layers", ctypes.c_int)]


class RopeT(ctypes.Structure):
    """Rotary positions, made by gqa_rope_init."""
    _fields_ = [("dims", ctypes.c_int), ("interleaved", ctypes.c_int), ("gain", ctypes.c_double),
                ("inv_freq", ctypes.c_double * 64)]


class PlanT(ctypes.Structure):
    _fields_ = [("ctas", ctypes.c_int), ("tile_tokens", ctypes.c_int),
                ("row_tiles", ctypes.c_int), ("stages", ctypes.c_int),
                ("threads", ctypes.c_int), ("smem_bytes", ctypes.c_int),
                ("max_tiles", ctypes.c_longlong)]


def load():
    """Builds (if the sources are newer) and loads libgqa_decode.so."""
    global _lib
    if _lib is not None:           # every call after the first: no lock
        return _lib
    with _lock:
        if _lib is None:
            path = _build.build()
            lib = ctypes.CDLL(path)
            vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
            shape = [i32] * 6
            lib.gqa_decode.argtypes = [vp, vp, vp, vp, f32, vp, vp, *shape, vp]
            lib.gqa_decode.restype = i32
            lib.gqa_decode_ex.argtypes = [vp, vp, vp, vp, f32, vp, vp, *shape, vp, sz, vp]
            lib.gqa_decode_ex.restype = i32
            lib.gqa_decode_append.argtypes = [vp, vp, vp, vp, vp, vp, f32, vp, vp, *shape, vp]
            lib.gqa_decode_append.restype = i32
            lib.gqa_decode_paged.argtypes = [vp, vp, vp, vp, vp, f32, vp, vp, *([i32] * 8), vp]
            lib.gqa_decode_paged.restype = i32
            lib.gqa_decode_fp8.argtypes = [vp, vp, vp, vp, vp, vp, f32, vp, vp, *shape, vp]
            lib.gqa_decode_fp8.restype = i32
            lib.gqa_prefill.argtypes = [vp, vp, vp, vp, f32, vp, vp, *shape, vp]
            lib.gqa_prefill.restype = i32
            paged = [i32] * 8
            lib.gqa_decode_paged_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, f32, vp, vp, *paged, vp, sz, vp]
            lib.gqa_decode_paged_fp8.restype = i32
            lib.gqa_decode_paged_fp8_workspace_bytes.argtypes = [i32] * 7
            lib.gqa_decode_paged_fp8_workspace_bytes.restype = sz
            lib.gqa_append_paged_fp8.argtypes = [vp] * 8 + [i32] * 7 + [vp]
            lib.gqa_append_paged_fp8.restype = i32
            lib.gqa_pages_workspace_bytes.argtypes = [i32, i32]
            lib.gqa_pages_workspace_bytes.restype = sz
            lib.gqa_pages_copy.argtypes = [vp, i32, vp, vp, i32, i32, vp]
            lib.gqa_pages_copy.restype = i32
            lib.gqa_pages_reserve.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, sz, vp]
            lib.gqa_pages_reserve.restype = i32
            lib.gqa_pages_fork.argtypes = [vp, i32] + [vp] * 8 + [i32] * 4 + [vp, sz, vp]
            lib.gqa_pages_fork.restype = i32
            lib.gqa_pages_free.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp]
            lib.gqa_pages_free.restype = i32
            lib.gqa_pages_compact.argtypes = [vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, vp, sz, vp]
            lib.gqa_pages_compact.restype = i32
            i64, f64 = ctypes.c_longlong, ctypes.c_double
            lib.gqa_rope_init.argtypes = [vp, i32, i32, i32, f64, i32, f64, f64, f64, f64]
            lib.gqa_rope_init.restype = i32
            lib.gqa_rope.argtypes = [vp] * 6 + [i32] * 4 + [i64] * 4 + [i32, vp]
            lib.gqa_rope.restype = i32
            lib.gqa_append_paged.argtypes = [vp] * 10 + [i32] * 5 + [i64] * 4 + [i32] * 3 + [vp]
            lib.gqa_append_paged.restype = i32
            lib.gqa_prefill_packed.argtypes = [vp] * 4 + [f32, vp, vp] + [i32] * 5 + [i64] * 3 + [vp, sz, vp]
            lib.gqa_prefill_packed.restype = i32
            lib.gqa_prefill_paged.argtypes = [vp] * 6 + [f32, vp, vp] + [i32] * 5 + [i64] + [i32] * 3 + [vp, sz, vp]
            lib.gqa_prefill_paged.restype = i32
            lib.gqa_prefill_ragged_workspace_bytes.argtypes = [i32] * 5
            lib.gqa_prefill_ragged_workspace_bytes.restype = sz
            lib.gqa_decode_noalloc.argtypes = [vp, vp, vp, vp, f32, vp, vp, *shape, vp]
            lib.gqa_decode_noalloc.restype = i32
            lib.gqa_decode_workspace_bytes.argtypes = shape
            lib.gqa_decode_workspace_bytes.restype = sz
            lib.gqa_decode_plan.argtypes = [*shape, i32, ctypes.POINTER(PlanT)]
            lib.gqa_decode_plan.restype = i32
            lib.gqa_decode_check_error.argtypes = [vp]
            lib.gqa_decode_check_error.restype = i32
            lib.gqa_decode_release_workspace.argtypes = [vp]
            lib.gqa_decode_release_workspace.restype = i32
            lib.gqa_decode_last_cuda_error.argtypes = []
            lib.gqa_decode_last_cuda_error.restype = i32
            lib.gqa_decode_strerror.argtypes = [i32]
            lib.gqa_decode_strerror.restype = ctypes.c_char_p
            _lib = lib
    return _lib


def strerror(status: int) -> str:
    return load().gqa_decode_strerror(int(status)).decode()


def gqa_decode_strerror(status: int) -> str:
    return strerror(status)


def gqa_decode_last_cuda_error() -> int:
    return int(load().gqa_decode_last_cuda_error())


def _stream_handle(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif hasattr(stream, "device_index") and stream.device_index != device:
        raise ValueError(f"stream is on cuda:{stream.device_index}, the tensors on cuda:{device}")
    return ctypes.c_void_p(int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream))


def _call(device, fn, *args):
    """Calls the library with `device` current (it launches on the current
    device); switches only when another device is current."""
    import torch
    if torch.cuda.current_device() == device:
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


def _check(dev, name, t, dt):
    """dtype, device (the CUDA device `dev`) and contiguity of one tensor; the
    device index doubles as the CUDA check (-1 for host tensors)."""
    if t.dtype != dt:
        raise TypeError(f"{name} must be {dt}, got {t.dtype}")
    d = t.get_device()
    if d < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    if d != dev:
        raise ValueError(f"{name} is on cuda:{d}, q on cuda:{dev}: all tensors must be on one device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_lse(dev, lse, B, sq, H):
    """lse is optional; when given it is float32 [B, sq, H] on q's device."""
    import torch
    if lse is None:
        return
    _check(dev, "lse", lse, torch.float32)
    if tuple(lse.shape) != (B, sq, H):
        raise ValueError("lse must be [B, sq, H]")


def _shapes(q, k_cache, v_cache, seq_lens, out, lse):
    """Checks the tensors of the contiguous-cache entry points (dtype, one
    CUDA device, contiguity, shapes); returns B, sq, H, G, D, Tmax and the
    device index."""
    import torch
    bf = torch.bfloat16
    dev = q.get_device()
    _check(dev, "q", q, bf)
    _check(dev, "k_cache", k_cache, bf)
    _check(dev, "v_cache", v_cache, bf)
    _check(dev, "seq_lens", seq_lens, torch.int32)
    _check(dev, "out", out, bf)
    if q.dim() != 4 or k_cache.dim() != 4:
        raise ValueError("q is [B, sq, H, D] and k_cache [B, G, Tmax, D]")
    B, sq, H, D = q.shape
    Bk, G, Tmax, Dk = k_cache.shape
    if (Bk, Dk) != (B, D) or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("k_cache / v_cache must be [B, G, Tmax, D] with q's B and D")
    if tuple(seq_lens.shape) != (B,) or tuple(out.shape) != (B, sq, H, D):
        raise ValueError("seq_lens must be [B] and out [B, sq, H, D]")
    _check_lse(dev, lse, B, sq, H)
    return B, sq, H, G, D, Tmax, dev


def gqa_decode(q, k_cache, v_cache, seq_lens, scale, out, lse=None, stream=None):
    """One decode step (library-owned workspace). See include/gqa_decode.h."""
    B, sq, H, G, D, Tmax, dev = _shapes(q, k_cache, v_cache, seq_lens, out, lse)
    rc = _call(dev, load().gqa_decode, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
               seq_lens.data_ptr(), float(scale), out.data_ptr(),
               None if lse is None else lse.data_ptr(), B, sq, H, G, D, Tmax,
               _stream_handle(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_decode")


def gqa_prefill(q, k_cache, v_cache, seq_lens, scale, out, lse=None, stream=None):
    """Prefill or chunked prefill: the same attention as gqa_decode for any
    number of new tokens sq (no limit on (H/G)*sq), on the tcgen05 kernel.
    The sq new tokens' K/V must already be in the cache; seq_lens counts them."""
    B, sq, H, G, D, Tmax, dev = _shapes(q, k_cache, v_cache, seq_lens, out, lse)
    rc = _call(dev, load().gqa_prefill, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
               seq_lens.data_ptr(), float(scale), out.data_ptr(),
               None if lse is None else lse.data_ptr(), B, sq, H, G, D, Tmax,
               _stream_handle(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_prefill")


def gqa_decode_append(q, k_new, v_new, k_cache, v_cache, seq_lens, scale, out, lse=None,
                      stream=None):
    """One decode step that first appends the sq new tokens' K/V ([B, sq, G, D]
    bf16) to the caches at positions seq_lens[b] - sq + s, in the same launch."""
    B, sq, H, G, D, Tmax, dev = _shapes(q, k_cache, v_cache, seq_lens, out, lse)
    import torch
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        _check(dev, name, t, torch.bfloat16)
        if tuple(t.shape) != (B, sq, G, D):
            raise ValueError(f"{name} must be [B, sq, G, D]")
    rc = _call(dev, load().gqa_decode_append, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
               k_cache.data_ptr(), v_cache.data_ptr(), seq_lens.data_ptr(),
               float(scale), out.data_ptr(),
               None if lse is None else lse.data_ptr(), B, sq, H, G, D, Tmax,
               _stream_handle(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_decode_append")


def gqa_decode_paged(q, k_pages, v_pages, block_table, seq_lens, scale, out, lse=None,
                     stream=None):
    """One decode step over a paged cache: k_pages/v_pages [num_pages, G,
    page_size, D] bf16, block_table [B, max_pages_per_seq] int32."""
    import torch
    dev = q.get_device()
    for name, t, dt in (("q", q, torch.bfloat16), ("k_pages", k_pages, torch.bfloat16),
                        ("v_pages", v_pages, torch.bfloat16), ("block_table", block_table, torch.int32),
                        ("seq_lens", seq_lens, torch.int32), ("out", out, torch.bfloat16)):
        _check(dev, name, t, dt)
    B, sq, H, D = q.shape
    num_pages, G, page_size, Dk = k_pages.shape
    if Dk != D or tuple(v_pages.shape) != tuple(k_pages.shape):
        raise ValueError("k_pages / v_pages must be [num_pages, G, page_size, D]")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages_per_seq]")
    if tuple(seq_lens.shape) != (B,) or tuple(out.shape) != (B, sq, H, D):
        raise ValueError("seq_lens must be [B] and out [B, sq, H, D]")
    _check_lse(dev, lse, B, sq, H)
    rc = _call(dev, load().gqa_decode_paged, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
               block_table.data_ptr(), seq_lens.data_ptr(), float(scale),
               out.data_ptr(), None if lse is None else lse.data_ptr(),
               B, sq, H, G, D, page_size, num_pages, block_table.shape[1],
               _stream_handle(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_decode_paged")


def gqa_decode_fp8(q, k_codes, v_codes, k_scale, v_scale, seq_lens, scale, out, lse=None,
                   stream=None):
    """One decode step over an fp8 cache: k_codes/v_codes [B, G, Tmax, 128]
    uint8 e4m3 codes, k_scale/v_scale [B, G, ceil(Tmax/64)] float32 (one scale
    per 64-token block)."""
    import torch
    dev = q.get_device()
    for name, t, dt in (("q", q, torch.bfloat16), ("k_codes", k_codes, torch.uint8),
                        ("v_codes", v_codes, torch.uint8), ("k_scale", k_scale, torch.float32),
                        ("v_scale", v_scale, torch.float32), ("seq_lens", seq_lens, torch.int32),
                        ("out", out, torch.bfloat16)):
        _check(dev, name, t, dt)
    B, sq, H, D = q.shape
    Bk, G, Tmax, Dk = k_codes.shape
    if (Bk, Dk) != (B, D) or tuple(v_codes.shape) != tuple(k_codes.shape):
        raise ValueError("k_codes / v_codes must be [B, G, Tmax, D]")
    nt = (Tmax + 63) // 64
    if tuple(k_scale.shape) != (B, G, nt) or tuple(v_scale.shape) != (B, G, nt):
        raise ValueError("k_scale / v_scale must be [B, G, ceil(Tmax/64)]")
    if tuple(seq_lens.shape) != (B,) or tuple(out.shape) != (B, sq, H, D):
        raise ValueError("seq_lens must be [B] and out [B, sq, H, D]")
    _check_lse(dev, lse, B, sq, H)
    rc = _call(dev, load().gqa_decode_fp8, q.data_ptr(), k_codes.data_ptr(), v_codes.data_ptr(),
               k_scale.data_ptr(), v_scale.data_ptr(), seq_lens.data_ptr(),
               float(scale), out.data_ptr(), None if lse is None else lse.data_ptr(),
               B, sq, H, G, D, Tmax, _stream_handle(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_decode_fp8")


def _check_all(dev, named):
    """dtype, device and contiguity of (name, tensor, dtype) triples: one pass
    that is quick when all is well (a decode step is a few microseconds), then
    the one that says what is wrong."""
    for _, t, dt in named:
        if not (t.dtype is dt and t.get_device() == dev and t.is_contiguous()):
            break
    else:
        if dev >= 0:
            return
    for name, t, dt in named:
        _check(dev, name, t, dt)


def _raw_stream(stream, dev):
    """The stream handle of a call: `stream`, or the device's current one."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(dev)
    return _stream_handle(stream, dev)


def _paged_fp8_cache(k_pages, v_pages, k_scale, v_scale, block_table, seq_lens):
    """Checks the shapes of a paged 8-bit cache; returns B, num_pages, G,
    page_size, D and max_pages_per_seq."""
    shape = k_pages.shape
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError("k_pages / v_pages must be [num_pages, G, page_size, D]")
    num_pages, G, page_size, D = shape
    blocks = (num_pages, G, (page_size + 63) // 64)
    if k_scale.shape != blocks or v_scale.shape != blocks:
        raise ValueError("k_scale / v_scale must be [num_pages, G, ceil(page_size/64)]")
    table = block_table.shape
    if len(table) != 2 or seq_lens.shape != table[:1]:
        raise ValueError("block_table must be [B, max_pages_per_seq] and seq_lens [B]")
    return table[0], num_pages, G, page_size, D, table[1]


class _Workspaces:
    """The workspaces that one host thread keeps, by (device, stream handle),
    grow-only: a thread's calls on a stream run in order. Threads share none, also
    on one stream: a call may be two launches, the second of which reads what the
    first one wrote, and another thread's call may come in between. (So
    cudaStreamPerThread, another stream in every thread, is a handle like any.)"""

    def __init__(self):
        self.by_stream = {}


_of_thread = threading.local()
_of_all_threads = weakref.WeakSet()


def _kept_workspaces():
    try:
        return _of_thread.workspaces.by_stream
    except AttributeError:
        mine = _of_thread.workspaces = _Workspaces()
        with _lock:
            _of_all_threads.add(mine)
        return mine.by_stream


def _workspace(nbytes, like, dev, stream):
    """A buffer for one call on the device of `like`, in the order of the call's
    stream. A call on the current stream takes the calling thread's own for that
    stream, kept from call to call; a call that is being captured takes new memory
    of its graph, which no other graph shares; one on a stream passed as an
    argument takes new memory too."""
    import torch
    if stream is None:
        if torch._C._cuda_getDevice() != dev or torch._C._cuda_isCurrentStreamCapturing():
            return torch.empty(nbytes, dtype=torch.uint8, device=like.device)
        kept = _kept_workspaces()
        key = (dev, torch._C._cuda_getCurrentRawStream(dev))
        buf = kept.get(key)
        if buf is None or buf.shape[0] < nbytes:
            buf = kept[key] = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
        return buf
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)


def gqa_decode_paged_fp8(q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, scale, out, lse=None,
                         stream=None, workspace=None):
    """Attention over a paged 8-bit cache, for any number of new tokens sq:
    k_pages/v_pages [num_pages, G, page_size, D] uint8 e4m3 codes, k_scale/
    v_scale [num_pages, G, ceil(page_size/64)] float32, block_table [B,
    max_pages_per_seq] int32. The workspace (a CUDA uint8 tensor of
    gqa_decode_paged_fp8_workspace_bytes(...)) comes from torch's allocator when
    not given: the calling thread's own for the stream, kept from call to call, or
    memory of the graph being captured."""
    import torch
    dev = q.get_device()
    bf, u8, f32, i32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
    named = [("q", q, bf), ("out", out, bf), ("k_pages", k_pages, u8), ("v_pages", v_pages, u8),
             ("k_scale", k_scale, f32), ("v_scale", v_scale, f32), ("block_table", block_table, i32),
             ("seq_lens", seq_lens, i32)]
    if lse is not None:
        named.append(("lse", lse, f32))
    if workspace is not None:
        named.append(("workspace", workspace, u8))
    _check_all(dev, named)
    Bt, num_pages, G, page_size, Dk, most = _paged_fp8_cache(k_pages, v_pages, k_scale, v_scale, block_table, seq_lens)
    shape = q.shape
    if len(shape) != 4 or shape[0] != Bt or shape[3] != Dk:
        raise ValueError("q must be [B, sq, H, D] with block_table's B and the pages' D")
    B, sq, H, D = shape
    if out.shape != shape:
        raise ValueError("out must be [B, sq, H, D]")
    if lse is not None and lse.shape != (B, sq, H):
        raise ValueError("lse must be [B, sq, H]")
    if workspace is None:
        workspace = _workspace(_paged_fp8_workspace_bytes(B, sq, H, G, D, page_size, most, dev) or 256, q, dev, stream)
    rc = _call(dev, load().gqa_decode_paged_fp8, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
               k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
               float(scale), out.data_ptr(), None if lse is None else lse.data_ptr(), B, sq, H, G, D,
               page_size, num_pages, most, workspace.data_ptr(), workspace.numel(), _raw_stream(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_decode_paged_fp8")


class _NoSize(Exception):
    """No workspace size: unsupported sizes, or a device that could not be asked
    just then. An exception, so that it is not kept."""


@functools.lru_cache(maxsize=4096)
def _known_paged_fp8_bytes(*sizes):
    n = int(_call(sizes[-1], load().gqa_decode_paged_fp8_workspace_bytes, *sizes[:-1]))
    if n == 0:
        raise _NoSize
    return n


def _paged_fp8_workspace_bytes(*sizes):
    """By B, sq, H, G, D, page_size, max_pages_per_seq and device."""
    try:
        return _known_paged_fp8_bytes(*sizes)
    except _NoSize:
        return 0


def gqa_decode_paged_fp8_workspace_bytes(B, sq, H, G, D, page_size, max_pages_per_seq, device=None) -> int:
    """Workspace bytes of gqa_decode_paged_fp8 on a device (0: unsupported sizes)."""
    if device is None:
        import torch
        device = torch.cuda.current_device()
    return _paged_fp8_workspace_bytes(B, sq, H, G, D, page_size, max_pages_per_seq, device)


def gqa_append_paged_fp8(k_new, v_new, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, stream=None):
    """Quantises the sq new tokens' K/V ([B, sq, G, D] bf16) into a paged
    8-bit cache at positions seq_lens[b] - sq + s, with one power-of-two scale
    per block of min(64, page_size) tokens and KV head."""
    import torch
    dev = k_new.get_device()
    bf, u8, f32, i32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
    _check_all(dev, (("k_new", k_new, bf), ("v_new", v_new, bf), ("k_pages", k_pages, u8), ("v_pages", v_pages, u8),
                     ("k_scale", k_scale, f32), ("v_scale", v_scale, f32), ("block_table", block_table, i32),
                     ("seq_lens", seq_lens, i32)))
    B, num_pages, G, page_size, D, most = _paged_fp8_cache(k_pages, v_pages, k_scale, v_scale, block_table, seq_lens)
    shape = k_new.shape
    if len(shape) != 4 or shape[0] != B or shape[2:] != (G, D) or v_new.shape != shape:
        raise ValueError("k_new / v_new must be [B, sq, G, D]")
    rc = _call(dev, load().gqa_append_paged_fp8, k_new.data_ptr(), v_new.data_ptr(), k_pages.data_ptr(),
               v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(),
               seq_lens.data_ptr(), B, shape[1], G, D, page_size, num_pages, most, _raw_stream(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_append_paged_fp8")


def _page_pools(dev, pools, num_pages, page_dim):
    """The pools of a page call as the library's array. Each is a tensor whose
    dimension `page_dim` counts the pages; dimensions before it are layers
    that share the page numbers."""
    pools = list(pools)
    arr = (PagePoolT * max(1, len(pools)))()
    _check_all(dev, [(f"pools[{i}]", t, t.dtype) for i, t in enumerate(pools)])
    for i, t in enumerate(pools):
        shape = t.shape
        if not 0 <= page_dim < len(shape) or shape[page_dim] != num_pages:
            raise ValueError(f"pools[{i}] must count {num_pages} pages in dimension {page_dim}")
        page, layers = t.element_size() * math.prod(shape[page_dim + 1:]), math.prod(shape[:page_dim])
        if page * layers == 0:
            raise ValueError(f"pools[{i}] is empty")
        arr[i] = (t.data_ptr(), page, page * num_pages, layers)
    return arr, len(pools)


def _page_sizes(block_table, seq_lens, ref_counts, counts=None):
    """Checks the shapes of a block table and its counts; returns B,
    max_pages_per_seq and num_pages."""
    table, pages = block_table.shape, ref_counts.shape
    if len(table) != 2 or (seq_lens is not None and seq_lens.shape != table[:1]):
        raise ValueError("block_table must be [B, max_pages_per_seq] and seq_lens [B]")
    if len(pages) != 1:
        raise ValueError("ref_counts must be [num_pages]")
    if counts is not None and counts.shape != (2,):
        raise ValueError("counts must be [2]")
    return table[0], table[1], pages[0]


@functools.lru_cache(maxsize=4096)
def gqa_pages_workspace_bytes(B, num_pages) -> int:
    """Workspace bytes of gqa_pages_reserve, gqa_pages_fork and
    gqa_pages_compact (the functions here take one from torch's allocator)."""
    return int(load().gqa_pages_workspace_bytes(B, num_pages))


def gqa_pages_copy(pools, src, dst, num_pages, page_dim=0, stream=None):
    """Copies page src[i] to page dst[i] (int32 [n]) in every pool: tensors
    whose dimension page_dim counts the pages (dimensions before it: layers).
    No page may be a source and a destination, or twice a destination."""
    import torch
    dev = src.get_device()
    _check_all(dev, (("src", src, torch.int32), ("dst", dst, torch.int32)))
    if src.dim() != 1 or dst.shape != src.shape:
        raise ValueError("src and dst must be [n]")
    arr, n = _page_pools(dev, pools, num_pages, page_dim)
    rc = _call(dev, load().gqa_pages_copy, arr, n, src.data_ptr(), dst.data_ptr(), src.shape[0], num_pages,
               _raw_stream(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_pages_copy")


def gqa_pages_reserve(block_table, seq_lens, ref_counts, page_size, counts, stream=None):
    """Gives every sequence, in place, the pages that seq_lens[b] tokens need:
    empty entries take the free pages (ref_counts <= 0) in ascending order.
    counts (int32 [2]) = pages needed, pages that were free; nothing changes
    if fewer are free than needed."""
    import torch
    dev, i32 = block_table.get_device(), torch.int32
    _check_all(dev, (("block_table", block_table, i32), ("seq_lens", seq_lens, i32), ("ref_counts", ref_counts, i32),
                     ("counts", counts, i32)))
    B, most, num_pages = _page_sizes(block_table, seq_lens, ref_counts, counts)
    ws = _workspace(gqa_pages_workspace_bytes(B, num_pages) or 256, block_table, dev, stream)
    rc = _call(dev, load().gqa_pages_reserve, block_table.data_ptr(), seq_lens.data_ptr(),
               ref_counts.data_ptr(), counts.data_ptr(), B, most, page_size, num_pages, ws.data_ptr(),
               ws.numel(), _raw_stream(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_pages_reserve")


def gqa_pages_fork(pools, src, block_table, seq_lens, ref_counts, page_size, block_table_out, seq_lens_out,
                   ref_counts_out, counts, page_dim=0, stream=None):
    """New row i goes on from old row src[i] (int32 [B]; outside [0, B): empty):
    full pages are shared, the partly filled last page stays with the lowest
    such row and is copied, in every pool, for the others; sequences that no
    row goes on from give their pages back. Holders outside the table keep full
    pages only: the lowest row writes on in a partly filled one. The outputs are
    other tensors than the inputs. counts (int32 [2]) = pages needed, pages that
    were free; the outputs are copies of the inputs if fewer are free than needed."""
    import torch
    dev, i32 = block_table.get_device(), torch.int32
    _check_all(dev, (("src", src, i32), ("block_table", block_table, i32), ("seq_lens", seq_lens, i32),
                     ("ref_counts", ref_counts, i32), ("block_table_out", block_table_out, i32),
                     ("seq_lens_out", seq_lens_out, i32), ("ref_counts_out", ref_counts_out, i32),
                     ("counts", counts, i32)))
    B, most, num_pages = _page_sizes(block_table, seq_lens, ref_counts, counts)
    if (block_table_out.shape != block_table.shape or seq_lens_out.shape != seq_lens.shape or
            ref_counts_out.shape != ref_counts.shape):
        raise ValueError("the outputs must have the inputs' shapes")
    if src.shape != (B,):
        raise ValueError("src must be [B]")
    arr, n = _page_pools(dev, pools, num_pages, page_dim)
    ws = _workspace(gqa_pages_workspace_bytes(B, num_pages) or 256, block_table, dev, stream)
    rc = _call(dev, load().gqa_pages_fork, arr, n, src.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
               ref_counts.data_ptr(), block_table_out.data_ptr(), seq_lens_out.data_ptr(),
               ref_counts_out.data_ptr(), counts.data_ptr(), B, most, page_size, num_pages, ws.data_ptr(),
               ws.numel(), _raw_stream(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_pages_fork")


def gqa_pages_free(done, block_table, seq_lens, ref_counts, stream=None):
    """Gives back the pages of every sequence with done[b] (bool or uint8 [B]),
    in place: counts go down by one, rows become -1, lengths 0."""
    import torch
    dev, i32 = block_table.get_device(), torch.int32
    _check_all(dev, (("done", done, torch.bool if done.dtype is torch.bool else torch.uint8),
                     ("block_table", block_table, i32), ("seq_lens", seq_lens, i32), ("ref_counts", ref_counts, i32)))
    B, most, num_pages = _page_sizes(block_table, seq_lens, ref_counts)
    if done.shape != (B,):
        raise ValueError("done must be [B]")
    rc = _call(dev, load().gqa_pages_free, done.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
               ref_counts.data_ptr(), B, most, num_pages, _raw_stream(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_pages_free")


def gqa_pages_compact(pools, block_table, ref_counts, block_table_out, ref_counts_out, counts, page_dim=0,
                      stream=None):
    """Moves the live pages (ref_counts > 0) to the lowest page numbers, in
    every pool; the block table and counts follow (the outputs may be the
    input tensors themselves). counts (int32 [2]) = pages moved, pages live."""
    import torch
    dev, i32 = block_table.get_device(), torch.int32
    _check_all(dev, (("block_table", block_table, i32), ("ref_counts", ref_counts, i32),
                     ("block_table_out", block_table_out, i32), ("ref_counts_out", ref_counts_out, i32),
                     ("counts", counts, i32)))
    B, most, num_pages = _page_sizes(block_table, None, ref_counts, counts)
    if block_table_out.shape != block_table.shape or ref_counts_out.shape != ref_counts.shape:
        raise ValueError("the outputs must have the inputs' shapes")
    arr, n = _page_pools(dev, pools, num_pages, page_dim)
    ws = _workspace(gqa_pages_workspace_bytes(B, num_pages) or 256, block_table, dev, stream)
    rc = _call(dev, load().gqa_pages_compact, arr, n, block_table.data_ptr(), ref_counts.data_ptr(),
               block_table_out.data_ptr(), ref_counts_out.data_ptr(), counts.data_ptr(), B, most, num_pages,
               ws.data_ptr(), ws.numel(), _raw_stream(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_pages_compact")


# ------------------------------------------------- packed batches over bf16

_SCALINGS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "yarn": 4}


def gqa_rope_init(D, dims=None, interleaved=False, base=10000.0, scaling="none", factor=1.0, original=0.0, low=1.0,
                  high=4.0) -> RopeT:
    """Rotary positions of the first `dims` (default: all D) elements of a head,
    in pairs (i, i + dims / 2) or, interleaved, (2 i, 2 i + 1). scaling lengthens
    the context by `factor`: "none", "linear", "base", "bands" or "yarn" (the last
    two with the original context and the turns low and high between which pairs
    are slowed in part). See include/gqa_decode.h."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(_SCALINGS)}")
    rope = RopeT()
    rc = load().gqa_rope_init(ctypes.byref(rope), D, D if dims is None else dims, bool(interleaved), float(base),
                              _SCALINGS[scaling], float(factor), float(original), float(low), float(high))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_rope_init")
    return rope


def _row_stride(name, t, dt, dev, shape):
    """Checks a packed tensor [N, heads, D] whose heads are dense; returns the
    distance of its tokens in elements."""
    if t.shape == shape and t.dtype is dt and t.get_device() == dev:      # the quick pass
        s = t.stride()
        if s[2] == 1 and s[1] == shape[2] and shape[0] > 1 and dev >= 0:
            return s[0]
    if t.dtype is not dt:
        raise TypeError(f"{name} must be {dt}, got {t.dtype}")
    if t.get_device() < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, others on cuda:{dev}: all tensors must be on one device")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, is {list(t.shape)}")
    N, heads, D = shape
    s = t.stride()
    if not t.is_contiguous() and (s[2] != 1 or (heads > 1 and s[1] != D)):
        raise ValueError(f"{name} must have dense heads (only its tokens may be apart)")
    return s[0] if N > 1 else heads * D


def _check_rope(rope):
    if not isinstance(rope, RopeT):
        raise TypeError("rope must come from gqa_rope_init")


def _launch(dev, fn, *args):
    """_call for tensors that are there, so that CUDA is initialised."""
    import torch
    if torch._C._cuda_getDevice() == dev:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def gqa_rope(rope, q, k, positions, q_out, k_out, inverse=False, stream=None):
    """Rotates q [N, H, D] and k [N, G, D] (bf16; either may be None) by
    positions (int32 [N]) into q_out and k_out, which may be the inputs
    themselves. inverse turns the other way (the transpose: the gradient's
    operator). Tokens may be apart, as in views of a fused projection's rows."""
    import torch
    _check_rope(rope)
    bf = torch.bfloat16
    if (q is None) != (q_out is None) or (k is None) != (k_out is None) or (q is None and k is None):
        raise ValueError("q comes with q_out and k with k_out, one of them at least")
    dev = positions.get_device()
    qp = qo = kp = ko = None
    H = G = qs = qos = ks = kos = 0
    for name, t in (("q", q), ("k", k)):
        if t is not None and t.dim() != 3:
            raise ValueError(f"{name} must be [N, heads, D]")
    if q is not None:
        shape = q.shape
        N, H, D = shape
        qs, qos = _row_stride("q", q, bf, dev, shape), _row_stride("q_out", q_out, bf, dev, shape)
        qp, qo = q.data_ptr(), q_out.data_ptr()
    if k is not None:
        shape = k.shape
        if q is not None and (shape[0] != N or shape[2] != D):
            raise ValueError("k must be [N, heads, D] with q's N and D")
        N, G, D = shape
        ks, kos = _row_stride("k", k, bf, dev, shape), _row_stride("k_out", k_out, bf, dev, shape)
        kp, ko = k.data_ptr(), k_out.data_ptr()
    _check_all(dev, (("positions", positions, torch.int32),))
    if positions.shape != (N,):
        raise ValueError("positions must be [N]")
    rc = _launch(dev, load().gqa_rope, ctypes.addressof(rope), qp, kp, positions.data_ptr(), qo, ko, N, H, G, D, qs, ks,
                 qos, kos, 1 if inverse else 0, _raw_stream(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_rope")


def _paged_bf16_cache(k_pages, v_pages, block_table, seq_lens, cu):
    """Checks the shapes of a paged bf16 cache and a packed batch; returns B,
    num_pages, G, page_size, D and max_pages_per_seq."""
    shape = k_pages.shape
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError("k_pages / v_pages must be [num_pages, G, page_size, D]")
    table = block_table.shape
    if len(table) != 2 or seq_lens.shape != table[:1]:
        raise ValueError("block_table must be [B, max_pages_per_seq] and seq_lens [B]")
    if cu.shape != (table[0] + 1,):
        raise ValueError("cu_new must be [B + 1]")
    return (table[0], *shape, table[1])


def gqa_append_paged(k_new, v_new, k_pages, v_pages, block_table, cu_new, seq_lens, rope=None, q=None, q_out=None,
                     stream=None):
    """Writes the new tokens k_new, v_new ([N, G, D] bf16, rows cu_new[b] to
    cu_new[b + 1] of sequence b) to bf16 pages, at the last positions of
    seq_lens[b]. With rope, keys are rotated on the way, and the queries q [N, H,
    D] where given, into q_out (which may be q)."""
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    if (q is None) != (q_out is None):
        raise ValueError("q comes with q_out")
    if rope is not None:
        _check_rope(rope)
    dev = k_new.get_device()
    _check_all(dev, (("k_pages", k_pages, bf), ("v_pages", v_pages, bf), ("block_table", block_table, i32),
                     ("cu_new", cu_new, i32), ("seq_lens", seq_lens, i32)))
    B, num_pages, G, page_size, D, most = _paged_bf16_cache(k_pages, v_pages, block_table, seq_lens, cu_new)
    N = k_new.shape[0]
    shape = (N, G, D)
    ks, vs = _row_stride("k_new", k_new, bf, dev, shape), _row_stride("v_new", v_new, bf, dev, shape)
    qp = qo = None
    H = qs = qos = 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [N, H, D]")
        H = q.shape[1]
        shape = (N, H, D)
        qs, qos = _row_stride("q", q, bf, dev, shape), _row_stride("q_out", q_out, bf, dev, shape)
        qp, qo = q.data_ptr(), q_out.data_ptr()
    rc = _launch(dev, load().gqa_append_paged, None if rope is None else ctypes.addressof(rope), qp, k_new.data_ptr(),
                 v_new.data_ptr(), qo, k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
                 cu_new.data_ptr(), seq_lens.data_ptr(), N, B, H, G, D, qs, ks, vs, qos, page_size, num_pages, most,
                 _raw_stream(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_append_paged")


@functools.lru_cache(maxsize=64)
def _known_ragged_bytes(D, device):
    n = int(_call(device, load().gqa_prefill_ragged_workspace_bytes, 1, 1, 1, 1, D))
    if n == 0:
        raise _NoSize
    return n


def _ragged_workspace_bytes(D, device):
    """Of any sizes that the calls take: a packed batch's workspace depends on D and the
    device's SMs alone, so that steps of changing sizes ask once."""
    try:
        return _known_ragged_bytes(D, device)
    except _NoSize:
        return 0


def gqa_prefill_ragged_workspace_bytes(N, B, H, G, D, device=None) -> int:
    """Workspace bytes of gqa_prefill_packed and gqa_prefill_paged on a device
    (0: unsupported sizes)."""
    if device is None:
        import torch
        device = torch.cuda.current_device()
    return int(_call(device, load().gqa_prefill_ragged_workspace_bytes, N, B, H, G, D))


def _ragged_outputs(dev, q, out, lse, workspace):
    """Checks q, out, lse and workspace of a packed batch; returns q's shape and
    the distance of its tokens."""
    import torch
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q must be [N, H, D]")
    qs = _row_stride("q", q, torch.bfloat16, dev, shape)
    _check_all(dev, (("out", out, torch.bfloat16),))
    if lse is not None:
        _check_all(dev, (("lse", lse, torch.float32),))
    if workspace is not None:
        _check_all(dev, (("workspace", workspace, torch.uint8),))
    if out.shape != shape or (lse is not None and lse.shape != shape[:2]):
        raise ValueError("out must be [N, H, D] and lse [N, H]")
    return shape, qs


def gqa_prefill_packed(q, k, v, cu_seqlens, scale, out, lse=None, stream=None, workspace=None):
    """Causal attention of whole prompts that lie behind one another: q [N, H, D],
    k and v [N, G, D] (tokens may be apart, as in views of a fused projection's
    rows), cu_seqlens [B + 1] int32; out [N, H, D], lse [N, H]. Rows behind
    cu_seqlens[B] are left as they are. The workspace is kept as for
    gqa_decode_paged_fp8 when not given (gqa_prefill_ragged_workspace_bytes)."""
    import torch
    bf = torch.bfloat16
    dev = q.get_device()
    (N, H, D), qs = _ragged_outputs(dev, q, out, lse, workspace)
    if k.dim() != 3:
        raise ValueError("k must be [N, G, D]")
    G = k.shape[1]
    shape = (N, G, D)
    ks, vs = _row_stride("k", k, bf, dev, shape), _row_stride("v", v, bf, dev, shape)
    _check_all(dev, (("cu_seqlens", cu_seqlens, torch.int32),))
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must be [B + 1]")
    B = cu_seqlens.shape[0] - 1
    if workspace is None:
        workspace = _workspace(_ragged_workspace_bytes(D, dev) or 256, q, dev, stream)
    rc = _launch(dev, load().gqa_prefill_packed, q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(),
                 float(scale), out.data_ptr(), None if lse is None else lse.data_ptr(), N, B, H, G, D, qs, ks, vs,
                 workspace.data_ptr(), workspace.numel(), _raw_stream(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_prefill_packed")


def gqa_prefill_paged(q, k_pages, v_pages, block_table, cu_new, seq_lens, scale, out, lse=None, stream=None,
                      workspace=None):
    """Attention of chunks of any length, single tokens among them, over a paged
    bf16 cache ([num_pages, G, page_size, D]): rows cu_new[b] to cu_new[b + 1] of
    q [N, H, D] are the last tokens of seq_lens[b]. out [N, H, D], lse [N, H];
    rows behind cu_new[B] are left as they are. Workspace as for
    gqa_prefill_packed."""
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    dev = q.get_device()
    (N, H, D), qs = _ragged_outputs(dev, q, out, lse, workspace)
    _check_all(dev, (("k_pages", k_pages, bf), ("v_pages", v_pages, bf), ("block_table", block_table, i32),
                     ("cu_new", cu_new, i32), ("seq_lens", seq_lens, i32)))
    B, num_pages, G, page_size, Dk, most = _paged_bf16_cache(k_pages, v_pages, block_table, seq_lens, cu_new)
    if Dk != D:
        raise ValueError("q must be [N, H, D] with the pages' D")
    if workspace is None:
        workspace = _workspace(_ragged_workspace_bytes(D, dev) or 256, q, dev, stream)
    rc = _launch(dev, load().gqa_prefill_paged, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                 block_table.data_ptr(), cu_new.data_ptr(), seq_lens.data_ptr(), float(scale), out.data_ptr(),
                 None if lse is None else lse.data_ptr(), N, B, H, G, D, qs, page_size, num_pages, most,
                 workspace.data_ptr(), workspace.numel(), _raw_stream(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_prefill_paged")


def gqa_decode_ex(q, k_cache, v_cache, seq_lens, scale, out, lse, workspace, stream=None):
    """One decode step with a caller-owned workspace (a CUDA uint8 tensor of at
    least gqa_decode_workspace_bytes(...) bytes)."""
    B, sq, H, G, D, Tmax, dev = _shapes(q, k_cache, v_cache, seq_lens, out, lse)
    import torch
    _check(dev, "workspace", workspace, torch.uint8)
    rc = _call(dev, load().gqa_decode_ex, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
               seq_lens.data_ptr(), float(scale), out.data_ptr(),
               None if lse is None else lse.data_ptr(), B, sq, H, G, D, Tmax,
               workspace.data_ptr(), workspace.numel() * workspace.element_size(),
               _stream_handle(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_decode_ex")


# Size of the fixed per-device scratch array gqa_decode_noalloc draws from.
GQA_NOALLOC_SCRATCH_BYTES = 8 << 20


def gqa_decode_noalloc(q, k_cache, v_cache, seq_lens, scale, out, lse=None, stream=None):
    """One decode step that allocates no device memory: the scratch comes from
    a fixed 8 MiB array the library keeps on each GPU. For callers that may not
    allocate once running (a pre-reserved memory pool, a framework plugin with
    no allocator, a loop that cannot take cudaMalloc's synchronisation). Calls
    on one device share that array, so calls that overlap on the GPU race."""
    B, sq, H, G, D, Tmax, dev = _shapes(q, k_cache, v_cache, seq_lens, out, lse)
    rc = _call(dev, load().gqa_decode_noalloc, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
               seq_lens.data_ptr(), float(scale), out.data_ptr(),
               None if lse is None else lse.data_ptr(), B, sq, H, G, D, Tmax,
               _stream_handle(stream, dev))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_decode_noalloc")


def gqa_decode_release_workspace(stream=None, device=None) -> None:
    """Frees the workspaces kept for (device, stream), those of every thread,
    after the work queued on the stream; the next call on that stream allocates
    again."""
    import torch
    if device is None:
        device = stream.device_index if hasattr(stream, "device_index") else torch.cuda.current_device()
    handle = _stream_handle(stream, device)
    index = device if isinstance(device, int) else torch.device(device).index
    key = (torch.cuda.current_device() if index is None else index, handle.value or 0)
    with _lock:
        everyone = list(_of_all_threads)
    for w in everyone:
        w.by_stream.pop(key, None)
    rc = _call(device, load().gqa_decode_release_workspace, handle)
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_decode_release_workspace")


def gqa_decode_workspace_bytes(B, sq, H, G, D, Tmax) -> int:
    return int(load().gqa_decode_workspace_bytes(B, sq, H, G, D, Tmax))


def gqa_decode_plan(B, sq, H, G, D, Tmax, num_sms) -> dict:
    plan = PlanT()
    rc = load().gqa_decode_plan(B, sq, H, G, D, Tmax, num_sms, ctypes.byref(plan))
    if rc != GQA_OK:
        raise GQADecodeError(rc, "gqa_decode_plan")
    return {f: getattr(plan, f) for f, _ in PlanT._fields_}


def gqa_decode_check_error(stream=None, device=None) -> int:
    """Synchronises the stream and returns (and clears) the device status."""
    import torch
    if device is None:
        device = stream.device_index if hasattr(stream, "device_index") else torch.cuda.current_device()
    dev = device if isinstance(device, int) else torch.device(device).index
    return int(_call(dev, load().gqa_decode_check_error, _stream_handle(stream, dev)))
