"""ctypes binding of libsmla.so (the C ABI in include/smla.h).

Argument marshalling only: every step of the decode runs in the library's
CUDA kernels.  torch tensors supply device memory and the current stream.
If the library is missing, calls raise -- there is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsmla.so")

DC, DR, D, PAGE_SIZE = 512, 64, 576, 64
MAX_HEADS, MAX_NSPLIT = 64, 1024
NOALLOC_SCRATCH_BYTES = 16 << 20
# Largest K (index-list width, dense longest visible length, indexer selection
# width): the library's split arithmetic (ceil(K / nsplit) rounded up to whole
# pages, then K + that split length) and its fill loops are 32-bit.  The
# library does not check this bound itself.
MAX_K = 2**30 - 64

STATUS = {
    0: "SMLA_OK", 1: "SMLA_ERR_INVALID_ARG", 2: "SMLA_ERR_UNSUPPORTED", 3: "SMLA_ERR_MISALIGNED",
    4: "SMLA_ERR_WORKSPACE_TOO_SMALL", 5: "SMLA_ERR_INDEX_RANGE", 6: "SMLA_ERR_CUDA",
    7: "SMLA_ERR_TIMEOUT",
}

# exported symbol -> (restype, argtypes)
_P, _I, _I64, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "smla_choose_nsplit": (_I, [_I, _I, _I, _I, _I]),
    "smla_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "smla_decode_partial": (_I, [_P, _P, _I64, _P, _I, _P, _I, _I, _I, _I, _I, _F, _I, _P, _P, _P,
                                 _P]),
    "smla_lse_combine": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P]),
    "smla_decode": (_I, [_P, _P, _I64, _P, _I, _P, _I, _I, _I, _I, _I, _F, _I, _P, _SZ, _P, _P,
                         _P]),
    "smla_decode_partial_ws": (_I, [_P, _P, _I64, _P, _I, _P, _I, _I, _I, _I, _I, _F, _I, _P, _SZ,
                                    _P]),
    "smla_decode_noalloc": (_I, [_P, _P, _I64, _P, _I, _P, _I, _I, _I, _I, _I, _F, _I, _P, _P,
                                 _P]),
    "smla_workspace_host_bytes": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "smla_decode_host": (_I, [_P, _P, _I64, _P, _I, _P, _I, _I, _I, _I, _I, _F, _I, _P, _SZ, _P, _P,
                              _P]),
    "smla_dense_nsplit": (_I, [_I, _I, _I, _I]),
    "smla_dense_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "smla_decode_dense": (_I, [_P, _P, _I64, _P, _I, _P, _I, _I, _I, _I, _I, _F, _I, _P, _SZ, _P,
                               _P, _P]),
    "smla_decode_dense_partial": (_I, [_P, _P, _I64, _P, _I, _P, _I, _I, _I, _I, _I, _F, _I, _P,
                                       _P, _P, _P]),
    "smla_indexer_workspace_bytes": (_SZ, [_I, _I, _I]),
    "smla_indexer_topk": (_I, [_P, _P, _P, _I64, _P, _I, _P, _I, _I, _I, _I, _I, _I, _P, _SZ, _P,
                               _P]),
    "smla_indexer_scores": (_I, [_P, _P, _P, _I64, _P, _I, _P, _I, _I, _I, _I, _I, _P, _SZ, _P,
                                 _P]),
    "smla_indexer_select": (_I, [_P, _P, _I, _I, _I, _I, _P, _SZ, _P, _P]),
    "smla_indexer_select_workspace_bytes": (_SZ, [_I, _I, _I]),
    "smla_q4_append": (_I, [_P, _I, _P, _P, _I, _P, _I64, _P, _I, _I, _P]),
    "smla_q4_read": (_I, [_P, _I64, _P, _I, _P, _I, _I, _I, _P, _P]),
    "smla_q4_nsplit": (_I, [_I, _I, _I, _I]),
    "smla_q4_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "smla_decode_q4": (_I, [_P, _P, _I64, _P, _I, _P, _I, _I, _I, _I, _I, _F, _I, _P, _SZ, _P, _P,
                            _P]),
    "smla_dense_q4_nsplit": (_I, [_I, _I, _I, _I]),
    "smla_dense_q4_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "smla_decode_dense_q4": (_I, [_P, _P, _I64, _P, _I, _P, _I, _I, _I, _I, _I, _F, _I, _P, _SZ, _P,
                                  _P, _P]),
    "smla_evict_accumulate": (_I, [_P, _P, _I64, _P, _I, _P, _P, _I, _I, _I, _I, _F, _P, _I, _P]),
    "smla_evict_accumulate_q4": (_I, [_P, _P, _I64, _P, _I, _P, _P, _I, _I, _I, _I, _F, _P, _I,
                                      _P]),
    "smla_evict_workspace_bytes": (_SZ, [_I, _I]),
    "smla_evict_plan": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _SZ, _P, _P, _P, _P, _P]),
    "smla_evict_apply": (_I, [_P, _I, _I, _P, _I, _I64, _I, _P, _P, _I, _P]),
    "smla_selftest_wait_timeout": (_I, [ctypes.c_ulonglong, _P]),
    "smla_check_device": (_I, [_I, ctypes.POINTER(ctypes.c_ulonglong), _P]),
    "smla_status_string": (ctypes.c_char_p, [_I]),
    "smla_last_error": (ctypes.c_char_p, []),
    "smla_version": (_I, []),
}


class SmlaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {STATUS.get(status, status)}"
        if status == 6:
            msg += f" ({lib().smla_last_error().decode()})"
        super().__init__(msg)


_lib = None


def lib():
    """Load libsmla.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m sparse_mla_decode_partial_b200.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _k_in_range(K: int) -> int:
    if K > MAX_K:
        raise ValueError(f"K = {K} is above the library's limit {MAX_K}")
    return K


def _check(status: int, where: str):
    if status != 0:
        raise SmlaError(status, where)


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need(t, dtype, name, device=None, shape=None):
    """Type, dtype, contiguity, shape (when given: the library reads or writes
    exactly that many elements through the pointer) and device of a tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    _on_device(t, name, device)


def _on_device(t, name, device):
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a CUDA tensor on {device}")


def _torch_stream(stream, dev):
    """``stream`` (a torch stream, a handle, or None) as torch takes it."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(_stream(stream), device=dev)


class _Memory:
    """Allocates the tensors that a launch on ``stream`` uses from that stream's
    own memory: a block that the current stream has let go of may still be written
    by work queued there, which nothing orders before the launch.  What is
    ``returned`` will be read on the current stream, which therefore holds the
    memory too.  (Streams are compared by handle and switched once per call: a
    switch costs some 8 us of host time.)"""
    __slots__ = ("dev", "side", "here", "switch")

    def __init__(self, stream, dev):
        self.dev, self.here, self.switch = dev, None, None
        other = stream is not None and _stream(stream) != torch._C._cuda_getCurrentRawStream(dev.index)
        self.side = _torch_stream(stream, dev) if other else None

    def __enter__(self):
        return self

    def __call__(self, shape, dtype, returned=True):
        if self.side is not None and self.switch is None:
            self.here = torch.cuda.current_stream(self.dev)
            self.switch = torch.cuda.stream(self.side)
            self.switch.__enter__()
        t = torch.empty(*shape, dtype=dtype, device=self.dev)  # (separate sizes parse 0.7 us faster than a tuple)
        if returned and self.here is not None:
            t.record_stream(self.here)
        return t

    def __exit__(self, *exc):
        if self.switch is not None:
            self.switch.__exit__(*exc)


_plain = {}  # by device: the same for calls without a stream


def _memory(stream, dev):
    if stream is not None:
        return _Memory(stream, dev)
    if dev not in _plain:
        _plain[dev] = contextlib.nullcontext(
            lambda shape, dtype, returned=True: torch.empty(*shape, dtype=dtype, device=dev))
    return _plain[dev]


def choose_nsplit(B: int, T: int, H: int, K: int, sm_count: int = 0) -> int:
    return int(lib().smla_choose_nsplit(B, T, H, _k_in_range(K), sm_count))


def workspace_bytes(B: int, T: int, H: int, nsplit: int) -> int:
    return int(lib().smla_workspace_bytes(B, T, H, nsplit))


def _decode_args(q, cache, page_table, idx):
    _need(q, torch.bfloat16, "q")
    dev = q.device
    _need(cache, torch.bfloat16, "cache", dev)
    _need(page_table, torch.int32, "page_table", dev)
    _need(idx, torch.int32, "idx", dev)
    if q.dim() != 4 or q.shape[-1] != D:
        raise ValueError(f"q must be [B,T,H,{D}]")
    B, T, H, _ = q.shape
    if idx.dim() != 3 or tuple(idx.shape[:2]) != (B, T):
        raise ValueError("idx must be [B,T,K]")
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B, pt_stride]")
    if cache.numel() % (PAGE_SIZE * D):
        raise ValueError("cache must be [num_pages, 64, 576]")
    num_pages = cache.numel() // (PAGE_SIZE * D)
    return B, T, H, _k_in_range(idx.shape[2]), page_table.shape[1], num_pages


def decode_partial(q, cache, page_table, idx, scale: float, nsplit: int, *, part_o=None,
                   part_m=None, part_lse=None, stream=None):
    """Partial pass; returns (part_o [B,T,H,S,512], part_m [B,T,H,S], part_lse [B,T,H,S])."""
    B, T, H, K, pt_stride, num_pages = _decode_args(q, cache, page_table, idx)
    dev = q.device
    with _memory(stream, dev) as new:
        if part_o is None:
            part_o = new((B, T, H, nsplit, DC), torch.float32)
        if part_m is None:
            part_m = new((B, T, H, nsplit), torch.float32)
        if part_lse is None:
            part_lse = new((B, T, H, nsplit), torch.float32)
    _need(part_o, torch.float32, "part_o", dev, (B, T, H, nsplit, DC))
    _need(part_m, torch.float32, "part_m", dev, (B, T, H, nsplit))
    _need(part_lse, torch.float32, "part_lse", dev, (B, T, H, nsplit))
    _check(lib().smla_decode_partial(_ptr(q), _ptr(cache), num_pages, _ptr(page_table), pt_stride,
                                     _ptr(idx), B, T, H, K, PAGE_SIZE, float(scale), int(nsplit),
                                     _ptr(part_o), _ptr(part_m), _ptr(part_lse),
                                     _stream(stream)), "smla_decode_partial")
    return part_o, part_m, part_lse


def lse_combine(part_o, part_m, part_lse, *, o=None, lse=None, stream=None):
    """LSE combine; returns (o bf16 [B,T,H,512], lse fp32 [B,T,H])."""
    _need(part_m, torch.float32, "part_m")
    dev = part_m.device
    _need(part_o, torch.float32, "part_o", dev)
    _need(part_lse, torch.float32, "part_lse", dev)
    if part_m.dim() != 4:
        raise ValueError("part_m must be [B,T,H,S]")
    B, T, H, S = part_m.shape
    if tuple(part_o.shape) != (B, T, H, S, DC) or part_lse.shape != part_m.shape:
        raise ValueError("partial shapes disagree")
    with _memory(stream, dev) as new:
        if o is None:
            o = new((B, T, H, DC), torch.bfloat16)
        if lse is None:
            lse = new((B, T, H), torch.float32)
    _need(o, torch.bfloat16, "o", dev, (B, T, H, DC))
    _need(lse, torch.float32, "lse", dev, (B, T, H))
    _check(lib().smla_lse_combine(_ptr(part_o), _ptr(part_m), _ptr(part_lse), B, T, H, S, _ptr(o),
                                  _ptr(lse), _stream(stream)), "smla_lse_combine")
    return o, lse


def decode(q, cache, page_table, idx, scale: float, nsplit: int = 0, *, workspace=None,
           o=None, lse=None, stream=None):
    """Whole decode (partial + combine); returns (o bf16 [B,T,H,512], lse fp32 [B,T,H]).

    nsplit = 0 uses the library's heuristic.  A workspace (uint8 CUDA tensor)
    is allocated here when not given.
    """
    B, T, H, K, pt_stride, num_pages = _decode_args(q, cache, page_table, idx)
    dev = q.device
    if nsplit == 0:
        nsplit = choose_nsplit(B, T, H, K, 0)
    need = workspace_bytes(B, T, H, nsplit) if nsplit > 1 else 0
    with _memory(stream, dev) as new:
        if workspace is None:
            workspace = new((max(need, 16),), torch.uint8, returned=False)
        _need(workspace, torch.uint8, "workspace", dev)
        if o is None:
            o = new((B, T, H, DC), torch.bfloat16)
        if lse is None:
            lse = new((B, T, H), torch.float32)
    _need(o, torch.bfloat16, "o", dev, (B, T, H, DC))
    _need(lse, torch.float32, "lse", dev, (B, T, H))
    _check(lib().smla_decode(_ptr(q), _ptr(cache), num_pages, _ptr(page_table), pt_stride,
                             _ptr(idx), B, T, H, K, PAGE_SIZE, float(scale), int(nsplit),
                             _ptr(workspace), workspace.numel(), _ptr(o), _ptr(lse),
                             _stream(stream)), "smla_decode")
    return o, lse


def decode_noalloc(q, cache, page_table, idx, scale: float, nsplit: int = 0, *, o, lse,
                   stream=None):
    """Whole decode through smla_decode_noalloc: no workspace argument and no
    allocation anywhere (the split-K partials use the library's own device
    scratch array).  For callers that cannot allocate device memory while they
    decode, so o and lse must be given.  Calls that overlap on the GPU race on
    the shared scratch."""
    B, T, H, K, pt_stride, num_pages = _decode_args(q, cache, page_table, idx)
    _need(o, torch.bfloat16, "o", q.device, (B, T, H, DC))
    _need(lse, torch.float32, "lse", q.device, (B, T, H))
    _check(lib().smla_decode_noalloc(_ptr(q), _ptr(cache), num_pages, _ptr(page_table),
                                     pt_stride, _ptr(idx), B, T, H, K, PAGE_SIZE, float(scale),
                                     int(nsplit), _ptr(o), _ptr(lse), _stream(stream)),
           "smla_decode_noalloc")
    return o, lse


def dense_nsplit(B: int, T: int, H: int, K: int) -> int:
    return int(lib().smla_dense_nsplit(B, T, H, _k_in_range(K)))


def dense_workspace_bytes(B: int, T: int, H: int, K: int, nsplit: int) -> int:
    return int(lib().smla_dense_workspace_bytes(B, T, H, K, nsplit))


def _longest(seq_lens, stream) -> int:
    """The longest length, as it stands on the stream of the launch."""
    if not seq_lens.numel():
        return 0
    with torch.cuda.stream(_torch_stream(stream, seq_lens.device)):
        return int(seq_lens.max().item())


def _dense_args(q, cache, page_table, seq_lens, K, stream):
    _need(q, torch.bfloat16, "q")
    dev = q.device
    _need(cache, torch.bfloat16, "cache", dev)
    _need(page_table, torch.int32, "page_table", dev)
    _need(seq_lens, torch.int32, "seq_lens", dev)
    if q.dim() != 4 or q.shape[-1] != D:
        raise ValueError(f"q must be [B,T,H,{D}]")
    B, T, H, _ = q.shape
    if tuple(seq_lens.shape) != (B, T):
        raise ValueError("seq_lens must be [B,T]")
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B, pt_stride]")
    if cache.numel() % (PAGE_SIZE * D):
        raise ValueError("cache must be [num_pages, 64, 576]")
    if K is None:
        K = _longest(seq_lens, stream)
    return B, T, H, _k_in_range(int(K)), page_table.shape[1], cache.numel() // (PAGE_SIZE * D)


def decode_dense(q, cache, page_table, seq_lens, scale: float, nsplit: int = 0, *, K=None,
                 workspace=None, o=None, lse=None, stream=None):
    """Dense-context decode (KV-split verify): query token (b, t) attends to
    positions 0 .. seq_lens[b, t] - 1 of sequence b.  K defaults to the longest
    length (read from seq_lens, which synchronises); pass it to stay
    asynchronous.  Returns (o bf16 [B,T,H,512], lse fp32 [B,T,H])."""
    B, T, H, K, pt_stride, num_pages = _dense_args(q, cache, page_table, seq_lens, K, stream)
    dev = q.device
    if nsplit == 0:
        nsplit = dense_nsplit(B, T, H, K)
    need = dense_workspace_bytes(B, T, H, K, nsplit)
    with _memory(stream, dev) as new:
        if workspace is None:
            workspace = new((max(need, 16),), torch.uint8, returned=False)
        _need(workspace, torch.uint8, "workspace", dev)
        if o is None:
            o = new((B, T, H, DC), torch.bfloat16)
        if lse is None:
            lse = new((B, T, H), torch.float32)
    _need(o, torch.bfloat16, "o", dev, (B, T, H, DC))
    _need(lse, torch.float32, "lse", dev, (B, T, H))
    _check(lib().smla_decode_dense(_ptr(q), _ptr(cache), num_pages, _ptr(page_table), pt_stride,
                                   _ptr(seq_lens), B, T, H, K, PAGE_SIZE, float(scale),
                                   int(nsplit), _ptr(workspace), workspace.numel(), _ptr(o),
                                   _ptr(lse), _stream(stream)), "smla_decode_dense")
    return o, lse


def decode_dense_partial(q, cache, page_table, seq_lens, scale: float, nsplit: int, *, K=None,
                         part_o=None, part_m=None, part_lse=None, stream=None):
    """Partial pass of the dense variant; returns (part_o [B,T,H,S,512],
    part_m [B,T,H,S], part_lse [B,T,H,S])."""
    B, T, H, K, pt_stride, num_pages = _dense_args(q, cache, page_table, seq_lens, K, stream)
    dev = q.device
    with _memory(stream, dev) as new:
        if part_o is None:
            part_o = new((B, T, H, nsplit, DC), torch.float32)
        if part_m is None:
            part_m = new((B, T, H, nsplit), torch.float32)
        if part_lse is None:
            part_lse = new((B, T, H, nsplit), torch.float32)
    _need(part_o, torch.float32, "part_o", dev, (B, T, H, nsplit, DC))
    _need(part_m, torch.float32, "part_m", dev, (B, T, H, nsplit))
    _need(part_lse, torch.float32, "part_lse", dev, (B, T, H, nsplit))
    _check(lib().smla_decode_dense_partial(_ptr(q), _ptr(cache), num_pages, _ptr(page_table),
                                           pt_stride, _ptr(seq_lens), B, T, H, K, PAGE_SIZE,
                                           float(scale), int(nsplit), _ptr(part_o), _ptr(part_m),
                                           _ptr(part_lse), _stream(stream)),
           "smla_decode_dense_partial")
    return part_o, part_m, part_lse


def workspace_host_bytes(B: int, T: int, H: int, K: int, pt_stride: int, nsplit: int) -> int:
    return int(lib().smla_workspace_host_bytes(B, T, H, K, pt_stride, nsplit))


def decode_host(q, cache, page_table, idx, scale: float, nsplit: int = 0, *, o, lse,
                workspace=None, stream=None):
    """Whole decode through smla_decode_host: q, page_table, idx, o and lse are
    pinned CPU tensors (the per-step data of a host-driven decode loop), cache
    and workspace live on the GPU.  The inputs are pulled over the host link
    by a copy kernel and o, lse are written straight back into host memory;
    both are asynchronous on the stream (synchronise before reading o)."""
    for t, n, dt in ((q, "q", torch.bfloat16), (page_table, "page_table", torch.int32),
                     (idx, "idx", torch.int32), (o, "o", torch.bfloat16), (lse, "lse", torch.float32)):
        if not isinstance(t, torch.Tensor) or t.dtype != dt or not t.is_contiguous():
            raise TypeError(f"{n} must be a contiguous {dt} tensor")
        if t.is_cuda or not t.is_pinned():
            raise ValueError(f"{n} must be a pinned CPU tensor")
    _need(cache, torch.bfloat16, "cache")
    dev = cache.device
    if q.dim() != 4 or q.shape[-1] != D:
        raise ValueError(f"q must be [B,T,H,{D}]")
    B, T, H, _ = q.shape
    if idx.dim() != 3 or tuple(idx.shape[:2]) != (B, T):
        raise ValueError("idx must be [B,T,K]")
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B, pt_stride]")
    K, pt_stride = _k_in_range(idx.shape[2]), page_table.shape[1]
    if tuple(o.shape) != (B, T, H, DC) or tuple(lse.shape) != (B, T, H):
        raise ValueError(f"o must be [{B}, {T}, {H}, {DC}] and lse [{B}, {T}, {H}]")
    if cache.numel() % (PAGE_SIZE * D):
        raise ValueError("cache must be [num_pages, 64, 576]")
    num_pages = cache.numel() // (PAGE_SIZE * D)
    if nsplit == 0:
        nsplit = choose_nsplit(B, T, H, K, 0)
    need = workspace_host_bytes(B, T, H, K, pt_stride, nsplit)
    with _memory(stream, dev) as new:
        if workspace is None:
            workspace = new((max(need, 16),), torch.uint8, returned=False)
    _need(workspace, torch.uint8, "workspace", dev)
    _check(lib().smla_decode_host(_ptr(q), _ptr(cache), num_pages, _ptr(page_table), pt_stride,
                                  _ptr(idx), B, T, H, K, PAGE_SIZE, float(scale), int(nsplit),
                                  _ptr(workspace), workspace.numel(), _ptr(o), _ptr(lse),
                                  _stream(stream)), "smla_decode_host")
    return o, lse


INDEXER_DIM, INDEXER_MAX_HEADS, INDEXER_MAX_N = 128, 64, 524288


def indexer_workspace_bytes(B: int, T: int, max_n: int) -> int:
    return int(lib().smla_indexer_workspace_bytes(B, T, max_n))


def indexer_select_workspace_bytes(B: int, T: int, max_n: int) -> int:
    return int(lib().smla_indexer_select_workspace_bytes(B, T, max_n))


def _indexer_args(q_index, w, k_index, page_table, n_vis):
    _need(q_index, torch.bfloat16, "q_index")
    dev = q_index.device
    _need(w, torch.float32, "w", dev)
    _need(k_index, torch.bfloat16, "k_index", dev)
    _need(page_table, torch.int32, "page_table", dev)
    _need(n_vis, torch.int32, "n_vis", dev)
    if q_index.dim() != 4 or q_index.shape[-1] != INDEXER_DIM:
        raise ValueError(f"q_index must be [B,T,HI,{INDEXER_DIM}]")
    B, T, HI, _ = q_index.shape
    if tuple(w.shape) != (B, T, HI) or tuple(n_vis.shape) != (B, T):
        raise ValueError("w must be [B,T,HI] and n_vis [B,T]")
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B, pt_stride]")
    if k_index.numel() % (PAGE_SIZE * INDEXER_DIM):
        raise ValueError("k_index must be [num_pages, 64, 128]")
    return B, T, HI, page_table.shape[1], k_index.numel() // (PAGE_SIZE * INDEXER_DIM)


def indexer_topk(q_index, w, k_index, page_table, n_vis, K: int, max_n: int, *, out=None,
                 workspace=None, stream=None):
    """Top-k indexer: the min(K, n) positions with the largest index score
    per query token, ascending then -1 (int32 [B, T, K]).  max_n bounds
    n_vis (it sizes the work and the score buffer)."""
    B, T, HI, pt_stride, num_pages = _indexer_args(q_index, w, k_index, page_table, n_vis)
    dev = q_index.device
    K = _k_in_range(int(K))
    with _memory(stream, dev) as new:
        if out is None:
            out = new((B, T, K), torch.int32)
        _need(out, torch.int32, "out", dev, (B, T, K))
        if workspace is None:
            workspace = new((max(16, indexer_workspace_bytes(B, T, max_n)),), torch.uint8, returned=False)
    _need(workspace, torch.uint8, "workspace", dev)
    _check(lib().smla_indexer_topk(_ptr(q_index), _ptr(w), _ptr(k_index), num_pages,
                                   _ptr(page_table), pt_stride, _ptr(n_vis), B, T, HI, int(max_n),
                                   int(K), PAGE_SIZE, _ptr(workspace), workspace.numel(),
                                   _ptr(out), _stream(stream)), "smla_indexer_topk")
    return out


def indexer_scores(q_index, w, k_index, page_table, n_vis, max_n: int, *, scores=None,
                   workspace=None, stream=None):
    """Index scores fp32 [B, T, max_n] for every visible position (NaN where
    a position is not a candidate; entries past n_vis are not written)."""
    B, T, HI, pt_stride, num_pages = _indexer_args(q_index, w, k_index, page_table, n_vis)
    dev = q_index.device
    with _memory(stream, dev) as new:
        if scores is None:
            scores = new((B, T, max(max_n, 1)), torch.float32)
            scores.fill_(float("nan"))  # (on the launch's stream, as the allocation)
        # rows of max_n scores, one per query token (nothing is written when max_n is 0)
        _need(scores, torch.float32, "scores", dev, (B, T, max_n) if max_n > 0 else None)
        if workspace is None:
            workspace = new((max(16, indexer_workspace_bytes(B, T, 0)),), torch.uint8, returned=False)
    _need(workspace, torch.uint8, "workspace", dev)
    _check(lib().smla_indexer_scores(_ptr(q_index), _ptr(w), _ptr(k_index), num_pages,
                                     _ptr(page_table), pt_stride, _ptr(n_vis), B, T, HI,
                                     int(max_n), PAGE_SIZE, _ptr(workspace), workspace.numel(),
                                     _ptr(scores), _stream(stream)), "smla_indexer_scores")
    return scores


def indexer_select(scores, n_vis, K: int, *, out=None, workspace=None, stream=None):
    """The indexer's selection rule on given scores fp32 [B, T, max_n]."""
    _need(scores, torch.float32, "scores")
    dev = scores.device
    if scores.dim() != 3:
        raise ValueError("scores must be [B, T, max_n]")
    B, T, max_n = scores.shape
    _need(n_vis, torch.int32, "n_vis", dev, (B, T))
    K = _k_in_range(int(K))
    with _memory(stream, dev) as new:
        if out is None:
            out = new((B, T, K), torch.int32)
        _need(out, torch.int32, "out", dev, (B, T, K))
        if workspace is None:
            workspace = new((max(16, indexer_select_workspace_bytes(B, T, max_n)),), torch.uint8, returned=False)
    _need(workspace, torch.uint8, "workspace", dev)
    _check(lib().smla_indexer_select(_ptr(scores), _ptr(n_vis), B, T, max_n, int(K),
                                     _ptr(workspace), workspace.numel(), _ptr(out),
                                     _stream(stream)), "smla_indexer_select")
    return out


# ---------------------------------------------------------------- 4-bit latent cache
Q4_ROW_BYTES = 416


def _launch(name, dev, stream, *args):
    """Call an entry point with the tensors' device current, on ``stream`` or on
    that device's current stream."""
    if dev.index != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return _launch(name, dev, stream, *args)
    # the stream's handle alone: building a torch.cuda.Stream costs a few
    # microseconds, as much as the launch
    raw = torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else _stream(stream)
    status = getattr(lib(), name)(*args, raw)
    if status != 0:
        raise SmlaError(status, name)


def _want(t, dtype, name, device, shape=None):
    """_need() for a tensor that must be on ``device``, with the checks that pass
    in one expression (a CPU tensor's get_device() is -1); what fails is left to
    _need to name."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_contiguous()
            and (shape is None or t.shape == shape) and t.get_device() == device.index):
        _need(t, dtype, name, device, shape)
        _on_device(t, name, device)


def _paged(cache, width, dtype, dev, page_table, B):
    """Pages of a paged cache [num_pages, 64, width], and the page table's width."""
    _want(cache, dtype, "cache", dev)
    shape = cache.shape
    if len(shape) != 3 or shape[1] != PAGE_SIZE or shape[2] != width:
        raise ValueError(f"cache must be [num_pages, {PAGE_SIZE}, {width}], got {list(shape)}")
    return shape[0], _table(page_table, B, dev)


def _table(page_table, B, dev):
    _want(page_table, torch.int32, "page_table", dev)
    shape = page_table.shape
    if len(shape) != 2 or shape[0] != B:
        raise ValueError("page_table must be [B, pt_stride]")
    return shape[1]


def _dims(t, n, what):
    """Shape of a tensor of n dimensions."""
    shape = t.shape
    if len(shape) != n:
        raise ValueError(what)
    return shape


def q4_append(rows, cache, page_table, cu_rows, start, *, stream=None):
    """Quantise new latent rows into the 4-bit cache: rows [cu_rows[b],
    cu_rows[b + 1]) of ``rows`` (bf16 [N, 576]) go to positions start[b],
    start[b] + 1, ... of sequence b.  cache is uint8 [num_pages, 64, 416],
    cu_rows int32 [B + 1], start int32 [B]; rows at or behind cu_rows[B] are
    left out.  Writes into cache and returns it."""
    _need(rows, torch.bfloat16, "rows")
    dev = rows.device
    n, width = _dims(rows, 2, f"rows must be [N, {D}]")
    if width != D:
        raise ValueError(f"rows must be [N, {D}]")
    _want(start, torch.int32, "start", dev)
    B, = _dims(start, 1, "start must be [B]")
    _want(cu_rows, torch.int32, "cu_rows", dev, (B + 1,))
    num_pages, pt_stride = _paged(cache, Q4_ROW_BYTES, torch.uint8, dev, page_table, B)
    _launch("smla_q4_append", dev, stream, rows.data_ptr(), _k_in_range(n), cu_rows.data_ptr(),
            start.data_ptr(), B, cache.data_ptr(), num_pages, page_table.data_ptr(), pt_stride, PAGE_SIZE)
    return cache


def q4_read(cache, page_table, positions, *, out=None, stream=None):
    """Rows of the 4-bit cache as bf16 [B, K, 576]: entry (b, j) is position
    positions[b, j] of sequence b (int32 [B, K]; -1 gives zeros)."""
    _need(cache, torch.uint8, "cache")
    dev = cache.device
    _want(positions, torch.int32, "positions", dev)
    B, K = _dims(positions, 2, "positions must be [B, K]")
    num_pages, pt_stride = _paged(cache, Q4_ROW_BYTES, torch.uint8, dev, page_table, B)
    with _memory(stream, dev) as new:
        if out is None:
            out = new((B, K, D), torch.bfloat16)
        else:
            _want(out, torch.bfloat16, "out", dev, (B, K, D))
    _launch("smla_q4_read", dev, stream, cache.data_ptr(), num_pages, page_table.data_ptr(), pt_stride,
            positions.data_ptr(), B, _k_in_range(K), PAGE_SIZE, out.data_ptr())
    return out


def q4_nsplit(B: int, T: int, H: int, K: int) -> int:
    return int(lib().smla_q4_nsplit(B, T, H, _k_in_range(K)))


def q4_workspace_bytes(B: int, T: int, H: int, K: int, nsplit: int = 0) -> int:
    return int(lib().smla_q4_workspace_bytes(B, T, H, _k_in_range(K), nsplit))


def dense_q4_nsplit(B: int, T: int, H: int, K: int) -> int:
    return int(lib().smla_dense_q4_nsplit(B, T, H, _k_in_range(K)))


def dense_q4_workspace_bytes(B: int, T: int, H: int, K: int, nsplit: int = 0) -> int:
    return int(lib().smla_dense_q4_workspace_bytes(B, T, H, _k_in_range(K), nsplit))


def _queries(q):
    """Device and [B, T, H] of a decode's queries."""
    _need(q, torch.bfloat16, "q")
    B, T, H, width = _dims(q, 4, f"q must be [B,T,H,{D}]")
    if width != D:
        raise ValueError(f"q must be [B,T,H,{D}]")
    return q.device, B, T, H


def _decode_out(dev, B, T, H, need, workspace, o, lse, stream):
    """Workspace and outputs of a decode, allocated where they are not given."""
    with _memory(stream, dev) as new:
        if workspace is None:
            workspace = new((max(need, 16),), torch.uint8, returned=False)
        else:
            _want(workspace, torch.uint8, "workspace", dev)
        if o is None:
            o = new((B, T, H, DC), torch.bfloat16)
        else:
            _want(o, torch.bfloat16, "o", dev, (B, T, H, DC))
        if lse is None:
            lse = new((B, T, H), torch.float32)
        else:
            _want(lse, torch.float32, "lse", dev, (B, T, H))
    return workspace, o, lse


def decode_q4(q, cache, page_table, idx, scale: float, nsplit: int = 0, *, workspace=None, o=None,
              lse=None, stream=None):
    """decode() over a 4-bit cache (uint8 [num_pages, 64, 416], as q4_append
    writes it); returns (o bf16 [B,T,H,512], lse fp32 [B,T,H])."""
    dev, B, T, H = _queries(q)
    num_pages, pt_stride = _paged(cache, Q4_ROW_BYTES, torch.uint8, dev, page_table, B)
    _want(idx, torch.int32, "idx", dev)
    b, t, K = _dims(idx, 3, "idx must be [B,T,K]")
    if b != B or t != T:
        raise ValueError("idx must be [B,T,K]")
    nsplit = int(nsplit)
    need = q4_workspace_bytes(B, T, H, K, nsplit) if workspace is None else 0
    workspace, o, lse = _decode_out(dev, B, T, H, need, workspace, o, lse, stream)
    _launch("smla_decode_q4", dev, stream, q.data_ptr(), cache.data_ptr(), num_pages, page_table.data_ptr(),
            pt_stride, idx.data_ptr(), B, T, H, _k_in_range(K), PAGE_SIZE, float(scale), nsplit,
            workspace.data_ptr(), workspace.numel(), o.data_ptr(), lse.data_ptr())
    return o, lse


def decode_dense_q4(q, cache, page_table, seq_lens, scale: float, nsplit: int = 0, *, K=None,
                    workspace=None, o=None, lse=None, stream=None):
    """decode_dense() over a 4-bit cache: query token (b, t) attends to
    positions 0 .. seq_lens[b, t] - 1 of sequence b.  K defaults to the longest
    length (read from seq_lens, which synchronises)."""
    dev, B, T, H = _queries(q)
    num_pages, pt_stride = _paged(cache, Q4_ROW_BYTES, torch.uint8, dev, page_table, B)
    _want(seq_lens, torch.int32, "seq_lens", dev, (B, T))
    if K is None:
        K = _longest(seq_lens, stream)
    K = _k_in_range(int(K))
    nsplit = int(nsplit)
    need = dense_q4_workspace_bytes(B, T, H, K, nsplit) if workspace is None else 0
    workspace, o, lse = _decode_out(dev, B, T, H, need, workspace, o, lse, stream)
    _launch("smla_decode_dense_q4", dev, stream, q.data_ptr(), cache.data_ptr(), num_pages,
            page_table.data_ptr(), pt_stride, seq_lens.data_ptr(), B, T, H, K, PAGE_SIZE, float(scale), nsplit,
            workspace.data_ptr(), workspace.numel(), o.data_ptr(), lse.data_ptr())
    return o, lse


# ---------------------------------------------------------------- eviction
EVICT_MAX_N, EVICT_MAX_CACHES, EVICT_MAX_ROW_BYTES = 524288, 4, 65536


class EvictPlan(NamedTuple):
    """What evict_plan returns: src int32 [B, K] (slot i takes the row of slot
    src[b, i]; -1 past the end), n int32 [B] (slots in use afterwards), acc and
    pos [B, max_n] carried along."""
    src: torch.Tensor
    n: torch.Tensor
    acc: torch.Tensor
    pos: torch.Tensor


def evict_workspace_bytes(B: int, max_n: int) -> int:
    return int(lib().smla_evict_workspace_bytes(B, max_n))


def evict_accumulate(q, cache, page_table, seq_lens, lse, scale: float, acc, *, stream=None):
    """Add to acc (fp32 [B, max_n], in place) the attention weight that the
    query tokens of a dense decode gave to each position: q, seq_lens and lse
    are that decode's.  cache is the bf16 or the 4-bit latent cache.  Returns
    acc."""
    dev, B, T, H = _queries(q)
    q4 = isinstance(cache, torch.Tensor) and cache.dtype is torch.uint8
    num_pages, pt_stride = _paged(cache, Q4_ROW_BYTES if q4 else D, torch.uint8 if q4 else torch.bfloat16, dev,
                                  page_table, B)
    _want(seq_lens, torch.int32, "seq_lens", dev, (B, T))
    _want(lse, torch.float32, "lse", dev, (B, T, H))
    _want(acc, torch.float32, "acc", dev)
    b, max_n = _dims(acc, 2, "acc must be [B, max_n]")
    if b != B:
        raise ValueError("acc must be [B, max_n]")
    _launch("smla_evict_accumulate_q4" if q4 else "smla_evict_accumulate", dev, stream, q.data_ptr(),
            cache.data_ptr(), num_pages, page_table.data_ptr(), pt_stride, seq_lens.data_ptr(), lse.data_ptr(),
            B, T, H, PAGE_SIZE, float(scale), acc.data_ptr(), _k_in_range(max_n))
    return acc


def evict_plan(acc, n, K: int, *, pos=None, n_sink: int = 0, n_recent: int = 0, src=None, n_new=None,
               acc_new=None, pos_new=None, stream=None) -> EvictPlan:
    """Choose the min(n[b], K) slots of each sequence that stay, by accumulated
    weight acc (fp32 [B, max_n]), and which row each slot takes.  pos (int32
    [B, max_n], default: the slot's number) is the token's original position:
    the first n_sink and the last n_recent always stay.  acc and pos come back
    carried along to the new slots; the inputs are left as they are."""
    _need(acc, torch.float32, "acc")
    dev = acc.device
    B, max_n = _dims(acc, 2, "acc must be [B, max_n]")
    K, n_sink, n_recent = _k_in_range(int(K)), _k_in_range(int(n_sink)), _k_in_range(int(n_recent))
    if K < 1:
        raise ValueError("K must be at least 1")
    _want(n, torch.int32, "n", dev, (B,))
    if pos is not None:
        _want(pos, torch.int32, "pos", dev, (B, max_n))
    with _memory(stream, dev) as new:
        if src is None:
            src = new((B, K), torch.int32)
        else:
            _want(src, torch.int32, "src", dev, (B, K))
        if n_new is None:
            n_new = new((B,), torch.int32)
        else:
            _want(n_new, torch.int32, "n_new", dev, (B,))
        if acc_new is None:
            acc_new = new((B, max_n), torch.float32)
        else:
            _want(acc_new, torch.float32, "acc_new", dev, (B, max_n))
        if pos_new is None:
            pos_new = new((B, max_n), torch.int32)
        else:
            _want(pos_new, torch.int32, "pos_new", dev, (B, max_n))
    _launch("smla_evict_plan", dev, stream, acc.data_ptr(), None if pos is None else pos.data_ptr(),
            n.data_ptr(), B, max_n, K, n_sink, n_recent, None, 0, src.data_ptr(), n_new.data_ptr(),
            acc_new.data_ptr(), pos_new.data_ptr())
    return EvictPlan(src, n_new, acc_new, pos_new)


def evict_apply(src, page_table, caches, *, stream=None):
    """Move the rows of a plan, in place, in every paged buffer of ``caches``
    (contiguous CUDA tensors [num_pages, 64, W] of any dtype, rows of a
    multiple of 16 bytes, one page table for all): the bf16 or 4-bit latent
    cache, the index keys.  Returns caches."""
    _need(src, torch.int32, "src")
    dev = src.device
    B, K = _dims(src, 2, "src must be [B, K]")
    pt_stride = _table(page_table, B, dev)
    if not 1 <= len(caches) <= EVICT_MAX_CACHES:
        raise ValueError(f"caches must be 1 to {EVICT_MAX_CACHES} tensors")
    ptrs, sizes, num_pages = [], [], None
    for t in caches:
        if not isinstance(t, torch.Tensor):
            raise TypeError("caches must be torch.Tensors")
        _want(t, t.dtype, "a cache", dev)
        shape = t.shape
        if len(shape) != 3 or shape[1] != PAGE_SIZE or num_pages not in (None, shape[0]):
            raise ValueError(f"caches must be [num_pages, {PAGE_SIZE}, width], the same pages in all")
        num_pages = shape[0]
        ptrs.append(t.data_ptr())
        sizes.append(shape[2] * t.element_size())
    n = len(ptrs)
    _launch("smla_evict_apply", dev, stream, src.data_ptr(), B, _k_in_range(K), page_table.data_ptr(), pt_stride,
            num_pages, PAGE_SIZE, (_P * n)(*ptrs), (ctypes.c_int32 * n)(*sizes), n)
    return caches


def check_device(clear: bool = True, stream=None):
    """Synchronise and read the sticky device status: (status, n_bad_index)."""
    n = ctypes.c_ulonglong(0)
    st = lib().smla_check_device(1 if clear else 0, ctypes.byref(n), _stream(stream))
    return int(st), int(n.value)


def selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    """Launch the bounded-wait self-test: one warp waits on a barrier that
    nothing arrives at and gives up after limit_ns, raising the timeout flag
    that check_device() then reports."""
    _check(lib().smla_selftest_wait_timeout(int(limit_ns), _stream(stream)),
           "smla_selftest_wait_timeout")


def status_string(status: int) -> str:
    return lib().smla_status_string(status).decode()
