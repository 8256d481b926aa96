"""Exact tiled attention forward for one NVIDIA GB300 (sm_103a).

A thin Python binding over the C ABI of ``libattn.so`` (declared in
``include/attn.h``): the functions here only check and marshal arguments;
every step of the computation runs in the library's CUDA kernels.  PyTorch
provides device memory and streams.  If the library has not been built the
import fails loudly; there is no CPU or PyTorch fallback.

    attn_fwd(q, k, v, causal=False, scale=None, Br=0, Bc=0, key_mask=None)
        -> (o, lse)          tiled exact forward (bf16 on tcgen05, or fp32 SIMT)
    attn_naive_fwd(...)      materialising baseline (S and P in the input dtype)
    attn_deviation(a, b)     max-abs, Wasserstein-1 (via sort), mean/std |a-b|

A paged key/value cache (``PagedCache``), of bf16, float32 or 4-bit values: pages
are handed out, shared and released on the device by attn_cache_reserve / _free /
_fork / _compact; new tokens are written by attn_cache_append, or with the position
rotation by attn_cache_append_rotated, attended to by attn_paged_fwd and copied out
by attn_cache_read.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libattn.so")

ATTN_F32, ATTN_BF16, ATTN_F64, ATTN_E2M1 = 0, 1, 2, 3
ATTN_OK = 0
ATTN_ERR_ARG = -1
ATTN_ERR_UNSUPPORTED = -2
ATTN_ERR_WORKSPACE = -3
ATTN_ERR_CUDA = -4
ATTN_ERR_DEVICE_TIMEOUT = -5

# Every symbol include/attn.h declares.
EXPORTS = ("attn_fwd", "attn_fwd_host_workspace_size", "attn_fwd_host", "attn_fwd_block_sparse", "attn_naive_workspace_size", "attn_naive_fwd", "attn_deviation_workspace_size",
           "attn_deviation", "attn_deviation_noalloc", "attn_decode_workspace_size", "attn_decode_fwd",
           "attn_cache_workspace_size", "attn_cache_reserve", "attn_cache_free", "attn_cache_fork", "attn_cache_compact",
           "attn_cache_append", "attn_cache_append_granted", "attn_paged_workspace_size", "attn_paged_fwd",
           "attn_paged_fwd_granted", "attn_cache_append_rotated", "attn_cache_read",
           "attn_bwd_workspace_size", "attn_bwd", "attn_emul_fwd", "attn_emul_round", "attn_status",
           "attn_strerror", "attn_last_variant", "attn_debug_wait_timeout")
DEVIATION_NOALLOC_MAX_N = 1 << 20

_DTYPE = {torch.float32: ATTN_F32, torch.bfloat16: ATTN_BF16, torch.float64: ATTN_F64}
_E2M1 = getattr(torch, "float4_e2m1fn_x2", object())   # (a torch without the type: equal to none, and calls with other types work)


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {strerror(status)} ({status})")
        self.status = status


class DevT(ctypes.Structure):
    _fields_ = [("max_abs", ctypes.c_double), ("w1", ctypes.c_double), ("mean_abs", ctypes.c_double),
                ("std_abs", ctypes.c_double), ("mean_signed", ctypes.c_double), ("n", ctypes.c_longlong)]


class CacheT(ctypes.Structure):
    """attn_cache_t"""
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("ref_counts", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("layers", ctypes.c_int), ("pages", ctypes.c_int), ("heads", ctypes.c_int), ("page_size", ctypes.c_int),
                ("d", ctypes.c_int), ("seqs", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("layer_stride", ctypes.c_longlong), ("page_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong), ("slot_stride", ctypes.c_longlong)]


class RotationT(ctypes.Structure):
    """attn_rotation_t"""
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("rows", ctypes.c_int), ("dims", ctypes.c_int),
                ("neighbours", ctypes.c_int)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built: run `python -c 'import __graft_entry__ as g; g.build()'` "
                          "(the CUDA library is required; there is no fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, f, sz, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
    lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, i, vp, vp]
    lib.attn_fwd_block_sparse.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, vp, vp]
    lib.attn_fwd_block_sparse.restype = i
    lib.attn_fwd.restype = i
    lib.attn_fwd_host_workspace_size.argtypes = [i, i, i, i, i, i]
    lib.attn_fwd_host_workspace_size.restype = sz
    lib.attn_fwd_host.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, i, vp, vp, sz, vp]
    lib.attn_fwd_host.restype = i
    lib.attn_naive_workspace_size.argtypes = [i, i, i, i]
    lib.attn_naive_workspace_size.restype = sz
    lib.attn_naive_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, vp, sz, vp]
    lib.attn_naive_fwd.restype = i
    lib.attn_deviation_workspace_size.argtypes = [ll]
    lib.attn_deviation_workspace_size.restype = sz
    lib.attn_deviation.argtypes = [vp, i, vp, i, ll, vp, sz, vp, ctypes.POINTER(DevT)]
    lib.attn_deviation.restype = i
    lib.attn_deviation_noalloc.argtypes = [vp, i, vp, i, ll, vp, ctypes.POINTER(DevT)]
    lib.attn_deviation_noalloc.restype = i
    lib.attn_decode_workspace_size.argtypes = [i, i, i, i]
    lib.attn_decode_workspace_size.restype = sz
    lib.attn_decode_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, vp, sz, vp]
    lib.attn_decode_fwd.restype = i
    cp = ctypes.POINTER(CacheT)
    lib.attn_cache_workspace_size.argtypes = [i, i]
    lib.attn_cache_workspace_size.restype = sz
    lib.attn_cache_reserve.argtypes = [cp, vp, vp, i, vp, vp, sz, vp]
    lib.attn_cache_reserve.restype = i
    lib.attn_cache_free.argtypes = [cp, vp, vp, i, vp]
    lib.attn_cache_free.restype = i
    lib.attn_cache_fork.argtypes = [cp, vp, vp, i, i, vp, vp, sz, vp]
    lib.attn_cache_fork.restype = i
    lib.attn_cache_compact.argtypes = [cp, vp, vp, vp, vp, sz, vp]
    lib.attn_cache_compact.restype = i
    lib.attn_cache_append.argtypes = [cp, i, vp, vp, ll, ll, i, vp, vp, i, vp]
    lib.attn_cache_append.restype = i
    lib.attn_cache_append_granted.argtypes = [cp, i, vp, vp, ll, ll, i, vp, vp, vp, i, vp]
    lib.attn_cache_append_granted.restype = i
    lib.attn_paged_workspace_size.argtypes = [i, i, i, i, i]
    lib.attn_paged_workspace_size.restype = sz
    lib.attn_paged_fwd.argtypes = [cp, i, vp, vp, vp, ll, ll, ll, ll, i, i, vp, vp, i, i, i, f, vp, sz, vp]
    lib.attn_paged_fwd.restype = i
    lib.attn_paged_fwd_granted.argtypes = [cp, i, vp, vp, vp, ll, ll, ll, ll, i, i, vp, vp, vp, i, i, i, f, vp, sz, vp]
    lib.attn_paged_fwd_granted.restype = i
    lib.attn_cache_append_rotated.argtypes = [cp, i, vp, vp, ll, ll, vp, vp, i, ll, ll, ll, ll, i, vp, vp, vp, i,
                                              ctypes.POINTER(RotationT), vp]
    lib.attn_cache_append_rotated.restype = i
    lib.attn_cache_read.argtypes = [cp, i, vp, vp, ll, ll, i, vp, vp, vp, i, vp]
    lib.attn_cache_read.restype = i
    lib.attn_bwd_workspace_size.argtypes = [i, i, i, i]
    lib.attn_bwd_workspace_size.restype = sz
    lib.attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, vp, sz, vp]
    lib.attn_bwd.restype = i
    lib.attn_emul_fwd.argtypes = [vp, vp, vp, i, vp, i, i, i, i, i, f, vp, i, i, i, i, vp, ll, vp]
    lib.attn_emul_fwd.restype = i
    lib.attn_emul_round.argtypes = [vp, vp, ll, i, i, vp]
    lib.attn_emul_round.restype = i
    lib.attn_status.argtypes = [vp]
    lib.attn_status.restype = i
    lib.attn_strerror.argtypes = [i]
    lib.attn_strerror.restype = ctypes.c_char_p
    lib.attn_last_variant.argtypes = [ctypes.c_char_p, i]
    lib.attn_last_variant.restype = i
    lib.attn_debug_wait_timeout.argtypes = [ctypes.c_uint, vp]
    lib.attn_debug_wait_timeout.restype = i
    return lib


lib = _load()


def strerror(status: int) -> str:
    return lib.attn_strerror(int(status)).decode()


def _check(rc: int, what: str) -> None:
    if rc != ATTN_OK:
        raise AttnError(rc, what)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _shape4(q):
    if q.dim() == 4:
        return q.shape
    if q.dim() == 3:
        return (1,) + tuple(q.shape)
    raise ValueError("q, k, v must be [B, H, N, d] or [H, N, d]")


BLOCK_SPARSE_BLOCK = 128
BLOCK_SPARSE_MAX_N = 131072


def attn_fwd_block_sparse(q, k, v, block_mask, causal: bool = False, scale: float | None = None, key_mask=None,
                          out=None, lse=None, stream=None, want_lse: bool = True):
    """Forward restricted to the marked 128 x 128 blocks.  block_mask: [B, H,
    nb, nb] uint8 (or bool) device tensor, nb = ceil(N / 128), non-zero = the
    block takes part.  Returns (o, lse)."""
    for t in (q, k, v):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous device tensors")
    if not (q.shape == k.shape == v.shape and q.dtype == k.dtype == v.dtype):
        raise ValueError("q, k, v must share shape and dtype")
    B, H, N, d = _shape4(q)
    nb = -(-N // BLOCK_SPARSE_BLOCK)
    if block_mask.dtype == torch.bool:
        block_mask = block_mask.to(torch.uint8)
    if (block_mask.dtype != torch.uint8 or not block_mask.is_cuda or not block_mask.is_contiguous()
            or block_mask.numel() != B * H * nb * nb):
        raise ValueError("block_mask must be a contiguous uint8 device tensor with B*H*nb*nb elements")
    if q.dtype not in _DTYPE:
        raise ValueError(f"unsupported dtype {q.dtype}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = out if out is not None else torch.empty_like(q)
    l = lse if lse is not None else (torch.empty((B, H, N), dtype=torch.float32, device=q.device)
                                     if want_lse else None)
    m = None
    if key_mask is not None:
        m = key_mask
        if m.dtype != torch.float32 or not m.is_contiguous() or m.numel() != B * H * N or not m.is_cuda:
            raise ValueError("key_mask must be a contiguous float32 device tensor with B*H*N elements")
    rc = lib.attn_fwd_block_sparse(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, H, N, d, int(bool(causal)),
                                   float(scale), _DTYPE[q.dtype], _ptr(block_mask), _ptr(m),
                                   ctypes.c_void_p(_stream(stream)))
    _check(rc, "attn_fwd_block_sparse")
    return o, l


def attn_fwd_host_workspace_size(B: int, H: int, N: int, d: int, dtype, with_mask: bool = False) -> int:
    return int(lib.attn_fwd_host_workspace_size(B, H, N, d, _DTYPE[dtype] if not isinstance(dtype, int) else dtype,
                                                int(bool(with_mask))))


def _attn_fwd_host(q, k, v, causal, scale, Br, Bc, key_mask, out, lse, stream, want_lse, sync, workspace):
    """attn_fwd on host tensors through the C ABI's attn_fwd_host: the library
    copies the inputs into a device workspace, runs the forward and copies O
    and LSE back, all on `stream`."""
    for t in (q, k, v):
        if t.device.type != "cpu" or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous host tensors")
    if not (q.shape == k.shape == v.shape and q.dtype == k.dtype == v.dtype) or q.dtype not in _DTYPE:
        raise ValueError("q, k, v must share shape and a supported dtype")
    B, H, N, d = _shape4(q)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    st = stream if stream is not None else torch.cuda.current_stream()
    if not isinstance(st, torch.cuda.Stream):
        st = torch.cuda.ExternalStream(int(st))
    m = None
    if key_mask is not None:
        m = key_mask
        if m.device.type != "cpu" or m.dtype != torch.float32 or not m.is_contiguous() or m.numel() != B * H * N:
            raise ValueError("key_mask must be a contiguous float32 host tensor with B*H*N elements")
    need = attn_fwd_host_workspace_size(B, H, N, d, q.dtype, m is not None)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", torch.cuda.current_device()))
        workspace.record_stream(st)
    ho = out if out is not None else torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
    hl = lse if lse is not None else (torch.empty((B, H, N), dtype=torch.float32, pin_memory=True)
                                      if want_lse else None)
    for t in (ho,) + ((hl,) if hl is not None else ()):
        if t.device.type != "cpu" or not t.is_contiguous():
            raise ValueError("out / lse must be contiguous host tensors")
    rc = lib.attn_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(ho), _ptr(hl), B, H, N, d, int(bool(causal)), float(scale),
                           int(Br), int(Bc), _DTYPE[q.dtype], _ptr(m), _ptr(workspace), workspace.numel(),
                           ctypes.c_void_p(st.cuda_stream))
    _check(rc, "attn_fwd_host")
    if sync:
        st.synchronize()
    return ho, hl


def attn_fwd(q, k, v, causal: bool = False, scale: float | None = None, Br: int = 0, Bc: int = 0,
             key_mask=None, out=None, lse=None, stream=None, want_lse: bool = True, sync: bool = True,
             workspace=None):
    """Tiled exact attention forward.  Returns (o, lse).

    Device tensors: the call is enqueued on `stream` (default: torch's current
    stream) and returns immediately.  Host tensors (pinned or not): the C ABI's
    attn_fwd_host copies the inputs into a device workspace (``workspace``, a
    uint8 device tensor of attn_fwd_host_workspace_size bytes, allocated here
    if not given), runs the kernel and copies o / lse back into host tensors,
    all on `stream`; with sync=False the call returns once that work is
    enqueued (o / lse are valid after the stream is synchronised), so calls on
    two streams overlap one's copies with the other's kernel.
    """
    if q.device.type == "cpu":
        return _attn_fwd_host(q, k, v, causal, scale, Br, Bc, key_mask, out, lse, stream, want_lse, sync, workspace)
    for t in (q, k, v):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous tensors on one device")
    if not (q.shape == k.shape == v.shape and q.dtype == k.dtype == v.dtype):
        raise ValueError("q, k, v must share shape and dtype")
    B, H, N, d = _shape4(q)
    if q.dtype not in _DTYPE:
        raise ValueError(f"unsupported dtype {q.dtype}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = out if out is not None else torch.empty_like(q)
    l = lse if lse is not None else (torch.empty((B, H, N), dtype=torch.float32, device=q.device)
                                     if want_lse else None)
    m = None
    if key_mask is not None:
        m = key_mask
        if m.dtype != torch.float32 or not m.is_contiguous() or m.numel() != B * H * N or not m.is_cuda:
            raise ValueError("key_mask must be a contiguous float32 device tensor with B*H*N elements")
    rc = lib.attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, H, N, d, int(bool(causal)),
                      float(scale), int(Br), int(Bc), _DTYPE[q.dtype], _ptr(m), ctypes.c_void_p(_stream(stream)))
    _check(rc, "attn_fwd")
    return o, l


def attn_naive_workspace_size(B: int, H: int, N: int, dtype) -> int:
    return int(lib.attn_naive_workspace_size(B, H, N, _DTYPE[dtype] if not isinstance(dtype, int) else dtype))


def attn_naive_fwd(q, k, v, causal: bool = False, scale: float | None = None, key_mask=None, workspace=None,
                   stream=None, out=None, lse=None):
    """Materialising baseline.  Returns (o, lse).  Allocates its workspace
    (uint8 device tensor) and outputs with torch unless they are passed."""
    B, H, N, d = _shape4(q)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = attn_naive_workspace_size(B, H, N, q.dtype)
    ws = workspace if workspace is not None else torch.empty(need, dtype=torch.uint8, device=q.device)
    o = out if out is not None else torch.empty_like(q)
    l = lse if lse is not None else torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    rc = lib.attn_naive_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, H, N, d, int(bool(causal)),
                            float(scale), _DTYPE[q.dtype], _ptr(key_mask), _ptr(ws), ws.numel(),
                            ctypes.c_void_p(_stream(stream)))
    _check(rc, "attn_naive_fwd")
    return o, l


def attn_deviation_workspace_size(n: int) -> int:
    return int(lib.attn_deviation_workspace_size(int(n)))


def _same_device(a, b):
    if a.numel() != b.numel():
        raise ValueError("a and b must have the same number of elements")
    if not (a.is_cuda and b.is_cuda) or a.device != b.device:
        raise ValueError("a and b must be tensors on one CUDA device")


def attn_deviation(a, b, workspace=None, stream=None) -> dict:
    """Deviation between two device tensors of equal size (synchronous)."""
    _same_device(a, b)
    a = a.contiguous()
    b = b.contiguous()
    n = a.numel()
    with torch.cuda.device(a.device):   # the library launches on the current device
        ws = workspace if workspace is not None else torch.empty(attn_deviation_workspace_size(n),
                                                                 dtype=torch.uint8, device=a.device)
        if not ws.is_cuda or ws.device != a.device:
            raise ValueError("workspace must be on the tensors' device")
        res = DevT()
        rc = lib.attn_deviation(_ptr(a), _DTYPE[a.dtype], _ptr(b), _DTYPE[b.dtype], n, _ptr(ws), ws.numel(),
                                ctypes.c_void_p(_stream(stream)), ctypes.byref(res))
    _check(rc, "attn_deviation")
    return {"max_abs": res.max_abs, "w1": res.w1, "mean_abs": res.mean_abs, "std_abs": res.std_abs,
            "mean_signed": res.mean_signed, "n": res.n}


def attn_deviation_noalloc(a, b, stream=None) -> dict:
    """attn_deviation without a workspace, for callers that cannot allocate
    device memory (the library's own fixed scratch array is used instead;
    n <= DEVIATION_NOALLOC_MAX_N; calls that overlap on the GPU race)."""
    _same_device(a, b)
    a = a.contiguous()
    b = b.contiguous()
    res = DevT()
    with torch.cuda.device(a.device):   # the scratch array and the launch follow the current device
        rc = lib.attn_deviation_noalloc(_ptr(a), _DTYPE[a.dtype], _ptr(b), _DTYPE[b.dtype], a.numel(),
                                        ctypes.c_void_p(_stream(stream)), ctypes.byref(res))
    _check(rc, "attn_deviation_noalloc")
    return {"max_abs": res.max_abs, "w1": res.w1, "mean_abs": res.mean_abs, "std_abs": res.std_abs,
            "mean_signed": res.mean_signed, "n": res.n}


DECODE_MAX_NQ = 8


def attn_decode_workspace_size(B: int, H: int, Nq: int, d: int) -> int:
    return int(lib.attn_decode_workspace_size(B, H, Nq, d))


def attn_decode_fwd(q, k, v, causal: bool = False, scale: float | None = None, key_mask=None, out=None, lse=None,
                    workspace=None, stream=None, want_lse: bool = True):
    """Decode with a key/value cache.  q: [B, H, Nq, d]; k, v: [B, H, Nk, d]
    contiguous device tensors of one dtype (bfloat16 or float32).  Causal:
    query row i is the token at position Nk - Nq + i.  Returns (o, lse)."""
    for t in (q, k, v):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous device tensors")
    if k.shape != v.shape or q.dtype != k.dtype or q.dtype != v.dtype:
        raise ValueError("k and v must share a shape, and q, k, v a dtype")
    B, H, Nq, d = _shape4(q)
    Bk, Hk, Nk, dk = _shape4(k)
    if (Bk, Hk, dk) != (B, H, d):
        raise ValueError("q and k/v disagree on B, H or d")
    if q.dtype not in _DTYPE:
        raise ValueError(f"unsupported dtype {q.dtype}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = out if out is not None else torch.empty_like(q)
    l = lse if lse is not None else (torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
                                     if want_lse else None)
    need = attn_decode_workspace_size(B, H, Nq, d)
    ws = workspace if workspace is not None else torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    m = None
    if key_mask is not None:
        m = key_mask
        if m.dtype != torch.float32 or not m.is_contiguous() or m.numel() != B * H * Nk or not m.is_cuda:
            raise ValueError("key_mask must be a contiguous float32 device tensor with B*H*Nk elements")
    rc = lib.attn_decode_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, H, Nq, Nk, d, int(bool(causal)),
                             float(scale), _DTYPE[q.dtype], _ptr(m), _ptr(ws), ws.numel(),
                             ctypes.c_void_p(_stream(stream)))
    _check(rc, "attn_decode_fwd")
    return o, l


# ---------------------------------------------------------------------------
# paged key/value cache
# ---------------------------------------------------------------------------
class PagedCache:
    """A paged key/value cache over the caller's device tensors (attn_cache_t).

    k, v: pools of pages, [layers, pages, heads, page_size, d], bfloat16 or
    float32, with equal strides; a page of one layer is one contiguous block,
    head by head (a contiguous tensor) or token by token (a tensor of
    [layers, pages, page_size, heads, d] seen through transpose(2, 3)).
    Or uint8, [layers, pages, heads, page_size, 9 * d / 16], head by head: a
    cache of 4-bit values.  The last two dimensions are one run of bytes, first
    the codes, page_size x d / 2, then the scales, page_size x d / 16 (views of
    both: ``parts``); what goes in and out of the cache is bfloat16.
    page_table: int32 [seqs, max_pages], -1 where a sequence has no page;
    seq_lens: int32 [seqs]; ref_counts: int32 [pages].  The object keeps the
    tensors; all are changed in place by the operators below.  dtype is that of
    rows that go in and out.
    """

    def __init__(self, k, v, page_table, seq_lens, ref_counts):
        if k.dim() != 5 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v must be [layers, pages, heads, page_size, d] with one shape, dtype and strides")
        four = k.dtype == torch.uint8
        if k.dtype not in _DTYPE and not four:
            raise ValueError(f"unsupported dtype {k.dtype}")
        if k.shape[4] > 1 and k.stride(4) != 1:
            raise ValueError("the last dimension of k and v must be contiguous")
        layers, pages, heads, page_size, d = k.shape
        slot_stride = k.stride(3)
        if four:
            if d % 18 or (page_size > 1 and slot_stride != d):
                raise ValueError("k and v of 4-bit values must be [layers, pages, heads, page_size, 9 * d / 16] bytes, "
                                 "the last two dimensions contiguous")
            d = d // 9 * 16
            slot_stride = d // 2
        for t, shape, name in ((page_table, 2, "page_table [seqs, max_pages]"), (seq_lens, 1, "seq_lens [seqs]"),
                               (ref_counts, 1, "ref_counts [pages]")):
            if t.dtype != torch.int32 or t.dim() != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 tensor")
        if seq_lens.shape[0] != page_table.shape[0] or ref_counts.shape[0] != pages:
            raise ValueError("page_table, seq_lens and ref_counts do not fit each other or the pools")
        for t in (k, v, page_table, seq_lens, ref_counts):
            if not t.is_cuda or t.device != k.device:
                raise ValueError("the tensors of a cache must be on one CUDA device")
        self.k, self.v, self.page_table, self.seq_lens, self.ref_counts = k, v, page_table, seq_lens, ref_counts
        self.device, self.dtype = k.device, torch.bfloat16 if four else k.dtype
        self.layers, self.pages, self.heads, self.page_size, self.d = layers, pages, heads, page_size, d
        self.seqs, self.max_pages = page_table.shape
        self._index = k.get_device()
        self._scale = 1.0 / math.sqrt(d)
        self._code = ATTN_E2M1 if four else _DTYPE[k.dtype]
        self._spaces = threading.local()   # workspaces of calls that bring none (_paged_workspace)
        self._c = CacheT(k.data_ptr(), v.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), ref_counts.data_ptr(),
                         self._code, layers, pages, heads, page_size, d, self.seqs, self.max_pages, k.stride(0),
                         k.stride(1), k.stride(2), slot_stride)
        self._p = ctypes.pointer(self._c)

    def parts(self, pool):
        """Views of a pool (``k`` or ``v``) of 4-bit values: codes [layers, pages,
        heads, page_size, d / 2], two columns to a byte, and scales [layers, pages,
        heads, page_size, d / 16], uint8."""
        if self._code != ATTN_E2M1:
            raise ValueError("only a cache of 4-bit values has codes and scales")
        block, S, d = pool.flatten(3), self.page_size, self.d
        return (block[..., :S * d // 2].unflatten(3, (S, d // 2)), block[..., S * d // 2:].unflatten(3, (S, d // 16)))

    @classmethod
    def empty(cls, layers: int, pages: int, heads: int, page_size: int, d: int, seqs: int, max_pages: int,
              dtype=torch.bfloat16, device="cuda", token_major: bool = False):
        """A new cache without sequences.  dtype: bfloat16, float32, or
        torch.float4_e2m1fn_x2 for 4-bit values.  token_major: pages lie token by
        token instead of head by head."""
        if dtype == _E2M1:
            if token_major or d % 32:
                raise ValueError("pages of 4-bit values lie head by head, with d a multiple of 32")
            dtype, d = torch.uint8, 9 * d // 16

        def pool():
            if token_major:
                return torch.empty((layers, pages, page_size, heads, d), dtype=dtype, device=device).transpose(2, 3)
            return torch.empty((layers, pages, heads, page_size, d), dtype=dtype, device=device)

        def ints(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=device)
        return cls(pool(), pool(), ints(seqs, max_pages) - 1, ints(seqs), ints(pages))


# The current device's index, and the raw handle of a device's current stream:
# torch's own binding functions where they exist (the public ones cost several
# microseconds a call, which is what a decode step is made of).
_device_index = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _paged_list(t, cache, name, n=None):
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.get_device() != cache._index:
        raise ValueError(f"{name} must be a contiguous int32 vector on the cache's device")
    if n is not None and t.shape[0] != n:
        raise ValueError(f"{name} must have {n} elements")
    return t.data_ptr()


_lib_reserve, _lib_free, _lib_fork = lib.attn_cache_reserve, lib.attn_cache_free, lib.attn_cache_fork
_lib_compact, _lib_append, _lib_paged_fwd = lib.attn_cache_compact, lib.attn_cache_append, lib.attn_paged_fwd
_lib_append_granted, _lib_paged_fwd_granted = lib.attn_cache_append_granted, lib.attn_paged_fwd_granted
_lib_append_rotated, _lib_read = lib.attn_cache_append_rotated, lib.attn_cache_read


@contextlib.contextmanager
def _paged_scope(cache, stream):
    """The cache's device is current, and `stream` too, so that memory
    allocated inside belongs to it.  Yields the stream's handle."""
    with torch.cuda.device(cache.device):
        if stream is None:
            yield torch.cuda.current_stream().cuda_stream
        else:
            st = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
            with torch.cuda.stream(st):
                yield st.cuda_stream


def _paged_here(cache, stream):
    """Whether a call can go out as things are: no stream of its own, and the
    cache's device current.  (A decode step is made of calls that take a few
    microseconds; entering _paged_scope costs as much.)"""
    return stream is None and _device_index() == cache._index


_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or torch.cuda.is_current_stream_capturing


def _paged_workspace(workspace, need, cache, st):
    """The caller's workspace, or one of the cache object's own: one for each
    thread and stream, whose calls run in order, so no two calls in flight
    share it.  It is kept as long as the thread and the cache are there (the
    stream that it was allocated on orders what comes after it).  A call that
    is being captured gets memory of its own, which belongs to the graph."""
    if workspace is None:
        if _capturing():
            t = torch.empty(need, dtype=torch.uint8, device=cache.device)
            return t, need, t.data_ptr()
        spaces = cache._spaces.__dict__   # (this thread's)
        ws = spaces.get(st)
        if ws is None or ws[1] < need:
            t = torch.empty(need, dtype=torch.uint8, device=cache.device)
            ws = spaces[st] = (t, need, t.data_ptr())
        return ws
    if workspace.get_device() != cache._index or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the cache's device")
    return workspace, workspace.numel(), workspace.data_ptr()


@functools.lru_cache(maxsize=256)
def attn_cache_workspace_size(pages: int, n: int) -> int:
    return int(lib.attn_cache_workspace_size(pages, n))


def _granted(granted, cache, n, like):
    if granted is None:
        return torch.empty_like(like)   # (the list: int32 [n], contiguous)
    _paged_list(granted, cache, "granted", n)
    return granted


def _reserve(cache, st, seqs, a, b, n, granted, workspace):
    g = _granted(granted, cache, n, seqs)
    ws = _paged_workspace(workspace, attn_cache_workspace_size(cache.pages, n), cache, st)
    _check(_lib_reserve(cache._p, a, b, n, g.data_ptr(), ws[2], ws[1], st), "attn_cache_reserve")
    return g


def attn_cache_reserve(cache, seqs, n_new, granted=None, workspace=None, stream=None):
    """Room for n_new[i] more tokens in sequence seqs[i] (int32 device
    vectors): free pages, lowest first, in list order; lengths grow.  Returns
    granted, int32 [n]: 1, or 0 for an entry that got nothing."""
    n = seqs.shape[0]
    a, b = _paged_list(seqs, cache, "seqs"), _paged_list(n_new, cache, "n_new", n)
    if _paged_here(cache, stream):
        return _reserve(cache, _raw_stream(cache._index), seqs, a, b, n, granted, workspace)
    with _paged_scope(cache, stream) as st:
        return _reserve(cache, st, seqs, a, b, n, granted, workspace)


def attn_cache_free(cache, seqs, keep=None, stream=None) -> None:
    """Cuts sequence seqs[i] to its first keep[i] tokens (None, or negative: to none)."""
    n = seqs.shape[0]
    a = _paged_list(seqs, cache, "seqs")
    b = None if keep is None else _paged_list(keep, cache, "keep", n)
    if _paged_here(cache, stream):
        rc = _lib_free(cache._p, a, b, n, _raw_stream(cache._index))
    else:
        with _paged_scope(cache, stream) as st:
            rc = _lib_free(cache._p, a, b, n, st)
    _check(rc, "attn_cache_free")


def _fork(cache, st, parents, a, b, n, copy, granted, workspace):
    g = _granted(granted, cache, n, parents)
    ws = _paged_workspace(workspace, attn_cache_workspace_size(cache.pages, n), cache, st)
    _check(_lib_fork(cache._p, a, b, n, copy, g.data_ptr(), ws[2], ws[1], st), "attn_cache_fork")
    return g


def attn_cache_fork(cache, parents, children, copy: bool = False, granted=None, workspace=None, stream=None):
    """Makes the empty sequence children[i] a copy of parents[i]: full pages
    shared and a partly filled last page copied, or (copy=True) every page
    copied.  Returns granted, int32 [n]."""
    n = parents.shape[0]
    a, b = _paged_list(parents, cache, "parents"), _paged_list(children, cache, "children", n)
    if _paged_here(cache, stream):
        return _fork(cache, _raw_stream(cache._index), parents, a, b, n, 1 if copy else 0, granted, workspace)
    with _paged_scope(cache, stream) as st:
        return _fork(cache, st, parents, a, b, n, 1 if copy else 0, granted, workspace)


def _compact(cache, st, inplace, workspace):
    table = cache.page_table if inplace else torch.empty_like(cache.page_table)
    refs = cache.ref_counts if inplace else torch.empty_like(cache.ref_counts)
    n_live = torch.empty(1, dtype=torch.int32, device=cache.device)
    ws = _paged_workspace(workspace, attn_cache_workspace_size(cache.pages, 0), cache, st)
    _check(_lib_compact(cache._p, table.data_ptr(), refs.data_ptr(), n_live.data_ptr(), ws[2], ws[1], st), "attn_cache_compact")
    return table, refs, n_live


def attn_cache_compact(cache, inplace: bool = True, workspace=None, stream=None):
    """Moves the live pages to the bottom of the pool.  Returns (page_table,
    ref_counts, n_live): the cache's own tensors, updated, or with
    inplace=False new ones, the cache's staying as they were (and valid, since
    only free pages are written); n_live is an int32 device tensor [1]."""
    if _paged_here(cache, stream):
        return _compact(cache, _raw_stream(cache._index), inplace, workspace)
    with _paged_scope(cache, stream) as st:
        return _compact(cache, st, inplace, workspace)


def _append(cache, st, layer, k, v, strides, T, a, b, c, n):
    if c is None:
        return _lib_append(cache._p, layer, k, v, strides[0], strides[1], T, a, b, n, st)
    return _lib_append_granted(cache._p, layer, k, v, strides[0], strides[1], T, a, b, c, n, st)


def _new_rows(cache, k, v, ks, vs):
    shape, strides = k.shape, k.stride()
    if (len(shape) != 3 or shape != v.shape or strides != v.stride() or shape[1] != cache.heads or
            shape[2] != cache.d or strides[2] != 1):
        raise ValueError(f"{ks} and {vs} must be [T, heads, d] with one shape and strides, the last dimension contiguous")
    if (k.dtype != cache.dtype or v.dtype != cache.dtype or k.get_device() != cache._index or
            v.get_device() != cache._index):
        raise ValueError(f"{ks} and {vs} must have the cache's dtype and device")
    return shape, strides


def attn_cache_append(cache, layer: int, k_new, v_new, seqs, q_start, stream=None, granted=None) -> None:
    """Writes the keys and values of new tokens into one layer.  k_new, v_new:
    [T, heads, d] of the cache's dtype, any strides with a contiguous last
    dimension (one pair of strides for both).  Entry i: sequence seqs[i]
    (seqs None: sequence i), tokens q_start[i] .. q_start[i+1] - 1, the last
    ones of the sequence (reserved before).  granted: what attn_cache_reserve
    returned for these entries; those that got no room are left out (without
    it they write over the sequence's last tokens)."""
    shape, strides = _new_rows(cache, k_new, v_new, "k_new", "v_new")
    n = q_start.shape[0] - 1
    a = None if seqs is None else _paged_list(seqs, cache, "seqs", n)
    b = _paged_list(q_start, cache, "q_start")
    c = None if granted is None else _paged_list(granted, cache, "granted", n)
    args = (layer, k_new.data_ptr(), v_new.data_ptr(), strides, shape[0], a, b, c, n)
    if _paged_here(cache, stream):
        rc = _append(cache, _raw_stream(cache._index), *args)
    else:
        with _paged_scope(cache, stream) as st:
            rc = _append(cache, st, *args)
    _check(rc, "attn_cache_append")


def _append_rotated(cache, st, layer, k, v, strides, q, q_out, Hq, T, a, b, c, n, rotation):
    qp, op, qs, os_ = None, None, (0, 0), (0, 0)
    if q is not None:
        if q_out is None:
            q_out = torch.empty_like(q) if q.is_contiguous() else torch.empty(q.shape, dtype=q.dtype, device=q.device)
        qp, op, qs, os_ = q.data_ptr(), q_out.data_ptr(), q.stride(), q_out.stride()
    _check(_lib_append_rotated(cache._p, layer, k, v, strides[0], strides[1], qp, op, Hq, qs[0], qs[1], os_[0], os_[1], T, a, b,
                               c, n, ctypes.byref(rotation), st), "attn_cache_append_rotated")
    return q_out


def attn_cache_append_rotated(cache, layer: int, k_new, v_new, seqs, q_start, table, q=None, q_out=None,
                              neighbours: bool = False, positions=None, granted=None, stream=None):
    """attn_cache_append with the position rotation applied to the keys on the
    way, and to the queries of the same tokens.  table: contiguous float32
    [positions, dims], of each position dims / 2 cosines and then as many sines;
    the first dims columns of a row turn, dims <= d.  Pair i is columns i and
    i + dims / 2, or (neighbours) 2 i and 2 i + 1.  A token's position is its
    index in its sequence, or positions[t] (int32 [T]).  q: [T, Hq, d] as for
    attn_paged_fwd, or None; q_out: where its rotated rows go (q itself: in
    place; default: a new tensor).  Returns q_out (None without q); its rows of
    tokens that are not written are as they were."""
    shape, strides = _new_rows(cache, k_new, v_new, "k_new", "v_new")
    T, Hq = shape[0], 0
    if table.dtype != torch.float32 or table.dim() != 2 or not table.is_contiguous() or table.get_device() != cache._index:
        raise ValueError("table must be a contiguous float32 tensor [positions, dims] on the cache's device")
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
    else:
        Hq = q.shape[1] if q.dim() == 3 else 0
        if Hq == 0 or q.shape[0] != T or q.shape[2] != cache.d or q.stride(2) != 1:
            raise ValueError("q must be [T, Hq, d] with a contiguous last dimension")
        if q.dtype != cache.dtype or q.get_device() != cache._index:
            raise ValueError("q must have the cache's dtype and device")
        if q_out is not None and (q_out.shape != q.shape or q_out.dtype != q.dtype or q_out.get_device() != cache._index or
                                  q_out.stride(2) != 1):
            raise ValueError("q_out must be like q, with a contiguous last dimension")
    n = q_start.shape[0] - 1
    a = None if seqs is None else _paged_list(seqs, cache, "seqs", n)
    b = _paged_list(q_start, cache, "q_start")
    c = None if granted is None else _paged_list(granted, cache, "granted", n)
    p = None if positions is None else _paged_list(positions, cache, "positions", T)
    # (positions are below 2^31: rows past them are never met)
    rotation = RotationT(table.data_ptr(), p, min(table.shape[0], 2 ** 31 - 1), table.shape[1], 1 if neighbours else 0)
    args = (layer, k_new.data_ptr(), v_new.data_ptr(), strides, q, q_out, Hq, T, a, b, c, n, rotation)
    if _paged_here(cache, stream):
        return _append_rotated(cache, _raw_stream(cache._index), *args)
    with _paged_scope(cache, stream) as st:
        return _append_rotated(cache, st, *args)


def _read(cache, st, layer, shape, k, v, T, a, b, c, n):
    if k is None:
        k = torch.empty(shape, dtype=cache.dtype, device=cache.device)
        v = torch.empty_like(k)
    s = k.stride()
    _check(_lib_read(cache._p, layer, k.data_ptr(), v.data_ptr(), s[0], s[1], T, a, b, c, n, st), "attn_cache_read")
    return k, v


def attn_cache_read(cache, layer: int, seqs, q_start, T: int | None = None, first=None, k_out=None, v_out=None, stream=None):
    """Copies tokens of one layer out of the cache (of 4-bit values: the values
    that they stand for, exact in bfloat16).  Entry i: sequence seqs[i] (seqs
    None: sequence i), whose tokens first[i], first[i] + 1, ... (first None: the
    last ones) go to rows q_start[i] .. q_start[i+1] - 1.  T: rows in all;
    k_out, v_out: [T, heads, d] of the cache's dtype with one pair of strides, or
    new tensors (T needed).  Returns (k, v); rows of no entry, of tokens that
    the cache does not hold, and of entries with a negative first are as they were."""
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out go together")
    if k_out is not None:
        shape, _ = _new_rows(cache, k_out, v_out, "k_out", "v_out")
        if T is not None and T != shape[0]:
            raise ValueError("k_out and v_out must have T rows")
        T = shape[0]
    elif T is None or T < 0:
        raise ValueError("T, the rows in all, is needed where k_out and v_out are not given")
    n = q_start.shape[0] - 1
    a = None if seqs is None else _paged_list(seqs, cache, "seqs", n)
    b = _paged_list(q_start, cache, "q_start")
    c = None if first is None else _paged_list(first, cache, "first", n)
    args = (layer, (T, cache.heads, cache.d), k_out, v_out, T, a, b, c, n)
    if _paged_here(cache, stream):
        return _read(cache, _raw_stream(cache._index), *args)
    with _paged_scope(cache, stream) as st:
        return _read(cache, st, *args)


@functools.lru_cache(maxsize=256)
def _paged_workspace_size(Hq, heads, max_q, d, dtype) -> int:
    return int(lib.attn_paged_workspace_size(Hq, heads, max_q, d, dtype))


def attn_paged_workspace_size(Hq: int, heads: int, max_q: int, d: int, dtype) -> int:
    """dtype: the cache's (torch.float4_e2m1fn_x2 for 4-bit values)."""
    code = dtype if isinstance(dtype, int) else ATTN_E2M1 if dtype == _E2M1 else _DTYPE[dtype]
    return _paged_workspace_size(Hq, heads, max_q, d, code)


def _paged_fwd(cache, st, q, layer, shape, a, b, c, n, max_q, causal, scale, o, l, want_lse, workspace):
    T, Hq, d = shape
    if o is None:
        o = torch.empty_like(q) if q.is_contiguous() else torch.empty(shape, dtype=cache.dtype, device=cache.device)
    if l is None and want_lse:
        l = torch.empty((T, Hq), dtype=torch.float32, device=cache.device)
    # (arguments the library rejects give a size of 0 here; it then says which)
    ws = _paged_workspace(workspace, _paged_workspace_size(Hq, cache.heads, max(max_q, 1), d, cache._code), cache, st)
    qs, os_ = q.stride(), o.stride()
    ptrs = (q.data_ptr(), o.data_ptr(), None if l is None else l.data_ptr(), qs[0], qs[1], os_[0], os_[1], T, Hq, a, b)
    rest = (n, max_q, causal, scale, ws[2], ws[1], st)
    rc = (_lib_paged_fwd(cache._p, layer, *ptrs, *rest) if c is None else
          _lib_paged_fwd_granted(cache._p, layer, *ptrs, c, *rest))
    _check(rc, "attn_paged_fwd")
    return o, l


def attn_paged_fwd(q, cache, layer: int, seqs, q_start, max_q: int | None = None, causal: bool = True,
                   scale: float | None = None, out=None, lse=None, workspace=None, stream=None, want_lse: bool = True,
                   granted=None):
    """Attention of new tokens over one layer of a paged cache.  q: [T, Hq, d]
    of the cache's dtype, any strides with a contiguous last dimension; Hq a
    multiple of the cache's heads (query head j reads kv head j // (Hq /
    heads)).  Entry i: sequence seqs[i] (seqs None: sequence i), whose last
    tokens are rows q_start[i] .. q_start[i+1] - 1 of q; causal: token t of the
    entry's n sees keys j <= len - n + t.  max_q: at least the most new tokens
    of an entry, at most T.  The default, T, is right for one entry only: it
    sends a decode batch to the kernel for chunks, which is slower there, takes
    a workspace of up to 42 MB, and rounds probabilities to bf16 once where
    decoding (Hq / heads * max_q <= 16) keeps two bf16 parts (over 4-bit values
    both round them once, to float16).  granted: what attn_cache_reserve
    returned for these entries; those that got no room are left out.  Returns (o, lse): o like q, lse [T,
    Hq] float32; rows of no entry, or of one left out, are as they were."""
    shape = q.shape
    if len(shape) != 3 or shape[2] != cache.d or q.stride(2) != 1:
        raise ValueError("q must be [T, Hq, d] with a contiguous last dimension")
    if q.dtype != cache.dtype or q.get_device() != cache._index:
        raise ValueError("q must have the cache's dtype and device")
    n = q_start.shape[0] - 1
    a = None if seqs is None else _paged_list(seqs, cache, "seqs", n)
    b = _paged_list(q_start, cache, "q_start")
    if out is not None and (out.shape != shape or out.dtype != q.dtype or out.get_device() != cache._index or
                            out.stride(2) != 1):
        raise ValueError("out must be like q, with a contiguous last dimension")
    if lse is not None and (lse.shape != shape[:2] or lse.dtype != torch.float32 or not lse.is_contiguous() or
                            lse.get_device() != cache._index):
        raise ValueError("lse must be a contiguous float32 tensor [T, Hq] on q's device")
    c = None if granted is None else _paged_list(granted, cache, "granted", n)
    args = (q, layer, shape, a, b, c, n, shape[0] if max_q is None else int(max_q), 1 if causal else 0,
            cache._scale if scale is None else float(scale), out, lse, want_lse, workspace)
    if _paged_here(cache, stream):
        return _paged_fwd(cache, _raw_stream(cache._index), *args)
    with _paged_scope(cache, stream) as st:
        return _paged_fwd(cache, st, *args)


def attn_bwd_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(lib.attn_bwd_workspace_size(B, H, N, d))


def attn_bwd(q, k, v, o, do, lse, causal: bool = False, scale: float | None = None, key_mask=None,
             dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients of attention.  q, k, v, o, do: [B, H, N, d] contiguous
    bfloat16 device tensors (o and lse from attn_fwd on the same inputs);
    lse: [B, H, N] float32.  Returns (dq, dk, dv)."""
    ts = (q, k, v, o, do)
    for t in ts:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v, o, do must be contiguous device tensors")
        if t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError("q, k, v, o, do must share one shape and dtype")
    B, H, N, d = _shape4(q)
    if q.dtype not in _DTYPE:
        raise ValueError(f"unsupported dtype {q.dtype}")
    if (lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous() or lse.numel() != B * H * N):
        raise ValueError("lse must be a contiguous float32 device tensor with B*H*N elements")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = dq if dq is not None else torch.empty_like(q)
    dk = dk if dk is not None else torch.empty_like(q)
    dv = dv if dv is not None else torch.empty_like(q)
    need = attn_bwd_workspace_size(B, H, N, d)
    ws = workspace if workspace is not None else torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    m = None
    if key_mask is not None:
        m = key_mask
        if m.dtype != torch.float32 or not m.is_contiguous() or m.numel() != B * H * N or not m.is_cuda:
            raise ValueError("key_mask must be a contiguous float32 device tensor with B*H*N elements")
    rc = lib.attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                      B, H, N, d, int(bool(causal)), float(scale), _DTYPE[q.dtype], _ptr(m), _ptr(ws), ws.numel(),
                      ctypes.c_void_p(_stream(stream)))
    _check(rc, "attn_bwd")
    return dq, dk, dv


# Number formats of the emulation (fraction bits, exponent bits).
EMUL_FORMATS = {"bf16": (7, 8), "fp16": (10, 5), "tf32": (10, 8), "fp32": (23, 8), "fp64": (52, 11)}
EMUL_BASELINE, EMUL_TILED = 0, 1


def attn_emul_fwd(q, k, v, causal: bool, scale: float, algo: int, Bc: int, mbits: int, ebits: int,
                  key_mask=None, rows=None, stream=None):
    """Attention with every tensor op rounded to a number format (the
    paper's numerical re-implementation; see include/attn.h).  q, k, v:
    contiguous device tensors [B, H, N, d] (float32, bfloat16 or float64).
    rows: None or a device int64 tensor of flat row ids.  Returns a float64
    device tensor [B, H, N, d] (all rows) or [nrows, d]."""
    for t in (q, k, v):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous device tensors")
    B, H, N, d = _shape4(q)
    if rows is None:
        o = torch.empty((B, H, N, d), dtype=torch.float64, device=q.device)
        nrows = 0
    else:
        if rows.dtype != torch.int64 or not rows.is_cuda or not rows.is_contiguous():
            raise ValueError("rows must be a contiguous int64 device tensor")
        nrows = rows.numel()
        o = torch.empty((nrows, d), dtype=torch.float64, device=q.device)
    m = None
    if key_mask is not None:
        m = key_mask
        if m.dtype != torch.float32 or not m.is_contiguous() or m.numel() != B * H * N or not m.is_cuda:
            raise ValueError("key_mask must be a contiguous float32 device tensor with B*H*N elements")
    rc = lib.attn_emul_fwd(_ptr(q), _ptr(k), _ptr(v), _DTYPE[q.dtype], _ptr(o), B, H, N, d, int(bool(causal)),
                           float(scale), _ptr(m), int(algo), int(Bc), int(mbits), int(ebits), _ptr(rows), nrows,
                           ctypes.c_void_p(_stream(stream)))
    _check(rc, "attn_emul_fwd")
    return o


def attn_emul_round(x, mbits: int, ebits: int, stream=None):
    """fl(x) for a contiguous float64 device tensor (new tensor)."""
    if x.dtype != torch.float64 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous float64 device tensor")
    y = torch.empty_like(x)
    rc = lib.attn_emul_round(_ptr(x), _ptr(y), x.numel(), int(mbits), int(ebits), ctypes.c_void_p(_stream(stream)))
    _check(rc, "attn_emul_round")
    return y


def attn_status(stream=None) -> int:
    return int(lib.attn_status(ctypes.c_void_p(_stream(stream))))


def attn_last_variant() -> str:
    buf = ctypes.create_string_buffer(128)
    lib.attn_last_variant(buf, 128)
    return buf.value.decode()


def attn_debug_wait_timeout(timeout_us: int, stream=None) -> int:
    return int(lib.attn_debug_wait_timeout(int(timeout_us), ctypes.c_void_p(_stream(stream))))
