"""GB300-native PISA pyramid Top-K block selection.

Thin Python binding over the C ABI of ``include/pisa.h`` (library
``_build/libpisa.so``, built in-tree by ``build.py``).  This module only
marshals arguments: PyTorch provides device memory and the current CUDA
stream; every step of the selection runs in the library's CUDA kernels.  There
is no CPU fallback: if the library cannot be loaded, every call raises.

Method: "Block Sparse Attention with Log-Linear Complexity" (§3.1 pyramid of
mean-pooled keys, §3.2 coarse-to-fine Top-K walk, "Scoring: LogSumExp", §4.1
GQA head sum, §5.1 prefill and decoding kernels).
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

import torch

from . import build as _build

__all__ = [
    "PisaError", "Pyramid", "load", "num_levels", "pyramid_nodes", "level_offset",
    "build_pyramid", "select_workspace_bytes", "select_prefill", "select_prefill_noalloc",
    "noalloc_prepare", "noalloc_device_status",
    "decode_workspace_bytes",
    "decode_append_and_select", "check_device_status", "status_string", "kernel_launches",
    "PagedCache", "cache_workspace", "cache_workspace_bytes", "cache_append", "cache_read", "cache_attention",
    "rotary_table",
    "prefill_phases", "set_phase_events", "D", "C", "G_MERGE",
]

D, C, G_MERGE = 64, 64, 2

_lib = None


class PisaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def load(path: str | None = None):
    """Load (building first if needed) the CUDA library and declare its ABI."""
    global _lib
    if _lib is not None:
        return _lib
    if path is None:
        path = _build.LIB if os.path.exists(_build.LIB) else _build.build()
    lib = ctypes.CDLL(path)
    i32, i64, sz, vp = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
    lib.pisa_num_levels.argtypes = [i64, i32, i32]
    lib.pisa_num_levels.restype = i32
    lib.pisa_pyramid_nodes.argtypes = [i64, i32, i32]
    lib.pisa_pyramid_nodes.restype = i64
    lib.pisa_level_offset.argtypes = [i64, i32, i32, i32]
    lib.pisa_level_offset.restype = i64
    lib.pisa_build_pyramid.argtypes = [vp, i64, vp]
    lib.pisa_build_pyramid.restype = i32
    lib.pisa_select_workspace_bytes.argtypes = [i32, i64, i32, i32, i32]
    lib.pisa_select_workspace_bytes.restype = sz
    lib.pisa_select_prefill.argtypes = [vp, i32, vp, i64, i32, i32, vp, vp, vp, sz, vp]
    lib.pisa_select_prefill.restype = i32
    lib.pisa_flat_workspace_bytes.argtypes = [i32, i64, i32, i32, i32]
    lib.pisa_flat_workspace_bytes.restype = sz
    lib.pisa_select_flat.argtypes = [vp, i32, vp, i64, i32, i32, vp, vp, vp, sz, vp]
    lib.pisa_select_flat.restype = i32
    lib.pisa_select_prefill_ex.argtypes = [vp, i32, vp, i64, i32, i32, vp, vp, vp, sz, vp, i32]
    lib.pisa_select_prefill_ex.restype = i32
    lib.pisa_select_prefill_host.argtypes = [vp, vp, i64, vp, vp, i32, i32, i32, vp, vp, vp, sz, vp, vp]
    lib.pisa_select_prefill_host.restype = i32
    lib.pisa_selftest_bounded_wait.argtypes = [vp, sz, i64, vp]
    lib.pisa_selftest_bounded_wait.restype = i32
    lib.pisa_select_flat_ex.argtypes = [vp, i32, vp, i64, i32, i32, vp, vp, vp, sz, vp, i32]
    lib.pisa_select_flat_ex.restype = i32
    lib.pisa_sparse_attention.argtypes = [vp, i32, vp, vp, i32, i64, i32, vp, i32, i32, vp, vp]
    lib.pisa_sparse_attention.restype = i32
    lib.pisa_build_pyramid_ragged.argtypes = [vp, vp]
    lib.pisa_build_pyramid_ragged.restype = i32
    lib.pisa_decode_workspace_bytes.argtypes = [i32, i32, i32, i32]
    lib.pisa_decode_workspace_bytes.restype = sz
    lib.pisa_decode_append_and_select.argtypes = [vp, vp, i32, vp, i32, vp, vp, vp, sz, vp]
    lib.pisa_decode_append_and_select.restype = i32
    lib.pisa_check_device_status.argtypes = [vp, vp]
    lib.pisa_check_device_status.restype = i32
    lib.pisa_status_string.argtypes = [i32]
    lib.pisa_status_string.restype = ctypes.c_char_p
    lib.pisa_kernel_launches.argtypes = []
    lib.pisa_kernel_launches.restype = ctypes.c_uint64
    lib.pisa_set_phase_events.argtypes = [ctypes.c_void_p, i32]
    lib.pisa_set_phase_events.restype = i32
    lib.pisa_prefill_phase_count.argtypes = []
    lib.pisa_prefill_phase_count.restype = i32
    lib.pisa_prefill_phase_name.argtypes = [i32]
    lib.pisa_prefill_phase_name.restype = ctypes.c_char_p
    lib.pisa_select_prefill_noalloc.argtypes = [vp, i32, vp, i64, i32, i32, vp, vp, vp]
    lib.pisa_select_prefill_noalloc.restype = i32
    lib.pisa_noalloc_prepare.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
    lib.pisa_noalloc_prepare.restype = i32
    lib.pisa_noalloc_device_status.argtypes = [vp]
    lib.pisa_noalloc_device_status.restype = i32
    lib.pisa_cache_page_bytes.argtypes = [i32, i32, i32]
    lib.pisa_cache_page_bytes.restype = sz
    lib.pisa_cache_workspace_bytes.argtypes = []
    lib.pisa_cache_workspace_bytes.restype = sz
    lib.pisa_cache_append.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp, vp, i64, i32, i32, vp, vp, vp, vp]
    lib.pisa_cache_append.restype = i32
    lib.pisa_cache_read.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp]
    lib.pisa_cache_read.restype = i32
    lib.pisa_cache_attention.argtypes = [vp, vp, i32, i32, vp, vp, i32, vp, i32, vp, sz, vp]
    lib.pisa_cache_attention.restype = i32
    lib.pisa_event_elapsed_ms.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_float)]
    lib.pisa_event_elapsed_ms.restype = i32
    _lib = lib
    return lib


class _PyrStruct(ctypes.Structure):
    _fields_ = [
        ("summaries", ctypes.c_void_p),
        ("keys", ctypes.c_void_p),
        ("lengths", ctypes.c_void_p),
        ("B", ctypes.c_int),
        ("Hkv", ctypes.c_int),
        ("d", ctypes.c_int),
        ("C", ctypes.c_int),
        ("g", ctypes.c_int),
        ("n_cap", ctypes.c_int),
    ]


def status_string(status: int) -> str:
    return load().pisa_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != 0:
        raise PisaError(status, what)


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def num_levels(n: int) -> int:
    return int(load().pisa_num_levels(n, C, G_MERGE))


def pyramid_nodes(n_cap: int) -> int:
    return int(load().pisa_pyramid_nodes(n_cap, C, G_MERGE))


def level_offset(n_cap: int, level: int) -> int:
    return int(load().pisa_level_offset(n_cap, C, G_MERGE, level))


@dataclass
class Pyramid:
    """Caller-owned pyramid storage: borrowed keys [B, n_cap, Hkv, 64] bf16,
    summaries [B, Hkv, nodes(n_cap), 64] fp32 and optional lengths [B] int32."""

    keys: torch.Tensor
    summaries: torch.Tensor
    lengths: torch.Tensor | None = None

    @classmethod
    def allocate(cls, keys: torch.Tensor, with_lengths: bool = False) -> "Pyramid":
        if keys.dtype != torch.bfloat16 or keys.dim() != 4 or not keys.is_cuda:
            raise ValueError("keys must be a CUDA bf16 tensor [B, n_cap, Hkv, d]")
        B, n_cap, Hkv, d = keys.shape
        nodes = pyramid_nodes(n_cap)
        summ = torch.empty(B, Hkv, nodes, d, dtype=torch.float32, device=keys.device)
        lengths = torch.zeros(B, dtype=torch.int32, device=keys.device) if with_lengths else None
        return cls(keys.contiguous(), summ, lengths)

    @property
    def B(self):
        return self.keys.shape[0]

    @property
    def n_cap(self):
        return self.keys.shape[1]

    @property
    def Hkv(self):
        return self.keys.shape[2]

    def struct(self) -> _PyrStruct:
        return _PyrStruct(self.summaries.data_ptr(), self.keys.data_ptr(),
                          self.lengths.data_ptr() if self.lengths is not None else None,
                          self.B, self.Hkv, self.keys.shape[3], C, G_MERGE, self.n_cap)

    def level(self, level: int, n: int | None = None) -> torch.Tensor:
        """View of the summaries of one level [B, Hkv, M_level(n), d]."""
        n = self.n_cap if n is None else n
        off = level_offset(self.n_cap, level)
        m = -(-n // (C << (level - 1)))
        return self.summaries[:, :, off:off + m]


def build_pyramid(keys: torch.Tensor | Pyramid, N: int | None = None, with_lengths: bool = False,
                  stream=None) -> Pyramid:
    """Mean pyramid over the first N tokens (§3.1).  Accepts raw keys or a Pyramid."""
    pyr = keys if isinstance(keys, Pyramid) else Pyramid.allocate(keys, with_lengths)
    N = pyr.n_cap if N is None else N
    st = pyr.struct()
    _check(load().pisa_build_pyramid(ctypes.byref(st), N, _stream(stream)), "pisa_build_pyramid")
    return pyr


def select_workspace_bytes(B: int, N: int, Hq: int, Hkv: int, K: int) -> int:
    return int(load().pisa_select_workspace_bytes(B, N, Hq, Hkv, K))


def select_prefill(Q: torch.Tensor, pyr: Pyramid, K: int, causal: bool = True, N: int | None = None,
                   with_scores: bool = True, workspace: torch.Tensor | None = None,
                   out: tuple | None = None, stream=None, mode: int = 0):
    """Coarse-to-fine Top-K for every query (§3.2).  mode: block score, 0 = LSE,
    1 = mean of the child logits (PISA-1), 2 = mean + half their variance (PISA-2).

    Q [B, N, Hq, 64] bf16 (CUDA).  Returns (idx [B, Hkv, N, K] int32, scores
    [B, Hkv, N, K] fp32 or None).
    """
    if Q.dtype != torch.bfloat16 or not Q.is_cuda or Q.dim() != 4:
        raise ValueError("Q must be a CUDA bf16 tensor [B, N, Hq, d]")
    B, NQ, Hq, _ = Q.shape
    N = NQ if N is None else N
    lib = load()
    need = lib.pisa_select_workspace_bytes(B, N, Hq, pyr.Hkv, K)
    if need == 0:
        _check(2, "pisa_select_workspace_bytes")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=Q.device)
    if out is None:
        idx = torch.empty(B, pyr.Hkv, N, K, dtype=torch.int32, device=Q.device)
        scores = torch.empty(B, pyr.Hkv, N, K, dtype=torch.float32, device=Q.device) if with_scores else None
    else:
        idx, scores = out
    st = pyr.struct()
    _check(lib.pisa_select_prefill_ex(_ptr(Q), Hq, ctypes.byref(st), N, K, int(causal), _ptr(idx),
                                      _ptr(scores), _ptr(workspace), workspace.numel(), _stream(stream),
                                      int(mode)),
           "pisa_select_prefill_ex")
    return idx, scores


_COPY_STREAMS: dict = {}


def select_prefill_host(q_host: torch.Tensor, k_host: torch.Tensor, pyr: Pyramid, K: int, causal: bool = True,
                        idx_host: torch.Tensor | None = None, q_dev: torch.Tensor | None = None,
                        idx_dev: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None, copy_stream=None) -> torch.Tensor:
    """Pyramid build + prefill selection for host-resident Q [B, N, Hq, 64] and K
    [B, N, Hkv, 64] (bf16, pinned for overlap): the library copies K into pyr.keys and
    Q into q_dev in runs of query chunks on copy_stream while `stream` selects, and
    copies each run's indices back into idx_host [B, Hkv, N, K] (int32, pinned) as soon
    as they are final.  Asynchronous: synchronise `stream` before reading idx_host.
    The device staging buffers are allocated here when not given.
    """
    if q_host.dtype != torch.bfloat16 or k_host.dtype != torch.bfloat16 or q_host.is_cuda or k_host.is_cuda:
        raise ValueError("q_host and k_host must be host bf16 tensors")
    if q_host.dim() != 4 or k_host.dim() != 4 or not q_host.is_contiguous() or not k_host.is_contiguous():
        raise ValueError("q_host [B, N, Hq, d] and k_host [B, N, Hkv, d] must be contiguous")
    B, N, Hq, _ = q_host.shape
    if k_host.shape[0] != B or k_host.shape[1] != N or k_host.shape[2] != pyr.Hkv:
        raise ValueError("k_host must be [B, N, Hkv, d] with the pyramid's B and Hkv")
    dev = pyr.keys.device
    lib = load()
    need = lib.pisa_select_workspace_bytes(B, N, Hq, pyr.Hkv, K)
    if need == 0:
        _check(2, "pisa_select_workspace_bytes")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if q_dev is None:
        q_dev = torch.empty(B, N, Hq, q_host.shape[3], dtype=torch.bfloat16, device=dev)
    if idx_dev is None:
        idx_dev = torch.empty(B, pyr.Hkv, N, K, dtype=torch.int32, device=dev)
    if idx_host is None:
        idx_host = torch.empty(B, pyr.Hkv, N, K, dtype=torch.int32, pin_memory=True)
    if copy_stream is None:  # a side stream of the library's own, one per device
        copy_stream = _COPY_STREAMS.get(dev.index)
        if copy_stream is None:
            copy_stream = _COPY_STREAMS[dev.index] = torch.cuda.Stream(device=dev)
    st = pyr.struct()
    _check(lib.pisa_select_prefill_host(ctypes.byref(st), _ptr(k_host), N, _ptr(q_host), _ptr(q_dev), Hq, K,
                                        int(causal), _ptr(idx_host), _ptr(idx_dev), _ptr(workspace),
                                        workspace.numel(), _stream(stream), _stream(copy_stream)),
           "pisa_select_prefill_host")
    return idx_host


def flat_workspace_bytes(B: int, N: int, Hq: int, Hkv: int, K: int) -> int:
    return int(load().pisa_flat_workspace_bytes(B, N, Hq, Hkv, K))


def build_pyramid_ragged(pyr: Pyramid, stream=None) -> Pyramid:
    """Build every sequence over its own length pyr.lengths[b] (set by the caller)."""
    if pyr.lengths is None:
        raise ValueError("a ragged build needs a Pyramid with lengths")
    st = pyr.struct()
    _check(load().pisa_build_pyramid_ragged(ctypes.byref(st), _stream(stream)), "pisa_build_pyramid_ragged")
    return pyr


def select_flat(Q: torch.Tensor, pyr: Pyramid, K: int, causal: bool = True, N: int | None = None,
                with_scores: bool = True, workspace: torch.Tensor | None = None,
                out: tuple | None = None, stream=None, mode: int = 0):
    """Flat selection: every eligible leaf scored exactly, the K best kept.
    Same arguments and outputs as select_prefill (only pyr.keys is read)."""
    if Q.dtype != torch.bfloat16 or not Q.is_cuda or Q.dim() != 4:
        raise ValueError("Q must be a CUDA bf16 tensor [B, N, Hq, d]")
    B, NQ, Hq, _ = Q.shape
    N = NQ if N is None else N
    lib = load()
    if workspace is None:
        need = lib.pisa_flat_workspace_bytes(B, N, Hq, pyr.Hkv, K)
        if need == 0:
            _check(2, "pisa_flat_workspace_bytes")
        workspace = torch.empty(need, dtype=torch.uint8, device=Q.device)
    if out is None:
        idx = torch.empty(B, pyr.Hkv, N, K, dtype=torch.int32, device=Q.device)
        scores = torch.empty(B, pyr.Hkv, N, K, dtype=torch.float32, device=Q.device) if with_scores else None
    else:
        idx, scores = out
    st = pyr.struct()
    _check(lib.pisa_select_flat_ex(_ptr(Q), Hq, ctypes.byref(st), N, K, int(causal), _ptr(idx),
                                   _ptr(scores), _ptr(workspace), workspace.numel(), _stream(stream),
                                   int(mode)),
           "pisa_select_flat_ex")
    return idx, scores


def sparse_attention(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, idx: torch.Tensor, causal: bool = True,
                     out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Stage-two block-sparse attention over the blocks in idx [B, Hkv, N, Ksel].
    Q [B, N, Hq, 64], K and V [B, N, Hkv, 64] bf16 CUDA; returns fp32 [B, N, Hq, 64]."""
    for x in (Q, K, V):
        if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 4 or not x.is_contiguous():
            raise ValueError("Q, K, V must be contiguous CUDA bf16 tensors [B, N, H, d]")
    if idx.dtype != torch.int32 or not idx.is_contiguous():
        raise ValueError("idx must be contiguous int32 [B, Hkv, N, Ksel]")
    B, N, Hq, d = Q.shape
    if out is None:
        out = torch.empty(B, N, Hq, d, dtype=torch.float32, device=Q.device)
    _check(load().pisa_sparse_attention(_ptr(Q), Hq, _ptr(K), _ptr(V), B, N, K.shape[2], _ptr(idx), idx.shape[-1],
                                        int(causal), _ptr(out), _stream(stream)),
           "pisa_sparse_attention")
    return out


def select_prefill_noalloc(Q: torch.Tensor, pyr: Pyramid, K: int, causal: bool = True,
                           with_scores: bool = True, out: tuple | None = None, stream=None):
    """select_prefill without a workspace: the library's built-in 32 MiB device
    scratch is used instead (for callers that cannot allocate device memory).
    Calls sharing that scratch must not overlap on the GPU."""
    B, N, Hq, _ = Q.shape
    if out is None:
        idx = torch.empty(B, pyr.Hkv, N, K, dtype=torch.int32, device=Q.device)
        scores = torch.empty(B, pyr.Hkv, N, K, dtype=torch.float32, device=Q.device) if with_scores else None
    else:
        idx, scores = out
    st = pyr.struct()
    _check(load().pisa_select_prefill_noalloc(_ptr(Q), Hq, ctypes.byref(st), N, K, int(causal), _ptr(idx),
                                              _ptr(scores), _stream(stream)),
           "pisa_select_prefill_noalloc")
    return idx, scores


def noalloc_prepare() -> int:
    """Set-up for select_prefill_noalloc on the current device (loads the library's
    device code there, which is when its scratch array comes into being); returns
    the scratch's device address."""
    p = ctypes.c_void_p()
    _check(load().pisa_noalloc_prepare(ctypes.byref(p)), "pisa_noalloc_prepare")
    return int(p.value or 0)


def noalloc_device_status(stream=None) -> int:
    """Synchronise the stream and return the status word of the last
    select_prefill_noalloc call on the current device (0 = ok)."""
    return int(load().pisa_noalloc_device_status(_stream(stream)))


def decode_workspace_bytes(B: int, Hq: int, Hkv: int, K: int) -> int:
    return int(load().pisa_decode_workspace_bytes(B, Hq, Hkv, K))


def decode_append_and_select(q_new: torch.Tensor, k_new: torch.Tensor, pyr: Pyramid, K: int,
                             with_scores: bool = True, workspace: torch.Tensor | None = None,
                             out: tuple | None = None, stream=None):
    """One decoding step: append k_new at lengths[b], refresh that leaf and its
    ancestors, then select for q_new.  Returns (idx [B, Hkv, K], scores)."""
    if pyr.lengths is None:
        raise ValueError("decode needs a Pyramid with lengths")
    B, Hq, _ = q_new.shape
    lib = load()
    need = lib.pisa_decode_workspace_bytes(B, Hq, pyr.Hkv, K)
    if need == 0:
        _check(2, "pisa_decode_workspace_bytes")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q_new.device)
    if out is None:
        idx = torch.empty(B, pyr.Hkv, K, dtype=torch.int32, device=q_new.device)
        scores = torch.empty(B, pyr.Hkv, K, dtype=torch.float32, device=q_new.device) if with_scores else None
    else:
        idx, scores = out
    st = pyr.struct()
    _check(lib.pisa_decode_append_and_select(_ptr(q_new), _ptr(k_new), Hq, ctypes.byref(st), K, _ptr(idx),
                                             _ptr(scores), _ptr(workspace), workspace.numel(),
                                             _stream(stream)),
           "pisa_decode_append_and_select")
    return idx, scores


class _CacheStruct(ctypes.Structure):
    _fields_ = [
        ("pages", ctypes.c_void_p),
        ("table", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64),
        ("B", ctypes.c_int),
        ("Hkv", ctypes.c_int),
        ("d", ctypes.c_int),
        ("page_size", ctypes.c_int),
        ("n_pages", ctypes.c_int),
        ("max_pages", ctypes.c_int),
        ("kind", ctypes.c_int),
        ("k_exp", ctypes.c_int),
        ("v_exp", ctypes.c_int),
    ]


class _RowsStruct(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("stride_b", ctypes.c_int64),
        ("stride_t", ctypes.c_int64),
        ("stride_h", ctypes.c_int64),
    ]


# a _RowsStruct as bytes: cheaper to make than the ctypes object, and as good an argument
_pack_rows = struct.Struct("Pqqq").pack


class PagedCache:
    """Caller-owned paged KV cache: the pages and the table that maps a sequence's tokens to them.

    pages: bf16 [n_pages, Hkv, page_size / U, 2, U, 64] (K, then V), or 4 bits as uint8
    [n_pages, Hkv, page_size / U, 72 U] (K codes [U, 32], K scales [U, 4], V codes, V scales; e2m1 codes, one
    e4m3 scale per 16 dims), U = min(page_size, 64).  Only the stride between pages may differ from dense (a
    pool that interleaves layers).  table: int32 [B, max_pages].  k_exp, v_exp (4 bits only): keys and values
    are held divided by 2^k_exp and 2^v_exp.  The descriptor is made once; the tensors' contents may change, the
    tensors may not.
    """

    __slots__ = ("pages", "table", "page_size", "B", "Hkv", "n_pages", "max_pages", "bits", "device", "_struct",
                 "_ref", "_index")

    def __init__(self, pages: torch.Tensor, table: torch.Tensor, page_size: int, k_exp: int = 0, v_exp: int = 0):
        if page_size not in (16, 32, 64, 128, 256):
            raise ValueError("page_size must be 16, 32, 64, 128 or 256")
        U = min(page_size, 64)
        if pages.dtype == torch.bfloat16 and pages.dim() == 6:
            bits, inner = 16, (page_size // U, 2, U, D)
        elif pages.dtype == torch.uint8 and pages.dim() == 4:
            bits, inner = 4, (page_size // U, 72 * U)
        else:
            raise ValueError("pages must be bf16 [n_pages, Hkv, page_size / U, 2, U, 64] or "
                             "uint8 [n_pages, Hkv, page_size / U, 72 U]")
        if tuple(pages.shape[2:]) != inner or pages.shape[0] < 1 or pages.shape[1] < 1:
            raise ValueError(f"pages of {page_size} tokens must be [n_pages, Hkv, {', '.join(map(str, inner))}]")
        if not pages[0].is_contiguous():
            raise ValueError("a page must be contiguous")
        if table.dtype != torch.int32 or table.dim() != 2 or not table.is_contiguous() or table.numel() < 1:
            raise ValueError("table must be a contiguous int32 tensor [B, max_pages]")
        if not pages.is_cuda or table.device != pages.device:
            raise ValueError("pages and table must be on the same CUDA device")
        self.pages, self.table, self.page_size, self.bits = pages, table, page_size, bits
        self.n_pages, self.Hkv = pages.shape[0], pages.shape[1]
        self.B, self.max_pages = table.shape
        self.device = pages.device
        self._index = pages.get_device()
        stride = pages.stride(0) if self.n_pages > 1 else pages[0].numel()
        self._struct = _CacheStruct(pages.data_ptr(), table.data_ptr(), stride * pages.element_size(), self.B,
                                    self.Hkv, D, page_size, self.n_pages, self.max_pages, 0 if bits == 16 else 1,
                                    k_exp, v_exp)
        self._ref = ctypes.byref(self._struct)

    @classmethod
    def allocate(cls, B: int, n_cap: int, Hkv: int, page_size: int = 64, bits: int = 16, device="cuda",
                 k_exp: int = 0, v_exp: int = 0) -> "PagedCache":
        """Pages (zeroed) and a table for B sequences of up to n_cap tokens, sequence b holding pages
        b * per .. (b + 1) * per - 1."""
        if page_size not in (16, 32, 64, 128, 256) or bits not in (4, 16) or B < 1 or n_cap < 1 or Hkv < 1:
            raise ValueError("page_size 16, 32, 64, 128 or 256, bits 4 or 16, B, n_cap and Hkv at least 1")
        U, per = min(page_size, 64), -(-n_cap // page_size)
        shape = (B * per, Hkv, page_size // U) + ((2, U, D) if bits == 16 else (72 * U,))
        pages = torch.zeros(shape, dtype=torch.bfloat16 if bits == 16 else torch.uint8, device=device)
        table = torch.arange(B * per, dtype=torch.int32, device=pages.device).view(B, per)
        return cls(pages, table, page_size, k_exp, v_exp)


def rotary_table(n: int, rot: int = D, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """Cosines and sines fp32 [n, rot] of positions 0 .. n - 1 at frequencies base^(-2 i / rot), the angles in 64
    bits (cache_append's `rotary`; any other table of that layout will do as well)."""
    if rot not in (16, 32, 48, 64) or n < 1:
        raise ValueError("rot must be 16, 32, 48 or 64 and n at least 1")
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=device)
    angle = torch.arange(n, dtype=torch.float64, device=device)[:, None] * base ** (-i / rot)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


_cache_ws_bytes = 0  # asked once: it is the same for every size


def cache_workspace_bytes() -> int:
    global _cache_ws_bytes
    _cache_ws_bytes = int(load().pisa_cache_workspace_bytes())
    return _cache_ws_bytes


def cache_workspace(cache: PagedCache) -> torch.Tensor:
    """A workspace for the cache calls on this cache's device, its status word zero.  One stream at a time; the
    word keeps the first error of all the calls (check_device_status)."""
    return torch.zeros(cache_workspace_bytes(), dtype=torch.uint8, device=cache.device)


# (the current stream's handle and the current device's number without the objects around them: a decoding step
# makes these calls once a layer, and the objects cost as much as the launch)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None
_get_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _on(cache: PagedCache, stream):
    """What has to be entered so that the cache's device, and `stream` if given, are current in a call (tensors
    that it allocates then belong to that stream); None where they are."""
    if stream is not None:
        if stream.device != cache.device:
            raise ValueError("the stream must be on the cache's device")
        return torch.cuda.stream(stream)
    return None if _get_device() == cache._index else torch.cuda.device(cache.device)


def _current(cache: PagedCache) -> int:
    return _raw_stream(cache._index) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


def _rows(x: torch.Tensor, what: str, cache: PagedCache, shape: tuple, written: bool = False) -> bytes:
    """The descriptor of rows of x [B, T, H, 64], checked to have that shape."""
    if x.dtype is not torch.bfloat16 or x.shape != shape or x.get_device() != cache._index:
        raise ValueError(f"{what} must be a bf16 tensor {list(shape)} on the cache's device")
    B, T, H, _ = shape
    sb, st, sh, sd = x.stride()
    if sd != 1:
        raise ValueError(f"the rows of {what} must be dense")
    # (the stride of a dimension of one entry is never used and may be anything)
    if B == 1:
        sb = 0
    elif written and sb == 0:
        raise ValueError(f"the rows of {what} must not share memory")
    if T == 1:
        st = 0
    elif written and st == 0:
        raise ValueError(f"the rows of {what} must not share memory")
    if H == 1:
        sh = 0
    elif written and sh == 0:
        raise ValueError(f"the rows of {what} must not share memory")
    return _pack_rows(x.data_ptr(), sb, st, sh)


def _per_sequence(x: torch.Tensor, what: str, cache: PagedCache) -> int:
    if (x.dtype is not torch.int32 or x.shape != (cache.B,) or x.get_device() != cache._index
            or not x.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous int32 tensor [{cache.B}] on the cache's device")
    return x.data_ptr()


def _cache_ws(workspace: torch.Tensor, cache: PagedCache, need: int) -> int:
    if workspace.dtype is not torch.uint8 or workspace.get_device() != cache._index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the cache's device")
    if workspace.numel() < need:
        raise PisaError(3, "workspace")
    return workspace.data_ptr()


def cache_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, cache: PagedCache, start: torch.Tensor,
                 rotary: torch.Tensor | None, counts: torch.Tensor | None = None, interleaved: bool = False,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None):
    """Rotate new queries and keys by their positions and put keys and values into the cache.

    q [B, T, Hq, 64] (or None), k and v [B, T, Hkv, 64] bf16, any strides that are multiples of 8; token t of
    sequence b goes to position start[b] + t (int32 [B]), t < counts[b] (int32 [B]; None: all T).  rotary fp32
    [n, rot], rot 16, 32, 48 or 64: cosines, then sines of each position (None: no rotation); pairs (i, i +
    rot / 2), or (2 i, 2 i + 1) when interleaved.  Returns (q_out, k_out): the rotated queries (None without q)
    and keys, allocated here when not given (rows t >= counts[b] are then not written); q_out may be q and
    k_out may be k.  workspace (of cache_workspace): for the status word only; without one, nothing tells of
    tokens that are left out because their position or page is out of range.
    """
    guard = _on(cache, stream)
    if guard is not None:
        with guard:
            return cache_append(q, k, v, cache, start, rotary, counts, interleaved, q_out, k_out, workspace)
    if k.dim() != 4:
        raise ValueError("k must be a bf16 tensor [B, T, Hkv, 64]")
    B, T = cache.B, k.shape[1]
    shape = (B, T, cache.Hkv, D)
    ks, vs = _rows(k, "k", cache, shape), _rows(v, "v", cache, shape)
    Hq, qs, qo = 0, None, None
    if q is not None:
        if q.dim() != 4:
            raise ValueError("q must be a bf16 tensor [B, T, Hq, 64]")
        Hq = q.shape[2]
        qshape = (B, T, Hq, D)
        qs = _rows(q, "q", cache, qshape)
        if q_out is None:
            q_out = torch.empty(qshape, dtype=torch.bfloat16, device=cache.device)
        qo = _rows(q_out, "q_out", cache, qshape, True)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k_out is None:
        k_out = torch.empty(shape, dtype=torch.bfloat16, device=cache.device)
    n_rot, rot, rp = 0, 0, None
    if rotary is not None:
        if (rotary.dtype is not torch.float32 or rotary.dim() != 2 or rotary.get_device() != cache._index
                or not rotary.is_contiguous()):
            raise ValueError("rotary must be a contiguous fp32 tensor [n, rot] on the cache's device")
        n_rot, rot = rotary.shape
        if rot not in (16, 32, 48, 64):
            raise ValueError("rotary must be [n, rot] with rot 16, 32, 48 or 64")
        rp = rotary.data_ptr()
    _check((_lib or load()).pisa_cache_append(
        cache._ref, T, qs, Hq, ks, vs, _per_sequence(start, "start", cache),
        None if counts is None else _per_sequence(counts, "counts", cache), rp, n_rot, rot, 1 if interleaved else 0,
        qo, _rows(k_out, "k_out", cache, shape, True), None if workspace is None else _cache_ws(workspace, cache, 4),
        _current(cache)), "pisa_cache_append")
    return q_out, k_out


def cache_read(cache: PagedCache, start: torch.Tensor, T: int, counts: torch.Tensor | None = None,
               k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None):
    """Cached tokens start[b] .. start[b] + counts[b] - 1 (T where counts is None) as dense bf16 (k, v)
    [B, T, Hkv, 64], exactly; allocated here when not given (rows t >= counts[b] are not written).  workspace
    as in cache_append."""
    guard = _on(cache, stream)
    if guard is not None:
        with guard:
            return cache_read(cache, start, T, counts, k_out, v_out, workspace)
    if T < 1:
        raise ValueError("T must be at least 1")
    shape = (cache.B, T, cache.Hkv, D)
    if k_out is None:
        k_out = torch.empty(shape, dtype=torch.bfloat16, device=cache.device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=torch.bfloat16, device=cache.device)
    _check((_lib or load()).pisa_cache_read(
        cache._ref, T, _per_sequence(start, "start", cache),
        None if counts is None else _per_sequence(counts, "counts", cache),
        _rows(k_out, "k_out", cache, shape, True), _rows(v_out, "v_out", cache, shape, True),
        None if workspace is None else _cache_ws(workspace, cache, 4), _current(cache)), "pisa_cache_read")
    return k_out, v_out


def cache_attention(q: torch.Tensor, cache: PagedCache, lengths: torch.Tensor, idx: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """The newest T tokens of every sequence attend over the cache: all of it, or the blocks of a selection.

    q [B, T, Hq, 64] bf16, 1 <= T <= 16; query t sits at position lengths[b] - T + t (lengths int32 [B], the new
    tokens included) and sees the tokens up to its own.  idx int32 [B, Hkv, T, Ksel] ([B, Hkv, Ksel] when T is
    1, as decode_append_and_select returns it): blocks of 64 tokens, -1 skipped.  out [B, T, Hq, 64], bf16
    (allocated here when not given) or fp32.  workspace (of cache_workspace, one stream at a time): a decoding
    program makes one and checks its status word (check_device_status); without one the call takes scratch of its
    own and nothing tells of errors: a length past the table's capacity is cut to it, and queries that see a page
    out of range are NaN.
    """
    guard = _on(cache, stream)
    if guard is not None:
        with guard:
            return cache_attention(q, cache, lengths, idx, out, workspace)
    if q.dim() != 4:
        raise ValueError("q must be a bf16 tensor [B, T, Hq, 64]")
    _, T, Hq, _ = q.shape
    B, Hkv = cache.B, cache.Hkv
    shape = (B, T, Hq, D)
    qs = _rows(q, "q", cache, shape)
    Ksel, ip = 0, None
    if idx is not None:
        Ksel = idx.shape[-1]
        if (idx.dtype is not torch.int32 or idx.get_device() != cache._index or not idx.is_contiguous() or Ksel < 1
                or not (idx.shape == (B, Hkv, T, Ksel) or (T == 1 and idx.shape == (B, Hkv, Ksel)))):
            raise ValueError(f"idx must be a contiguous int32 tensor [{B}, {Hkv}, {T}, Ksel], Ksel at least 1, on the "
                             "cache's device")
        ip = idx.data_ptr()
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=cache.device)
    elif ((out.dtype is not torch.bfloat16 and out.dtype is not torch.float32) or out.get_device() != cache._index
          or out.shape != shape or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous bf16 or fp32 tensor {list(shape)}")
    lib = _lib or load()
    need = _cache_ws_bytes or cache_workspace_bytes()
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=cache.device)
    _check(lib.pisa_cache_attention(cache._ref, qs, T, Hq,
                                    _per_sequence(lengths, "lengths", cache), ip, Ksel, out.data_ptr(),
                                    1 if out.dtype is torch.float32 else 0, _cache_ws(workspace, cache, need), need,
                                    _current(cache)), "pisa_cache_attention")
    return out


def kernel_launches() -> int:
    """Kernels the library has launched since it was loaded."""
    return int(load().pisa_kernel_launches())


def prefill_phases() -> list[str]:
    lib = load()
    return [lib.pisa_prefill_phase_name(i).decode() for i in range(lib.pisa_prefill_phase_count())]


def set_phase_events(events: list | None) -> None:
    """Attach torch.cuda.Event objects recorded at the prefill phase boundaries
    (len = number of phases + 1), or None to detach."""
    lib = load()
    if not events:
        _check(lib.pisa_set_phase_events(None, 0), "pisa_set_phase_events")
        return
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    set_phase_events._keep = arr
    _check(lib.pisa_set_phase_events(arr, len(events)), "pisa_set_phase_events")


def event_elapsed_ms(start, end) -> float:
    """Milliseconds between two torch.cuda.Event objects, either of which may
    have been recorded by the library (phase events)."""
    out = ctypes.c_float()
    _check(load().pisa_event_elapsed_ms(ctypes.c_void_p(start.cuda_event), ctypes.c_void_p(end.cuda_event),
                                        ctypes.byref(out)), "pisa_event_elapsed_ms")
    return float(out.value)


def selftest_bounded_wait(workspace: torch.Tensor, delay_cycles: int = 2_000_000, stream=None) -> None:
    """Make a kernel's bounded barrier wait run out (nothing arrives; an abort flag goes
    up after delay_cycles): its status word in `workspace` then reads the timeout code."""
    _check(load().pisa_selftest_bounded_wait(_ptr(workspace), workspace.numel(), int(delay_cycles), _stream(stream)),
           "pisa_selftest_bounded_wait")


def check_device_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise the stream and return the kernels' status word (0 = ok)."""
    return int(load().pisa_check_device_status(_ptr(workspace), _stream(stream)))
