"""Thin ctypes binding of ``libdeltakv.so`` (argument marshalling only).

Every computation runs in the library's CUDA kernels.  This module converts torch tensors to raw
pointers and sizes, checks their dtypes/devices/contiguity, calls the C entry point of the same name and
raises on a non-OK status.  There is no fallback: if the library is missing or fails to load, every call
raises ``RuntimeError``.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass
from functools import lru_cache
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdeltakv.so")

DKV_OK, DKV_ERR_INVALID_ARG, DKV_ERR_UNSUPPORTED, DKV_ERR_WORKSPACE, DKV_ERR_CUDA, DKV_ERR_OUT_OF_BLOCKS = range(6)
DKV_F32, DKV_BF16, DKV_BF16_Q4 = 0, 1, 2
DEVERR_NAMES = {0: "none", 1: "block id out of range", 2: "reference index out of range",
                3: "length over host bound", 4: "pipeline wait timed out"}

# every symbol include/deltakv.h declares
EXPORTED = ("deltakv_status_string", "deltakv_check_shape", "deltakv_block_bytes", "deltakv_cache_bytes",
            "deltakv_compress_workspace", "deltakv_decode_workspace", "deltakv_compress",
            "deltakv_decode_attention", "deltakv_profile_kernel", "deltakv_profile_count",
            "deltakv_get_device_error", "deltakv_decode_attention_noalloc", "deltakv_decode_sparse_workspace",
            "deltakv_decode_attention_sparse", "deltakv_compress_topk", "deltakv_decode_topk_workspace",
            "deltakv_decode_attention_topk", "deltakv_selftest_wait_timeout", "deltakv_kv8_cache_bytes",
            "deltakv_kv8_append", "deltakv_kv8_attention_workspace", "deltakv_kv8_attention",
            "deltakv_merge_attention")
KV8_CODES = {"int8": 0, "e4m3": 1}
MERGE_MAX_PARTS = 8
NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024
KERNEL_CENTER, KERNEL_REFPREP, KERNEL_SEARCH, KERNEL_DECODE_PROLOGUE, KERNEL_DECODE_SPLIT, KERNEL_DECODE_COMBINE = range(6)


class DkvShape(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("ref_stride", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class DkvParams(ctypes.Structure):
    _fields_ = [("mu", ctypes.c_void_p), ("basis", ctypes.c_void_p)]


class DkvCache(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("ref_idx", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("num_blocks", ctypes.c_int32)]


class DkvKv8Shape(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_tokens", ctypes.c_int32), ("dtype", ctypes.c_int32), ("code", ctypes.c_int32)]


class DkvKv8Cache(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("num_blocks", ctypes.c_int32)]


class DkvKv8Rope(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("max_pos", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("pairs", ctypes.c_int32)]


class DkvKv8Score(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int32), ("alibi_slopes", ctypes.c_void_p),
                ("prefix_lens", ctypes.c_void_p), ("first_key", ctypes.c_void_p)]


_lib = None


def load_library() -> ctypes.CDLL:
    """Load ``libdeltakv.so`` (built in-tree by ``build.py``); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libdeltakv.so not built ({LIB_PATH}); run residual_kv_cache_delta_b200/build.py")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    pshape, pparams, pcache = ctypes.POINTER(DkvShape), ctypes.POINTER(DkvParams), ctypes.POINTER(DkvCache)
    lib.deltakv_status_string.argtypes = [ctypes.c_int]
    lib.deltakv_status_string.restype = ctypes.c_char_p
    lib.deltakv_check_shape.argtypes = [pshape]
    lib.deltakv_check_shape.restype = ctypes.c_int
    lib.deltakv_block_bytes.argtypes = [pshape]
    lib.deltakv_block_bytes.restype = SZ
    lib.deltakv_cache_bytes.argtypes = [pshape, I32, ctypes.POINTER(SZ), ctypes.POINTER(SZ), ctypes.POINTER(SZ)]
    lib.deltakv_cache_bytes.restype = ctypes.c_int
    lib.deltakv_compress_workspace.argtypes = [pshape, I32, I64, I32, I32, ctypes.POINTER(SZ)]
    lib.deltakv_compress_workspace.restype = ctypes.c_int
    lib.deltakv_decode_workspace.argtypes = [pshape, I32, I32, ctypes.POINTER(SZ)]
    lib.deltakv_decode_workspace.restype = ctypes.c_int
    lib.deltakv_compress.argtypes = [pshape, pparams, pcache, P, P, P, P, P, I32, I32, I64, I32, I32, P, SZ, P]
    lib.deltakv_compress.restype = ctypes.c_int
    lib.deltakv_decode_attention.argtypes = [pshape, pparams, pcache, P, P, P, I32, I32, I32, ctypes.c_float, P, P,
                                             P, SZ, P]
    lib.deltakv_decode_attention.restype = ctypes.c_int
    lib.deltakv_profile_kernel.argtypes = [I32, P, P, I32]
    lib.deltakv_profile_kernel.restype = ctypes.c_int
    lib.deltakv_profile_count.argtypes = [I32, ctypes.POINTER(I32)]
    lib.deltakv_profile_count.restype = ctypes.c_int
    lib.deltakv_decode_attention_noalloc.argtypes = [pshape, pparams, pcache, P, P, P, I32, I32, I32, ctypes.c_float,
                                                     P, P, P]
    lib.deltakv_decode_attention_noalloc.restype = ctypes.c_int
    lib.deltakv_decode_sparse_workspace.argtypes = [pshape, I32, I32, I32, ctypes.POINTER(SZ)]
    lib.deltakv_decode_sparse_workspace.restype = ctypes.c_int
    lib.deltakv_decode_attention_sparse.argtypes = [pshape, pparams, pcache, P, P, P, I32, P, P, I32, I32, I32,
                                                    ctypes.c_float, P, P, P, SZ, P]
    lib.deltakv_decode_attention_sparse.restype = ctypes.c_int
    lib.deltakv_compress_topk.argtypes = [pshape, I32, pparams, pcache, P, P, P, P, P, I32, I32, I64, I32, I32, P,
                                          SZ, P]
    lib.deltakv_compress_topk.restype = ctypes.c_int
    lib.deltakv_decode_topk_workspace.argtypes = [pshape, I32, I32, I32, ctypes.POINTER(SZ)]
    lib.deltakv_decode_topk_workspace.restype = ctypes.c_int
    lib.deltakv_decode_attention_topk.argtypes = [pshape, I32, pparams, pcache, P, P, P, I32, I32, I32, ctypes.c_float,
                                                  P, P, P, SZ, P]
    lib.deltakv_decode_attention_topk.restype = ctypes.c_int
    lib.deltakv_get_device_error.argtypes = [P, ctypes.POINTER(I32)]
    lib.deltakv_get_device_error.restype = ctypes.c_int
    lib.deltakv_selftest_wait_timeout.argtypes = [ctypes.c_uint64, P, P]
    lib.deltakv_selftest_wait_timeout.restype = ctypes.c_int
    pkshape, pkcache = ctypes.POINTER(DkvKv8Shape), ctypes.POINTER(DkvKv8Cache)
    lib.deltakv_kv8_cache_bytes.argtypes = [pkshape, I32, ctypes.POINTER(SZ), ctypes.POINTER(SZ)]
    lib.deltakv_kv8_cache_bytes.restype = ctypes.c_int
    lib.deltakv_kv8_append.argtypes = [pkshape, pkcache, ctypes.POINTER(DkvKv8Rope), P, I64, P, I64, P, P, P, I32, I32,
                                       I64, I32, P, I64, P, P]
    lib.deltakv_kv8_append.restype = ctypes.c_int
    lib.deltakv_kv8_attention_workspace.argtypes = [pkshape, I32, I64, I32, I32, ctypes.POINTER(SZ)]
    lib.deltakv_kv8_attention_workspace.restype = ctypes.c_int
    lib.deltakv_kv8_attention.argtypes = [pkshape, pkcache, ctypes.POINTER(DkvKv8Score), P, I64, P, P, P, I32, I32, I64,
                                          I32, I32, ctypes.c_float, P, P, P, SZ, P]
    lib.deltakv_kv8_attention.restype = ctypes.c_int
    lib.deltakv_merge_attention.argtypes = [I32, I32, I64, I32, ctypes.POINTER(P), ctypes.POINTER(P), P, P, P]
    lib.deltakv_merge_attention.restype = ctypes.c_int
    _lib = lib
    return lib


class DeltaKVError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


def status_string(status: int) -> str:
    return load_library().deltakv_status_string(status).decode()


def _check(status: int, what: str):
    if status != DKV_OK:
        raise DeltaKVError(status, what)


@dataclass(frozen=True)
class Shape:
    """Head geometry of one layer (mirrors ``dkv_shape``)."""

    num_q_heads: int
    num_kv_heads: int
    head_dim: int
    rank: int
    ref_stride: int
    dtype: torch.dtype = torch.bfloat16
    q4: bool = False  # 4-bit residual codes (bf16 storage otherwise; see include/deltakv.h)

    @property
    def c(self) -> DkvShape:
        dt = DKV_F32 if self.dtype == torch.float32 else (DKV_BF16_Q4 if self.q4 else DKV_BF16)
        return DkvShape(self.num_q_heads, self.num_kv_heads, self.head_dim, self.rank, self.ref_stride, dt)

    @property
    def group(self) -> int:
        return self.num_q_heads // self.num_kv_heads


def check_shape(shape: Shape) -> int:
    return load_library().deltakv_check_shape(ctypes.byref(shape.c))


def block_bytes(shape: Shape) -> int:
    return int(load_library().deltakv_block_bytes(ctypes.byref(shape.c)))


def cache_bytes(shape: Shape, num_blocks: int) -> tuple[int, int, int]:
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().deltakv_cache_bytes(ctypes.byref(shape.c), num_blocks, ctypes.byref(a), ctypes.byref(b),
                                              ctypes.byref(c)), "deltakv_cache_bytes")
    return a.value, b.value, c.value


def compress_workspace(shape: Shape, num_seqs: int, total_new: int, max_new: int, max_ctx: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().deltakv_compress_workspace(ctypes.byref(shape.c), num_seqs, total_new, max_new, max_ctx,
                                                     ctypes.byref(n)), "deltakv_compress_workspace")
    return n.value


def decode_workspace(shape: Shape, num_seqs: int, max_ctx: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().deltakv_decode_workspace(ctypes.byref(shape.c), num_seqs, max_ctx, ctypes.byref(n)),
           "deltakv_decode_workspace")
    return n.value


def decode_sparse_workspace(shape: Shape, num_seqs: int, max_ctx: int, max_sel: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().deltakv_decode_sparse_workspace(ctypes.byref(shape.c), num_seqs, max_ctx, max_sel,
                                                          ctypes.byref(n)), "deltakv_decode_sparse_workspace")
    return n.value


@dataclass
class Cache:
    """Caller-owned device arrays of one layer's compressed cache (layout in include/deltakv.h)."""

    codes: torch.Tensor    # [num_blocks, H_kv, R, 2r] dtype
    ref_idx: torch.Tensor  # [num_blocks, H_kv, R] int32
    refs: torch.Tensor     # [num_blocks, H_kv, 2, d] dtype

    @property
    def num_blocks(self) -> int:
        return self.codes.shape[0]

    @property
    def c(self) -> DkvCache:
        return DkvCache(self.codes.data_ptr(), self.ref_idx.data_ptr(), self.refs.data_ptr(), self.num_blocks)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.codes, self.ref_idx, self.refs))


def alloc_cache(shape: Shape, num_blocks: int, device="cuda", topk: int = 0) -> Cache:
    """Zeroed cache arrays.  With 4-bit codes, ``codes`` is uint8 [num_blocks, H_kv, R*(r+4)] (per block and
    kv head: R packed rows of r bytes, then R pairs of bf16 scales).  topk > 0 (the k-nearest compress):
    ``ref_idx`` is [num_blocks, H_kv, R, k]."""
    H, R, r, d = shape.num_kv_heads, shape.ref_stride, shape.rank, shape.head_dim
    if topk > 0:
        return Cache(torch.zeros((num_blocks, H, R, 2 * r), dtype=shape.dtype, device=device),
                     torch.zeros((num_blocks, H, R, topk), dtype=torch.int32, device=device),
                     torch.zeros((num_blocks, H, 2, d), dtype=shape.dtype, device=device))
    if shape.q4:
        return Cache(torch.zeros((num_blocks, H, R * (r + 4)), dtype=torch.uint8, device=device),
                     torch.zeros((num_blocks, H, R), dtype=torch.int32, device=device),
                     torch.zeros((num_blocks, H, 2, d), dtype=shape.dtype, device=device))
    return Cache(torch.zeros((num_blocks, H, R, 2 * r), dtype=shape.dtype, device=device),
                 torch.zeros((num_blocks, H, R), dtype=torch.int32, device=device),
                 torch.zeros((num_blocks, H, 2, d), dtype=shape.dtype, device=device))


def alloc_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A 256-byte-aligned byte buffer (torch's caching allocator returns 512-byte-aligned blocks)."""
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def _ptr(t: Optional[torch.Tensor], dtype: Optional[torch.dtype] = None, name: str = "") -> int:
    if t is None:
        return 0
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def deltakv_compress(shape: Shape, mu: torch.Tensor, basis: torch.Tensor, cache: Cache, k_new: torch.Tensor,
                     v_new: torch.Tensor, cu_new: torch.Tensor, start_pos: torch.Tensor, block_tables: torch.Tensor,
                     max_new: int, max_ctx: int, workspace: torch.Tensor, stream=None) -> None:
    """Enqueue ``deltakv_compress`` (see include/deltakv.h).  Shapes: k_new/v_new [total_new, H_kv, d];
    cu_new [num_seqs+1]; start_pos [num_seqs]; block_tables [num_seqs, max_blocks] (all int32)."""
    sc = shape.c
    params = DkvParams(_ptr(mu, torch.float32, "mu"), _ptr(basis, shape.dtype, "basis"))
    cc = cache.c
    num_seqs, max_blocks = block_tables.shape
    st = load_library().deltakv_compress(
        ctypes.byref(sc), ctypes.byref(params), ctypes.byref(cc), _ptr(k_new, shape.dtype, "k_new"),
        _ptr(v_new, shape.dtype, "v_new"), _ptr(cu_new, torch.int32, "cu_new"),
        _ptr(start_pos, torch.int32, "start_pos"), _ptr(block_tables, torch.int32, "block_tables"), max_blocks,
        num_seqs, k_new.shape[0], max_new, max_ctx, _ptr(workspace, torch.uint8, "workspace"),
        workspace.numel(), _stream(stream))
    _check(st, "deltakv_compress")


def deltakv_decode_attention(shape: Shape, mu: torch.Tensor, basis: torch.Tensor, cache: Cache, q: torch.Tensor,
                             context_lens: torch.Tensor, block_tables: torch.Tensor, max_ctx: int,
                             out: torch.Tensor, lse: Optional[torch.Tensor], workspace: torch.Tensor,
                             softmax_scale: float = 0.0, stream=None) -> None:
    """Enqueue ``deltakv_decode_attention``.  q/out [num_seqs, H_q, d]; lse [num_seqs, H_q] fp32 or None."""
    sc = shape.c
    params = DkvParams(_ptr(mu, torch.float32, "mu"), _ptr(basis, shape.dtype, "basis"))
    cc = cache.c
    num_seqs, max_blocks = block_tables.shape
    st = load_library().deltakv_decode_attention(
        ctypes.byref(sc), ctypes.byref(params), ctypes.byref(cc), _ptr(q, shape.dtype, "q"),
        _ptr(context_lens, torch.int32, "context_lens"), _ptr(block_tables, torch.int32, "block_tables"),
        max_blocks, num_seqs, max_ctx, float(softmax_scale), _ptr(out, shape.dtype, "out"),
        _ptr(lse, torch.float32, "lse"), _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
        _stream(stream))
    _check(st, "deltakv_decode_attention")


def deltakv_decode_attention_noalloc(shape: Shape, mu: torch.Tensor, basis: torch.Tensor, cache: Cache,
                                     q: torch.Tensor, context_lens: torch.Tensor, block_tables: torch.Tensor,
                                     max_ctx: int, out: torch.Tensor, lse: Optional[torch.Tensor],
                                     softmax_scale: float = 0.0, stream=None) -> None:
    """Enqueue ``deltakv_decode_attention_noalloc``: decode attention with the library's own fixed scratch
    array instead of a caller workspace (no device allocation anywhere; see include/deltakv.h)."""
    sc = shape.c
    params = DkvParams(_ptr(mu, torch.float32, "mu"), _ptr(basis, shape.dtype, "basis"))
    cc = cache.c
    num_seqs, max_blocks = block_tables.shape
    st = load_library().deltakv_decode_attention_noalloc(
        ctypes.byref(sc), ctypes.byref(params), ctypes.byref(cc), _ptr(q, shape.dtype, "q"),
        _ptr(context_lens, torch.int32, "context_lens"), _ptr(block_tables, torch.int32, "block_tables"),
        max_blocks, num_seqs, max_ctx, float(softmax_scale), _ptr(out, shape.dtype, "out"),
        _ptr(lse, torch.float32, "lse"), _stream(stream))
    _check(st, "deltakv_decode_attention_noalloc")


def deltakv_decode_attention_sparse(shape: Shape, mu: torch.Tensor, basis: torch.Tensor, cache: Cache,
                                    q: torch.Tensor, context_lens: torch.Tensor, block_tables: torch.Tensor,
                                    token_idx: torch.Tensor, cu_tokens: torch.Tensor, max_sel: int, max_ctx: int,
                                    out: torch.Tensor, lse: Optional[torch.Tensor], workspace: torch.Tensor,
                                    softmax_scale: float = 0.0, stream=None) -> None:
    """Enqueue ``deltakv_decode_attention_sparse``: decode over the positions token_idx[cu_tokens[s] ..
    cu_tokens[s+1]-1] of each sequence (int32 device tensors); other arguments as in the dense call."""
    sc = shape.c
    params = DkvParams(_ptr(mu, torch.float32, "mu"), _ptr(basis, shape.dtype, "basis"))
    cc = cache.c
    num_seqs, max_blocks = block_tables.shape
    tok = _ptr(token_idx, torch.int32, "token_idx") if token_idx.numel() > 0 else 0
    st = load_library().deltakv_decode_attention_sparse(
        ctypes.byref(sc), ctypes.byref(params), ctypes.byref(cc), _ptr(q, shape.dtype, "q"),
        _ptr(context_lens, torch.int32, "context_lens"), _ptr(block_tables, torch.int32, "block_tables"),
        max_blocks, tok, _ptr(cu_tokens, torch.int32, "cu_tokens"), max_sel, num_seqs, max_ctx,
        float(softmax_scale), _ptr(out, shape.dtype, "out"), _ptr(lse, torch.float32, "lse"),
        _ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream))
    _check(st, "deltakv_decode_attention_sparse")


def decode_topk_workspace(shape: Shape, k: int, num_seqs: int, max_ctx: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().deltakv_decode_topk_workspace(ctypes.byref(shape.c), k, num_seqs, max_ctx, ctypes.byref(n)),
           "deltakv_decode_topk_workspace")
    return n.value


def deltakv_compress_topk(shape: Shape, k: int, mu: torch.Tensor, basis: torch.Tensor, cache: Cache,
                          k_new: torch.Tensor, v_new: torch.Tensor, cu_new: torch.Tensor, start_pos: torch.Tensor,
                          block_tables: torch.Tensor, max_new: int, max_ctx: int, workspace: torch.Tensor,
                          stream=None) -> None:
    """Enqueue ``deltakv_compress_topk`` (the k nearest references by L2, residual against their mean); the
    cache's ref_idx holds k slots per token (alloc_cache(..., topk=k))."""
    sc = shape.c
    params = DkvParams(_ptr(mu, torch.float32, "mu"), _ptr(basis, shape.dtype, "basis"))
    cc = cache.c
    num_seqs, max_blocks = block_tables.shape
    st = load_library().deltakv_compress_topk(
        ctypes.byref(sc), k, ctypes.byref(params), ctypes.byref(cc), _ptr(k_new, shape.dtype, "k_new"),
        _ptr(v_new, shape.dtype, "v_new"), _ptr(cu_new, torch.int32, "cu_new"),
        _ptr(start_pos, torch.int32, "start_pos"), _ptr(block_tables, torch.int32, "block_tables"), max_blocks,
        num_seqs, k_new.shape[0], max_new, max_ctx, _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
        _stream(stream))
    _check(st, "deltakv_compress_topk")


def deltakv_decode_attention_topk(shape: Shape, k: int, mu: torch.Tensor, basis: torch.Tensor, cache: Cache,
                                  q: torch.Tensor, context_lens: torch.Tensor, block_tables: torch.Tensor,
                                  max_ctx: int, out: torch.Tensor, lse: Optional[torch.Tensor],
                                  workspace: torch.Tensor, softmax_scale: float = 0.0, stream=None) -> None:
    """Enqueue ``deltakv_decode_attention_topk`` over a cache written by deltakv_compress_topk with the same k."""
    sc = shape.c
    params = DkvParams(_ptr(mu, torch.float32, "mu"), _ptr(basis, shape.dtype, "basis"))
    cc = cache.c
    num_seqs, max_blocks = block_tables.shape
    st = load_library().deltakv_decode_attention_topk(
        ctypes.byref(sc), k, ctypes.byref(params), ctypes.byref(cc), _ptr(q, shape.dtype, "q"),
        _ptr(context_lens, torch.int32, "context_lens"), _ptr(block_tables, torch.int32, "block_tables"),
        max_blocks, num_seqs, max_ctx, float(softmax_scale), _ptr(out, shape.dtype, "out"),
        _ptr(lse, torch.float32, "lse"), _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
        _stream(stream))
    _check(st, "deltakv_decode_attention_topk")


class KV8Shape(NamedTuple):
    """Head geometry of one layer of the 8-bit cache (mirrors ``dkv_kv8_shape``); code "int8" or "e4m3"."""

    num_q_heads: int
    num_kv_heads: int
    head_dim: int
    block_tokens: int
    dtype: torch.dtype = torch.bfloat16
    code: str = "int8"

    @property
    def c(self) -> DkvKv8Shape:
        if self.dtype not in (torch.bfloat16, torch.float32) or self.code not in KV8_CODES:
            raise ValueError(f"KV8Shape: dtype {self.dtype}, code {self.code!r}")
        return DkvKv8Shape(self.num_q_heads, self.num_kv_heads, self.head_dim, self.block_tokens,
                           DKV_F32 if self.dtype == torch.float32 else DKV_BF16, KV8_CODES[self.code])

    @property
    def code_dtype(self) -> torch.dtype:
        return torch.int8 if self.code == "int8" else torch.float8_e4m3fn


@lru_cache(maxsize=64)
def _kv8_shape(shape: KV8Shape):
    """(pointer to the shape's structure, dtype of its codes): what every call needs of a shape."""
    return ctypes.byref(shape.c), shape.code_dtype


@dataclass
class KV8Cache:
    """Caller-owned device arrays of one layer's 8-bit cache."""

    codes: torch.Tensor   # [num_blocks, H_kv, 2, B, d] int8 or float8_e4m3fn
    scales: torch.Tensor  # [num_blocks, H_kv, 2] float32

    @property
    def num_blocks(self) -> int:
        return self.codes.shape[0]

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.codes, self.scales))


def alloc_kv8_cache(shape: KV8Shape, num_blocks: int, device="cuda") -> KV8Cache:
    """Zeroed cache arrays (append writes a block before anything reads it, so their contents do not matter)."""
    H, B, d = shape.num_kv_heads, shape.block_tokens, shape.head_dim
    return KV8Cache(torch.zeros((num_blocks, H, 2, B, d), dtype=torch.uint8, device=device).view(shape.code_dtype),
                    torch.zeros((num_blocks, H, 2), dtype=torch.float32, device=device))


def kv8_cache_bytes(shape: KV8Shape, num_blocks: int) -> tuple[int, int]:
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().deltakv_kv8_cache_bytes(ctypes.byref(shape.c), num_blocks, ctypes.byref(a), ctypes.byref(b)),
           "deltakv_kv8_cache_bytes")
    return a.value, b.value


def kv8_attention_workspace(shape: KV8Shape, num_seqs: int, total_q: int, max_q: int, max_ctx: int) -> int:
    """Bytes of workspace for every call within these bounds (the size never falls as a bound grows)."""
    n = ctypes.c_size_t()
    _check(load_library().deltakv_kv8_attention_workspace(ctypes.byref(shape.c), num_seqs, total_q, max_q, max_ctx,
                                                          ctypes.byref(n)), "deltakv_kv8_attention_workspace")
    return n.value


def _refuse(t, dims: tuple, dtype: torch.dtype, name: str, dev: int):
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name} must be on {'a GPU' if dev < 0 else f'cuda:{dev}'}, got {t.device}")
    if t.shape != dims:
        raise ValueError(f"{name} must have shape {dims}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous")


def _sized(t: torch.Tensor, dims: tuple, dtype: torch.dtype, name: str, dev: int) -> int:
    """Pointer of a contiguous tensor of exactly these dimensions on GPU ``dev``."""
    if dev < 0 or t.get_device() != dev or t.shape != dims or t.dtype is not dtype or not t.is_contiguous():
        _refuse(t, dims, dtype, name, dev)
    return t.data_ptr()


def _rows(t: torch.Tensor, n: int, heads: int, shape: KV8Shape, name: str, dev: int) -> tuple[int, int]:
    """Pointer and row stride of [n, heads, d] whose rows may lie apart (a view of a fused projection)."""
    d = shape.head_dim
    if dev < 0 or t.get_device() != dev or t.shape != (n, heads, d) or t.dtype is not shape.dtype:
        _refuse(t, (n, heads, d), shape.dtype, name, dev)
    st = t.stride()
    if n > 0 and (st[2] != 1 or (heads > 1 and st[1] != d)):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return t.data_ptr(), (st[0] if n > 1 else heads * d)


def _kv8_cache(shape: KV8Shape, cache: KV8Cache, code: torch.dtype, dev: int):
    codes, H = cache.codes, shape.num_kv_heads
    nb = codes.shape[0]
    return ctypes.byref(DkvKv8Cache(
        _sized(codes, (nb, H, 2, shape.block_tokens, shape.head_dim), code, "cache.codes", dev),
        _sized(cache.scales, (nb, H, 2), torch.float32, "cache.scales", dev), nb))


# the current stream's handle, without a Stream object for each call where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _call_on(dev: int, stream, fn, *args) -> int:
    """fn(*args, stream) with GPU ``dev`` current; its current stream unless one is given."""
    if torch.cuda.current_device() == dev:
        return fn(*args, _raw_stream(dev) if stream is None else _stream(stream))
    with torch.cuda.device(dev):
        return fn(*args, _raw_stream(dev) if stream is None else _stream(stream))


def deltakv_kv8_append(shape: KV8Shape, cache: KV8Cache, k_new: torch.Tensor, v_new: torch.Tensor,
                       cu_new: torch.Tensor, start_pos: torch.Tensor, block_tables: torch.Tensor, max_new: int,
                       rope: Optional[torch.Tensor] = None, rope_pairs: bool = False,
                       positions: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                       q_out: Optional[torch.Tensor] = None, stream=None) -> None:
    """Enqueue ``deltakv_kv8_append``.  k_new/v_new [total_new, H_kv, d] (rows may be strided); cu_new [num_seqs+1],
    start_pos [num_seqs], block_tables [num_seqs, max_blocks] int32; rope [max_pos, rot_dim] fp32 (cosines, then
    sines); positions [total_new] int32 or None; q [total_new, H_q, d] with q_out of the same shape, or None."""
    dev, n = cache.codes.get_device(), k_new.shape[0]
    cs, code = _kv8_shape(shape)
    cc = _kv8_cache(shape, cache, code, dev)
    num_seqs, max_blocks = block_tables.shape
    kp, ks = _rows(k_new, n, shape.num_kv_heads, shape, "k_new", dev)
    vp, vs = _rows(v_new, n, shape.num_kv_heads, shape, "v_new", dev)
    qp, qs, qo, cr = 0, 0, 0, None
    if rope is not None:
        max_pos, rot = rope.shape
        pp = 0 if positions is None else _sized(positions, (n,), torch.int32, "positions", dev)
        cr = ctypes.byref(DkvKv8Rope(_sized(rope, (max_pos, rot), torch.float32, "rope", dev), pp, max_pos, rot,
                                     int(rope_pairs)))
    elif positions is not None:
        raise ValueError("positions without rope")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q is not None:
        qp, qs = _rows(q, n, shape.num_q_heads, shape, "q", dev)
        qo = _sized(q_out, (n, shape.num_q_heads, shape.head_dim), shape.dtype, "q_out", dev)
    st = _call_on(dev, stream, load_library().deltakv_kv8_append, cs, cc, cr, kp, ks, vp,
                  vs, _sized(cu_new, (num_seqs + 1,), torch.int32, "cu_new", dev),
                  _sized(start_pos, (num_seqs,), torch.int32, "start_pos", dev),
                  _sized(block_tables, (num_seqs, max_blocks), torch.int32, "block_tables", dev), max_blocks, num_seqs, n,
                  max_new, qp, qs, qo)
    _check(st, "deltakv_kv8_append")


def deltakv_kv8_attention(shape: KV8Shape, cache: KV8Cache, q: torch.Tensor, cu_q: Optional[torch.Tensor],
                          context_lens: torch.Tensor, block_tables: torch.Tensor, max_q: int, max_ctx: int,
                          out: torch.Tensor, lse: Optional[torch.Tensor], workspace: Optional[torch.Tensor],
                          softmax_scale: float = 0.0, softcap: float = 0.0, window: int = 0,
                          alibi_slopes: Optional[torch.Tensor] = None, prefix_lens: Optional[torch.Tensor] = None,
                          first_key: Optional[torch.Tensor] = None, stream=None) -> None:
    """Enqueue ``deltakv_kv8_attention``.  q [total_q, H_q, d] (rows may be strided), out the same shape, lse [total_q,
    H_q] fp32 or None; cu_q [num_seqs+1] or None (one query token per sequence), context_lens [num_seqs], block_tables
    [num_seqs, max_blocks] int32; alibi_slopes [H_q] fp32, prefix_lens [num_seqs] and first_key [total_q] int32."""
    dev, n = cache.codes.get_device(), q.shape[0]
    cs, code = _kv8_shape(shape)
    cc, i32, f32 = _kv8_cache(shape, cache, code, dev), torch.int32, torch.float32
    num_seqs, max_blocks = block_tables.shape
    H = shape.num_q_heads
    qp, qs = _rows(q, n, H, shape, "q", dev)
    score = None
    if softcap or window or alibi_slopes is not None or prefix_lens is not None or first_key is not None:
        score = ctypes.byref(DkvKv8Score(
            softcap, window, 0 if alibi_slopes is None else _sized(alibi_slopes, (H,), f32, "alibi_slopes", dev),
            0 if prefix_lens is None else _sized(prefix_lens, (num_seqs,), i32, "prefix_lens", dev),
            0 if first_key is None else _sized(first_key, (n,), i32, "first_key", dev)))
    wsn = 0 if workspace is None else workspace.numel()
    st = _call_on(dev, stream, load_library().deltakv_kv8_attention, cs, cc, score, qp,
                  qs, 0 if cu_q is None else _sized(cu_q, (num_seqs + 1,), i32, "cu_q", dev),
                  _sized(context_lens, (num_seqs,), i32, "context_lens", dev),
                  _sized(block_tables, (num_seqs, max_blocks), i32, "block_tables", dev), max_blocks, num_seqs, n, max_q,
                  max_ctx, softmax_scale, _sized(out, (n, H, shape.head_dim), shape.dtype, "out", dev),
                  0 if lse is None else _sized(lse, (n, H), f32, "lse", dev),
                  0 if workspace is None else _sized(workspace, (wsn,), torch.uint8, "workspace", dev), wsn)
    _check(st, "deltakv_kv8_attention")


def deltakv_merge_attention(outs, lses, out: torch.Tensor, lse: Optional[torch.Tensor], stream=None) -> None:
    """Enqueue ``deltakv_merge_attention``: outs, lses are lists of [..., d] and [...] (fp32) tensors, the results of
    the same queries over disjoint keys (deltakv_decode_attention*, deltakv_kv8_attention); out/lse of the same shapes."""
    n = len(outs)
    if len(lses) != n or not 1 <= n <= MERGE_MAX_PARTS:
        raise ValueError(f"1 to {MERGE_MAX_PARTS} parts, as many lses as outs: got {n} and {len(lses)}")
    dev, dims, dt, f32 = out.get_device(), tuple(out.shape), out.dtype, torch.float32
    if dt not in (torch.bfloat16, f32) or not dims:
        raise ValueError(f"out: {dt} of shape {dims}")
    rdims = dims[:-1]
    P = ctypes.c_void_p * n
    po = P(*[_sized(t, dims, dt, "outs", dev) for t in outs])
    pl = P(*[_sized(t, rdims, f32, "lses", dev) for t in lses])
    st = _call_on(dev, stream, load_library().deltakv_merge_attention, DKV_F32 if dt is f32 else DKV_BF16, dims[-1],
                  math.prod(rdims), n, po, pl, _sized(out, dims, dt, "out", dev),
                  0 if lse is None else _sized(lse, rdims, f32, "lse", dev))
    _check(st, "deltakv_merge_attention")


class KernelTimer:
    """Records CUDA events around the next ``n`` launches of one library kernel (deltakv_profile_kernel)."""

    def __init__(self, kernel_id: int, n: int):
        self.kernel_id = kernel_id
        self.starts = [torch.cuda.Event(enable_timing=True) for _ in range(n)]
        self.stops = [torch.cuda.Event(enable_timing=True) for _ in range(n)]
        for e in self.starts + self.stops:
            e.record()  # materialise the underlying cudaEvent_t
        torch.cuda.synchronize()
        self._a = (ctypes.c_void_p * n)(*[e.cuda_event for e in self.starts])
        self._b = (ctypes.c_void_p * n)(*[e.cuda_event for e in self.stops])
        _check(load_library().deltakv_profile_kernel(kernel_id, self._a, self._b, n), "deltakv_profile_kernel")

    def count(self) -> int:
        c = ctypes.c_int32()
        _check(load_library().deltakv_profile_count(self.kernel_id, ctypes.byref(c)), "deltakv_profile_count")
        return c.value

    def times_ms(self) -> list:
        torch.cuda.synchronize()
        return [a.elapsed_time(b) for a, b in zip(self.starts[: self.count()], self.stops[: self.count()])]

    def close(self):
        _check(load_library().deltakv_profile_kernel(self.kernel_id, None, None, 0), "deltakv_profile_kernel")


def deltakv_get_device_error(stream=None) -> int:
    """Synchronise ``stream`` and return (and clear) the device error word (0 = none)."""
    code = ctypes.c_int32()
    _check(load_library().deltakv_get_device_error(_stream(stream), ctypes.byref(code)), "deltakv_get_device_error")
    return code.value


def deltakv_selftest_wait_timeout(limit_ns: int, result: torch.Tensor, stream=None) -> None:
    """One bounded wait on a phase that nothing completes, with limit ``limit_ns``; ``result`` is a device int64
    tensor of 2 elements: [completed, waited ns]."""
    assert result.is_cuda and result.dtype == torch.int64 and result.numel() >= 2
    _check(load_library().deltakv_selftest_wait_timeout(int(limit_ns), _ptr(result), _stream(stream)),
           "deltakv_selftest_wait_timeout")
