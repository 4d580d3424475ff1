"""Thin Python binding of libkvq (the C ABI declared in include/kvq.h,
include/kvq_fp8_block.h and include/kvq_latent.h).

Argument marshalling only: every step of the path runs in the CUDA kernels of
libkvq.so.  PyTorch is used for device memory and streams.  There is no CPU
fallback -- if libkvq.so is missing, ``load()`` raises.

Names follow the header: ``append`` (kvq_append), ``fp8_set_scales``
(kvq_fp8_set_scales), ``decode_attn`` (kvq_decode_attn), ``dequant``
(kvq_dequant), ``decode_workspace_bytes`` (kvq_decode_workspace_bytes),
``rope_append`` (kvq_rope_append).  ``append``, ``decode_attn``,
``prefill_attn`` and ``dequant`` take an ``Fp8BlockCache`` as well and then call
kvq_fp8_block_append, _decode_attn, _prefill_attn and _dequant; the last three
take a ``LatentCache`` too (kvq_latent_attn, kvq_latent_dequant), which
``latent_append`` fills.  ``expanded_attn`` is kvq_expanded_attn.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvq.so")

FORMAT_FP4 = 1
FORMAT_FP8 = 2
FORMAT_NVFP4 = 3
FORMAT_FP8_BLOCK = 4
FLAG_NONFINITE = 0x1
FLAG_PAGE_OOB = 0x2
FLAG_TIMEOUT = 0x4
FLAG_BAD_LENGTH = 0x8
FLAG_POSITION = 0x20
LAYOUT_FP8_TENSOR = 1
LAYOUT_INT_PER_TOKEN = 2
LAYOUT_INT_PER_CHANNEL = 3
LAYOUT_FP4_G16 = 4

_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None


class KvqError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {_status_string(status)} (status {status})")
        self.status = status


class KvqCacheStruct(ctypes.Structure):
    _fields_ = [
        ("format", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int64),
        ("max_pages_per_seq", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("page_table", ctypes.c_void_p),
        ("data", ctypes.c_void_p),
        ("v_data", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
    ]


class KvqLatentStruct(ctypes.Structure):
    _fields_ = [
        ("latent_dim", ctypes.c_int32),
        ("rope_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32),
        ("num_pages", ctypes.c_int64),
        ("page_table", ctypes.c_void_p),
        ("data", ctypes.c_void_p),
    ]


_P = ctypes.c_void_p
_CP = ctypes.POINTER(KvqCacheStruct)
_LP = ctypes.POINTER(KvqLatentStruct)
_I32, _I64, _F = ctypes.c_int32, ctypes.c_int64, ctypes.c_float


def load() -> ctypes.CDLL:
    """Load libkvq.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m fp4_kv_cache_kvq_gb300.build` (nvcc, sm_103a)")
            L = ctypes.CDLL(LIB_PATH)
            L.kvq_append.restype = ctypes.c_int
            L.kvq_append.argtypes = [_CP, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P, _P]
            L.kvq_fp8_set_scales.restype = ctypes.c_int
            L.kvq_fp8_set_scales.argtypes = [_CP, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P]
            L.kvq_decode_workspace_bytes.restype = ctypes.c_size_t
            L.kvq_decode_workspace_bytes.argtypes = [ctypes.c_int32] * 4
            L.kvq_decode_attn.restype = ctypes.c_int
            L.kvq_decode_attn.argtypes = [_CP, _CP, ctypes.c_int32, ctypes.c_int32, _P, _P, ctypes.c_float,
                                          _P, _P, ctypes.c_size_t, _P, _P]
            L.kvq_decode_attn_tc.restype = ctypes.c_int
            L.kvq_decode_attn_tc.argtypes = L.kvq_decode_attn.argtypes
            L.kvq_test_set_wait_limit_ns.restype = None
            L.kvq_test_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
            L.kvq_append_decode_attn.restype = ctypes.c_int
            L.kvq_append_decode_attn.argtypes = [_CP, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P, ctypes.c_float,
                                                 _P, _P, ctypes.c_size_t, _P, _P]
            L.kvq_dequant.restype = ctypes.c_int
            L.kvq_dequant.argtypes = [_CP, ctypes.c_int32, _P, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P]
            L.kvq_status_string.restype = ctypes.c_char_p
            L.kvq_status_string.argtypes = [ctypes.c_int]
            L.kvq_version.restype = ctypes.c_int32
            L.kvq_version.argtypes = []
            L.kvq_prefill_attn.restype = ctypes.c_int
            L.kvq_prefill_attn.argtypes = [_CP, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, _P,
                                           ctypes.c_float, _P, _P, _P]
            L.kvq_fake_quant.restype = ctypes.c_int
            L.kvq_fake_quant.argtypes = [ctypes.c_int32] * 6 + [_P] * 6
            L.kvq_attn_dense.restype = ctypes.c_int
            L.kvq_attn_dense.argtypes = [ctypes.c_int32] * 5 + [_P, _P, _P, ctypes.c_float, _P, _P, _P]
            L.kvq_swa_replay_workspace_bytes.restype = ctypes.c_size_t
            L.kvq_swa_replay_workspace_bytes.argtypes = [ctypes.c_int32, ctypes.c_int64, ctypes.c_int32]
            L.kvq_swa_replay.restype = ctypes.c_int
            L.kvq_swa_replay.argtypes = [_P, ctypes.c_int32, ctypes.c_int32, _P, ctypes.c_int64, ctypes.c_int32,
                                         _P, _P, _P, ctypes.c_size_t, _P]
            L.kvq_fp4_pool_bytes.restype = ctypes.c_size_t
            L.kvq_fp4_pool_bytes.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
            L.kvq_fp8_block_pool_bytes.restype = ctypes.c_size_t
            L.kvq_fp8_block_pool_bytes.argtypes = [_I64, _I32, _I32, _I32]
            L.kvq_rope_table.restype = ctypes.c_int
            L.kvq_rope_table.argtypes = [_I64, _I32, ctypes.c_double, _P, _P]
            L.kvq_rope_append.restype = ctypes.c_int
            L.kvq_rope_append.argtypes = [_CP, _I32, _I32, _P, _P, _I32, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _I32,
                                          _I32, _P, _P, _P, _P]
            L.kvq_fp8_block_append.restype = ctypes.c_int
            L.kvq_fp8_block_append.argtypes = [_CP, _I32, _I32, _P, _P, _P, _P, _P, _P]
            L.kvq_fp8_block_dequant.restype = ctypes.c_int
            L.kvq_fp8_block_dequant.argtypes = L.kvq_dequant.argtypes
            L.kvq_fp8_block_decode_attn.restype = ctypes.c_int
            L.kvq_fp8_block_decode_attn.argtypes = [_CP, _I32, _I32, _P, _P, _F, _P, _I32, _P, ctypes.c_size_t, _P, _P]
            L.kvq_fp8_block_prefill_workspace_bytes.restype = ctypes.c_size_t
            L.kvq_fp8_block_prefill_workspace_bytes.argtypes = [_I32] * 5
            L.kvq_fp8_block_prefill_attn.restype = ctypes.c_int
            L.kvq_fp8_block_prefill_attn.argtypes = [_CP, _I32, _I32, _I32, _P, _P, _P, _F, _P, _I32, _P,
                                                     ctypes.c_size_t, _P, _P]
            L.kvq_latent_pool_bytes.restype = ctypes.c_size_t
            L.kvq_latent_pool_bytes.argtypes = [_I64, _I32, _I32, _I32]
            L.kvq_latent_append.restype = ctypes.c_int
            L.kvq_latent_append.argtypes = [_LP, _I32, _I32, _P, _P, _I32, _P, _I64, _I64, _P, _I64, _P, _I64, _P, _I64,
                                            _I32, _P, _I64, _I64, _P, _P, _P]
            L.kvq_latent_dequant.restype = ctypes.c_int
            L.kvq_latent_dequant.argtypes = [_LP, _I32, _P, _I32, _I32, _P, _P, _P, _P]
            L.kvq_latent_attn_workspace_bytes.restype = ctypes.c_size_t
            L.kvq_latent_attn_workspace_bytes.argtypes = [_I32] * 4
            L.kvq_latent_attn.restype = ctypes.c_int
            L.kvq_latent_attn.argtypes = [_LP, _I32, _I32, _I32, _P, _P, _P, _F, _P, _I32, _P, ctypes.c_size_t, _P, _P]
            L.kvq_expanded_attn.restype = ctypes.c_int
            L.kvq_expanded_attn.argtypes = [_I32] * 6 + [_P, _P, _P, _P, _I64, _I64, _P, _I64, _P, _I64, _I64, _F, _P,
                                                         _I32, _P, _P]
            _lib = L
    return _lib


def _status_string(status: int) -> str:
    try:
        return load().kvq_status_string(status).decode()
    except Exception:  # pragma: no cover
        return "unknown"


def _check(status: int, what: str) -> None:
    if status != 0:
        raise KvqError(status, what)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# The current stream's handle without a torch.cuda.Stream object around it
# (0.3 us a call instead of 3).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _need(t: torch.Tensor, dtype: torch.dtype, name: str) -> None:
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of dtype {dtype}")


class Fp4Cache:
    """FP4 (E2M1 codes, E4M3 scale per 16 channels) paged cache for K and V.

    pool  uint8 [num_pages][num_kv_heads][page_size / G][G * 9 * head_dim / 8],
          G = min(page_size, 128): one contiguous block per group of G tokens
          of one kv head (K codes, K scales, V codes in token pairs, V scales;
          the byte layout is documented in include/kvq.h).
    page_table int32 [batch][max_pages_per_seq] or None (contiguous).
    nvfp4=True adds one fp32 second-level scale per kv head for K and for V
    (k_gscale, v_gscale: float [num_kv_heads], 1 until set by fp8_set_scales).
    """

    def __init__(self, num_kv_heads: int, head_dim: int, page_size: int, num_pages: int,
                 max_pages_per_seq: int, page_table: Optional[torch.Tensor] = None, device="cuda",
                 nvfp4: bool = False):
        self.num_kv_heads, self.head_dim, self.page_size = num_kv_heads, head_dim, page_size
        self.num_pages, self.max_pages_per_seq = num_pages, max_pages_per_seq
        self.group = min(page_size, 128)
        nbytes = load().kvq_fp4_pool_bytes(num_pages, num_kv_heads, page_size, head_dim)
        if nbytes == 0:
            raise ValueError("invalid FP4 cache geometry (head_dim 64/128/256, page_size 16..256)")
        shape = (num_pages, num_kv_heads, page_size // self.group, self.group * 9 * head_dim // 8)
        self.pool = torch.zeros(shape, dtype=torch.uint8, device=device)
        assert self.pool.numel() == nbytes
        if page_table is not None:
            _need(page_table, torch.int32, "page_table")
        self.page_table = page_table
        self.nvfp4 = nvfp4
        self.k_gscale = torch.ones(num_kv_heads, dtype=torch.float32, device=device) if nvfp4 else None
        self.v_gscale = torch.ones(num_kv_heads, dtype=torch.float32, device=device) if nvfp4 else None

    def struct(self, page_table: Optional[torch.Tensor] = None) -> KvqCacheStruct:
        """The kvq_cache description (kept between calls while the pointers in
        it are those of the tensors; a page_table argument overrides the cache's
        own for one call)."""
        pt = self.page_table if page_table is None else page_table
        key = (_ptr(pt), _ptr(self.pool), _ptr(self.k_gscale), _ptr(self.v_gscale))
        cached = self.__dict__.get("_struct")
        if cached is not None and cached[0] == key:
            return cached[1]
        s = KvqCacheStruct(FORMAT_NVFP4 if self.nvfp4 else FORMAT_FP4, self.num_kv_heads, self.head_dim,
                           self.page_size, self.num_pages, self.max_pages_per_seq, 0, key[0], key[1], None, *key[2:])
        if page_table is None:
            self._struct = (key, s)
        return s

    @property
    def nbytes(self) -> int:
        return self.pool.numel()


class Fp8WindowCache:
    """FP8 E4M3 sliding-window cache: one ring of `window` slots per sequence,
    one fp32 scale per kv head (K and V apart).

    codes  uint8 [num_seqs][num_kv_heads][window][head_dim]
    scales float32 [num_kv_heads]
    """

    def __init__(self, num_seqs: int, num_kv_heads: int, head_dim: int, window: int, device="cuda"):
        self.num_seqs, self.num_kv_heads, self.head_dim, self.window = num_seqs, num_kv_heads, head_dim, window
        shape = (num_seqs, num_kv_heads, window, head_dim)
        self.k_codes = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.v_codes = torch.zeros_like(self.k_codes)
        self.k_scales = torch.ones(num_kv_heads, dtype=torch.float32, device=device)
        self.v_scales = torch.ones_like(self.k_scales)

    def struct(self) -> KvqCacheStruct:
        """The kvq_cache description (kept while the pointers in it are those of
        the tensors)."""
        key = (_ptr(self.k_codes), _ptr(self.v_codes), _ptr(self.k_scales), _ptr(self.v_scales))
        cached = self.__dict__.get("_struct")
        if cached is not None and cached[0] == key:
            return cached[1]
        s = KvqCacheStruct(FORMAT_FP8, self.num_kv_heads, self.head_dim, self.window, self.num_seqs, 0, 0, None, *key)
        self._struct = (key, s)
        return s



class Fp8BlockCache:
    """8-bit paged cache for K and V: FP8 E4M3 codes, one fp32 scale per 16
    positions of one kv head (K and V apart), head_dim 64 or 128.

    pool  uint8 [num_pages][num_kv_heads][page_size / G][group bytes],
          G = min(page_size, 64) (the byte layout is documented in
          include/kvq_fp8_block.h); one given by the caller is used as it is.
    page_table int32 [batch][max_pages_per_seq] or None (contiguous).
    """

    def __init__(self, num_kv_heads: int, head_dim: int, page_size: int, num_pages: int, max_pages_per_seq: int,
                 page_table: Optional[torch.Tensor] = None, device="cuda", pool: Optional[torch.Tensor] = None):
        self.num_kv_heads, self.head_dim, self.page_size = num_kv_heads, head_dim, page_size
        self.num_pages, self.max_pages_per_seq = num_pages, max_pages_per_seq
        self.group = min(page_size, 64)
        nbytes = load().kvq_fp8_block_pool_bytes(num_pages, num_kv_heads, page_size, head_dim)
        if nbytes == 0:
            raise ValueError("invalid 8-bit cache geometry (head_dim 64/128, page_size 16..256)")
        groups = num_pages * num_kv_heads * (page_size // self.group)
        shape = (num_pages, num_kv_heads, page_size // self.group, nbytes // groups)
        if pool is None:
            pool = torch.zeros(shape, dtype=torch.uint8, device=device)
        _need(pool, torch.uint8, "pool")
        if tuple(pool.shape) != shape:
            raise ValueError(f"pool must have shape {shape}")
        if page_table is not None:
            _need_table(page_table, max_pages_per_seq)
        self.pool, self.page_table = pool, page_table
        self._struct = KvqCacheStruct(FORMAT_FP8_BLOCK, num_kv_heads, head_dim, page_size, num_pages, max_pages_per_seq,
                                      0, None, None, None, None, None)

    def struct(self, page_table: Optional[torch.Tensor] = None) -> KvqCacheStruct:
        """The kvq_cache description of the cache as it is now, a new one each time
        (calls from several threads do not share it); a page_table argument
        overrides the cache's own for one call."""
        s = KvqCacheStruct.from_buffer_copy(self._struct)
        s.page_table, s.data = _ptr(self.page_table if page_table is None else page_table), self.pool.data_ptr()
        return s

    @property
    def nbytes(self) -> int:
        return self.pool.numel()


class LatentCache:
    """8-bit paged cache of one latent vector per token, key and value of all
    heads at once, and of the key's rotated position part: E4M3 codes (two per
    value of the position part) with one power-of-two scale per token.
    latent_dim 128, 256 or 512, rope_dim 32 or 64.

    pool  uint8 [num_pages][page_size / G][G * (latent_dim + 2 * rope_dim + 1)],
          G = min(page_size, 64) (the byte layout is documented in
          include/kvq_latent.h); one given by the caller is used as it is.
    page_table int32 [batch][max_pages_per_seq] or None (contiguous).
    """

    def __init__(self, latent_dim: int, rope_dim: int, page_size: int, num_pages: int, max_pages_per_seq: int,
                 page_table: Optional[torch.Tensor] = None, device="cuda", pool: Optional[torch.Tensor] = None):
        self.latent_dim, self.rope_dim, self.page_size = latent_dim, rope_dim, page_size
        self.num_pages, self.max_pages_per_seq = num_pages, max_pages_per_seq
        self.group = min(page_size, 64)
        nbytes = load().kvq_latent_pool_bytes(num_pages, page_size, latent_dim, rope_dim)
        if nbytes == 0:
            raise ValueError("invalid latent cache geometry (latent_dim 128/256/512, rope_dim 32/64, page_size 16..256)")
        shape = (num_pages, page_size // self.group, self.group * (latent_dim + 2 * rope_dim + 1))
        if pool is None:
            pool = torch.zeros(shape, dtype=torch.uint8, device=device)
        _need(pool, torch.uint8, "pool")
        if tuple(pool.shape) != shape:
            raise ValueError(f"pool must have shape {shape}")
        if page_table is not None:
            _need_table(page_table, max_pages_per_seq)
        self.pool, self.page_table = pool, page_table

    def struct(self, page_table: Optional[torch.Tensor] = None) -> KvqLatentStruct:
        """The kvq_latent_cache description of the cache as it is now, a new one
        each time; a page_table argument overrides the cache's own for one call."""
        return KvqLatentStruct(self.latent_dim, self.rope_dim, self.page_size, self.max_pages_per_seq, self.num_pages,
                               _ptr(self.page_table if page_table is None else page_table), self.pool.data_ptr())

    @property
    def nbytes(self) -> int:
        return self.pool.numel()


def _need_table(t: torch.Tensor, max_pages: int) -> None:
    _need(t, torch.int32, "page_table")
    if t.dim() != 2 or t.shape[1] != max_pages:
        raise ValueError("page_table must have shape [batch, max_pages_per_seq]")


# Checks of the calls on an Fp8BlockCache or LatentCache and of rope_append: a few
# hundred nanoseconds each, since a decode step makes them once a layer.
def _device(cache) -> int:
    """The cache's device, which has to be the current one."""
    dev = cache.pool.get_device()
    if dev != _current_device():
        raise ValueError(f"the cache is on {cache.pool.device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return dev


def _stream_on(dev: int, stream) -> Optional[int]:
    return _raw_stream(dev) if stream is None and _raw_stream is not None else _stream(stream)


def _on(dev: int, t: torch.Tensor, dtype: torch.dtype, name: str) -> None:
    """t is contiguous, of this type, on the cache's device."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of dtype {dtype} on cuda:{dev}")


def _per_seq(dev: int, t: torch.Tensor, batch: int, name: str) -> None:
    _on(dev, t, torch.int32, name)
    if t.numel() != batch:
        raise ValueError(f"{name} must hold one value per sequence ({batch})")


def _table_rows(dev: int, cache, page_table: Optional[torch.Tensor], batch: int) -> None:
    """The page table of a call has a row for every sequence."""
    if page_table is not None:
        _on(dev, page_table, torch.int32, "page_table")
        if page_table.dim() != 2 or page_table.shape[1] != cache.max_pages_per_seq:
            raise ValueError("page_table must have shape [batch, max_pages_per_seq]")
    pt = cache.page_table if page_table is None else page_table
    if pt is not None and pt.shape[0] < batch:
        raise ValueError("the page table has fewer rows than sequences")


def _alloc(stream, shape, dtype: torch.dtype, dev: int, zero: bool = False) -> torch.Tensor:
    """A buffer of a call on `stream` (None: the current one): from that stream's
    memory, so that nothing still running on another stream uses it."""
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=f"cuda:{dev}")
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=f"cuda:{dev}")


def _err_ptr(dev: int, err: Optional[torch.Tensor]) -> Optional[int]:
    if err is None:
        return None
    _on(dev, err, torch.int32, "err")
    if err.numel() < 1:
        raise ValueError("err must hold one int32")
    return err.data_ptr()


def append(cache, start_pos: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
           err: Optional[torch.Tensor] = None, stream=None, page_table: Optional[torch.Tensor] = None,
           new_lens: Optional[torch.Tensor] = None) -> None:
    """kvq_append: k, v bf16 [batch][n_new][Hkv][head_dim]; start_pos int32 [batch].
    An Fp8BlockCache (kvq_fp8_block_append) also takes new_lens, int32 [batch]:
    sequence b has new_lens[b] <= n_new new tokens."""
    if isinstance(cache, LatentCache):
        raise ValueError("a LatentCache is filled by latent_append")
    _need(k, torch.bfloat16, "k")
    _need(v, torch.bfloat16, "v")
    _need(start_pos, torch.int32, "start_pos")
    if k.dim() != 4 or k.shape != v.shape:
        raise ValueError("k and v must have shape [batch, n_new, num_kv_heads, head_dim]")
    if isinstance(cache, Fp8BlockCache):
        if tuple(k.shape[2:]) != (cache.num_kv_heads, cache.head_dim):
            raise ValueError("k and v must have the cache's heads and head_dim")
        B = k.shape[0]
        dev = _device(cache)
        _on(dev, k, torch.bfloat16, "k")
        _on(dev, v, torch.bfloat16, "v")
        _table_rows(dev, cache, page_table, B)
        _per_seq(dev, start_pos, B, "start_pos")
        if new_lens is not None:
            _per_seq(dev, new_lens, B, "new_lens")
        s = cache.struct(page_table)
        st = load().kvq_fp8_block_append(ctypes.byref(s), B, k.shape[1], _ptr(start_pos), _ptr(new_lens), _ptr(k),
                                         _ptr(v), _err_ptr(dev, err), _stream(stream))
        return _check(st, "kvq_fp8_block_append")
    if new_lens is not None:
        raise ValueError("new_lens needs an Fp8BlockCache (or rope_append)")
    s = cache.struct(page_table) if isinstance(cache, Fp4Cache) else cache.struct()
    st = load().kvq_append(ctypes.byref(s), k.shape[0], k.shape[1], _ptr(start_pos), _ptr(k), _ptr(v),
                           _ptr(err), _stream(stream))
    _check(st, "kvq_append")


def rope_table(num_positions: int, rotary_dim: int, base: float = 10000.0, device="cuda", stream=None) -> torch.Tensor:
    """kvq_rope_table: float32 [num_positions][rotary_dim], of each position
    the rotary_dim/2 cosines, then the sines."""
    where, dev = torch.device(device), torch.cuda.current_device()
    if where.type != "cuda" or where.index not in (None, dev):
        raise ValueError(f"device {where} is not the current one, cuda:{dev}")
    table = _alloc(stream, (num_positions, rotary_dim), torch.float32, dev)
    _check(load().kvq_rope_table(num_positions, rotary_dim, float(base), _ptr(table), _stream(stream)),
           "kvq_rope_table")
    return table


def _token_stride(dev: int, t: torch.Tensor, name: str):
    """Elements from one token to the next of a bf16 [batch][n][heads][d] tensor
    whose tokens' values are contiguous and evenly spaced (a contiguous tensor,
    or a part of a packed projection), and its shape."""
    shape = t.shape
    if t.dtype is not torch.bfloat16 or t.get_device() != dev or len(shape) != 4:
        raise ValueError(f"{name} must be a bfloat16 tensor [batch, n_new, heads, head_dim] on cuda:{dev}")
    B, n, H, d = shape
    if t.is_contiguous():
        return H * d, shape
    sb, sn, sh, sd = t.stride()
    step = sn if n > 1 else sb
    if t.numel() and not ((sd == 1 or d == 1) and (H == 1 or sh == d) and step >= H * d and
                          (n == 1 or B == 1 or sb == n * sn)):
        raise ValueError(f"{name}: the values of a token must be contiguous and the tokens evenly spaced")
    return step, shape


def rope_append(cache, start_pos: torch.Tensor, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                table: Optional[torch.Tensor], interleaved: bool = False, new_lens: Optional[torch.Tensor] = None,
                q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                err: Optional[torch.Tensor] = None, stream=None,
                page_table: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """kvq_rope_append: rotate q and k, bf16 [batch][n_new][heads][head_dim], by
    their positions start_pos[b] + t and append k and v to an Fp4Cache (NVFP4
    too) or Fp8BlockCache.  Returns the rotated queries (q_out, made when not
    given; None without q); k_out, when given, receives the rotated keys.  q, k
    and v may be parts of one packed projection.  table: rope_table(...), its
    width the rotated channels; None: no rotation.  new_lens, int32 [batch]: the
    new tokens of each sequence of a padded batch."""
    if not isinstance(cache, (Fp4Cache, Fp8BlockCache)):
        raise ValueError("rope_append needs an Fp4Cache or Fp8BlockCache (append k_out to a window ring)")
    dev = _device(cache)
    (ks, shape), (vs, v_shape) = _token_stride(dev, k, "k"), _token_stride(dev, v, "v")
    B, n, hkv, d = shape
    if shape != v_shape or hkv != cache.num_kv_heads or d != cache.head_dim:
        raise ValueError("k and v must have shape [batch, n_new, num_kv_heads, head_dim]")
    hq = qs = 0
    q_ptr = out_ptr = None
    if q is not None:
        qs, q_shape = _token_stride(dev, q, "q")
        hq = q_shape[2]
        if q_shape[0] != B or q_shape[1] != n or q_shape[3] != d:
            raise ValueError("q must have shape [batch, n_new, num_q_heads, head_dim]")
        if q_out is None:
            q_out = _alloc(stream, q_shape, torch.bfloat16, dev)
        else:
            _on(dev, q_out, torch.bfloat16, "q_out")
            if q_out.shape != q_shape:
                raise ValueError("q_out must have q's shape")
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k_out is not None:
        _on(dev, k_out, torch.bfloat16, "k_out")
        if k_out.shape != shape:
            raise ValueError("k_out must have k's shape")
    rows = rd = 0
    if table is not None:
        _on(dev, table, torch.float32, "table")
        rows, rd = table.shape
    _table_rows(dev, cache, page_table, B)
    _per_seq(dev, start_pos, B, "start_pos")
    if new_lens is not None:
        _per_seq(dev, new_lens, B, "new_lens")
    s = cache.struct(page_table)
    st = load().kvq_rope_append(ctypes.byref(s), B, n, start_pos.data_ptr(), _ptr(new_lens), hq, q_ptr, qs,
                                k.data_ptr(), ks, v.data_ptr(), vs, _ptr(table), rows, rd, 1 if interleaved else 0,
                                out_ptr, _ptr(k_out), _err_ptr(dev, err), _stream_on(dev, stream))
    _check(st, "kvq_rope_append")
    return q_out


def _row_strides(dev: int, t: torch.Tensor, name: str, heads: bool):
    """Elements from token to token and from head to head of a bf16
    [batch][n][heads][width] (or [batch][n][width]) tensor whose rows are
    contiguous and whose tokens are evenly spaced, and its shape."""
    shape = t.shape
    if t.dtype is not torch.bfloat16 or t.get_device() != dev or len(shape) != (4 if heads else 3):
        raise ValueError(f"{name} must be a bfloat16 tensor [batch, n, {'heads, ' if heads else ''}width] on cuda:{dev}")
    if heads:
        (B, n, H, w), (sb, sn, sh, sw) = shape, t.stride()
    else:
        (B, n, w), (sb, sn, sw), H, sh = shape, t.stride(), 1, shape[2]
    if H == 1:
        sh = w
    step = sn if n > 1 else sb if B > 1 else H * max(sh, w)
    if (sw != 1 or sh < w or step < (H - 1) * sh + w or (n > 1 and B > 1 and sb != n * sn)) and t.numel():
        raise ValueError(f"{name}: rows must be contiguous, heads and tokens evenly spaced and without overlap")
    return step, sh, shape


def latent_append(cache: LatentCache, start_pos: torch.Tensor, q: Optional[torch.Tensor], c: torch.Tensor,
                  k: torch.Tensor, table: Optional[torch.Tensor], interleaved: bool = False,
                  new_lens: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                  k_out: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None, stream=None,
                  page_table: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """kvq_latent_append: rotate the query parts q, bf16 [batch][n_new][heads][rope_dim],
    and key parts k, bf16 [batch][n_new][rope_dim], by their positions start_pos[b]
    + t and append latents c, bf16 [batch][n_new][latent_dim], and key parts to a
    LatentCache.  Returns the rotated query parts (q_out, made when not given; None
    without q); k_out, when given, receives the rotated key parts.  q, c, k and q_out
    may be parts of larger tensors (a packed projection; the tails of the absorbed
    queries, which is where q_out belongs for decode_attn and prefill_attn).  table:
    rope_table(n, rope_dim, ...); None: no rotation.  new_lens, int32 [batch]: the new
    tokens of each sequence of a padded batch."""
    if not isinstance(cache, LatentCache):
        raise ValueError("latent_append needs a LatentCache")
    dev = _device(cache)
    L, R = cache.latent_dim, cache.rope_dim
    (cs, _, shape), (ks, _, k_shape) = _row_strides(dev, c, "c", False), _row_strides(dev, k, "k", False)
    B, n, w = shape
    if w != L or k_shape[0] != B or k_shape[1] != n or k_shape[2] != R:
        raise ValueError("c and k must have shape [batch, n_new, latent_dim] and [batch, n_new, rope_dim]")
    hq = qt = qh = ot = oh = 0
    q_ptr = out_ptr = None
    if q is not None:
        qt, qh, q_shape = _row_strides(dev, q, "q", True)
        hq = q_shape[2]
        if q_shape[0] != B or q_shape[1] != n or hq < 1 or q_shape[3] != R:
            raise ValueError("q must have shape [batch, n_new, num_q_heads, rope_dim]")
        if q_out is None:
            q_out = _alloc(stream, q_shape, torch.bfloat16, dev)
        ot, oh, o_shape = _row_strides(dev, q_out, "q_out", True)
        if o_shape != q_shape:
            raise ValueError("q_out must have q's shape")
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k_out is not None:
        _on(dev, k_out, torch.bfloat16, "k_out")
        if k_out.shape != k_shape:
            raise ValueError("k_out must have k's shape")
    rows = 0
    if table is not None:
        _on(dev, table, torch.float32, "table")
        if table.dim() != 2 or table.shape[1] != R:
            raise ValueError("table must have shape [positions, rope_dim]")
        rows = table.shape[0]
    _table_rows(dev, cache, page_table, B)
    _per_seq(dev, start_pos, B, "start_pos")
    if new_lens is not None:
        _per_seq(dev, new_lens, B, "new_lens")
    s = cache.struct(page_table)
    st = load().kvq_latent_append(ctypes.byref(s), B, n, start_pos.data_ptr(), _ptr(new_lens), hq, q_ptr, qt, qh,
                                  c.data_ptr(), cs, k.data_ptr(), ks, _ptr(table), rows, 1 if interleaved else 0,
                                  out_ptr, ot, oh, _ptr(k_out), _err_ptr(dev, err), _stream_on(dev, stream))
    _check(st, "kvq_latent_append")
    return q_out


def fp8_set_scales(cache, k: torch.Tensor, v: torch.Tensor,
                   err: Optional[torch.Tensor] = None, stream=None) -> None:
    """kvq_fp8_set_scales over k, v bf16 [batch][n][Hkv][D]: an FP8 window
    cache gets s_h = amax/448 per head, an NVFP4 cache its second-level
    scales S_h = amax/(6*448)."""
    _need(k, torch.bfloat16, "k")
    _need(v, torch.bfloat16, "v")
    s = cache.struct()
    st = load().kvq_fp8_set_scales(ctypes.byref(s), k.shape[0], k.shape[1], _ptr(k), _ptr(v), _ptr(err),
                                   _stream(stream))
    _check(st, "kvq_fp8_set_scales")


def decode_workspace_bytes(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(load().kvq_decode_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim))


def decode_attn(cache: Fp4Cache, seq_lens: torch.Tensor, q: torch.Tensor, softmax_scale: Optional[float] = None,
                swa: Optional[Fp8WindowCache] = None, out: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None,
                stream=None, kernel: str = "mma") -> torch.Tensor:
    """kvq_decode_attn: q bf16 [batch][Hq][head_dim] -> out float32 [batch][Hq][head_dim].
    kernel="tcgen05" calls kvq_decode_attn_tc instead (head_dim 128: both
    products on the tensor-memory MMA; a measured, slower alternative).
    An Fp8BlockCache (kvq_fp8_block_decode_attn) takes a float32 or bfloat16
    out and neither swa nor kernel="tcgen05".  So does a LatentCache
    (kvq_latent_attn), with q [batch][Hq][latent_dim + rope_dim], out
    [batch][Hq][latent_dim], a workspace of latent_workspace_bytes(...) bytes and a
    softmax_scale, which the latent does not show."""
    if kernel not in ("mma", "tcgen05"):
        raise ValueError(f"unknown decode kernel {kernel!r}")
    if isinstance(cache, LatentCache):
        if swa is not None or kernel != "mma":
            raise ValueError("a LatentCache takes neither swa nor kernel=\"tcgen05\"")
        return _attend_latent(cache, seq_lens, q, softmax_scale, out, err, stream, None, workspace, False)
    if isinstance(cache, Fp8BlockCache):
        if swa is not None or kernel != "mma":
            raise ValueError("an Fp8BlockCache takes neither swa nor kernel=\"tcgen05\"")
        return _decode_block8(cache, seq_lens, q, softmax_scale, out, workspace, err, stream)
    _need(q, torch.bfloat16, "q")
    _need(seq_lens, torch.int32, "seq_lens")
    batch, hq, d = q.shape
    if out is None:
        out = torch.empty((batch, hq, d), dtype=torch.float32, device=q.device)
    _need(out, torch.float32, "out")
    if workspace is None:  # a caller's workspace is size-checked by the library
        need = decode_workspace_bytes(batch, hq, cache.num_kv_heads, d)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    g = cache.struct()
    w = swa.struct() if swa is not None else None
    fn = load().kvq_decode_attn_tc if kernel == "tcgen05" else load().kvq_decode_attn
    st = fn(ctypes.byref(g), ctypes.byref(w) if w is not None else None, batch, hq, _ptr(seq_lens), _ptr(q),
            float(softmax_scale), _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
            _ptr(err), _stream(stream))
    _check(st, "kvq_decode_attn_tc" if kernel == "tcgen05" else "kvq_decode_attn")
    return out


_OUT_DTYPES = {torch.float32: 0, torch.bfloat16: 1}


def _attn_out(dev: int, cache, q: torch.Tensor, shape, out: Optional[torch.Tensor], padded: bool, stream):
    """(out, its KVQ_DTYPE_*) of an attention over an Fp8BlockCache; shape: q's."""
    _on(dev, q, torch.bfloat16, "q")
    if shape[-1] != cache.head_dim:
        raise ValueError("q must have the cache's head_dim")
    if out is None:  # rows of a padded batch's padding are not written
        out = _alloc(stream, shape, torch.float32, dev, zero=padded)
    code = _OUT_DTYPES.get(out.dtype)
    if code is None or out.get_device() != dev or not out.is_contiguous() or out.shape != shape:
        raise ValueError("out must be a contiguous float32 or bfloat16 tensor of q's shape on the cache's device")
    return out, code


def _workspace(dev: int, workspace: Optional[torch.Tensor], stream, need, *sizes) -> torch.Tensor:
    if workspace is None:
        return _alloc(stream, max(16, need(*sizes)), torch.uint8, dev)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    return workspace  # its size is checked by the library


def _decode_block8(cache, seq_lens, q, softmax_scale, out, workspace, err, stream) -> torch.Tensor:
    dev = _device(cache)
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q must have shape [batch, num_q_heads, head_dim]")
    out, code = _attn_out(dev, cache, q, shape, out, False, stream)
    B, hq, d = shape
    _per_seq(dev, seq_lens, B, "seq_lens")
    _table_rows(dev, cache, None, B)
    ws = _workspace(dev, workspace, stream, decode_workspace_bytes, B, hq, cache.num_kv_heads, d)
    s = cache.struct()
    st = load().kvq_fp8_block_decode_attn(ctypes.byref(s), B, hq, seq_lens.data_ptr(), q.data_ptr(),
                                          1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale),
                                          out.data_ptr(), code, ws.data_ptr(), ws.nbytes, _err_ptr(dev, err),
                                          _stream_on(dev, stream))
    _check(st, "kvq_fp8_block_decode_attn")
    return out


def append_decode_attn(cache: Fp4Cache, seq_lens: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                       q: torch.Tensor, softmax_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """kvq_append_decode_attn: append k_new/v_new bf16 [batch][Hkv][head_dim] at
    position seq_lens[b] - 1, then decode attention over seq_lens[b] positions."""
    _need(q, torch.bfloat16, "q")
    _need(seq_lens, torch.int32, "seq_lens")
    _need(k_new, torch.bfloat16, "k_new")
    _need(v_new, torch.bfloat16, "v_new")
    batch, hq, d = q.shape
    if out is None:
        out = torch.empty((batch, hq, d), dtype=torch.float32, device=q.device)
    _need(out, torch.float32, "out")
    if workspace is None:
        need = decode_workspace_bytes(batch, hq, cache.num_kv_heads, d)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    g = cache.struct()
    st = load().kvq_append_decode_attn(ctypes.byref(g), batch, hq, _ptr(seq_lens), _ptr(k_new), _ptr(v_new), _ptr(q),
                                       float(softmax_scale), _ptr(out), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _ptr(err), _stream(stream))
    _check(st, "kvq_append_decode_attn")
    return out


def prefill_workspace_bytes(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, chunk: int) -> int:
    """kvq_fp8_block_prefill_workspace_bytes."""
    return int(load().kvq_fp8_block_prefill_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, chunk))


def _prefill_block8(cache, seq_lens, q, softmax_scale, out, err, stream, chunk_lens, workspace) -> torch.Tensor:
    dev = _device(cache)
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must have shape [batch, chunk, num_q_heads, head_dim]")
    out, code = _attn_out(dev, cache, q, shape, out, chunk_lens is not None, stream)
    B, chunk, hq, d = shape
    _per_seq(dev, seq_lens, B, "seq_lens")
    if chunk_lens is not None:
        _per_seq(dev, chunk_lens, B, "chunk_lens")
    _table_rows(dev, cache, None, B)
    ws = _workspace(dev, workspace, stream, prefill_workspace_bytes, B, hq, cache.num_kv_heads, d, chunk)
    s = cache.struct()
    st = load().kvq_fp8_block_prefill_attn(ctypes.byref(s), B, hq, chunk, seq_lens.data_ptr(), _ptr(chunk_lens),
                                           q.data_ptr(),
                                           1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale),
                                           out.data_ptr(), code, ws.data_ptr(), ws.nbytes, _err_ptr(dev, err),
                                           _stream_on(dev, stream))
    _check(st, "kvq_fp8_block_prefill_attn")
    return out


def latent_workspace_bytes(batch: int, num_q_heads: int, latent_dim: int, chunk: int = 1) -> int:
    """kvq_latent_attn_workspace_bytes."""
    return int(load().kvq_latent_attn_workspace_bytes(batch, num_q_heads, latent_dim, chunk))


def _out_like(dev: int, out: Optional[torch.Tensor], shape, zero: bool, stream):
    """(out, its KVQ_DTYPE_*), made as float32 when not given."""
    if out is None:  # rows of a padded batch's padding are not written
        out = _alloc(stream, shape, torch.float32, dev, zero=zero)
    code = _OUT_DTYPES.get(out.dtype)
    if code is None or out.get_device() != dev or not out.is_contiguous() or out.shape != shape:
        raise ValueError(f"out must be a contiguous float32 or bfloat16 tensor of shape {list(shape)} on cuda:{dev}")
    return out, code


def _attend_latent(cache, seq_lens, q, softmax_scale, out, err, stream, chunk_lens, workspace, chunked) -> torch.Tensor:
    dev = _device(cache)
    shape = q.shape
    if len(shape) != (4 if chunked else 3) or shape[-1] != cache.latent_dim + cache.rope_dim:
        raise ValueError(f"q must have shape [batch, {'chunk, ' if chunked else ''}num_q_heads, latent_dim + rope_dim]")
    if softmax_scale is None:
        raise ValueError("a LatentCache needs softmax_scale")
    _on(dev, q, torch.bfloat16, "q")
    out, code = _out_like(dev, out, shape[:-1] + (cache.latent_dim,), chunk_lens is not None, stream)
    B, chunk, hq = shape[0], shape[1] if chunked else 1, shape[-2]
    _per_seq(dev, seq_lens, B, "seq_lens")
    if chunk_lens is not None:
        _per_seq(dev, chunk_lens, B, "chunk_lens")
    _table_rows(dev, cache, None, B)
    ws = _workspace(dev, workspace, stream, latent_workspace_bytes, B, hq, cache.latent_dim, chunk)
    s = cache.struct()
    st = load().kvq_latent_attn(ctypes.byref(s), B, hq, chunk, seq_lens.data_ptr(), _ptr(chunk_lens), q.data_ptr(),
                                float(softmax_scale), out.data_ptr(), code, ws.data_ptr(), ws.nbytes,
                                _err_ptr(dev, err), _stream_on(dev, stream))
    _check(st, "kvq_latent_attn")
    return out


def expanded_attn(q: torch.Tensor, k: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor, seq_lens: torch.Tensor,
                  softmax_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  err: Optional[torch.Tensor] = None, stream=None,
                  chunk_lens: Optional[torch.Tensor] = None) -> torch.Tensor:
    """kvq_expanded_attn: causal attention of a chunk over keys and values multiplied
    out per head.  q bf16 [batch][chunk][heads][d + 64], k and v bf16
    [batch][max_len][heads][d] (parts of one packed projection as they are), k_rope
    bf16 [batch][max_len][64], shared by the heads, rotated as q's last 64 values are;
    sequence b holds seq_lens[b] positions, the chunk's included.  Returns out
    [batch][chunk][heads][d], float32 unless a bfloat16 out is given.  chunk_lens,
    int32 [batch]: the chunk's tokens of each sequence of a padded batch, whose other
    rows of out are left as they were (0 in an out made here)."""
    dev = q.get_device()
    if dev < 0 or dev != _current_device():
        raise ValueError(f"q must be on the current device, cuda:{torch.cuda.current_device()}")
    _on(dev, q, torch.bfloat16, "q")
    (kt, kh, shape), (vt, vh, v_shape) = _row_strides(dev, k, "k", True), _row_strides(dev, v, "v", True)
    rt, _, r_shape = _row_strides(dev, k_rope, "k_rope", False)
    if q.dim() != 4:
        raise ValueError("q must have shape [batch, chunk, heads, head_dim + rope_dim]")
    B, chunk, H, w = q.shape
    d, T = shape[3], shape[1]
    if shape != v_shape or shape[0] != B or shape[2] != H or tuple(r_shape) != (B, T, w - d):
        raise ValueError("k and v must have shape [batch, max_len, heads, head_dim], k_rope [batch, max_len, rope_dim]")
    out, code = _out_like(dev, out, q.shape[:-1] + (d,), chunk_lens is not None, stream)
    _per_seq(dev, seq_lens, B, "seq_lens")
    if chunk_lens is not None:
        _per_seq(dev, chunk_lens, B, "chunk_lens")
    st = load().kvq_expanded_attn(B, H, d, w - d, chunk, T, seq_lens.data_ptr(), _ptr(chunk_lens), q.data_ptr(),
                                  k.data_ptr(), kt, kh, k_rope.data_ptr(), rt, v.data_ptr(), vt, vh,
                                  1.0 / math.sqrt(w) if softmax_scale is None else float(softmax_scale),
                                  out.data_ptr(), code, _err_ptr(dev, err), _stream_on(dev, stream))
    _check(st, "kvq_expanded_attn")
    return out


def prefill_attn(cache, seq_lens: torch.Tensor, q: torch.Tensor, softmax_scale: Optional[float] = None,
                 out: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None, stream=None,
                 chunk_lens: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """kvq_prefill_attn: q bf16 [batch][chunk][Hq][head_dim] (their keys and
    values already appended) -> out float32, same shape; causal over the cache.
    An Fp8BlockCache (kvq_fp8_block_prefill_attn) takes a float32 or bfloat16
    out, a workspace of prefill_workspace_bytes(...) bytes, and chunk_lens, int32
    [batch]: the chunk's tokens of each sequence of a padded batch, whose other
    rows of out are left as they were (0 in an out made here).  So does a LatentCache
    (kvq_latent_attn), with q [batch][chunk][Hq][latent_dim + rope_dim], out
    [batch][chunk][Hq][latent_dim], a workspace of latent_workspace_bytes(...) bytes
    and a softmax_scale."""
    if isinstance(cache, LatentCache):
        return _attend_latent(cache, seq_lens, q, softmax_scale, out, err, stream, chunk_lens, workspace, True)
    if isinstance(cache, Fp8BlockCache):
        return _prefill_block8(cache, seq_lens, q, softmax_scale, out, err, stream, chunk_lens, workspace)
    if chunk_lens is not None or workspace is not None:
        raise ValueError("chunk_lens and workspace need an Fp8BlockCache")
    _need(q, torch.bfloat16, "q")
    _need(seq_lens, torch.int32, "seq_lens")
    batch, chunk, hq, d = q.shape
    if out is None:
        out = torch.empty((batch, chunk, hq, d), dtype=torch.float32, device=q.device)
    _need(out, torch.float32, "out")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    c = cache.struct()
    st = load().kvq_prefill_attn(ctypes.byref(c), batch, hq, chunk, _ptr(seq_lens), _ptr(q), float(softmax_scale),
                                 _ptr(out), _ptr(err), _stream(stream))
    _check(st, "kvq_prefill_attn")
    return out


def swa_replay(w: torch.Tensor, emb: torch.Tensor, n_win: int, want_hidden: bool = True,
               workspace: Optional[torch.Tensor] = None, states: Optional[torch.Tensor] = None, stream=None):
    """kvq_swa_replay: the toy sliding-window network over the positions whose
    inputs are emb (float32 [n][d]) with weights w (float32 [L][4][d][d]:
    Wq, Wk, Wv, Wo).  Returns (states float32 [L][2][n_win][d] -- each
    layer's K then V rows of the last n_win positions --, hidden float32
    [n][d] or None)."""
    _need(w, torch.float32, "w")
    _need(emb, torch.float32, "emb")
    L, four, d, _ = w.shape
    n = emb.shape[0]
    if states is None:
        states = torch.empty((L, 2, n_win, d), dtype=torch.float32, device=emb.device)
    _need(states, torch.float32, "states")
    hidden = torch.empty((n, d), dtype=torch.float32, device=emb.device) if want_hidden else None
    need = load().kvq_swa_replay_workspace_bytes(L, n, d)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=emb.device)
    st = load().kvq_swa_replay(_ptr(w), L, d, _ptr(emb), n, int(n_win), _ptr(states), _ptr(hidden), _ptr(workspace),
                               workspace.numel(), _stream(stream))
    _check(st, "kvq_swa_replay")
    return states, hidden


def _dequant_latent(cache, seq_lens, max_len, dtype, err, stream):
    dev = _device(cache)
    B = seq_lens.numel()
    _per_seq(dev, seq_lens, B, "seq_lens")
    _table_rows(dev, cache, None, B)
    if dtype not in _OUT_DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    c, k = (_alloc(stream, (B, max_len, w), dtype, dev) for w in (cache.latent_dim, cache.rope_dim))
    s = cache.struct()
    st = load().kvq_latent_dequant(ctypes.byref(s), B, seq_lens.data_ptr(), max_len, _OUT_DTYPES[dtype], c.data_ptr(),
                                   k.data_ptr(), _err_ptr(dev, err), _stream_on(dev, stream))
    _check(st, "kvq_latent_dequant")
    return c, k


def dequant(cache, seq_lens: Optional[torch.Tensor], max_len: int, dtype: torch.dtype = torch.float32,
            err: Optional[torch.Tensor] = None, stream=None):
    """kvq_dequant: dense K, V [batch][max_len][Hkv][head_dim] (FP8 ring: max_len
    == window, slot order; Fp8BlockCache: kvq_fp8_block_dequant).  LatentCache:
    kvq_latent_dequant, latents [batch][max_len][latent_dim] and key parts
    [batch][max_len][rope_dim]."""
    if isinstance(cache, LatentCache):
        return _dequant_latent(cache, seq_lens, max_len, dtype, err, stream)
    block8 = isinstance(cache, Fp8BlockCache)
    if block8:
        dev = _device(cache)
        _per_seq(dev, seq_lens, seq_lens.numel(), "seq_lens")
        _table_rows(dev, cache, None, seq_lens.numel())
        _err_ptr(dev, err)
    if isinstance(cache, (Fp4Cache, Fp8BlockCache)):
        batch = seq_lens.shape[0]
        s = cache.struct()
        device = cache.pool.device
    else:
        batch = cache.num_seqs
        s = cache.struct()
        device = cache.k_codes.device
    code = {torch.float32: 0, torch.bfloat16: 1}[dtype]
    shape = (batch, max_len, cache.num_kv_heads, cache.head_dim)
    if block8:
        k, v = _alloc(stream, shape, dtype, dev), _alloc(stream, shape, dtype, dev)
    else:
        k = torch.empty(shape, dtype=dtype, device=device)
        v = torch.empty(shape, dtype=dtype, device=device)
    fn = load().kvq_fp8_block_dequant if block8 else load().kvq_dequant
    st = fn(ctypes.byref(s), batch, _ptr(seq_lens), max_len, code, _ptr(k), _ptr(v), _ptr(err), _stream(stream))
    _check(st, "kvq_fp8_block_dequant" if block8 else "kvq_dequant")
    return k, v


# ---------------------------------------------------------------- bit-width sweep
def fake_quant(x: torch.Tensor, layout: int, bits: int, want_codes: bool = False,
               err: Optional[torch.Tensor] = None, stream=None):
    """kvq_fake_quant: x bf16 [batch][tokens][heads][head_dim] -> (x_hat float
    like x, codes int8 like x or None, scales or None).  Scales: FP8 tensor ->
    float[2] (s in [1]); INT per token -> uint16-as-int16 [batch][tokens][heads];
    INT per channel -> [batch][heads][head_dim]; FP4 -> uint8 [numel/16]."""
    _need(x, torch.bfloat16, "x")
    B, T, H, d = x.shape
    xh = torch.empty(x.shape, dtype=torch.float32, device=x.device)
    codes = torch.empty(x.shape, dtype=torch.int8, device=x.device) if want_codes else None
    if layout == LAYOUT_FP8_TENSOR:
        scales = torch.empty(2, dtype=torch.float32, device=x.device)
    elif layout == LAYOUT_INT_PER_TOKEN:
        scales = torch.empty((B, T, H), dtype=torch.int16, device=x.device)
    elif layout == LAYOUT_INT_PER_CHANNEL:
        scales = torch.empty((B, H, d), dtype=torch.int16, device=x.device)
    else:
        scales = torch.empty(x.numel() // 16, dtype=torch.uint8, device=x.device)
    st = load().kvq_fake_quant(layout, bits, B, T, H, d, _ptr(x), _ptr(xh), _ptr(codes), _ptr(scales), _ptr(err),
                               _stream(stream))
    _check(st, "kvq_fake_quant")
    return xh, codes, scales


def attn_dense(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, softmax_scale: Optional[float] = None,
               want_top: bool = False, stream=None):
    """kvq_attn_dense: q bf16 [batch][Hq][d], k, v float [batch][T][Hkv][d] ->
    (out float [batch][Hq][d], top int32 [batch][Hq] or None)."""
    _need(q, torch.bfloat16, "q")
    _need(k, torch.float32, "k")
    _need(v, torch.float32, "v")
    B, Hq, d = q.shape
    T, Hkv = k.shape[1], k.shape[2]
    out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
    top = torch.empty((B, Hq), dtype=torch.int32, device=q.device) if want_top else None
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else softmax_scale
    st = load().kvq_attn_dense(B, T, Hq, Hkv, d, _ptr(q), _ptr(k), _ptr(v), float(scale), _ptr(out), _ptr(top),
                               _stream(stream))
    _check(st, "kvq_attn_dense")
    return out, top
