"""Thin ctypes binding over the C ABI of ``libpagedkv.so`` (include/pagedkv.h).

Argument marshalling only: tensors are checked for device, dtype, shape and contiguity and
passed as raw device pointers together with torch's current CUDA stream.  Every step of the
hot path runs in the library's kernels.  If the library has not been built, every call
raises ``RuntimeError``: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

from .rotary import Rotary

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libpagedkv.so")

PKV_F16, PKV_BF16, PKV_FP8_E4M3, PKV_INT4 = 0, 1, 2, 3
_DT = {"f16": PKV_F16, "bf16": PKV_BF16, "fp8": PKV_FP8_E4M3, "int4": PKV_INT4}
_TORCH = {PKV_F16: torch.float16, PKV_BF16: torch.bfloat16}
DEVERR = {1: "block id", 2: "slot", 4: "length", 8: "cu_seqlens", 16: "timeout"}

_lock = threading.Lock()
_lib = None


class PagedKVError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"pagedkv status {status}: {msg}")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load the CUDA library (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"CUDA library {LIB_PATH} is not built; run __graft_entry__.build() "
                               "(paged_kv_cache_134_gb300.build.build()) on a machine with nvcc")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.kv_cache_create.argtypes = [i64, i32, i32, i32, i32, i32, ctypes.POINTER(vp)]
        L.kv_cache_destroy.argtypes = [vp]
        L.kv_cache_set_scales.argtypes = [vp, vp, vp, vp]
        L.kv_cache_view.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(i64), ctypes.POINTER(i64)]
        L.kv_cache_reserve.argtypes = [vp, i32, i32, i32]
        L.kv_cache_reserve_mass.argtypes = [vp, i32, i32, i32, i64]
        L.kv_cache_reserve_window.argtypes = [vp, i32, i32, i32, i32, i32]
        L.kv_cache_reserve_chunk.argtypes = [vp, i32, i64, i32, i32, i32]
        L.kv_cache_release_workspaces.argtypes = [vp, i32]
        L.kv_cache_check_error.argtypes = [vp, ctypes.POINTER(i32)]
        L.pkv_last_error.restype = ctypes.c_char_p
        L.paged_slot_mapping.argtypes = [vp, i32, i32, vp, vp, i64, i32, vp, vp]
        L.paged_kv_append.argtypes = [vp, vp, vp, vp, i64, vp]
        L.paged_kv_append_at.argtypes = [vp, vp, vp, vp, i32, i32, vp, vp, i64, vp, vp]
        L.paged_kv_append_rotary.argtypes = [vp, vp, i64, vp, i64, vp, i64, i32, vp, i32, i32, vp, vp, vp, i64, vp, vp, vp,
                                             ctypes.c_float, vp, i64, vp, vp]
        L.paged_decode_attention.argtypes = [vp, vp, vp, i32, vp, i32, i32, ctypes.c_float, vp, vp]
        L.paged_decode_attention_noalloc.argtypes = [vp, vp, vp, i32, vp, i32, i32, ctypes.c_float, vp, vp]
        L.paged_decode_attention_window.argtypes = [vp, vp, vp, i32, vp, i32, i32, ctypes.c_float, i32, i32, vp, vp]
        L.paged_kv_gather.argtypes = [vp, vp, i64, vp, vp, vp]
        L.paged_decode_attention_mass.argtypes = [vp, vp, vp, i32, vp, i32, i32, ctypes.c_float, ctypes.c_float, vp,
                                                  i64, vp, vp]
        L.paged_kv_evict.argtypes = [vp, vp, i32, vp, i32, vp, i64, i32, i32, vp, i32, vp, vp, vp, i64, vp]
        L.paged_chunk_attention.argtypes = [vp, vp, vp, i32, vp, vp, i32, i32, i64, i32, ctypes.c_float, i32, i32, vp, vp]
        L.packed_prefill_attention.argtypes = [vp, vp, vp, vp, i32, i32, i64, vp, i32, vp, i32, ctypes.c_float, vp,
                                               vp]
        L.paged_prefill_attention.argtypes = [vp, vp, vp, vp, vp, i32, i32, i64, vp, i32, vp, i32, ctypes.c_float, vp,
                                              vp]
        L.paged_block_copy.argtypes = [vp, vp, vp, i64, vp]
        L.paged_decode_attention_cascade.argtypes = [vp, vp, vp, i32, vp, i32, i32, i32, ctypes.c_float, vp, vp]
        L.pkv_block_hashes.argtypes = [vp, i64, i32, vp, i64, vp, vp, ctypes.POINTER(i64)]
        L.pkv_prefix_cache_create.argtypes = [i64, ctypes.POINTER(vp)]
        L.pkv_prefix_cache_destroy.argtypes = [vp]
        L.pkv_prefix_cache_match.argtypes = [vp, vp, i64, vp, ctypes.POINTER(i64)]
        L.pkv_prefix_cache_allocate.argtypes = [vp, i64, vp]
        L.pkv_prefix_cache_insert.argtypes = [vp, vp, vp, i64]
        L.pkv_prefix_cache_release.argtypes = [vp, vp, i64]
        L.pkv_prefix_cache_stats.argtypes = [vp, vp]
        L.paged_block_swap_out.argtypes = [vp, vp, i64, vp, vp]
        L.paged_block_swap_in.argtypes = [vp, vp, i64, vp, vp]
        L.kv_cache_profile_start.argtypes = [vp, ctypes.c_uint]
        L.kv_cache_profile_start_sampled.argtypes = [vp, ctypes.c_uint, ctypes.c_int]
        L.kv_cache_profile_read.argtypes = [vp, ctypes.c_void_p]
        L.pkv_kernel_launches.restype = i64
        L.kv_cache_selftest_wait_timeout.argtypes = [vp, ctypes.c_uint64, vp]
        _lib = L
        return L


class _Profile(ctypes.Structure):
    _fields_ = [("decode_launches", ctypes.c_int64), ("prefill_launches", ctypes.c_int64),
                ("append_launches", ctypes.c_int64), ("merge_launches", ctypes.c_int64),
                ("decode_ms", ctypes.c_double), ("prefill_ms", ctypes.c_double), ("append_ms", ctypes.c_double),
                ("merge_ms", ctypes.c_double), ("copy_launches", ctypes.c_int64), ("copy_ms", ctypes.c_double)]


def _check(status: int):
    if status:
        raise PagedKVError(status, lib().pkv_last_error().decode(errors="replace"))


def _stream(stream=None) -> int:
    """The stream's handle: the current stream's of the current device by default.

    (Raw handles and plain ints: building torch.cuda.Stream and ctypes objects took several of a small
    call's microseconds.)"""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return t.data_ptr() if t is not None else None


def _req(t: torch.Tensor, name: str, dtype=None, ndim=None):
    if type(t) is torch.Tensor and t.dtype is dtype and t.is_cuda and t.dim() == ndim and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def _take(cache: "KVCache", t: torch.Tensor, name: str, dtype, ndim: int) -> int:
    """The address of a checked tensor on the cache's device."""
    if (type(t) is torch.Tensor and t.dtype is dtype and t.dim() == ndim and t.get_device() == cache.device
            and t.is_contiguous()):
        return t.data_ptr()
    _req(t, name, dtype, ndim)
    if t.get_device() != cache.device:
        raise ValueError(f"{name} is on {t.device}, the cache on cuda:{cache.device}")
    return t.data_ptr()


class _DevMem:
    """Exposes a raw device range through __cuda_array_interface__ for a zero-copy torch view."""

    def __init__(self, ptr: int, nbytes: int, owner):
        self.__cuda_array_interface__ = {"shape": (int(nbytes),), "typestr": "|u1", "data": (int(ptr), False),
                                         "version": 3, "strides": None}
        self._owner = owner


class KVCache:
    """A block pool on the current CUDA device (kv_cache_create)."""

    def __init__(self, num_blocks: int, block_size: int, num_kv_heads: int, head_dim: int,
                 kv_dtype: str = "f16", model_dtype: Optional[str] = None):
        L = lib()
        self.num_blocks, self.block_size = int(num_blocks), int(block_size)
        self.num_kv_heads, self.head_dim = int(num_kv_heads), int(head_dim)
        self.kv_dtype = kv_dtype
        self.model_dtype = model_dtype or (kv_dtype if kv_dtype not in ("fp8", "int4") else "bf16")
        h = ctypes.c_void_p()
        _check(L.kv_cache_create(self.num_blocks, self.block_size, self.num_kv_heads, self.head_dim,
                                 _DT[kv_dtype], _DT[self.model_dtype], ctypes.byref(h)))
        self._h = h
        self.device = torch.cuda.current_device()
        self.torch_dtype = _TORCH[_DT[self.model_dtype]]

    @property
    def handle(self) -> ctypes.c_void_p:
        if self._h is None:
            raise RuntimeError("cache is closed")
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None:
            lib().kv_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def view(self):
        """(uint8 tensor over the whole pool, element strides of (block, K|V, head, offset, dim))."""
        base = ctypes.c_void_p()
        st = (ctypes.c_int64 * 5)()
        nbytes = ctypes.c_int64()
        _check(lib().kv_cache_view(self.handle, ctypes.byref(base), st, ctypes.byref(nbytes)))
        raw = torch.as_tensor(_DevMem(base.value, nbytes.value, self), device="cuda")
        return raw, [int(x) for x in st]

    def pool_elems(self) -> torch.Tensor:
        """The pool as a flat tensor of raw elements (int16 for 16-bit caches, uint8 for FP8; the bytes of a
        4-bit cache)."""
        raw, _ = self.view()
        return raw if self.kv_dtype in ("fp8", "int4") else raw.view(torch.int16)

    def set_scales(self, k_scale: torch.Tensor, v_scale: torch.Tensor):
        _req(k_scale, "k_scale", torch.float32, 1)
        _req(v_scale, "v_scale", torch.float32, 1)
        if k_scale.numel() != self.num_kv_heads or v_scale.numel() != self.num_kv_heads:
            raise ValueError("one scale per KV head")
        _check(lib().kv_cache_set_scales(self.handle, _ptr(k_scale), _ptr(v_scale), _stream()))

    def reserve(self, max_seqs: int, max_q_heads: int, max_blocks_per_seq: int):
        """Allocate the decode's workspace for calls of at most these sizes (4-bit caches: one more workspace a call,
        for one stream or stream capture)."""
        _check(lib().kv_cache_reserve(self.handle, int(max_seqs), int(max_q_heads), int(max_blocks_per_seq)))

    def reserve_mass(self, max_seqs: int, max_q_heads: int, max_blocks_per_seq: int, max_mass_len: int):
        """Allocate a workspace for paged_decode_attention_mass calls of at most these sizes (any cache type), for one
        stream or stream capture."""
        _check(lib().kv_cache_reserve_mass(self.handle, int(max_seqs), int(max_q_heads), int(max_blocks_per_seq),
                                           int(max_mass_len)))

    def reserve_window(self, max_seqs: int, max_q_heads: int, max_blocks_per_seq: int, max_window: int, max_sinks: int = 0):
        """Allocate a workspace for paged_decode_attention_window calls of at most these sizes, for one stream or stream
        capture."""
        window, sinks = _window(max_window, max_sinks, 1)
        _check(lib().kv_cache_reserve_window(self.handle, int(max_seqs), int(max_q_heads), int(max_blocks_per_seq), window,
                                             sinks))

    def reserve_chunk(self, max_seqs: int, max_tokens: int, max_seqlen: int, max_q_heads: int, max_blocks_per_seq: int):
        """Allocate a workspace for paged_chunk_attention calls of at most these sizes, for one stream or stream capture."""
        _check(lib().kv_cache_reserve_chunk(self.handle, int(max_seqs), int(max_tokens), _c_int(max_seqlen),
                                            int(max_q_heads), int(max_blocks_per_seq)))

    def release_workspaces(self, graphs: bool = False):
        """Synchronise and free the workspaces that the mass and windowed decodes, the chunk attention and the
        decode of 4-bit caches keep for streams; with ``graphs`` also those of stream captures, whose graphs must not be
        replayed again."""
        _check(lib().kv_cache_release_workspaces(self.handle, int(graphs)))

    def check_error(self) -> int:
        """Synchronise and return (and clear) the device error bits; 0 when clean."""
        code = ctypes.c_int(0)
        st = lib().kv_cache_check_error(self.handle, ctypes.byref(code))
        if st not in (0, -5):
            _check(st)
        return int(code.value)

    def selftest_wait_timeout(self, limit_ns: int = 1_000_000):
        """Enqueue the bounded-wait self-test: a kernel waits on an mbarrier that never completes
        and gives up after limit_ns, setting the timeout bit that check_error then returns."""
        _check(lib().kv_cache_selftest_wait_timeout(self.handle, int(limit_ns), _stream()))

    PROFILE = {"decode": 1, "prefill": 2, "append": 4, "merge": 8, "copy": 16}

    @property
    def block_bytes(self) -> int:
        """Bytes of one physical block (K and V of every KV head)."""
        if self.kv_dtype == "int4":
            return self.num_kv_heads * self.block_size * (self.head_dim + 8)
        return 2 * self.num_kv_heads * self.block_size * self.head_dim * (1 if self.kv_dtype == "fp8" else 2)

    def profile_start(self, kinds=("decode", "prefill", "append", "merge"), every: int = 1):
        """Record CUDA events around the named kernels (events between kernels stop their overlap);
        with every > 1 only around every n-th launch of each kind."""
        mask = 0
        for k in kinds:
            mask |= self.PROFILE[k]
        _check(lib().kv_cache_profile_start_sampled(self.handle, mask, int(every)))

    def profile_read(self) -> dict:
        p = _Profile()
        _check(lib().kv_cache_profile_read(self.handle, ctypes.byref(p)))
        return {k: getattr(p, k) for k, _ in _Profile._fields_}


def kernel_launches() -> int:
    return int(lib().pkv_kernel_launches())


def paged_slot_mapping(block_tables: torch.Tensor, seq_ids: torch.Tensor, positions: torch.Tensor,
                       block_size: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    _req(block_tables, "block_tables", torch.int32, 2)
    _req(seq_ids, "seq_ids", torch.int32, 1)
    _req(positions, "positions", torch.int32, 1)
    n = positions.numel()
    if seq_ids.numel() != n:
        raise ValueError("seq_ids and positions differ in length")
    if out is None:
        out = torch.empty(n, dtype=torch.int64, device=positions.device)
    _req(out, "out", torch.int64, 1)
    _check(lib().paged_slot_mapping(_ptr(block_tables), block_tables.shape[0], block_tables.shape[1],
                                    _ptr(seq_ids), _ptr(positions), n, int(block_size), _ptr(out), _stream()))
    return out


def paged_kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor) -> None:
    _req(k, "k", cache.torch_dtype, 3)
    _req(v, "v", cache.torch_dtype, 3)
    _req(slot_mapping, "slot_mapping", torch.int64, 1)
    n = k.shape[0]
    if k.shape != (n, cache.num_kv_heads, cache.head_dim) or k.shape != v.shape:
        raise ValueError(f"k/v must be [T, {cache.num_kv_heads}, {cache.head_dim}]")
    if slot_mapping.numel() != n:
        raise ValueError("slot_mapping length != number of tokens")
    _check(lib().paged_kv_append(cache.handle, _ptr(k), _ptr(v), _ptr(slot_mapping), n, _stream()))


def paged_kv_append_at(cache: KVCache, k: torch.Tensor, v: torch.Tensor, block_tables: torch.Tensor,
                       seq_ids: torch.Tensor, positions: torch.Tensor,
                       slot_mapping: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Slot indexing + append in one launch; fills ``slot_mapping`` (int64) when given."""
    _req(k, "k", cache.torch_dtype, 3)
    _req(v, "v", cache.torch_dtype, 3)
    _req(block_tables, "block_tables", torch.int32, 2)
    _req(seq_ids, "seq_ids", torch.int32, 1)
    _req(positions, "positions", torch.int32, 1)
    n = k.shape[0]
    if k.shape != (n, cache.num_kv_heads, cache.head_dim) or k.shape != v.shape:
        raise ValueError(f"k/v must be [T, {cache.num_kv_heads}, {cache.head_dim}]")
    if seq_ids.numel() != n or positions.numel() != n:
        raise ValueError("seq_ids/positions length != number of tokens")
    if slot_mapping is not None:
        _req(slot_mapping, "slot_mapping", torch.int64, 1)
        if slot_mapping.numel() != n:
            raise ValueError("slot_mapping length != number of tokens")
    _check(lib().paged_kv_append_at(cache.handle, _ptr(k), _ptr(v), _ptr(block_tables), block_tables.shape[0],
                                    block_tables.shape[1], _ptr(seq_ids), _ptr(positions), n, _ptr(slot_mapping),
                                    _stream()))
    return slot_mapping


def _take_rows(cache: "KVCache", t: torch.Tensor, name: str, heads: Optional[int], n: Optional[int]):
    """Address and token stride (elements) of [T, heads, head_dim] rows whose tokens may lie apart."""
    d = cache.head_dim
    if type(t) is torch.Tensor and t.dtype is cache.torch_dtype and t.get_device() == cache.device:
        shape = t.shape
        if len(shape) == 3 and shape[2] == d and (heads is None or shape[1] == heads) and (n is None or shape[0] == n):
            stride, head, elem = t.stride()
            if elem == 1 and head == d and shape[0] > 1:
                return t.data_ptr(), stride
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.get_device() != cache.device:
        raise ValueError(f"{name} is on {t.device}, the cache on cuda:{cache.device}")
    if t.dtype != cache.torch_dtype:
        raise TypeError(f"{name} must be {cache.torch_dtype}, got {t.dtype}")
    if t.dim() != 3 or t.shape[2] != d or (heads is not None and t.shape[1] != heads) or \
            (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must be [{'T' if n is None else n}, {'H' if heads is None else heads}, {d}], got "
                         f"{list(t.shape)}")
    stride, head, elem = t.stride()
    if elem != 1 or (t.shape[1] > 1 and head != d):
        raise ValueError(f"{name}'s heads must be contiguous")
    if t.shape[0] <= 1:
        return t.data_ptr(), t.shape[1] * d
    return t.data_ptr(), stride


def paged_kv_append_rotary(cache: KVCache, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                           block_tables: torch.Tensor, seq_ids: torch.Tensor, positions: torch.Tensor, rotary: Rotary,
                           q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                           eps: float = 1e-6, rotary_positions: Optional[torch.Tensor] = None,
                           slot_mapping: Optional[torch.Tensor] = None,
                           q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """paged_kv_append_at of rows as the projections leave them: q and k normed per head (where a weight is given),
    rotated, k and v written to their slots, q returned.

    q, k and v may be slices of one [T, (Hq + 2 Hkv) * D] projection (tokens apart, heads contiguous).
    ``rotary_positions`` (int32 [T]) where the rotation's position is not the place in the cache; ``q_out`` may be
    ``q``.  ``q`` None: k and v alone (returns None)."""
    n = k.shape[0] if isinstance(k, torch.Tensor) and k.dim() == 3 else None
    kp, ks = _take_rows(cache, k, "k", cache.num_kv_heads, None)
    vp, vs = _take_rows(cache, v, "v", cache.num_kv_heads, n)
    tables = _take(cache, block_tables, "block_tables", torch.int32, 2)
    seqs = _take(cache, seq_ids, "seq_ids", torch.int32, 1)
    pos = _take(cache, positions, "positions", torch.int32, 1)
    if seq_ids.shape[0] != n or positions.shape[0] != n:
        raise ValueError("seq_ids/positions length != number of tokens")
    if not isinstance(rotary, Rotary):
        raise TypeError("rotary must be a Rotary")
    angles = None
    if rotary_positions is not None:
        angles = _take(cache, rotary_positions, "rotary_positions", torch.int32, 1)
        if rotary_positions.shape[0] != n:
            raise ValueError("rotary_positions length != number of tokens")
    slots = None
    if slot_mapping is not None:
        slots = _take(cache, slot_mapping, "slot_mapping", torch.int64, 1)
        if slot_mapping.shape[0] != n:
            raise ValueError("slot_mapping length != number of tokens")
    weights = []
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        weights.append(None if w is None else _take(cache, w, name, cache.torch_dtype, 1))
        if w is not None and w.shape[0] != cache.head_dim:
            raise ValueError(f"{name} must be [{cache.head_dim}]")
    if q is None:
        if q_out is not None or q_weight is not None:
            raise ValueError("q_out and q_weight need q")
        qp, qs, hq, op, os_ = None, 0, 0, None, 0
    else:
        qp, qs = _take_rows(cache, q, "q", None, n)
        hq = q.shape[1]
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        op, os_ = _take_rows(cache, q_out, "q_out", hq, n)
    _check(lib().paged_kv_append_rotary(cache.handle, qp, qs, kp, ks, vp, vs, hq, tables, block_tables.shape[0],
                                        block_tables.shape[1], seqs, pos, angles, n, rotary._ref, weights[0],
                                        weights[1], float(eps), op, os_, slots, _stream()))
    return q_out


def paged_kv_gather(cache: KVCache, slot_mapping: torch.Tensor, k: Optional[torch.Tensor] = None,
                    v: Optional[torch.Tensor] = None):
    """K and V at ``slot_mapping`` as (k, v), each [T, num_kv_heads, head_dim] in the model dtype: the
    stored values of any cache type (a negative slot gives zeros)."""
    slots = _take(cache, slot_mapping, "slot_mapping", torch.int64, 1)
    n = slot_mapping.shape[0]
    shape = (n, cache.num_kv_heads, cache.head_dim)
    for name, t in (("k", k), ("v", v)):
        if t is not None:
            _take(cache, t, name, cache.torch_dtype, 3)
            if t.shape != shape:
                raise ValueError(f"{name} must be {list(shape)}")
    if k is None:
        k = slot_mapping.new_empty(shape, dtype=cache.torch_dtype)
    if v is None:
        v = torch.empty_like(k)
    _check(lib().paged_kv_gather(cache.handle, slots, n, k.data_ptr(), v.data_ptr(), _stream()))
    return k, v


def paged_decode_attention_mass(q: torch.Tensor, cache: KVCache, block_tables: torch.Tensor,
                                context_lens: torch.Tensor, scale: float, attn_mass: torch.Tensor,
                                decay: float = 1.0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """paged_decode_attention that also adds every token's attention weight, summed over the query heads
    of its KV head, to ``attn_mass`` (float32 [S, num_kv_heads, T], in place, after multiplying by
    ``decay``); T must reach every length.  A token's entry starts at 0."""
    qp = _take(cache, q, "q", cache.torch_dtype, 3)
    tables = _take(cache, block_tables, "block_tables", torch.int32, 2)
    lens = _take(cache, context_lens, "context_lens", torch.int32, 1)
    mass = _take(cache, attn_mass, "attn_mass", torch.float32, 3)
    S, hq, d = q.shape
    table_rows, width = block_tables.shape
    if d != cache.head_dim or table_rows != S or context_lens.shape[0] != S:
        raise ValueError("shape mismatch between q, block_tables and context_lens")
    rows, heads, mass_len = attn_mass.shape
    if rows != S or heads != cache.num_kv_heads:
        raise ValueError(f"attn_mass must be [{S}, {cache.num_kv_heads}, T]")
    if out is None:
        out = torch.empty_like(q)
    else:
        _take(cache, out, "out", cache.torch_dtype, 3)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    _check(lib().paged_decode_attention_mass(qp, cache.handle, tables, width, lens, S, hq, float(scale), float(decay),
                                             mass, mass_len, out.data_ptr(), _stream()))
    return out


def paged_kv_evict(cache: KVCache, block_tables: torch.Tensor, context_lens: torch.Tensor, attn_mass: torch.Tensor,
                   budget: int, recent: int, dst_block_tables: torch.Tensor, kept: Optional[torch.Tensor] = None,
                   new_lens: Optional[torch.Tensor] = None, new_mass: Optional[torch.Tensor] = None):
    """Keep per (sequence, KV head) the last ``recent`` tokens and the ``budget - recent`` others of largest
    ``attn_mass``, copied in order to the blocks of ``dst_block_tables`` (blocks of no table of this call).

    Returns (kept int32 [S, Hkv, budget]: the positions that stay, -1 behind them; new_lens int32 [S];
    new_mass float32 [S, Hkv, T']: their mass, 0 behind them, T' = attn_mass's T unless given).  The old
    blocks are unchanged; the caller releases them."""
    tables = _take(cache, block_tables, "block_tables", torch.int32, 2)
    dst = _take(cache, dst_block_tables, "dst_block_tables", torch.int32, 2)
    lens = _take(cache, context_lens, "context_lens", torch.int32, 1)
    mass = _take(cache, attn_mass, "attn_mass", torch.float32, 3)
    S, hkv, budget, recent = context_lens.shape[0], cache.num_kv_heads, int(budget), int(recent)
    table_rows, width = block_tables.shape
    dst_rows, dst_width = dst_block_tables.shape
    rows, heads, mass_len = attn_mass.shape
    if not table_rows == dst_rows == rows == S or heads != hkv:
        raise ValueError("shape mismatch between tables, context_lens and attn_mass")
    if not 0 <= recent <= budget or not 1 <= budget <= 1 << 30:
        raise ValueError(f"recent {recent} and budget {budget}: 0 <= recent <= budget, 1 <= budget <= 2^30")
    if kept is None:
        kept = context_lens.new_empty((S, hkv, budget))
    else:
        _take(cache, kept, "kept", torch.int32, 3)
        if kept.shape != (S, hkv, budget):
            raise ValueError(f"kept must be {[S, hkv, budget]}")
    if new_lens is None:
        new_lens = torch.empty_like(context_lens)
    else:
        _take(cache, new_lens, "new_lens", torch.int32, 1)
        if new_lens.shape[0] != S:
            raise ValueError(f"new_lens must be {[S]}")
    if new_mass is None:
        new_mass = torch.empty_like(attn_mass)
    else:
        _take(cache, new_mass, "new_mass", torch.float32, 3)
        if new_mass.shape[:2] != (S, hkv):
            raise ValueError(f"new_mass must be [{S}, {hkv}, T']")
    _check(lib().paged_kv_evict(cache.handle, tables, width, lens, S, mass, mass_len, budget, recent, dst, dst_width,
                                kept.data_ptr(), new_lens.data_ptr(), new_mass.data_ptr(), new_mass.shape[2],
                                _stream()))
    return kept, new_lens, new_mass


def paged_decode_attention(q: torch.Tensor, cache: KVCache, block_tables: torch.Tensor,
                           context_lens: torch.Tensor, scale: float,
                           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    _req(q, "q", cache.torch_dtype, 3)
    _req(block_tables, "block_tables", torch.int32, 2)
    _req(context_lens, "context_lens", torch.int32, 1)
    S, hq, d = q.shape
    if d != cache.head_dim or block_tables.shape[0] != S or context_lens.numel() != S:
        raise ValueError("shape mismatch between q, block_tables and context_lens")
    if out is None:
        out = torch.empty_like(q)
    else:
        _req(out, "out", cache.torch_dtype, 3)
    _check(lib().paged_decode_attention(_ptr(q), cache.handle, _ptr(block_tables), block_tables.shape[1],
                                        _ptr(context_lens), S, hq, float(scale), _ptr(out), _stream()))
    return out


def paged_decode_attention_window(q: torch.Tensor, cache: KVCache, block_tables: torch.Tensor,
                                  context_lens: torch.Tensor, scale: float, window: int, sinks: int = 0,
                                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """paged_decode_attention over the last ``window`` tokens of each sequence and its first ``sinks``; blocks that
    hold none of them are not read."""
    qp = _take(cache, q, "q", cache.torch_dtype, 3)
    tables = _take(cache, block_tables, "block_tables", torch.int32, 2)
    lens = _take(cache, context_lens, "context_lens", torch.int32, 1)
    S, hq, d = q.shape
    rows, width = block_tables.shape
    if d != cache.head_dim or rows != S or context_lens.shape[0] != S:
        raise ValueError("shape mismatch between q, block_tables and context_lens")
    window, sinks = _window(window, sinks, 1)
    if out is None:
        out = torch.empty_like(q)
    else:
        _take(cache, out, "out", cache.torch_dtype, 3)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    _check(lib().paged_decode_attention_window(qp, cache.handle, tables, width, lens, S, hq, float(scale), window, sinks,
                                               out.data_ptr(), _stream()))
    return out


def _c_int(n):
    """The nearest number a C int holds (ctypes would take its low 32 bits): for sizes that may be larger than need be."""
    return min(max(int(n), -2 ** 31), 2 ** 31 - 1)


def _window(window, sinks, least):
    window, sinks = int(window), int(sinks)
    if window < least or sinks < 0 or (window == 0 and sinks):
        raise ValueError(f"window {window} and sinks {sinks}: window >= {least}, sinks >= 0 and 0 without a window")
    return min(window, 2 ** 31 - 1), min(sinks, 2 ** 31 - 1)


def paged_decode_attention_cascade(q: torch.Tensor, cache: KVCache, block_tables: torch.Tensor,
                                   context_lens: torch.Tensor, shared_prefix_len: int, scale: float,
                                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """paged_decode_attention for a batch whose tables share their first ``shared_prefix_len`` tokens."""
    _req(q, "q", cache.torch_dtype, 3)
    _req(block_tables, "block_tables", torch.int32, 2)
    _req(context_lens, "context_lens", torch.int32, 1)
    S, hq, d = q.shape
    if d != cache.head_dim or block_tables.shape[0] != S or context_lens.numel() != S:
        raise ValueError("shape mismatch between q, block_tables and context_lens")
    if out is None:
        out = torch.empty_like(q)
    _req(out, "out", cache.torch_dtype, 3)
    _check(lib().paged_decode_attention_cascade(_ptr(q), cache.handle, _ptr(block_tables), block_tables.shape[1],
                                                _ptr(context_lens), S, hq, int(shared_prefix_len),
                                                float(scale), _ptr(out), _stream()))
    return out


def paged_decode_attention_noalloc(q: torch.Tensor, cache: KVCache, block_tables: torch.Tensor,
                                   context_lens: torch.Tensor, scale: float, out: torch.Tensor) -> torch.Tensor:
    """paged_decode_attention for callers that must not allocate device memory.

    The library keeps the split-K partials in a fixed 16 MiB array of its own (made resident when
    the cache was created) instead of the cache's growable workspace, so this call allocates
    nothing (the caller provides ``out``).  Calls that can overlap on the GPU share that array and
    must be serialised by the caller."""
    _req(q, "q", cache.torch_dtype, 3)
    _req(block_tables, "block_tables", torch.int32, 2)
    _req(context_lens, "context_lens", torch.int32, 1)
    _req(out, "out", cache.torch_dtype, 3)
    S, hq, d = q.shape
    if d != cache.head_dim or block_tables.shape[0] != S or context_lens.numel() != S or out.shape != q.shape:
        raise ValueError("shape mismatch between q, out, block_tables and context_lens")
    _check(lib().paged_decode_attention_noalloc(_ptr(q), cache.handle, _ptr(block_tables), block_tables.shape[1],
                                                _ptr(context_lens), S, hq, float(scale), _ptr(out),
                                                _stream()))
    return out


def packed_prefill_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                             max_seqlen: int, block_tables: torch.Tensor, cache: KVCache, scale: float,
                             out: Optional[torch.Tensor] = None) -> torch.Tensor:
    for name, t in (("q", q), ("k", k), ("v", v)):
        _req(t, name, cache.torch_dtype, 3)
    _req(cu_seqlens, "cu_seqlens", torch.int32, 1)
    _req(block_tables, "block_tables", torch.int32, 2)
    T, hq, d = q.shape
    if k.shape != (T, cache.num_kv_heads, d) or v.shape != k.shape or d != cache.head_dim:
        raise ValueError("q/k/v shape mismatch")
    nseq = cu_seqlens.numel() - 1
    if block_tables.shape[0] != nseq:
        raise ValueError("one block-table row per sequence")
    if out is None:
        out = torch.empty_like(q)
    _req(out, "out", cache.torch_dtype, 3)
    _check(lib().packed_prefill_attention(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), nseq, int(max_seqlen), T,
                                          _ptr(block_tables), block_tables.shape[1], cache.handle, hq,
                                          float(scale), _ptr(out), _stream()))
    return out


def paged_chunk_attention(q: torch.Tensor, cache: KVCache, block_tables: torch.Tensor, context_lens: torch.Tensor,
                          cu_seqlens: torch.Tensor, max_seqlen: int, scale: float, window: int = 0, sinks: int = 0,
                          out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of the last tokens of each sequence over everything the cache holds of it.

    Sequence i holds ``context_lens[i]`` tokens, its new ones included (append them first); its rows
    [cu_seqlens[i], cu_seqlens[i + 1]) of q are the queries of the last of them.  Causal; with ``window`` > 0 a query sees the
    last ``window`` tokens up to its own and the first ``sinks``.  Any mix of single tokens, drafted tokens and
    pieces of prompts; ``max_seqlen`` is at least the longest piece."""
    qp = _take(cache, q, "q", cache.torch_dtype, 3)
    tables = _take(cache, block_tables, "block_tables", torch.int32, 2)
    lens = _take(cache, context_lens, "context_lens", torch.int32, 1)
    cu = _take(cache, cu_seqlens, "cu_seqlens", torch.int32, 1)
    T, hq, d = q.shape
    rows, width = block_tables.shape
    nseq = context_lens.shape[0]
    if d != cache.head_dim or rows != nseq or cu_seqlens.shape[0] != nseq + 1:
        raise ValueError("shape mismatch between q, block_tables, context_lens and cu_seqlens")
    window, sinks = _window(window, sinks, 0)
    if out is None:
        out = torch.empty_like(q)
    else:
        _take(cache, out, "out", cache.torch_dtype, 3)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    _check(lib().paged_chunk_attention(qp, cache.handle, tables, width, lens, cu, nseq, _c_int(max_seqlen), T, hq,
                                       float(scale), window, sinks, out.data_ptr(), _stream()))
    return out


def _req_buffer(t: torch.Tensor, name: str, nbytes: int):
    """A contiguous byte buffer the GPU can reach: a CUDA tensor or page-locked host memory."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, {nbytes} needed")


def paged_block_copy(cache: KVCache, src_blocks: torch.Tensor, dst_blocks: torch.Tensor) -> None:
    """Copy-on-write: block dst_blocks[i] := block src_blocks[i] (whole blocks)."""
    _req(src_blocks, "src_blocks", torch.int32, 1)
    _req(dst_blocks, "dst_blocks", torch.int32, 1)
    if src_blocks.numel() != dst_blocks.numel():
        raise ValueError("src_blocks and dst_blocks differ in length")
    _check(lib().paged_block_copy(cache.handle, _ptr(src_blocks), _ptr(dst_blocks), src_blocks.numel(), _stream()))


def paged_block_swap_out(cache: KVCache, block_ids: torch.Tensor, dst: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gather whole blocks into ``dst`` (uint8, CUDA or pinned host; block i at i * block_bytes)."""
    _req(block_ids, "block_ids", torch.int32, 1)
    n = block_ids.numel()
    if dst is None:
        dst = torch.empty(n * cache.block_bytes, dtype=torch.uint8).pin_memory()
    _req_buffer(dst, "dst", n * cache.block_bytes)
    _check(lib().paged_block_swap_out(cache.handle, _ptr(block_ids), n, _ptr(dst), _stream()))
    return dst


def paged_block_swap_in(cache: KVCache, block_ids: torch.Tensor, src: torch.Tensor) -> None:
    """Scatter whole blocks back: block block_ids[i] := src[i * block_bytes : (i + 1) * block_bytes]."""
    _req(block_ids, "block_ids", torch.int32, 1)
    n = block_ids.numel()
    _req_buffer(src, "src", n * cache.block_bytes)
    _check(lib().paged_block_swap_in(cache.handle, _ptr(block_ids), n, _ptr(src), _stream()))


def paged_prefill_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                            context_lens: torch.Tensor, max_seqlen: int, block_tables: torch.Tensor, cache: KVCache,
                            scale: float, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Prefill of each prompt's tail over the prefix its blocks already hold (writes the tail's K/V)."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        _req(t, name, cache.torch_dtype, 3)
    _req(cu_seqlens, "cu_seqlens", torch.int32, 1)
    _req(context_lens, "context_lens", torch.int32, 1)
    _req(block_tables, "block_tables", torch.int32, 2)
    T, hq, d = q.shape
    if k.shape != (T, cache.num_kv_heads, d) or v.shape != k.shape or d != cache.head_dim:
        raise ValueError("q/k/v shape mismatch")
    nseq = cu_seqlens.numel() - 1
    if block_tables.shape[0] != nseq or context_lens.numel() != nseq:
        raise ValueError("one block-table row and one context length per sequence")
    if out is None:
        out = torch.empty_like(q)
    _req(out, "out", cache.torch_dtype, 3)
    _check(lib().paged_prefill_attention(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), _ptr(context_lens), nseq,
                                         int(max_seqlen), T, _ptr(block_tables), block_tables.shape[1], cache.handle,
                                         hq, float(scale), _ptr(out), _stream()))
    return out


# ----------------------------------------------------------------------------- prefix cache (host)

def _np(a, dtype):
    import numpy as np
    return np.ascontiguousarray(a, dtype=dtype)


def block_hashes(tokens, block_size: int, extra: bytes = b"", init: Optional[bytes] = None):
    """Chained SHA-256 hashes of the full blocks of ``tokens`` (host); returns uint8 [n, 32]."""
    import numpy as np
    tok = _np(tokens, np.int32)
    n = len(tok) // int(block_size)
    out = np.zeros((n, 32), np.uint8)
    got = ctypes.c_int64(0)
    ex = ctypes.create_string_buffer(bytes(extra), len(extra)) if extra else None
    ini = ctypes.create_string_buffer(bytes(init), 32) if init is not None else None
    _check(lib().pkv_block_hashes(tok.ctypes.data, len(tok), int(block_size), ex, len(extra), ini,
                                  out.ctypes.data, ctypes.byref(got)))
    assert got.value == n
    return out


class PrefixCache:
    """Host prefix cache: hash -> physical block map, reference counts, LRU retention."""

    def __init__(self, num_blocks: int):
        h = ctypes.c_void_p()
        _check(lib().pkv_prefix_cache_create(int(num_blocks), ctypes.byref(h)))
        self._h = h

    def close(self):
        if getattr(self, "_h", None) is not None:
            lib().pkv_prefix_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def match(self, hashes):
        """Blocks of the longest cached prefix (attached: reference count + 1)."""
        import numpy as np
        hs = _np(hashes, np.uint8).reshape(-1, 32)
        out = np.zeros(len(hs), np.int32)
        hit = ctypes.c_int64(0)
        _check(lib().pkv_prefix_cache_match(self._h, hs.ctypes.data, len(hs), out.ctypes.data, ctypes.byref(hit)))
        return out[: hit.value]

    def allocate(self, n: int):
        import numpy as np
        out = np.zeros(int(n), np.int32)
        _check(lib().pkv_prefix_cache_allocate(self._h, int(n), out.ctypes.data))
        return out

    def insert(self, hashes, blocks):
        import numpy as np
        hs = _np(hashes, np.uint8).reshape(-1, 32)
        bl = _np(blocks, np.int32)
        assert len(hs) == len(bl)
        _check(lib().pkv_prefix_cache_insert(self._h, hs.ctypes.data, bl.ctypes.data, len(bl)))

    def release(self, blocks):
        import numpy as np
        bl = _np(blocks, np.int32)
        _check(lib().pkv_prefix_cache_release(self._h, bl.ctypes.data, len(bl)))

    def stats(self) -> dict:
        import numpy as np
        out = np.zeros(4, np.int64)
        _check(lib().pkv_prefix_cache_stats(self._h, out.ctypes.data))
        return dict(free=int(out[0]), cached_free=int(out[1]), in_use=int(out[2]), hashed=int(out[3]))
