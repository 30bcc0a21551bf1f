"""Hybrid-SWA attention with sinks over a ring KV cache, for GB300 (sm_103a).

Thin Python binding over the C ABI of ``libkvring.so`` (``include/kvring.h``).
It only marshals arguments: every step of the attention path runs in the
library's CUDA kernels.  PyTorch supplies device memory and streams.  There
is no fallback: if the library is missing, every call raises.

The five calls (colibri "MiMo-V2.6", "What the engine implements";
gaudi-cookbook "MiMo-V2.6-Flash on Gaudi 2", "What was built"):

  kv_ring_append_rope     RoPE k (dims 0..63), scale v, write ring / pages / rows
  swa_sink_decode         one token over a 128-slot ring with a per-head sink
  full_attn_decode        one token over a paged pool, split-K + LSE combine
  swa_sink_prefill_chunk  a chunk over ring + chunk rows, sink in the softmax
  full_attn_prefill_chunk a chunk over a paged pool, causal

and the batched forms of the two prefill calls, ``swa_sink_prefill_varlen``
and ``full_attn_prefill_varlen``: n chunks of different lengths in one call
(multi-token-prediction draft verification, mixed prefill/decode batches).

A full layer's pool may be kept in 4 bits (``Kv4Layout``):

  kv4_append_rope         the KV write into it
  full_attn_decode_kv4    one token over it
  kv4_unpack              positions of it back to bf16 pages or rows

or in 8 bits (``Kv8Layout``: ``kv8_append_rope``, ``full_attn_decode_kv8``,
``kv8_unpack``), and ``kv_pages_grow`` builds a step's block tables and slot map
on the device from the requests' lengths, taking blocks from the free list that
``kv_pages_release_window`` fills.  Pages may be shared:

  kv_pages_fork           a sequence starts with another's positions
  kv_pages_free           a sequence, or a part of one, gives its blocks up
  kv_pages_compact        the used blocks move together at the pool's start
  kv_pages_copy           the block copies of either, in any pools
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

__all__ = [
    "KvrError", "RingLayout", "PagedLayout", "LinearLayout", "lib", "rope_table",
    "kv_ring_append_rope", "swa_sink_decode", "full_attn_decode", "full_attn_decode_workspace_size",
    "swa_sink_prefill_chunk", "full_attn_prefill_chunk", "device_status", "full_attn_decode_noalloc",
    "kv_ring_snapshot", "kv_ring_restore", "ring_snapshot_alloc",
    "full_attn_prefill_varlen", "swa_sink_prefill_varlen", "full_attn_prefill_varlen_workspace_size",
    "swa_sink_prefill_varlen_workspace_size",
    "Kv4Layout", "kv4_append_rope", "full_attn_decode_kv4", "full_attn_decode_kv4_workspace_size", "kv4_unpack",
    "kv_pages_grow",
    "Kv8Layout", "kv8_append_rope", "full_attn_decode_kv8", "full_attn_decode_kv8_workspace_size", "kv8_unpack",
    "kv_pages_fork", "kv_pages_free", "kv_pages_compact", "kv_pages_copy",
    "DQK", "DV", "DROT", "WINDOW",
]

DQK, DV, DROT, WINDOW = 192, 128, 64, 128
LAYOUT_RING, LAYOUT_PAGED, LAYOUT_LINEAR = 1, 2, 3
DEV_BAD_POS, DEV_BAD_SEQ, DEV_BAD_BLOCK, DEV_TIMEOUT, DEV_BAD_ROWS, DEV_FREE_FULL = 1, 2, 4, 8, 16, 32
DEV_NO_BLOCKS = 64
KV4_TILE = 2912  # bytes of 16 positions of one KV head in a 4-bit pool
KV8_TILE = 5136  # the same in an 8-bit pool

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvring.so")
_lib = None
_lock = threading.Lock()


class KvrError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"kvring error {code}: {msg}")
        self.code = code


class _Layout(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("slot_pos", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("num_seqs", ctypes.c_int32),
        ("max_blocks", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("num_rows", ctypes.c_int64),
    ]


class _Layout4(ctypes.Structure):  # (and that of an 8-bit pool: the same fields)
    _fields_ = [
        ("num_kv_heads", ctypes.c_int32),
        ("num_seqs", ctypes.c_int32),
        ("max_blocks", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("data", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
    ]


def lib():
    """The loaded libkvring.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise ImportError(f"{LIB_PATH} is missing: build it with sinks_kv_ring_gb300.build.build()")
                L = ctypes.CDLL(LIB_PATH)
                p, i32, i64, f32, f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double
                L.kvr_last_error.restype = ctypes.c_char_p
                L.kvr_last_error.argtypes = []
                L.kvr_device_status.restype = ctypes.c_int
                L.kvr_device_status.argtypes = [p, ctypes.c_int]
                L.kvr_debug_stall_next.restype = ctypes.c_int
                L.kvr_debug_stall_next.argtypes = [i32, i64]
                L.kvr_rope_table_build.restype = ctypes.c_int
                L.kvr_rope_table_build.argtypes = [f64, i64, p, ctypes.c_int]
                L.kv_ring_append_rope.restype = ctypes.c_int
                L.kv_ring_append_rope.argtypes = [p, p, p, p, i32, i32, p, i64, f32, p, p]
                L.swa_sink_decode.restype = ctypes.c_int
                L.swa_sink_decode.argtypes = [p, p, p, i32, i32, p, p, p, i64, f32, p, p]
                L.full_attn_decode_workspace_size.restype = ctypes.c_size_t
                L.full_attn_decode_workspace_size.argtypes = [i32, i32, i32, i64]
                L.full_attn_decode.restype = ctypes.c_int
                L.full_attn_decode.argtypes = [p, p, p, i32, i32, p, p, i64, f32, i64, p, ctypes.c_size_t, p, p]
                L.kv_ring_snapshot.restype = ctypes.c_int
                L.kv_ring_snapshot.argtypes = [p, p, i32, p, p, p, p]
                L.kv_ring_restore.restype = ctypes.c_int
                L.kv_ring_restore.argtypes = [p, p, i32, p, p, p, p]
                L.full_attn_decode_noalloc.restype = ctypes.c_int
                L.full_attn_decode_noalloc.argtypes = [p, p, p, i32, i32, p, p, i64, f32, i64, p, p]
                L.swa_sink_prefill_chunk.restype = ctypes.c_int
                L.swa_sink_prefill_chunk.argtypes = [p, i64, i32, i32, i32, p, p, p, p, i64, f32, p, p]
                L.full_attn_prefill_chunk.restype = ctypes.c_int
                L.full_attn_prefill_chunk.argtypes = [p, i64, i32, i32, i32, p, p, i64, f32, p, p]
                L.full_attn_prefill_varlen_workspace_size.restype = ctypes.c_size_t
                L.full_attn_prefill_varlen_workspace_size.argtypes = [i32, i64, i32, i32, i64]
                L.full_attn_prefill_varlen.restype = ctypes.c_int
                L.full_attn_prefill_varlen.argtypes = [p, p, p, p, i32, i64, i32, p, p, i64, f32, i64, p,
                                                       ctypes.c_size_t, p, p]
                L.swa_sink_prefill_varlen_workspace_size.restype = ctypes.c_size_t
                L.swa_sink_prefill_varlen_workspace_size.argtypes = [i32]
                L.swa_sink_prefill_varlen.restype = ctypes.c_int
                L.swa_sink_prefill_varlen.argtypes = [p, p, p, p, i32, i64, i32, p, p, p, p, i64, f32, p,
                                                      ctypes.c_size_t, p, p]
                L.kv_pages_release_window.restype = ctypes.c_int
                L.kv_pages_release_window.argtypes = [p, i32, i32, i32, i32, p, p, p, i32, i32, p, p, i32, p]
                L.kv_ring_gather_pages.restype = ctypes.c_int
                L.kv_ring_gather_pages.argtypes = [p, p, p, p, p, i32, p]
                L.kv_pages_grow.restype = ctypes.c_int
                L.kv_pages_grow.argtypes = [p, i32, i32, i32, i32, p, p, p, i32, p, p, p, i32, p, p, p, p, i64, p]
                L.kv4_append_rope.restype = ctypes.c_int
                L.kv4_append_rope.argtypes = [p, p, p, p, p, i32, i32, p, i64, f32, p, p]
                L.full_attn_decode_kv4_workspace_size.restype = ctypes.c_size_t
                L.full_attn_decode_kv4_workspace_size.argtypes = [i32, i32, i32, i64]
                L.full_attn_decode_kv4.restype = ctypes.c_int
                L.full_attn_decode_kv4.argtypes = [p, p, p, i32, i32, p, p, i64, f32, i64, p, ctypes.c_size_t, p, p]
                L.kv4_unpack.restype = ctypes.c_int
                L.kv4_unpack.argtypes = [p, p, p, p, i32, i64, p, p, p]
                L.kv8_append_rope.restype = ctypes.c_int
                L.kv8_append_rope.argtypes = [p, p, p, p, p, i32, i64, i32, p, i64, f32, p, p]
                L.full_attn_decode_kv8_workspace_size.restype = ctypes.c_size_t
                L.full_attn_decode_kv8_workspace_size.argtypes = [i32, i32, i32, i64]
                L.full_attn_decode_kv8.restype = ctypes.c_int
                L.full_attn_decode_kv8.argtypes = [p, p, p, i32, i32, p, p, i64, f32, i64, p, ctypes.c_size_t, p, p]
                L.kv8_unpack.restype = ctypes.c_int
                L.kv8_unpack.argtypes = [p, p, p, p, i32, i64, p, p, p]
                L.kv_pages_free.restype = ctypes.c_int
                L.kv_pages_free.argtypes = [p, i32, i32, i32, i32, p, p, p, p, i32, p, p, i32, p]
                L.kv_pages_fork.restype = ctypes.c_int
                L.kv_pages_fork.argtypes = [p, i32, i32, i32, i32, p, p, p, p, i32, p, p, p, i32, p, p, p, p]
                L.kv_pages_compact.restype = ctypes.c_int
                L.kv_pages_compact.argtypes = [p, p, i32, i32, i32, i32, p, p, p, p, p, i32, p, p, p, p]
                L.kv_pages_copy.restype = ctypes.c_int
                L.kv_pages_copy.argtypes = [p, p, i32, i32, p, p, p, i32, p]
                _lib = L
    return _lib


def _check(rc: int):
    if rc != 0:
        raise KvrError(rc, lib().kvr_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:  # the raw handle: a Stream object costs as much as the rest of a small call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _want(t, name, dtype, dim=None, cuda=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dims, got shape {tuple(t.shape)}")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# The C ABI takes bare pointers, so the sizes the kernels index by are
# checked here, before any launch.  Calls of a few microseconds first ask in one
# expression whether everything is as it should be (`fine`); the checks one by
# one, which say what is not, cost half as much as such a call again.

_BF, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
# what such an expression raises over something that is no tensor of its dims, and where there is no GPU
_ODD = (AttributeError, TypeError, ValueError, RuntimeError, AssertionError)


def _want_q(q):
    _want(q, "q", torch.bfloat16, 3)
    if q.shape[2] != DQK:
        raise ValueError(f"q must be [rows, Hq, {DQK}], got shape {tuple(q.shape)}")


def _want_table(table):
    _want(table, "table", torch.float32, 3)
    if table.shape[1:] != (DROT // 2, 2):
        raise ValueError(f"table must be [max_pos, {DROT // 2}, 2] (cos, sin), got shape {tuple(table.shape)}")


def _want_len(t, name, n):
    if t.shape[0] != n:
        raise ValueError(f"{name} must have {n} entries, got {t.shape[0]}")


def _empty(shape, dtype, like, stream):
    """Memory of a call's own, from the stream that the call runs on: a block that the current stream handed back may
    still be in use there.  The current stream, which is where the caller goes on, may use it as well."""
    cur = None if stream is None else torch.cuda.current_stream()
    if stream == cur:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if isinstance(getattr(stream, "cuda_stream", None), int) and not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=like.device)  # (a handle is all the calls ask for)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(cur)
    return t


def _out(out, rows, hq, like, stream):
    if out is None:
        return _empty((rows, hq, DV), torch.bfloat16, like, stream)
    _want(out, "out", torch.bfloat16, 3)
    if out.shape != (rows, hq, DV):
        raise ValueError(f"out must be [{rows}, {hq}, {DV}], got shape {tuple(out.shape)}")
    return out


def _same_device(first, *rest):
    """The library launches on the current CUDA device and reads every pointer
    of a call there, so all of the call's tensors must live on that device."""
    cur = torch.cuda.current_device()
    for t in rest:
        if t is not None and t.get_device() != cur:
            break
    else:
        if first.get_device() == cur:
            return
    dev = first.device
    if dev.index != cur:
        raise ValueError(f"the call's tensors are on {dev} but the current device is cuda:{cur} "
                         "(make it current with torch.cuda.device)")
    for t in rest:
        if t is not None and t.device != dev:
            raise ValueError(f"a tensor of the call is on {t.device}, the others on {dev}")


class RingLayout:
    """SWA pool of one layer: k [S, Hkv, 128, 192], v [S, Hkv, 128, 128] bf16,
    slot_pos [S, 128] int32 (-1 = empty)."""

    def __init__(self, k, v, slot_pos):
        _want(k, "ring.k", torch.bfloat16, 4)
        _want(v, "ring.v", torch.bfloat16, 4)
        _want(slot_pos, "ring.slot_pos", torch.int32, 2)
        S, H, W, D = k.shape
        if W != WINDOW or D != DQK or tuple(v.shape) != (S, H, WINDOW, DV) or tuple(slot_pos.shape) != (S, WINDOW):
            raise ValueError("ring tensors have inconsistent shapes")
        self.k, self.v, self.slot_pos = k, v, slot_pos
        self.num_seqs, self.num_kv_heads = S, H

    def tensors(self):
        return self.k, self.v, self.slot_pos

    @classmethod
    def empty(cls, num_seqs, num_kv_heads, device="cuda"):
        k = torch.zeros(num_seqs, num_kv_heads, WINDOW, DQK, dtype=torch.bfloat16, device=device)
        v = torch.zeros(num_seqs, num_kv_heads, WINDOW, DV, dtype=torch.bfloat16, device=device)
        sp = torch.full((num_seqs, WINDOW), -1, dtype=torch.int32, device=device)
        return cls(k, v, sp)

    @staticmethod
    def bytes_per_layer(num_seqs, num_kv_heads, elem_bytes=2):
        """Ring K+V bytes of one layer (slot tags not counted)."""
        return num_seqs * num_kv_heads * WINDOW * (DQK + DV) * elem_bytes

    def c(self):
        return _Layout(LAYOUT_RING, self.num_kv_heads, self.k.data_ptr(), self.v.data_ptr(),
                       self.slot_pos.data_ptr(), None, self.num_seqs, 0, 0, 0, 0)


class PagedLayout:
    """Full pool of one layer: k [nblk, Hkv, Bsz, 192], v [nblk, Hkv, Bsz, 128]
    bf16, block_table [S, max_blocks] int32."""

    def __init__(self, k, v, block_table):
        _want(k, "pool.k", torch.bfloat16, 4)
        _want(v, "pool.v", torch.bfloat16, 4)
        _want(block_table, "pool.block_table", torch.int32, 2)
        nb, H, bsz, D = k.shape
        if D != DQK or tuple(v.shape) != (nb, H, bsz, DV):
            raise ValueError("pool tensors have inconsistent shapes")
        self.k, self.v, self.block_table = k, v, block_table
        self.num_blocks, self.num_kv_heads, self.block_size = nb, H, bsz
        self.num_seqs, self.max_blocks = block_table.shape

    def tensors(self):
        return self.k, self.v, self.block_table

    @classmethod
    def contiguous(cls, num_seqs, num_kv_heads, max_ctx, block_size=64, device="cuda", zero=True):
        """A pool where sequence s owns blocks s*mb .. s*mb+mb-1 in order."""
        mb = (max_ctx + block_size - 1) // block_size
        nb = num_seqs * mb
        alloc = torch.zeros if zero else torch.empty
        k = alloc(nb, num_kv_heads, block_size, DQK, dtype=torch.bfloat16, device=device)
        v = alloc(nb, num_kv_heads, block_size, DV, dtype=torch.bfloat16, device=device)
        bt = torch.arange(nb, dtype=torch.int32, device=device).reshape(num_seqs, mb)
        return cls(k, v, bt)

    @staticmethod
    def bytes_per_token(num_kv_heads, elem_bytes=2, v_width=DV):
        """Pool K+V bytes one token adds per layer (v_width=192 models V zero-padded to 192)."""
        return num_kv_heads * (DQK + v_width) * elem_bytes

    def c(self):
        return _Layout(LAYOUT_PAGED, self.num_kv_heads, self.k.data_ptr(), self.v.data_ptr(), None,
                       self.block_table.data_ptr(), self.num_seqs, self.max_blocks, self.block_size,
                       self.num_blocks, 0)


class LinearLayout:
    """Staging rows: k [T, Hkv, 192], v [T, Hkv, 128] bf16."""

    def __init__(self, k, v):
        _want(k, "linear.k", torch.bfloat16, 3)
        _want(v, "linear.v", torch.bfloat16, 3)
        T, H, D = k.shape
        if D != DQK or v.shape != (T, H, DV):
            raise ValueError("linear tensors have inconsistent shapes")
        self.k, self.v = k, v
        self.num_rows, self.num_kv_heads = T, H

    def tensors(self):
        return self.k, self.v

    @classmethod
    def empty(cls, rows, num_kv_heads, device="cuda"):
        return cls(torch.empty(rows, num_kv_heads, DQK, dtype=torch.bfloat16, device=device),
                   torch.empty(rows, num_kv_heads, DV, dtype=torch.bfloat16, device=device))

    def c(self):
        return _Layout(LAYOUT_LINEAR, self.num_kv_heads, self.k.data_ptr(), self.v.data_ptr(), None, None,
                       0, 0, 0, 0, self.num_rows)


class _TileLayout:
    """A pool of tiles of 16 positions of one KV head: data [nblk, Hkv, Bsz / 16, TILE] uint8, block_table
    [S, max_blocks] int32."""

    TILE = 0

    def __init__(self, data, block_table):
        _want(data, "pool.data", torch.uint8, 4)
        _want(block_table, "pool.block_table", torch.int32, 2)
        nb, H, tiles, nbytes = data.shape
        if nbytes != self.TILE:
            raise ValueError(f"pool.data must be [blocks, Hkv, block_size / 16, {self.TILE}], got {tuple(data.shape)}")
        self.data, self.block_table = data, block_table
        self.num_blocks, self.num_kv_heads, self.block_size = nb, H, 16 * tiles
        self.num_seqs, self.max_blocks = block_table.shape
        self._c = _Layout4(H, self.num_seqs, self.max_blocks, 16 * tiles, nb)

    def tensors(self):
        return self.data, self.block_table

    @classmethod
    def contiguous(cls, num_seqs, num_kv_heads, max_ctx, block_size=64, device="cuda", zero=True):
        """A pool where sequence s owns blocks s*mb .. s*mb+mb-1 in order."""
        if block_size % 16:
            raise ValueError(f"block_size {block_size} is not a multiple of 16")
        mb = (max_ctx + block_size - 1) // block_size
        nb = num_seqs * mb
        alloc = torch.zeros if zero else torch.empty
        data = alloc(nb, num_kv_heads, block_size // 16, cls.TILE, dtype=torch.uint8, device=device)
        bt = torch.arange(nb, dtype=torch.int32, device=device).reshape(num_seqs, mb)
        return cls(data, bt)

    @classmethod
    def bytes_per_token(cls, num_kv_heads):
        """Pool bytes one token adds per layer."""
        return num_kv_heads * cls.TILE // 16

    def c(self):
        self._c.data, self._c.block_table = self.data.data_ptr(), self.block_table.data_ptr()
        return self._c


class Kv4Layout(_TileLayout):
    """Full pool of one layer in 4 bits: data [nblk, Hkv, Bsz / 16, 2912]
    uint8 (tiles of 16 positions, see kvr_kv4_layout in kvring.h), block_table
    [S, max_blocks] int32."""

    TILE = KV4_TILE


class Kv8Layout(_TileLayout):
    """Full pool of one layer in 8 bits: data [nblk, Hkv, Bsz / 16, 5136]
    uint8 (tiles of 16 positions, see kvr_kv8_layout in kvring.h), block_table
    [S, max_blocks] int32."""

    TILE = KV8_TILE


def rope_table(theta: float, max_pos: int, device="cuda", nthreads: int = 0) -> torch.Tensor:
    """[max_pos, 32, 2] fp32 (cos, sin) table, evaluated on the host in fp64
    by the library, then copied to `device`."""
    host = torch.empty((max_pos, 32, 2), dtype=torch.float32)
    _check(lib().kvr_rope_table_build(float(theta), int(max_pos), _ptr(host), int(nthreads)))
    return host if str(device) == "cpu" else host.to(device)


def kv_ring_append_rope(k, v, pos, seq, table, value_scale, dst, stream=None):
    _want(k, "k", torch.bfloat16, 3)
    _want(v, "v", torch.bfloat16, 3)
    _want(pos, "pos", torch.int64, 1)
    if seq is not None:
        _want(seq, "seq", torch.int32, 1)
    _want_table(table)
    T, H = k.shape[0], k.shape[1]
    if tuple(k.shape) != (T, H, DQK) or tuple(v.shape) != (T, H, DV) or pos.shape[0] != T:
        raise ValueError("k/v/pos shapes disagree")
    if seq is not None and seq.shape[0] != T:
        raise ValueError("seq shape disagrees")
    _same_device(k, v, pos, seq, table, *dst.tensors())
    c = dst.c()
    _check(lib().kv_ring_append_rope(_ptr(k), _ptr(v), _ptr(pos), _ptr(seq), T, H, _ptr(table),
                                     table.shape[0], float(value_scale), ctypes.byref(c), _stream(stream)))


def swa_sink_decode(q, pos, seq, ring, sinks, table, softmax_scale, out=None, stream=None):
    _want_q(q)
    _want(pos, "pos", torch.int64, 1)
    _want(seq, "seq", torch.int32, 1)
    _want(sinks, "sinks", torch.float32, 1)
    _want_table(table)
    B, Hq, _ = q.shape
    _want_len(pos, "pos", B)
    _want_len(seq, "seq", B)
    _want_len(sinks, "sinks", Hq)
    out = _out(out, B, Hq, q, stream)
    _same_device(q, pos, seq, sinks, table, out, *ring.tensors())
    c = ring.c()
    _check(lib().swa_sink_decode(_ptr(q), _ptr(pos), _ptr(seq), B, Hq, ctypes.byref(c), _ptr(sinks),
                                 _ptr(table), table.shape[0], float(softmax_scale), _ptr(out), _stream(stream)))
    return out


def full_attn_decode_workspace_size(B, Hq, Hkv, max_ctx) -> int:
    return int(lib().full_attn_decode_workspace_size(int(B), int(Hq), int(Hkv), int(max_ctx)))


def full_attn_decode(q, pos, seq, pool, table, softmax_scale, max_ctx, workspace=None, out=None, stream=None):
    _want_q(q)
    _want(pos, "pos", torch.int64, 1)
    _want(seq, "seq", torch.int32, 1)
    _want_table(table)
    B, Hq, _ = q.shape
    _want_len(pos, "pos", B)
    _want_len(seq, "seq", B)
    if workspace is None:
        n = full_attn_decode_workspace_size(B, Hq, pool.num_kv_heads, max_ctx)
        workspace = _empty(max(n, 1), torch.uint8, q, stream)
    _want(workspace, "workspace", torch.uint8, 1)
    out = _out(out, B, Hq, q, stream)
    _same_device(q, pos, seq, table, workspace, out, *pool.tensors())
    c = pool.c()
    _check(lib().full_attn_decode(_ptr(q), _ptr(pos), _ptr(seq), B, Hq, ctypes.byref(c), _ptr(table),
                                  table.shape[0], float(softmax_scale), int(max_ctx), _ptr(workspace),
                                  workspace.numel(), _ptr(out), _stream(stream)))
    return out


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


def full_attn_decode_noalloc(q, pos, seq, pool, table, softmax_scale, max_ctx, out=None, stream=None):
    """full_attn_decode for callers that may not allocate device memory: the
    split partials go to a fixed 32 MiB array inside the library instead of a
    workspace.  Calls that may run at the same time on the GPU share that
    array and must be ordered (e.g. one stream).  The first call on a device
    looks the array up; make it before any stream capture."""
    _want_q(q)
    _want(pos, "pos", torch.int64, 1)
    _want(seq, "seq", torch.int32, 1)
    _want_table(table)
    B, Hq, _ = q.shape
    _want_len(pos, "pos", B)
    _want_len(seq, "seq", B)
    out = _out(out, B, Hq, q, stream)
    _same_device(q, pos, seq, table, out, *pool.tensors())
    c = pool.c()
    _check(lib().full_attn_decode_noalloc(_ptr(q), _ptr(pos), _ptr(seq), B, Hq, ctypes.byref(c), _ptr(table),
                                          table.shape[0], float(softmax_scale), int(max_ctx), _ptr(out),
                                          _stream(stream)))
    return out


def swa_sink_prefill_chunk(q, P0, seq, chunk_kv, ring, sinks, table, softmax_scale, out=None, stream=None):
    _want_q(q)
    _want(sinks, "sinks", torch.float32, 1)
    _want_table(table)
    C, Hq, _ = q.shape
    _want_len(sinks, "sinks", Hq)
    out = _out(out, C, Hq, q, stream)
    _same_device(q, sinks, table, out, *chunk_kv.tensors(), *ring.tensors())
    cc, rc = chunk_kv.c(), ring.c()
    _check(lib().swa_sink_prefill_chunk(_ptr(q), int(P0), C, int(seq), Hq, ctypes.byref(cc), ctypes.byref(rc),
                                        _ptr(sinks), _ptr(table), table.shape[0], float(softmax_scale), _ptr(out),
                                        _stream(stream)))
    return out


def full_attn_prefill_chunk(q, P0, seq, pool, table, softmax_scale, out=None, stream=None):
    _want_q(q)
    _want_table(table)
    C, Hq, _ = q.shape
    out = _out(out, C, Hq, q, stream)
    _same_device(q, table, out, *pool.tensors())
    c = pool.c()
    _check(lib().full_attn_prefill_chunk(_ptr(q), int(P0), C, int(seq), Hq, ctypes.byref(c), _ptr(table),
                                         table.shape[0], float(softmax_scale), _ptr(out), _stream(stream)))
    return out


def full_attn_prefill_varlen_workspace_size(n, T, Hq, Hkv, max_ctx) -> int:
    return int(lib().full_attn_prefill_varlen_workspace_size(int(n), int(T), int(Hq), int(Hkv), int(max_ctx)))


def swa_sink_prefill_varlen_workspace_size(n) -> int:
    return int(lib().swa_sink_prefill_varlen_workspace_size(int(n)))


def _varlen_args(q, cu_rows, P0, seq):
    _want_q(q)
    _want(cu_rows, "cu_rows", torch.int32, 1)
    _want(P0, "P0", torch.int64, 1)
    _want(seq, "seq", torch.int32, 1)
    n = seq.numel()
    if cu_rows.numel() != n + 1 or P0.numel() != n:
        raise ValueError(f"cu_rows must have n+1 = {n + 1} entries and P0 n = {n}")
    return n


def full_attn_prefill_varlen(q, cu_rows, P0, seq, pool, table, softmax_scale, max_ctx, workspace=None, out=None,
                             stream=None):
    """n chunks over a full layer's paged pool: chunk s is q rows
    cu_rows[s]..cu_rows[s+1]-1 at positions P0[s].. of sequence seq[s]
    (device int32 / int64 / int32 tensors)."""
    n = _varlen_args(q, cu_rows, P0, seq)
    _want_table(table)
    T, Hq, _ = q.shape
    if workspace is None:
        nb = full_attn_prefill_varlen_workspace_size(n, T, Hq, pool.num_kv_heads, max_ctx)
        workspace = _empty(max(nb, 1), torch.uint8, q, stream)
    _want(workspace, "workspace", torch.uint8, 1)
    out = _out(out, T, Hq, q, stream)
    _same_device(q, cu_rows, P0, seq, table, workspace, out, *pool.tensors())
    c = pool.c()
    _check(lib().full_attn_prefill_varlen(_ptr(q), _ptr(cu_rows), _ptr(P0), _ptr(seq), n, T, Hq, ctypes.byref(c),
                                          _ptr(table), table.shape[0], float(softmax_scale), int(max_ctx),
                                          _ptr(workspace), workspace.numel(), _ptr(out), _stream(stream)))
    return out


def swa_sink_prefill_varlen(q, cu_rows, P0, seq, chunk_kv, ring, sinks, table, softmax_scale, workspace=None,
                            out=None, stream=None):
    """n chunks over a windowed layer: ring state before each chunk plus the
    batch's own rows in chunk_kv (row cu_rows[s] + i for chunk s)."""
    n = _varlen_args(q, cu_rows, P0, seq)
    _want(sinks, "sinks", torch.float32, 1)
    _want_table(table)
    T, Hq, _ = q.shape
    _want_len(sinks, "sinks", Hq)
    if workspace is None:
        nb = swa_sink_prefill_varlen_workspace_size(n)
        workspace = _empty(max(nb, 1), torch.uint8, q, stream)
    _want(workspace, "workspace", torch.uint8, 1)
    out = _out(out, T, Hq, q, stream)
    _same_device(q, cu_rows, P0, seq, sinks, table, workspace, out, *chunk_kv.tensors(), *ring.tensors())
    cc, rc = chunk_kv.c(), ring.c()
    _check(lib().swa_sink_prefill_varlen(_ptr(q), _ptr(cu_rows), _ptr(P0), _ptr(seq), n, T, Hq, ctypes.byref(cc),
                                         ctypes.byref(rc), _ptr(sinks), _ptr(table), table.shape[0],
                                         float(softmax_scale), _ptr(workspace), workspace.numel(), _ptr(out),
                                         _stream(stream)))
    return out


def ring_snapshot_alloc(n, num_kv_heads, device="cuda"):
    """Snapshot buffers for n rings: (k [n, Hkv, 128, 192], v [n, Hkv, 128, 128], tags [n, 128])."""
    return (torch.empty(n, num_kv_heads, WINDOW, DQK, dtype=torch.bfloat16, device=device),
            torch.empty(n, num_kv_heads, WINDOW, DV, dtype=torch.bfloat16, device=device),
            torch.empty(n, WINDOW, dtype=torch.int32, device=device))


def _ring_copy(fn, ring, seqs, snap, stream):
    _want(seqs, "seqs", torch.int32, 1)
    k, v, t = snap
    n = seqs.shape[0]
    _want(k, "k_snap", torch.bfloat16, 4)
    _want(v, "v_snap", torch.bfloat16, 4)
    _want(t, "tags_snap", torch.int32, 2)
    if k.shape[0] < n or v.shape[0] < n or t.shape[0] < n or k.shape[1] != ring.num_kv_heads:
        raise ValueError("snapshot buffers too small for the ring / sequence list")
    _same_device(seqs, k, v, t, *ring.tensors())
    c = ring.c()
    _check(fn(ctypes.byref(c), _ptr(seqs), n, _ptr(k), _ptr(v), _ptr(t), _stream(stream)))


def kv_ring_snapshot(ring, seqs, snap, stream=None):
    """Copy the rings (slots + tags) of sequences `seqs` into snapshot buffers."""
    _ring_copy(lib().kv_ring_snapshot, ring, seqs, snap, stream)


def kv_ring_restore(ring, seqs, snap, stream=None):
    """Copy snapshot buffers back into the rings of sequences `seqs`."""
    _ring_copy(lib().kv_ring_restore, ring, seqs, snap, stream)


def kv_pages_release_window(block_table, num_blocks, block_size, seqs, next_pos, free_ids, free_count, lo=None,
                            window=WINDOW, stream=None):
    """Release the pages of a windowed layer kept in pages that no query at or
    after next_pos[i] reads: their ids (entries of block_table, int32
    [num_seqs, max_blocks], ids < num_blocks) are appended to free_ids (int32
    [cap]) at free_count (int32 [1], advanced), their entries set to -1, and
    lo (int32 [num_seqs], optional) advanced.  Everything stays on the
    device."""
    _want(block_table, "block_table", torch.int32, 2)
    _want(seqs, "seqs", torch.int32, 1)
    _want(next_pos, "next_pos", torch.int64, 1)
    _want(free_ids, "free_ids", torch.int32, 1)
    _want(free_count, "free_count", torch.int32, 1)
    S, mb = block_table.shape
    if lo is not None:
        _want(lo, "lo", torch.int32, 1)
        if lo.shape[0] != S:
            raise ValueError("lo must have one entry per sequence of the block table")
    n = seqs.shape[0]
    if next_pos.shape[0] != n or free_count.shape[0] != 1:
        raise ValueError("seqs/next_pos/free_count shapes disagree")
    _same_device(block_table, seqs, next_pos, free_ids, free_count, lo)
    _check(lib().kv_pages_release_window(_ptr(block_table), S, mb, int(block_size), int(num_blocks), _ptr(seqs),
                                         _ptr(next_pos), _ptr(lo), n, int(window), _ptr(free_ids),
                                         _ptr(free_count), free_ids.shape[0], _stream(stream)))


def kv_ring_gather_pages(pages, ring, src_seqs, dst_seqs, end, stream=None):
    """Fill ring rows dst_seqs[i] with the window of paged sequence
    src_seqs[i] that ends before position end[i] (slot p mod 128 <- row p)."""
    _want(src_seqs, "src_seqs", torch.int32, 1)
    _want(dst_seqs, "dst_seqs", torch.int32, 1)
    _want(end, "end", torch.int64, 1)
    n = src_seqs.shape[0]
    if dst_seqs.shape[0] != n or end.shape[0] != n:
        raise ValueError("src_seqs/dst_seqs/end shapes disagree")
    _same_device(src_seqs, dst_seqs, end, *pages.tensors(), *ring.tensors())
    pc, rc = pages.c(), ring.c()
    _check(lib().kv_ring_gather_pages(ctypes.byref(pc), ctypes.byref(rc), _ptr(src_seqs), _ptr(dst_seqs), _ptr(end),
                                      n, _stream(stream)))


def kv_pages_grow(block_table, num_blocks, block_size, seqs, lens, add, free_ids, free_count, cu_rows, pos, row_seq,
                  slots, free_count_out=None, stream=None):
    """The block tables and slot map of a step in which request i (sequence
    seqs[i], int32 [n]) holds lens[i] (int64) positions and gains add[i]
    (int32) tokens: the blocks they need are taken from the end of the free
    list (free_ids int32 [cap], free_count int32 [1]) and written to
    block_table (int32 [num_seqs, max_blocks]); cu_rows (int32 [n + 1]) and the
    rows' pos (int64 [T]), row_seq (int32 [T]) and slots (int64 [T]) are filled
    (-1 past the last token).  The remaining count goes to free_count_out
    (default: free_count itself).  Everything stays on the device."""
    _want(block_table, "block_table", torch.int32, 2)
    _want(seqs, "seqs", torch.int32, 1)
    _want(lens, "lens", torch.int64, 1)
    _want(add, "add", torch.int32, 1)
    _want(free_ids, "free_ids", torch.int32, 1)
    _want(free_count, "free_count", torch.int32, 1)
    _want(cu_rows, "cu_rows", torch.int32, 1)
    _want(pos, "pos", torch.int64, 1)
    _want(row_seq, "row_seq", torch.int32, 1)
    _want(slots, "slots", torch.int64, 1)
    if free_count_out is None:
        free_count_out = free_count
    _want(free_count_out, "free_count_out", torch.int32, 1)
    S, mb = block_table.shape
    n, T = seqs.shape[0], pos.shape[0]
    _want_len(lens, "lens", n)
    _want_len(add, "add", n)
    _want_len(cu_rows, "cu_rows", n + 1)
    _want_len(row_seq, "row_seq", T)
    _want_len(slots, "slots", T)
    _want_len(free_count, "free_count", 1)
    _want_len(free_count_out, "free_count_out", 1)
    _same_device(block_table, seqs, lens, add, free_ids, free_count, free_count_out, cu_rows, pos, row_seq, slots)
    _check(lib().kv_pages_grow(_ptr(block_table), S, mb, int(block_size), int(num_blocks), _ptr(seqs), _ptr(lens),
                               _ptr(add), n, _ptr(free_ids), _ptr(free_count), _ptr(free_count_out),
                               free_ids.shape[0], _ptr(cu_rows), _ptr(pos), _ptr(row_seq), _ptr(slots), T,
                               _stream(stream)))


def kv4_append_rope(k, v, pos, seq, table, value_scale, dst, slots=None, stream=None):
    """kv_ring_append_rope into a 4-bit pool (Kv4Layout).  Token t goes to
    position pos[t] of sequence seq[t], or, with seq None, to slot slots[t]
    (block id * block_size + row, int64, as kv_pages_grow makes them).  seq -1
    or a negative slot marks padding."""
    _want(k, "k", torch.bfloat16, 3)
    _want(v, "v", torch.bfloat16, 3)
    _want(pos, "pos", torch.int64, 1)
    if (seq is None) == (slots is None):
        raise ValueError("exactly one of seq and slots names where the tokens go")
    if seq is not None:
        _want(seq, "seq", torch.int32, 1)
        _want_len(seq, "seq", k.shape[0])
    else:
        _want(slots, "slots", torch.int64, 1)
        _want_len(slots, "slots", k.shape[0])
    _want_table(table)
    T, H = k.shape[:2]
    if k.shape[2] != DQK or v.shape != (T, H, DV) or pos.shape[0] != T:
        raise ValueError("k/v/pos shapes disagree")
    _want_pool(dst, Kv4Layout)
    _same_device(k, v, pos, seq, slots, table, *dst.tensors())
    c = dst.c()
    _check(lib().kv4_append_rope(_ptr(k), _ptr(v), _ptr(pos), _ptr(seq), _ptr(slots), T, H, _ptr(table),
                                 table.shape[0], float(value_scale), ctypes.byref(c), _stream(stream)))


def full_attn_decode_kv4_workspace_size(B, Hq, Hkv, max_ctx) -> int:
    return int(lib().full_attn_decode_kv4_workspace_size(int(B), int(Hq), int(Hkv), int(max_ctx)))


def full_attn_decode_kv4(q, pos, seq, pool, table, softmax_scale, max_ctx, workspace=None, out=None, stream=None):
    """full_attn_decode over a 4-bit pool (Kv4Layout).  Rows may share a
    sequence (draft tokens at their own positions)."""
    return _decode_tiles(Kv4Layout, lib().full_attn_decode_kv4, full_attn_decode_kv4_workspace_size, q, pos, seq, pool,
                         table, softmax_scale, max_ctx, workspace, out, stream)


def _decode_tiles(kind, fn, size, q, pos, seq, pool, table, softmax_scale, max_ctx, workspace, out, stream):
    try:
        cur = torch.cuda.current_device()
        B, Hq, D = q.shape
        P, half, two = table.shape
        fine = (D == DQK and half == DROT // 2 and two == 2 and q.dtype is _BF and pos.dtype is _I64 and seq.dtype is _I32
                and table.dtype is _F32 and pos.shape == (B,) and seq.shape == (B,) and q.is_contiguous()
                and pos.is_contiguous() and seq.is_contiguous() and table.is_contiguous() and q.get_device() == cur
                and pos.get_device() == cur and seq.get_device() == cur and table.get_device() == cur
                and pool.data.get_device() == cur and pool.block_table.get_device() == cur)
    except _ODD:
        fine = False
    if not fine:
        _want_q(q)
        _want(pos, "pos", torch.int64, 1)
        _want(seq, "seq", torch.int32, 1)
        _want_table(table)
        B, Hq, _ = q.shape
        P = table.shape[0]
        _want_len(pos, "pos", B)
        _want_len(seq, "seq", B)
    _want_pool(pool, kind)
    given = workspace is not None or out is not None
    if workspace is None:
        n = size(B, Hq, pool.num_kv_heads, max_ctx)
        if n:  # (short contexts need none)
            workspace = _empty(n, torch.uint8, q, stream)
    else:
        _want(workspace, "workspace", torch.uint8, 1)
    out = _out(out, B, Hq, q, stream)
    if not fine:
        _same_device(q, pos, seq, table, workspace, out, *pool.tensors())
    elif given:
        _same_device(q, workspace, out)
    c = pool.c()
    _check(fn(q.data_ptr(), pos.data_ptr(), seq.data_ptr(), B, Hq, ctypes.byref(c), table.data_ptr(), P,
              float(softmax_scale), int(max_ctx), None if workspace is None else workspace.data_ptr(),
              0 if workspace is None else workspace.numel(), out.data_ptr(), _stream(stream)))
    return out


def _want_pool(pool, kind):
    """The quantised layouts' structs look alike to the library, so a pool says by TILE which it is; one of the caller's own
    kind that does not say is a 4-bit one."""
    tile = getattr(pool, "TILE", None)
    if tile is None and not isinstance(pool, (RingLayout, PagedLayout, LinearLayout)):
        tile = KV4_TILE
    if tile != kind.TILE:
        raise TypeError(f"a {kind.__name__} is wanted, got {type(pool).__name__}")


def kv4_unpack(src, src_seqs, lo, cu_rows, dst, dst_seqs=None, T=None, stream=None):
    """Positions lo[i] .. lo[i] + cu_rows[i+1] - cu_rows[i] - 1 of sequence
    src_seqs[i] of a 4-bit pool as bf16: into the same positions of sequence
    dst_seqs[i] of a PagedLayout, or into rows cu_rows[i] .. of a LinearLayout.
    T bounds the rows of the call (cu_rows' last entry); by default it is all
    that dst, or its block table, can name."""
    _unpack_tiles(Kv4Layout, lib().kv4_unpack, src, src_seqs, lo, cu_rows, dst, dst_seqs, T, stream)


def _unpack_tiles(kind, fn, src, src_seqs, lo, cu_rows, dst, dst_seqs, T, stream):
    try:
        cur = torch.cuda.current_device()
        n, = src_seqs.shape
        fine = (dst_seqs is None and src_seqs.dtype is _I32 and lo.dtype is _I64 and cu_rows.dtype is _I32
                and lo.shape == (n,) and cu_rows.shape == (n + 1,) and src_seqs.is_contiguous() and lo.is_contiguous()
                and cu_rows.is_contiguous() and src_seqs.get_device() == cur and lo.get_device() == cur
                and cu_rows.get_device() == cur and src.data.get_device() == cur and src.block_table.get_device() == cur
                and dst.k.get_device() == cur and dst.v.get_device() == cur)
    except _ODD:
        fine = False
    if not fine:
        _want(src_seqs, "src_seqs", torch.int32, 1)
        _want(lo, "lo", torch.int64, 1)
        _want(cu_rows, "cu_rows", torch.int32, 1)
        n = src_seqs.shape[0]
        _want_len(lo, "lo", n)
        _want_len(cu_rows, "cu_rows", n + 1)
    if isinstance(dst, LinearLayout):
        most = dst.num_rows
    elif isinstance(dst, PagedLayout):
        if dst_seqs is None:
            raise ValueError("dst_seqs names the sequences of a PagedLayout")
        most = min(dst.num_seqs * dst.max_blocks * dst.block_size, 2 ** 31 - 1)
    else:
        raise TypeError("dst must be a PagedLayout or a LinearLayout")
    _want_pool(src, kind)
    if not fine:
        if dst_seqs is not None:
            _want(dst_seqs, "dst_seqs", torch.int32, 1)
            _want_len(dst_seqs, "dst_seqs", n)
        _same_device(src_seqs, lo, cu_rows, dst_seqs, *src.tensors(), *dst.tensors())
    T = most if T is None else int(T)
    sc, dc = src.c(), dst.c()
    _check(fn(ctypes.byref(sc), src_seqs.data_ptr(), lo.data_ptr(), cu_rows.data_ptr(), n, T, _ptr(dst_seqs),
              ctypes.byref(dc), _stream(stream)))


def kv8_append_rope(k, v, cu_rows, P0, seqs, table, value_scale, dst, stream=None):
    """KV write into an 8-bit pool (Kv8Layout) of a batch of chunks: rows
    cu_rows[i] .. cu_rows[i+1]-1 of k and v (int32 [n + 1]) go to positions
    P0[i] .. (int64) of sequence seqs[i] (int32; -1 marks padding).  Positions are
    written in order: those ahead of P0[i] in its tile of 16 are there already,
    those behind the chunk in its last tile mean nothing afterwards."""
    _want_pool(dst, Kv8Layout)
    try:
        cur = torch.cuda.current_device()
        T, H, D = k.shape
        n, = seqs.shape
        P, half, two = table.shape
        fine = (D == DQK and half == DROT // 2 and two == 2 and v.shape == (T, H, DV) and cu_rows.shape == (n + 1,)
                and P0.shape == (n,) and k.dtype is _BF and v.dtype is _BF and cu_rows.dtype is _I32 and P0.dtype is _I64
                and seqs.dtype is _I32 and table.dtype is _F32 and k.is_contiguous() and v.is_contiguous()
                and cu_rows.is_contiguous() and P0.is_contiguous() and seqs.is_contiguous() and table.is_contiguous()
                and k.get_device() == cur and v.get_device() == cur and cu_rows.get_device() == cur
                and P0.get_device() == cur and seqs.get_device() == cur and table.get_device() == cur
                and dst.data.get_device() == cur and dst.block_table.get_device() == cur)
    except _ODD:
        fine = False
    if not fine:
        _want(k, "k", torch.bfloat16, 3)
        _want(v, "v", torch.bfloat16, 3)
        _want(cu_rows, "cu_rows", torch.int32, 1)
        _want(P0, "P0", torch.int64, 1)
        _want(seqs, "seqs", torch.int32, 1)
        _want_table(table)
        T, H = k.shape[:2]
        n, P = seqs.shape[0], table.shape[0]
        if k.shape[2] != DQK or v.shape != (T, H, DV):
            raise ValueError("k/v shapes disagree")
        _want_len(cu_rows, "cu_rows", n + 1)
        _want_len(P0, "P0", n)
        _same_device(k, v, cu_rows, P0, seqs, table, *dst.tensors())
    c = dst.c()
    _check(lib().kv8_append_rope(k.data_ptr(), v.data_ptr(), cu_rows.data_ptr(), P0.data_ptr(), seqs.data_ptr(), n, T, H,
                                 table.data_ptr(), P, float(value_scale), ctypes.byref(c), _stream(stream)))


def full_attn_decode_kv8_workspace_size(B, Hq, Hkv, max_ctx) -> int:
    return int(lib().full_attn_decode_kv8_workspace_size(int(B), int(Hq), int(Hkv), int(max_ctx)))


def full_attn_decode_kv8(q, pos, seq, pool, table, softmax_scale, max_ctx, workspace=None, out=None, stream=None):
    """full_attn_decode over an 8-bit pool (Kv8Layout).  Rows may share a
    sequence (draft tokens at their own positions)."""
    return _decode_tiles(Kv8Layout, lib().full_attn_decode_kv8, full_attn_decode_kv8_workspace_size, q, pos, seq, pool,
                         table, softmax_scale, max_ctx, workspace, out, stream)


def kv8_unpack(src, src_seqs, lo, cu_rows, dst, dst_seqs=None, T=None, stream=None):
    """kv4_unpack from an 8-bit pool (Kv8Layout)."""
    _unpack_tiles(Kv8Layout, lib().kv8_unpack, src, src_seqs, lo, cu_rows, dst, dst_seqs, T, stream)


def _fine_ints(cur, *tensors):
    """Whether all are contiguous int32 vectors on device cur."""
    for t in tensors:
        if t.dtype is not _I32 or t.dim() != 1 or not t.is_contiguous() or t.get_device() != cur:
            return False
    return True


def _fine_pages(cur, block_table, num_blocks, refs, free_ids, free_count):
    return (block_table.dtype is _I32 and block_table.dim() == 2 and block_table.is_contiguous()
            and block_table.get_device() == cur and refs.numel() == num_blocks and free_count.numel() == 1
            and _fine_ints(cur, refs, free_ids, free_count))


def _want_free_list(free_ids, free_count, refs, num_blocks):
    _want(free_ids, "free_ids", torch.int32, 1)
    _want(free_count, "free_count", torch.int32, 1)
    _want_len(free_count, "free_count", 1)
    _want(refs, "refs", torch.int32, 1)
    _want_len(refs, "refs", int(num_blocks))


def _want_pairs(copy_src, copy_dst, copy_count, least):
    _want(copy_src, "copy_src", torch.int32, 1)
    _want(copy_dst, "copy_dst", torch.int32, 1)
    _want(copy_count, "copy_count", torch.int32, 1)
    _want_len(copy_count, "copy_count", 1)
    if copy_src.shape[0] < least or copy_dst.shape[0] < least:
        raise ValueError(f"copy_src and copy_dst must have {least} entries, got {copy_src.shape[0]} and {copy_dst.shape[0]}")


def kv_pages_free(block_table, num_blocks, block_size, refs, seqs, free_ids, free_count, keep_lo=None, keep_hi=None,
                  stream=None):
    """Sequences seqs[i] (int32 [n]) give up their blocks -- all of them, or with
    keep_hi (and keep_lo, default 0; int64 [n]) those without a position of
    [keep_lo[i], keep_hi[i]): the entries of block_table (int32 [num_seqs,
    max_blocks]) become -1, refs (int32 [num_blocks], the holders of a block
    beyond the first) goes down, and the blocks that nobody holds are added to the
    free list (free_ids int32 [cap], free_count int32 [1]) in ascending order."""
    try:
        cur = torch.cuda.current_device()
        fine = (keep_lo is None and keep_hi is None
                and _fine_pages(cur, block_table, num_blocks, refs, free_ids, free_count) and _fine_ints(cur, seqs))
    except _ODD:
        fine = False
    if not fine:
        _want(block_table, "block_table", torch.int32, 2)
        _want(seqs, "seqs", torch.int32, 1)
        _want_free_list(free_ids, free_count, refs, num_blocks)
        for t, name in ((keep_lo, "keep_lo"), (keep_hi, "keep_hi")):
            if t is not None:
                _want(t, name, torch.int64, 1)
                _want_len(t, name, seqs.shape[0])
        _same_device(block_table, refs, seqs, free_ids, free_count, keep_lo, keep_hi)
    S, mb = block_table.shape
    _check(lib().kv_pages_free(block_table.data_ptr(), S, mb, int(block_size), int(num_blocks), refs.data_ptr(),
                               seqs.data_ptr(), _ptr(keep_lo), _ptr(keep_hi), seqs.shape[0], free_ids.data_ptr(),
                               free_count.data_ptr(), free_ids.shape[0], _stream(stream)))


def kv_pages_fork(block_table, num_blocks, block_size, refs, src_seqs, dst_seqs, lens, free_ids, free_count, copy_src,
                  copy_dst, copy_count, free_count_out=None, stream=None):
    """Sequence dst_seqs[i] (int32 [n]) receives the first lens[i] (int64)
    positions of src_seqs[i]: whole blocks are shared (refs goes up), a last block
    that is filled in part gets a new one from the end of the free list, and the
    copies to be made (kv_pages_copy) are copy_src[k] -> copy_dst[k] (int32, n
    entries), copy_count (int32 [1]) of them.  The remaining count goes to
    free_count_out (default: free_count itself).  Everything stays on the
    device."""
    if free_count_out is None:
        free_count_out = free_count
    try:
        cur = torch.cuda.current_device()
        n, = src_seqs.shape
        fine = (_fine_pages(cur, block_table, num_blocks, refs, free_ids, free_count) and lens.dtype is _I64
                and lens.shape == (n,) and lens.is_contiguous() and lens.get_device() == cur and dst_seqs.numel() == n
                and free_count_out.numel() == 1 and copy_count.numel() == 1 and copy_src.numel() >= n
                and copy_dst.numel() >= n
                and _fine_ints(cur, src_seqs, dst_seqs, free_count_out, copy_src, copy_dst, copy_count))
    except _ODD:
        fine = False
    if not fine:
        _want(block_table, "block_table", torch.int32, 2)
        _want(src_seqs, "src_seqs", torch.int32, 1)
        _want(dst_seqs, "dst_seqs", torch.int32, 1)
        _want(lens, "lens", torch.int64, 1)
        _want_free_list(free_ids, free_count, refs, num_blocks)
        _want(free_count_out, "free_count_out", torch.int32, 1)
        _want_len(free_count_out, "free_count_out", 1)
        n = src_seqs.shape[0]
        _want_len(dst_seqs, "dst_seqs", n)
        _want_len(lens, "lens", n)
        _want_pairs(copy_src, copy_dst, copy_count, n)
        _same_device(block_table, refs, src_seqs, dst_seqs, lens, free_ids, free_count, free_count_out, copy_src,
                     copy_dst, copy_count)
    S, mb = block_table.shape
    _check(lib().kv_pages_fork(block_table.data_ptr(), S, mb, int(block_size), int(num_blocks), refs.data_ptr(),
                               src_seqs.data_ptr(), dst_seqs.data_ptr(), lens.data_ptr(), n, free_ids.data_ptr(),
                               free_count.data_ptr(), free_count_out.data_ptr(), free_ids.shape[0], copy_src.data_ptr(),
                               copy_dst.data_ptr(), copy_count.data_ptr(), _stream(stream)))


def kv_pages_compact(block_table, num_blocks, refs, free_ids, free_count, copy_src, copy_dst, copy_count, limit=0,
                     table_out=None, refs_out=None, free_ids_out=None, stream=None):
    """The pool's used blocks move below `limit` (0: as low as they fit): the
    copies to be made (kv_pages_copy) are copy_src[k] -> copy_dst[k] (int32,
    num_blocks // 2 entries), copy_count (int32 [1]) of them; block_table, refs
    and the free list (then in descending order) name the new places, in
    table_out, refs_out and free_ids_out (default: the arrays themselves).
    Everything stays on the device."""
    table_out = block_table if table_out is None else table_out
    refs_out = refs if refs_out is None else refs_out
    free_ids_out = free_ids if free_ids_out is None else free_ids_out
    try:
        cur = torch.cuda.current_device()
        fine = (_fine_pages(cur, block_table, num_blocks, refs, free_ids, free_count) and table_out.dtype is _I32
                and table_out.shape == block_table.shape and table_out.is_contiguous() and table_out.get_device() == cur
                and refs_out.shape == refs.shape and free_ids_out.shape == free_ids.shape and copy_count.numel() == 1
                and copy_src.numel() >= num_blocks // 2 and copy_dst.numel() >= num_blocks // 2
                and _fine_ints(cur, refs_out, free_ids_out, copy_src, copy_dst, copy_count))
    except _ODD:
        fine = False
    if not fine:
        _want(block_table, "block_table", torch.int32, 2)
        _want_free_list(free_ids, free_count, refs, num_blocks)
        _want_pairs(copy_src, copy_dst, copy_count, int(num_blocks) // 2)
        for t, src, name in ((table_out, block_table, "table_out"), (refs_out, refs, "refs_out"),
                             (free_ids_out, free_ids, "free_ids_out")):
            _want(t, name, torch.int32, src.dim())
            if t.shape != src.shape:
                raise ValueError(f"{name} must have the shape {tuple(src.shape)}, got {tuple(t.shape)}")
        _same_device(block_table, refs, free_ids, free_count, copy_src, copy_dst, copy_count, table_out, refs_out,
                     free_ids_out)
    S, mb = block_table.shape
    _check(lib().kv_pages_compact(block_table.data_ptr(), table_out.data_ptr(), S, mb, int(num_blocks), int(limit),
                                  refs.data_ptr(), refs_out.data_ptr(), free_ids.data_ptr(), free_count.data_ptr(),
                                  free_ids_out.data_ptr(), free_ids.shape[0], copy_src.data_ptr(), copy_dst.data_ptr(),
                                  copy_count.data_ptr(), _stream(stream)))


def kv_pages_copy(pools, copy_src, copy_dst, copy_count, stream=None):
    """Copy block copy_src[k] to copy_dst[k], k < copy_count, in every pool of
    `pools` (one PagedLayout, Kv4Layout or Kv8Layout, or a list of them: the
    layers that share a block table), in one launch."""
    if isinstance(pools, (PagedLayout, _TileLayout)):
        pools = [pools]
    planes = []
    for p in pools:
        if isinstance(p, PagedLayout):
            planes += [p.k, p.v]
        elif isinstance(p, _TileLayout):
            planes.append(p.data)
        else:
            raise TypeError(f"pools must be PagedLayout, Kv4Layout or Kv8Layout, got {type(p).__name__}")
    if not planes:
        return
    nb = planes[0].shape[0]
    for t in planes:
        if t.shape[0] != nb:
            raise ValueError(f"the pools have {nb} and {t.shape[0]} blocks: they do not share a block table")
    try:
        cur = torch.cuda.current_device()
        fine = copy_count.numel() == 1 and _fine_ints(cur, copy_src, copy_dst, copy_count)
    except _ODD:
        fine = False
    if not fine:
        _want_pairs(copy_src, copy_dst, copy_count, 0)
    _same_device(copy_src, copy_dst, copy_count, *planes)
    n = len(planes)
    ptrs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in planes])
    sizes = (ctypes.c_int64 * n)(*[t.numel() // max(nb, 1) * t.element_size() for t in planes])
    _check(lib().kv_pages_copy(ptrs, sizes, n, nb, copy_src.data_ptr(), copy_dst.data_ptr(), copy_count.data_ptr(),
                               min(copy_src.shape[0], copy_dst.shape[0]), _stream(stream)))


def debug_stall_next(launches: int, limit_ns: int) -> None:
    """Test hook: the next `launches` windowed decodes (ring layout), 4-bit and
    8-bit decodes or single-chunk full-attention prefills stall on purpose and leave
    by their bounded-wait exit after limit_ns, setting DEV_TIMEOUT (kvr_debug_stall_next)."""
    _check(lib().kvr_debug_stall_next(int(launches), int(limit_ns)))


def device_status(reset: bool = True) -> int:
    """Device status bits (DEV_BAD_POS | DEV_BAD_SEQ | DEV_BAD_BLOCK); synchronises."""
    flags = ctypes.c_uint32(0)
    _check(lib().kvr_device_status(ctypes.byref(flags), 1 if reset else 0))
    return int(flags.value)
