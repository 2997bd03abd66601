"""Thin Python binding of libhs2 (argument marshalling only).

Functions carry the C names (``hs2_fa_select``, ``hs2_sa_reuse``,
``hs2_hier_reindex``, the ``*_workspace`` queries) and take torch CUDA tensors;
every step of the path runs in the library's kernels. PyTorch only provides
device memory and the current stream. There is no fallback: if the library
cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import operator
import os
from dataclasses import dataclass

import torch

from . import build as _build

ABI_VERSION = 6  # include/hs2.h HS2_ABI_VERSION this binding marshals for
F32, BF16, FP8_E4M3, FP4_E2M1 = 0, 1, 2, 3
FULL, REINDEX = 0, 1
DEV_BAD_PAGE, DEV_BAD_INDEX, DEV_TIMEOUT, DEV_BAD_LENGTH, DEV_SELECT = 1, 2, 4, 8, 16
EXPORTS = (
    "hs2_fa_select_workspace", "hs2_fa_select", "hs2_fa_select_ex", "hs2_sa_reuse_workspace", "hs2_sa_reuse", "hs2_sa_reuse_ex",
    "hs2_hier_reindex_workspace", "hs2_hier_reindex", "hs2_strerror", "hs2_last_cuda_error",
    "hs2_abi_version", "hs2_profile_next", "hs2_selftest_wait_timeout", "hs2_fa_select_noalloc", "hs2_fa_select_noalloc_capacity",
    "hs2_kv_append", "hs2_fa_select_append", "hs2_fa_select_launches", "hs2_sa_reuse_launches",
    "hs2_kv_write", "hs2_kv_read", "hs2_fa_chunk_workspace", "hs2_fa_chunk", "hs2_pages_grow", "hs2_pages_free",
    "hs2_pages_fork", "hs2_pages_compact_workspace", "hs2_pages_compact",
)
STAGE_FA_SCAN, STAGE_SA_GATHER, STAGE_INDEXER = 0, 1, 2
SA_OVERLAP = 1  # HS2_SA_OVERLAP


class hs2_kv(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
        ("seq_len", ctypes.c_void_p), ("batch", ctypes.c_int32), ("num_pages", ctypes.c_int32),
        ("max_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("Hkv", ctypes.c_int32),
        ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("k_sf", ctypes.c_void_p), ("v_sf", ctypes.c_void_p),
    ]


class hs2_pages(ctypes.Structure):
    _fields_ = [("ref", ctypes.c_void_p), ("free_list", ctypes.c_void_p), ("n_free", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32)]


class HS2Error(RuntimeError):
    pass


_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libhs2.so (built in-tree by ``build.build()``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or _build.LIB
    if not os.path.exists(path):
        raise HS2Error(f"libhs2 not built ({path}); run top_hs2_fa_gb300.build.build()")
    lib = ctypes.CDLL(path)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    kvp = ctypes.POINTER(hs2_kv)
    lib.hs2_fa_select_workspace.argtypes = [i32, i32, kvp, i32, i32, i32]
    lib.hs2_fa_select_workspace.restype = sz
    lib.hs2_fa_select.argtypes = [vp, i32, i32, kvp, i32, i32, i32, f32, i32, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.hs2_fa_select.restype = i32
    lib.hs2_fa_select_ex.argtypes = [vp, i32, i32, kvp, i32, i32, i32, f32, i32, i32, vp, vp, vp, vp, vp, sz, vp,
                                     vp]
    lib.hs2_fa_select_ex.restype = i32
    lib.hs2_sa_reuse_workspace.argtypes = [i32, i32, kvp, i32, i32, i32]
    lib.hs2_sa_reuse_workspace.restype = sz
    lib.hs2_sa_reuse.argtypes = [vp, i32, i32, kvp, i32, vp, vp, i32, f32, i32, vp, vp, sz, vp, vp]
    lib.hs2_sa_reuse.restype = i32
    lib.hs2_sa_reuse_ex.argtypes = [vp, i32, i32, kvp, i32, vp, vp, i32, f32, i32, vp, vp, i32, vp, vp, sz, vp, vp]
    lib.hs2_sa_reuse_ex.restype = i32
    lib.hs2_hier_reindex_workspace.argtypes = [i32, i32, kvp, i32, i32, i32, i32]
    lib.hs2_hier_reindex_workspace.restype = sz
    lib.hs2_hier_reindex.argtypes = [i32, vp, vp, i32, kvp, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.hs2_hier_reindex.restype = i32
    lib.hs2_selftest_wait_timeout.argtypes = [i32, vp, vp]
    lib.hs2_selftest_wait_timeout.restype = i32
    lib.hs2_strerror.argtypes = [i32]
    lib.hs2_strerror.restype = ctypes.c_char_p
    lib.hs2_last_cuda_error.restype = i32
    lib.hs2_abi_version.restype = i32
    lib.hs2_profile_next.argtypes = [i32, vp, vp]
    lib.hs2_profile_next.restype = None
    lib.hs2_fa_select_noalloc.argtypes = [vp, i32, i32, kvp, i32, i32, i32, f32, i32, vp, vp, vp, vp, vp, vp]
    lib.hs2_fa_select_noalloc.restype = i32
    lib.hs2_kv_append.argtypes = [i32, kvp, ctypes.POINTER(vp), ctypes.POINTER(vp), vp, vp]
    lib.hs2_kv_append.restype = i32
    lib.hs2_fa_select_append.argtypes = [vp, i32, i32, kvp, i32, i32, i32, f32, i32, vp, vp, vp, vp, vp, vp, vp, sz,
                                         vp, vp]
    lib.hs2_fa_select_append.restype = i32
    lib.hs2_fa_select_noalloc_capacity.argtypes = []
    lib.hs2_fa_select_noalloc_capacity.restype = sz
    lib.hs2_fa_select_launches.argtypes = [i32, i32, kvp, i32, i32, i32, i32, i32, i32]
    lib.hs2_fa_select_launches.restype = i32
    lib.hs2_sa_reuse_launches.argtypes = [i32, i32, kvp, i32, i32, i32]
    lib.hs2_sa_reuse_launches.restype = i32
    i64, pgp = ctypes.c_int64, ctypes.POINTER(hs2_pages)
    lib.hs2_kv_write.argtypes = [kvp, vp, vp, i32, i64, vp, i32, vp, vp]
    lib.hs2_kv_write.restype = i32
    lib.hs2_kv_read.argtypes = [kvp, vp, vp, i32, i64, vp, i32, vp, vp]
    lib.hs2_kv_read.restype = i32
    lib.hs2_fa_chunk_workspace.argtypes = [i32, i32, kvp, i32, i32, i32]
    lib.hs2_fa_chunk_workspace.restype = sz
    lib.hs2_fa_chunk.argtypes = [vp, vp, i32, i32, i32, kvp, i32, i32, f32, vp, vp, i32, vp, vp, sz, vp, vp]
    lib.hs2_fa_chunk.restype = i32
    lib.hs2_pages_grow.argtypes = [pgp, vp, vp, vp, i32, i32, vp, vp]
    lib.hs2_pages_grow.restype = i32
    lib.hs2_pages_free.argtypes = [pgp, vp, vp, vp, i32, i32, vp, vp]
    lib.hs2_pages_free.restype = i32
    lib.hs2_pages_fork.argtypes = [pgp, i32, kvp, vp, i32, vp, vp, vp, vp]
    lib.hs2_pages_fork.restype = i32
    lib.hs2_pages_compact_workspace.argtypes = [pgp]
    lib.hs2_pages_compact_workspace.restype = sz
    lib.hs2_pages_compact.argtypes = [pgp, i32, kvp, vp, sz, vp, vp]
    lib.hs2_pages_compact.restype = i32
    if lib.hs2_abi_version() != ABI_VERSION:
        raise HS2Error(f"libhs2 ABI {lib.hs2_abi_version()} != binding ABI {ABI_VERSION}: rebuild the library")
    _lib = lib
    return lib


def _check(st: int) -> None:
    if st != 0:
        lib = load()
        msg = lib.hs2_strerror(st).decode()
        if st == -3:
            msg += f" (cudaError {lib.hs2_last_cuda_error()})"
        raise HS2Error(f"hs2 status {st}: {msg}")


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


_data_ptr, _size, _contiguous = torch.Tensor.data_ptr, torch.Tensor.size, torch.Tensor.is_contiguous
_dtype = operator.attrgetter("dtype")


class _Handle:
    """Base of the handles whose C struct is kept between calls: setting an attribute drops it,
    and a tensor whose storage, shape, type or strides have changed makes a new one (or an error)."""

    # (struct, device, tensors it was made from, their pointers, the first three's shapes and types)
    _c = None

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_c":
            object.__setattr__(self, "_c", None)

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_c"}

    def _cached(self):
        got = self._c
        if (got is None or got[3] != tuple(map(_data_ptr, got[2])) or got[4] != tuple(map(_size, got[2][:3]))
                or got[5] != tuple(map(_dtype, got[2][:3])) or not all(map(_contiguous, got[2]))):
            ts = self._tensors()
            got = (self._make(), _device_of(ts), ts, tuple(map(_data_ptr, ts)), tuple(map(_size, ts[:3])),
                   tuple(map(_dtype, ts[:3])))
            object.__setattr__(self, "_c", got)
        return got


@dataclass
class KV(_Handle):
    """Device tensors of one group's paged KV cache."""

    k: torch.Tensor  # [num_pages][Hkv][64][d], float32, bfloat16 or uint8 (FP8 E4M3 codes);
    v: torch.Tensor | None  # FP4: uint8 [num_pages][Hkv][64][d/2], two E2M1 codes per byte
    block_table: torch.Tensor  # int32 [B][max_pages]
    seq_len: torch.Tensor  # int32 [B]
    k_scale: torch.Tensor | None = None  # FP8 / FP4: float32 [num_pages][Hkv]
    v_scale: torch.Tensor | None = None
    k_sf: torch.Tensor | None = None  # FP4: uint8 E4M3 [num_pages][Hkv][64][d/16]
    v_sf: torch.Tensor | None = None

    def _tensors(self):
        return tuple(t for t in (self.k, self.block_table, self.seq_len, self.v, self.k_scale, self.v_scale,
                                 self.k_sf, self.v_sf) if t is not None)

    def _make(self) -> hs2_kv:
        return self.c()

    def c(self) -> hs2_kv:
        d = int(self.k.shape[3])
        if self.k.dtype == torch.uint8 and self.k_sf is not None:
            dt, d = FP4_E2M1, 2 * d
            if self.k_scale is None or (self.v is not None and (self.v_scale is None or self.v_sf is None)):
                raise HS2Error("an FP4 KV cache needs k_scale, v_scale, k_sf and v_sf")
        elif self.k.dtype == torch.uint8:
            dt = FP8_E4M3
            if self.k_scale is None or (self.v is not None and self.v_scale is None):
                raise HS2Error("an FP8 KV cache needs k_scale and v_scale")
        elif self.k.dtype in (torch.bfloat16, torch.float32):
            dt = BF16 if self.k.dtype == torch.bfloat16 else F32
        else:
            raise HS2Error(f"unsupported KV dtype {self.k.dtype}")
        for t in (self.k, self.v, self.block_table, self.seq_len, self.k_scale, self.v_scale, self.k_sf, self.v_sf):
            if t is not None and not t.is_contiguous():
                raise HS2Error("KV tensors must be contiguous")
        return hs2_kv(_ptr(self.k), _ptr(self.v), _ptr(self.block_table), _ptr(self.seq_len),
                      int(self.seq_len.shape[0]), int(self.k.shape[0]), int(self.block_table.shape[1]),
                      int(self.k.shape[2]), int(self.k.shape[1]), d, dt,
                      _ptr(self.k_scale), _ptr(self.v_scale), _ptr(self.k_sf), _ptr(self.v_sf))


def _workspace(nbytes: int, device, ws):
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise HS2Error("workspace too small")
        return ws
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def hs2_fa_select_workspace(B_or_n: int, Hq: int, kv: KV, max_t: int, k: int, prefill: bool = False) -> int:
    c = kv.c()
    return int(load().hs2_fa_select_workspace(B_or_n, Hq, ctypes.byref(c), max_t, k, int(prefill)))


def hs2_fa_select_launches(B_or_n: int, Hq: int, kv: KV, max_t: int, w: int, k: int, prefill: bool = False,
                           sel_block: int = 1, append: bool = False) -> int:
    """Kernels one hs2_fa_select call with these arguments launches (-1: rejected)."""
    c = kv.c()
    return int(load().hs2_fa_select_launches(B_or_n, Hq, ctypes.byref(c), max_t, w, k, int(prefill), sel_block,
                                              int(append)))


def hs2_sa_reuse_launches(B_or_n: int, Hq: int, kv: KV, w: int, k: int, prefill: bool = False) -> int:
    """Kernels one hs2_sa_reuse call with these arguments launches (-1: rejected)."""
    c = kv.c()
    return int(load().hs2_sa_reuse_launches(B_or_n, Hq, ctypes.byref(c), w, k, int(prefill)))


def hs2_kv_append(kvs, k_new, v_new=None, dev_err=None, stream=None) -> None:
    """Decode KV append for several caches in one launch: row t-1 (t = seq_len[b]) of
    every sequence of cache c takes k_new[c][b] / v_new[c][b] ([batch][Hkv][d], the cache's
    dtype). ``kvs``: list of KV (bf16 or f32 pools, written in place)."""
    lib = load()
    n = len(kvs)
    if n != len(k_new) or (v_new is not None and n != len(v_new)):
        raise HS2Error("one k_new (and v_new) tensor per cache")
    for kv, kn, vn in zip(kvs, k_new, v_new if v_new is not None else [None] * n):
        for x in (kn, vn):
            if x is not None and (not x.is_contiguous() or x.dtype != kv.k.dtype):
                raise HS2Error("new rows must be contiguous and of the cache's dtype")
    cs = (hs2_kv * n)(*[kv.c() for kv in kvs])
    kp = (ctypes.c_void_p * n)(*[_ptr(x) for x in k_new])
    vpa = (ctypes.c_void_p * n)(*[_ptr(x) for x in v_new]) if v_new is not None else None
    _check(lib.hs2_kv_append(n, cs, kp, vpa, _ptr(dev_err), _stream(stream)))


def hs2_fa_select(q: torch.Tensor, kv: KV, w: int, k: int, scale: float, prefill: bool = False,
                  max_t: int | None = None, out=None, workspace=None, dev_err=None, stream=None,
                  sel_block: int = 1, k_new: torch.Tensor | None = None, v_new: torch.Tensor | None = None):
    """FA layer + window-excluding top-k. Returns (o, lse, idx, idx_cnt) (float32, float32,
    int32, int32). ``max_t`` defaults to the table's capacity (decode) or n (prefill).
    ``sel_block`` > 1 selects whole blocks of that many far positions (``hs2_fa_select_ex``).
    ``k_new`` / ``v_new`` ([B][Hkv][d], decode): the current token's rows, appended to the
    cache at position t-1 by the same call (``hs2_fa_select_append``).
    ``dev_err`` (int32 device tensor) collects the device-side error bits (``DEV_*``). Every
    row gets its exact top-k: a prefill row whose streamed candidates cannot prove it is
    recomputed over its whole far range in the same call."""
    lib = load()
    Bq, Hq, d = q.shape
    c = kv.c()
    Hkv = c.Hkv
    if max_t is None:
        max_t = Bq if prefill else c.max_pages * c.page_size
    dev = q.device
    if out is None:
        o = torch.empty((Bq, Hq, d), dtype=torch.float32, device=dev)
        lse = torch.empty((Bq, Hq), dtype=torch.float32, device=dev)
        idx = torch.empty((Bq, Hkv, k), dtype=torch.int32, device=dev)
        cnt = torch.empty((Bq, Hkv), dtype=torch.int32, device=dev)
    else:
        o, lse, idx, cnt = out
    nb = int(lib.hs2_fa_select_workspace(Bq, Hq, ctypes.byref(c), max_t, k, int(prefill)))
    ws = _workspace(nb, dev, workspace)
    if k_new is not None:
        if prefill:
            raise HS2Error("the fused append is decode only")
        for x in (k_new, v_new):
            if x is None or not x.is_contiguous() or x.dtype != kv.k.dtype:
                raise HS2Error("k_new and v_new must be contiguous and of the cache's dtype")
        st = lib.hs2_fa_select_append(_ptr(q), Bq, Hq, ctypes.byref(c), max_t, w, k, float(scale), int(sel_block),
                                      _ptr(k_new), _ptr(v_new), _ptr(o), _ptr(lse), _ptr(idx), _ptr(cnt), _ptr(ws),
                                      ws.numel() * ws.element_size(), _ptr(dev_err), _stream(stream))
    elif sel_block == 1:
        st = lib.hs2_fa_select(_ptr(q), Bq, Hq, ctypes.byref(c), max_t, w, k, float(scale), int(prefill),
                               _ptr(o), _ptr(lse), _ptr(idx), _ptr(cnt), _ptr(ws), ws.numel() * ws.element_size(),
                               _ptr(dev_err), _stream(stream))
    else:
        st = lib.hs2_fa_select_ex(_ptr(q), Bq, Hq, ctypes.byref(c), max_t, w, k, float(scale), int(prefill),
                                  int(sel_block), _ptr(o), _ptr(lse), _ptr(idx), _ptr(cnt), _ptr(ws),
                                  ws.numel() * ws.element_size(), _ptr(dev_err), _stream(stream))
    _check(st)
    return o, lse, idx, cnt


def hs2_sa_reuse_workspace(B_or_n: int, Hq: int, kv: KV, w: int, k: int, prefill: bool = False) -> int:
    c = kv.c()
    return int(load().hs2_sa_reuse_workspace(B_or_n, Hq, ctypes.byref(c), w, k, int(prefill)))


def hs2_sa_reuse(q: torch.Tensor, kv: KV, w: int, idx: torch.Tensor, idx_cnt: torch.Tensor, k: int,
                 scale: float, prefill: bool = False, out=None, workspace=None, dev_err=None, stream=None,
                 sink: torch.Tensor | None = None, gate: torch.Tensor | None = None, overlap: bool = False):
    """SA layer reusing the FA's KV and indices with its own query. Returns o (float32).

    ``sink`` (float32 [Hq]) and ``gate`` (float32 [Bq][Hq][d]) are the optional per-head sink
    logits and output gate logits. ``overlap`` (``HS2_SA_OVERLAP``, the SA layers of a group
    after the first): idx, idx_cnt, the block table and the lengths were complete before the
    previous launch on the stream began, and ``workspace`` is the one the previous SA call on
    this stream used with the same sizes, so the decode kernel is one launch that may read
    them while that launch finishes. Without these three this is ``hs2_sa_reuse``, else
    ``hs2_sa_reuse_ex``."""
    lib = load()
    Bq, Hq, d = q.shape
    c = kv.c()
    o = out if out is not None else torch.empty((Bq, Hq, d), dtype=torch.float32, device=q.device)
    nb = int(lib.hs2_sa_reuse_workspace(Bq, Hq, ctypes.byref(c), w, k, int(prefill)))
    if overlap and workspace is None:
        raise HS2Error("overlap continues the previous SA call's workspace: pass it")
    ws = _workspace(nb, q.device, workspace)
    if sink is not None:
        assert sink.dtype == torch.float32 and sink.is_contiguous() and sink.numel() == Hq
    if gate is not None:
        assert gate.dtype == torch.float32 and gate.is_contiguous() and tuple(gate.shape) == (Bq, Hq, d)
    if sink is None and gate is None and not overlap:
        st = lib.hs2_sa_reuse(_ptr(q), Bq, Hq, ctypes.byref(c), w, _ptr(idx), _ptr(idx_cnt), k, float(scale),
                              int(prefill), _ptr(o), _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_err),
                              _stream(stream))
    else:
        st = lib.hs2_sa_reuse_ex(_ptr(q), Bq, Hq, ctypes.byref(c), w, _ptr(idx), _ptr(idx_cnt), k, float(scale),
                                 int(prefill), _ptr(sink), _ptr(gate), SA_OVERLAP if overlap else 0, _ptr(o),
                                 _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_err), _stream(stream))
    _check(st)
    return o


def hs2_hier_reindex_workspace(mode: int, Hi: int, k_idx: KV, max_t: int, k_top: int, blk: int,
                               max_blocks: int) -> int:
    c = k_idx.c()
    return int(load().hs2_hier_reindex_workspace(mode, Hi, ctypes.byref(c), max_t, k_top, blk, max_blocks))


def hs2_hier_reindex(mode: int, q_idx: torch.Tensor, w_idx: torch.Tensor, k_idx: KV, k_top: int, blk: int,
                     max_blocks: int, pool_blocks=None, pool_cnt=None, max_t: int | None = None, out=None,
                     workspace=None, dev_err=None, stream=None):
    """CSA2 hierarchical indexer (Full or Reindex). Returns (idx, idx_cnt, pool_blocks, pool_cnt)."""
    lib = load()
    B, Hi, di = q_idx.shape
    c = k_idx.c()
    dev = q_idx.device
    if max_t is None:
        max_t = c.max_pages * c.page_size
    if pool_blocks is None:
        pool_blocks = torch.empty((B, max_blocks), dtype=torch.int32, device=dev)
        pool_cnt = torch.empty((B,), dtype=torch.int32, device=dev)
    if out is None:
        idx = torch.empty((B, k_top), dtype=torch.int32, device=dev)
        cnt = torch.empty((B,), dtype=torch.int32, device=dev)
    else:
        idx, cnt = out
    nb = int(lib.hs2_hier_reindex_workspace(mode, Hi, ctypes.byref(c), max_t, k_top, blk, max_blocks))
    ws = _workspace(nb, dev, workspace)
    st = lib.hs2_hier_reindex(mode, _ptr(q_idx), _ptr(w_idx), Hi, ctypes.byref(c), max_t, k_top, blk,
                              max_blocks, _ptr(pool_blocks), _ptr(pool_cnt), _ptr(idx), _ptr(cnt), _ptr(ws),
                              ws.numel() * ws.element_size(), _ptr(dev_err), _stream(stream))
    _check(st)
    return idx, cnt, pool_blocks, pool_cnt


def hs2_profile_next(stage: int, start, stop) -> None:
    """Have the next call running ``stage`` record torch.cuda.Event ``start``/``stop`` around
    its main kernel (events must already have been recorded once so that they exist)."""
    load().hs2_profile_next(stage, start.cuda_event if start is not None else None,
                            stop.cuda_event if stop is not None else None)


def hs2_fa_select_noalloc(q: torch.Tensor, kv: KV, w: int, k: int, scale: float, prefill: bool = False,
                          max_t: int | None = None, out=None, dev_err=None, stream=None):
    """hs2_fa_select without a workspace, for callers that cannot allocate device memory:
    the library's own static scratch (hs2_fa_select_noalloc_capacity() bytes) is used.
    Only the outputs are allocated here when ``out`` is None; pass ``out`` to allocate
    nothing. Concurrent calls on the GPU race on the shared scratch."""
    lib = load()
    Bq, Hq, d = q.shape
    c = kv.c()
    if max_t is None:
        max_t = Bq if prefill else c.max_pages * c.page_size
    if out is None:
        dev = q.device
        out = (torch.empty((Bq, Hq, d), dtype=torch.float32, device=dev),
               torch.empty((Bq, Hq), dtype=torch.float32, device=dev),
               torch.empty((Bq, c.Hkv, k), dtype=torch.int32, device=dev),
               torch.empty((Bq, c.Hkv), dtype=torch.int32, device=dev))
    o, lse, idx, cnt = out
    st = lib.hs2_fa_select_noalloc(_ptr(q), Bq, Hq, ctypes.byref(c), max_t, w, k, float(scale), int(prefill),
                                   _ptr(o), _ptr(lse), _ptr(idx), _ptr(cnt), _ptr(dev_err), _stream(stream))
    _check(st)
    return o, lse, idx, cnt


def hs2_selftest_wait_timeout(timeout_us: int, dev_err: torch.Tensor, stream=None) -> None:
    """One warp waits (bounded, timeout_us) on an mbarrier nothing arrives on: the wait must
    give up and set DEV_TIMEOUT in dev_err."""
    _check(load().hs2_selftest_wait_timeout(int(timeout_us), _ptr(dev_err), _stream(stream)))


# ---------------------------------------------------------------------------- paged-cache operators
_ROW_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


def _i32(t: torch.Tensor, name: str, *shape) -> None:
    """t is an int32 contiguous tensor of that shape, or an error."""
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous():
        raise HS2Error(f"{name} must be a contiguous int32 tensor of shape {list(shape)}")


def _table(t: torch.Tensor, name: str):
    """(rows, columns) of an int32 contiguous table, or an error."""
    if t.dtype is not torch.int32 or t.dim() != 2 or not t.is_contiguous():
        raise HS2Error(f"{name} must be a contiguous int32 matrix")
    return t.shape


def _device_of(tensors) -> int:
    """The one device of the tensors (None: left out), or an error."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise HS2Error("tensors on several devices")
    return dev


def _launch_stream(stream, dev: int, *tensors) -> int:
    """The stream to launch on, once every tensor is on device `dev` and that is the current
    device (and the stream's)."""
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise HS2Error("tensors on several devices")
    if dev < 0 or dev != torch._C._cuda_getDevice() or (stream is not None and stream.device.index != dev):
        raise HS2Error("the tensors must be on the current CUDA device (and the stream's)")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _new(shape, dtype, device, stream) -> torch.Tensor:
    """A tensor that a call on `stream` may write: memory of that stream's own, which what is
    still running on the current stream does not use, kept until the current stream is done
    with it too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def _scratch(nbytes: int, device, stream) -> torch.Tensor:
    """A workspace of this call's own."""
    return _new(max(nbytes, 256), torch.uint8, device, stream)


def _token_stride(shape, stride, n: int, c: hs2_kv) -> int:
    """Elements from one token of rows to the next, or an error."""
    if shape != (n, c.Hkv, c.d) or stride[2] != 1 or (c.Hkv > 1 and stride[1] != c.d):
        raise HS2Error("rows must be [n_rows][Hkv][d] with contiguous tokens")
    return stride[0] if n > 1 else c.Hkv * c.d  # one token: its stride reaches nothing


def _side(c: hs2_kv, v: bool) -> hs2_kv:
    """The K (V) half of the cache as a key-only cache."""
    half = hs2_kv.from_buffer_copy(c)
    if v:
        half.k, half.k_scale, half.k_sf = c.v, c.v_scale, c.v_sf
    half.v = half.v_scale = half.v_sf = None
    return half


def _kv_rows(call, kv: KV, k_rows, v_rows, row_start, dev_err, stream) -> None:
    c, dev = kv._cached()[:2]
    dtype = k_rows.dtype
    if (v_rows is None) != (kv.v is None):
        raise HS2Error("v_rows goes with a cache that has V")
    if dtype not in _ROW_DTYPES or (v_rows is not None and v_rows.dtype is not dtype):
        raise HS2Error("rows must be float32 or bfloat16, K and V alike")
    shape, stride = k_rows.shape, k_rows.stride()
    n = shape[0]
    ks = vs = _token_stride(shape, stride, n, c)
    if v_rows is not None and (v_rows.stride() != stride or v_rows.shape != shape):
        vs = _token_stride(v_rows.shape, v_rows.stride(), n, c)
    _i32(row_start, "row_start", c.batch + 1)
    st = _launch_stream(stream, dev, k_rows, v_rows, row_start, dev_err)
    dt, rs, err = _ROW_DTYPES[dtype], row_start.data_ptr(), _ptr(dev_err)
    if vs == ks:
        _check(call(ctypes.byref(c), k_rows.data_ptr(), _ptr(v_rows), dt, ks, rs, n, err, st))
        return
    # a call takes one stride: a call for each side, once it is sure that neither will be refused
    for x, stride in ((k_rows, ks), (v_rows, vs)):
        if (x.data_ptr() | stride * x.element_size()) % 16 or stride < c.Hkv * c.d:
            raise HS2Error("rows must start on 16 bytes, their tokens a multiple of 16 bytes apart and disjoint")
    for v, x, stride in ((False, k_rows, ks), (True, v_rows, vs)):
        _check(call(ctypes.byref(_side(c, v)), x.data_ptr(), 0, dt, stride, rs, n, err, st))


def hs2_kv_write(kv: KV, k_rows: torch.Tensor, v_rows: torch.Tensor | None, row_start: torch.Tensor, dev_err=None,
                 stream=None) -> None:
    """Rows of a ragged batch into the cache, quantised to its type: rows [row_start[b],
    row_start[b+1]) are sequence b's last positions (seq_len already counts them). ``k_rows``
    / ``v_rows``: float32 or bfloat16 (both alike) [n_rows][Hkv][d], each with a token stride
    of its own (a multiple of 16 bytes; one launch where they agree, else two); the cache's
    k_scale / v_scale are inputs."""
    _kv_rows(load().hs2_kv_write, kv, k_rows, v_rows, row_start, dev_err, stream)


def hs2_kv_read(kv: KV, row_start: torch.Tensor, n_rows: int, dtype: torch.dtype = torch.float32, out=None,
                dev_err=None, stream=None):
    """The values of the rows hs2_kv_write with this ``row_start`` would write, as (k_rows,
    v_rows) of ``dtype`` [n_rows][Hkv][d] (v_rows None for a key-only cache). Rows outside
    every sequence are left as they are in ``out``."""
    if out is None:
        c = kv.c()
        k, v = (_new((n_rows, c.Hkv, c.d), dtype, kv.k.device, stream) if t is not None else None for t in (kv.k, kv.v))
        out = (k, v)
    elif out[0].shape[0] != n_rows or out[0].dtype != dtype:
        raise HS2Error("out must hold n_rows rows of the dtype")
    _kv_rows(load().hs2_kv_read, kv, out[0], out[1], row_start, dev_err, stream)
    return out


def hs2_fa_chunk_workspace(n_rows: int, Hq: int, kv: KV, max_n: int, max_t: int, w: int = 0) -> int:
    return load().hs2_fa_chunk_workspace(n_rows, Hq, ctypes.byref(kv.c()), max_n, max_t, w)


def hs2_fa_chunk(q: torch.Tensor, row_start: torch.Tensor, kv: KV, scale: float, max_n: int,
                 max_t: int | None = None, w: int = 0, sink: torch.Tensor | None = None,
                 o_dtype: torch.dtype = torch.float32, out=None, workspace=None, dev_err=None, stream=None):
    """Causal attention of a ragged batch of query chunks over the cache; returns (o, lse).

    ``q`` [n_rows][Hq][d] (bf16; float32 with an F32 cache): rows [row_start[b],
    row_start[b+1]) are sequence b's last positions. ``max_n`` bounds the rows of a sequence,
    ``max_t`` its keys (default: the table's capacity). ``w`` > 0: a sliding window of that
    many keys; ``sink``: float32 [Hq] logits of one more key with a zero value. ``o_dtype``
    float32 or bfloat16; lse is float32 [n_rows][Hq]."""
    lib = load()
    c, dev = kv._cached()[:2]
    n, Hq, d = q.shape
    if max_t is None:
        max_t = c.max_pages * c.page_size
    if q.dtype is not (torch.float32 if c.dtype == F32 else torch.bfloat16) or d != c.d or not q.is_contiguous():
        raise HS2Error("q must be contiguous [n_rows][Hq][d], bfloat16 (float32 with an F32 cache)")
    if sink is not None and (sink.dtype is not torch.float32 or not sink.is_contiguous() or sink.numel() != Hq):
        raise HS2Error("sink must be float32 [Hq]")
    if o_dtype not in _ROW_DTYPES:
        raise HS2Error("o_dtype must be float32 or bfloat16")
    _i32(row_start, "row_start", c.batch + 1)
    if out is None:
        o = _new((n, Hq, d), o_dtype, q.device, stream)
        lse = _new((n, Hq), torch.float32, q.device, stream)
    else:
        o, lse = out
        if o.dtype is not o_dtype or o.shape != (n, Hq, d) or not o.is_contiguous() or (
                lse is not None and (lse.dtype is not torch.float32 or lse.shape != (n, Hq)
                                     or not lse.is_contiguous())):
            raise HS2Error("out must be contiguous (o [n_rows][Hq][d] of o_dtype, lse float32 [n_rows][Hq] or None)")
    st = _launch_stream(stream, dev, q, row_start, sink, o, lse, workspace, dev_err)
    ws = workspace
    if ws is None:
        ws = _scratch(lib.hs2_fa_chunk_workspace(n, Hq, ctypes.byref(c), max_n, max_t, w), q.device, stream)
    _check(lib.hs2_fa_chunk(q.data_ptr(), row_start.data_ptr(), n, max_n, Hq, ctypes.byref(c), max_t, w, scale,
                            _ptr(sink), o.data_ptr(), _ROW_DTYPES[o_dtype], _ptr(lse), ws.data_ptr(), ws.nbytes,
                            _ptr(dev_err), st))
    return o, lse


@dataclass
class Pages(_Handle):
    """The books of a page pool: references per page and the stack of free pages."""

    ref: torch.Tensor  # int32 [num_pages], table entries that hold the page (0: free)
    free_list: torch.Tensor  # int32 [num_pages], of which the first n_free are free pages
    n_free: torch.Tensor  # int32 [1]

    @classmethod
    def make(cls, num_pages: int, device="cuda") -> "Pages":
        """A pool with every page free; the lowest are taken first."""
        return cls(ref=torch.zeros(num_pages, dtype=torch.int32, device=device),
                   free_list=torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device),
                   n_free=torch.full((1,), num_pages, dtype=torch.int32, device=device))

    def _tensors(self):
        return self.ref, self.free_list, self.n_free

    def _make(self) -> hs2_pages:
        return self.c()

    def c(self) -> hs2_pages:
        n = int(self.ref.shape[0])
        for t, name, size in ((self.ref, "ref", n), (self.free_list, "free_list", n), (self.n_free, "n_free", 1)):
            _i32(t, name, size)
        return hs2_pages(self.ref.data_ptr(), self.free_list.data_ptr(), self.n_free.data_ptr(), n)


def hs2_pages_grow(pages: Pages, block_table: torch.Tensor, seq_len: torch.Tensor, n_new: torch.Tensor, dev_err=None,
                   stream=None) -> None:
    """seq_len += n_new, with free pages for the positions that need them, in place."""
    b, mp = _table(block_table, "block_table")
    _i32(seq_len, "seq_len", b)
    _i32(n_new, "n_new", b)
    c, dev = pages._cached()[:2]
    st = _launch_stream(stream, dev, block_table, seq_len, n_new, dev_err)
    _check(load().hs2_pages_grow(ctypes.byref(c), block_table.data_ptr(), seq_len.data_ptr(),
                                 n_new.data_ptr(), b, mp, _ptr(dev_err), st))


def hs2_pages_free(pages: Pages, block_table: torch.Tensor, seq_len: torch.Tensor, drop: torch.Tensor, dev_err=None,
                   stream=None) -> None:
    """The pages of every sequence with drop[b] != 0 lose a reference; those left with none
    return to the free list."""
    b, mp = _table(block_table, "block_table")
    _i32(seq_len, "seq_len", b)
    _i32(drop, "drop", b)
    c, dev = pages._cached()[:2]
    st = _launch_stream(stream, dev, block_table, seq_len, drop, dev_err)
    _check(load().hs2_pages_free(ctypes.byref(c), block_table.data_ptr(), seq_len.data_ptr(),
                                 drop.data_ptr(), b, mp, _ptr(dev_err), st))


def _kv_array(kvs, dev: int):
    """The caches' C structs as an array, all on device `dev`."""
    if not kvs:
        raise HS2Error("at least one cache")
    got = [kv._cached() for kv in kvs]
    if any(x[1] != dev for x in got):
        raise HS2Error("tensors on several devices")
    return ctypes.byref(got[0][0]) if len(got) == 1 else (hs2_kv * len(got))(*[x[0] for x in got])


def hs2_pages_fork(pages: Pages, kvs, src: torch.Tensor, out=None, dev_err=None, stream=None):
    """Branches of the caches' sequences: branch c continues sequence src[c] (-1: none), with
    its full pages shared and the last, partly filled one copied. ``kvs``: the caches of one
    block table. Returns (child_table, child_len)."""
    c, dev = pages._cached()[:2]
    cs = _kv_array(kvs, dev)
    n, mp = src.numel(), kvs[0].block_table.shape[1]
    _i32(src, "src", n)
    if out is None:
        out = _new((n, mp), torch.int32, src.device, stream), _new((n,), torch.int32, src.device, stream)
    else:
        _i32(out[0], "child_table", n, mp)
        _i32(out[1], "child_len", n)
    st = _launch_stream(stream, dev, src, out[0], out[1], dev_err)
    _check(load().hs2_pages_fork(ctypes.byref(c), len(kvs), cs, src.data_ptr(), n, out[0].data_ptr(),
                                 out[1].data_ptr(), _ptr(dev_err), st))
    return out


def hs2_pages_compact_workspace(pages: Pages) -> int:
    return load().hs2_pages_compact_workspace(ctypes.byref(pages.c()))


def hs2_pages_compact(pages: Pages, kvs, workspace=None, dev_err=None, stream=None) -> None:
    """The pool's referenced pages to its front, in place in every cache of ``kvs`` (which
    share one block table holding every sequence), with tables and books updated."""
    c, dev = pages._cached()[:2]
    cs = _kv_array(kvs, dev)
    st = _launch_stream(stream, dev, workspace, dev_err)
    ws = workspace if workspace is not None else _scratch(hs2_pages_compact_workspace(pages), pages.ref.device, stream)
    _check(load().hs2_pages_compact(ctypes.byref(c), len(kvs), cs, ws.data_ptr(), ws.nbytes, _ptr(dev_err), st))
