"""ctypes binding of libmapflow.so (argument marshalling only).

Every step of the path runs in the library's CUDA kernels; this module only
turns torch tensors into pointers, allocates caller-owned outputs and
workspaces with torch, and passes torch's current stream.  There is no CPU
fallback: if the shared library is missing, loading raises.  Nothing here is
recorded for autograd: outputs never require gradients, whatever the inputs do.

Names follow the C ABI in include/mapflow.h.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass

import numpy as np
import torch

from .build import marshal_key

_HERE = os.path.dirname(os.path.abspath(__file__))
# the in-tree build; MAPFLOW_LIB names another build of the same library
LIB_PATH = os.environ.get("MAPFLOW_LIB") or os.path.join(_HERE, "libmapflow.so")

MF_OK, MF_ERR_INVALID_ARG, MF_ERR_UNSUPPORTED, MF_ERR_WORKSPACE = 0, 1, 2, 3
MF_ERR_CUDA, MF_ERR_TIMEOUT, MF_ERR_NOT_FOUND, MF_ERR_CAPACITY = 4, 5, 6, 7
MF_BF16, MF_F32 = 0, 1

EXPORTED = [
    "mf_version", "mf_last_error", "mf_layout_sizes", "mf_block_stats_workspace",
    "mf_block_stats", "mf_block_stats_range", "mf_select_extract_workspace",
    "mf_select_extract", "mf_select_extract_range", "mf_extract_workspace", "mf_extract",
    "mf_select_rounds_workspace", "mf_select_rounds", "mf_cache_offload", "mf_cache_fetch",
    "mf_mapped_av_workspace", "mf_mapped_av", "mf_mapped_av_range", "mf_block_stats_noalloc",
    "mf_block_stats_noalloc_max_workspace",
    "mf_rope_freqs", "mf_rope_phases", "mf_rope", "mf_kv_append", "mf_paged_attn_workspace",
    "mf_paged_attn",
    "mf_mapped_av_plan", "mf_path_info", "mf_exp2_fma_eval", "mf_selftest_timeout", "mf_sync_status", "mf_prefix_hash",
    "mf_index_create",
    "mf_index_destroy",
    "mf_index_insert", "mf_index_lookup", "mf_index_size",
]


class AttnDesc(C.Structure):
    _fields_ = [("nseq", C.c_int32), ("cu_seqlens", C.c_void_p),
                ("cu_seqlens_host", C.c_void_p), ("Hs", C.c_int32), ("d", C.c_int32),
                ("B", C.c_int32), ("band_bias", C.c_float), ("band_width", C.c_int32),
                ("dt", C.c_int)]


class CsrCache(C.Structure):
    _fields_ = [("nqb_total", C.c_int64), ("nnz_capacity", C.c_int64),
                ("row_ptr", C.c_void_p), ("col_idx", C.c_void_p), ("qb_seq", C.c_void_p),
                ("qb_idx", C.c_void_p), ("values", C.c_void_p), ("Hs", C.c_int32),
                ("B", C.c_int32), ("dt", C.c_int), ("nseq", C.c_int32),
                ("cu_seqlens", C.c_void_p)]


class VDesc(C.Structure):
    _fields_ = [("V", C.c_void_p), ("page_table", C.c_void_p), ("page_size", C.c_int32),
                ("max_pages_per_seq", C.c_int32), ("npages", C.c_int64), ("Hkv", C.c_int32),
                ("d", C.c_int32)]


class RopeDesc(C.Structure):
    _fields_ = [("rot_dim", C.c_int32), ("interleaved", C.c_int32), ("phases", C.c_void_p),
                ("scale", C.c_float)]


class TokenBatch(C.Structure):
    _fields_ = [("ntok", C.c_int64), ("nseq", C.c_int32), ("cu_seqlens", C.c_void_p),
                ("start", C.c_void_p)]


class KvCacheDesc(C.Structure):
    _fields_ = [("K", C.c_void_p), ("V", C.c_void_p), ("page_table", C.c_void_p),
                ("npages", C.c_int64), ("page_size", C.c_int32),
                ("max_pages_per_seq", C.c_int32), ("nseq", C.c_int32), ("Hkv", C.c_int32),
                ("d", C.c_int32), ("dt", C.c_int)]


class PagedAttnDesc(C.Structure):
    _fields_ = [("Hq", C.c_int32), ("scale", C.c_float), ("band_bias", C.c_float),
                ("band_width", C.c_int32), ("window", C.c_int32), ("len_add", C.c_int32)]


class MapflowError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"mapflow status {status}: {msg}")
        self.status = status


_lib = None
_fast = None  # the decode calls' marshalling in C++ (csrc_py/marshal.cpp)


def load_library(path: str = LIB_PATH):
    """Load libmapflow.so and declare its signatures (no GPU needed)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m cross_model_attention_block_b200.build`")
    L = C.CDLL(path)
    P, I32, I64, SZ = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
    sig = {
        "mf_version": (C.c_char_p, []),
        "mf_last_error": (C.c_char_p, []),
        "mf_layout_sizes": (C.c_int, [I32, P, I32, P, P]),
        "mf_block_stats_workspace": (SZ, [P]),
        "mf_block_stats": (C.c_int, [P, P, P, P, P, P, SZ, P]),
        "mf_block_stats_range": (C.c_int, [P, P, P, P, P, I64, I64, P, SZ, P]),
        "mf_select_extract_workspace": (SZ, [P]),
        "mf_select_extract": (C.c_int, [P, P, P, P, P, C.c_double, P, P, SZ, P]),
        "mf_select_extract_range": (C.c_int, [P, P, P, P, P, C.c_double, P, I64, I64, P, SZ,
                                              P]),
        "mf_extract_workspace": (SZ, [P]),
        "mf_extract": (C.c_int, [P, P, P, P, P, P, SZ, P]),
        "mf_select_rounds_workspace": (SZ, [P, I32, P]),
        "mf_select_rounds": (C.c_int, [P, P, I32, P, P, C.c_double, P, P, SZ, P]),
        "mf_cache_offload": (C.c_int, [P, P, P]),
        "mf_cache_fetch": (C.c_int, [P, P, I64, I64, P]),
        "mf_mapped_av_workspace": (SZ, [P, P, I32, P]),
        "mf_mapped_av": (C.c_int, [P, P, I32, P, P, P, P, SZ, P]),
        "mf_mapped_av_range": (C.c_int, [P, P, I32, P, P, P, I64, I64, P, SZ, P]),
        "mf_block_stats_noalloc_max_workspace": (SZ, []),
        "mf_block_stats_noalloc": (C.c_int, [P, P, P, P, P, P]),
        "mf_rope_freqs": (C.c_int, [I32, C.c_double, C.c_int, C.c_double, C.c_double, C.c_double,
                                    C.c_double, P]),
        "mf_rope_phases": (C.c_int, [P, I32, P]),
        "mf_rope": (C.c_int, [P, P, I32, C.c_int, I32, P, I64, P, I64, I32, P, I64, P, I64, I32,
                              P]),
        "mf_kv_append": (C.c_int, [P, P, P, P, I64, P, I64, I32, P, I64, P, I64, P]),
        "mf_paged_attn_workspace": (SZ, [P, P]),
        "mf_paged_attn": (C.c_int, [P, P, P, P, I64, P, I64, P, P, SZ, P]),
        "mf_mapped_av_plan": (C.c_int, [I32, I32, I32, P]),
        "mf_path_info": (C.c_int, [P, I32, P, P]),
        "mf_exp2_fma_eval": (C.c_int, [P, P, I64, P]),
        "mf_selftest_timeout": (C.c_int, [I32, P]),
        "mf_sync_status": (C.c_int, [P]),
        "mf_prefix_hash": (C.c_int, [P, I64, I32, C.c_uint64, P]),
        "mf_index_create": (C.c_int, [P]),
        "mf_index_destroy": (None, [P]),
        "mf_index_insert": (C.c_int, [P, P, I64, I32, I32, P]),
        "mf_index_lookup": (C.c_int, [P, P, I64, I32, P, P, P]),
        "mf_index_size": (I64, [P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def _check(status):
    if status != MF_OK:
        raise MapflowError(status, load_library().mf_last_error().decode())


def _stream():
    # without a CUDA device only the library's argument checks can run (they
    # return before anything is enqueued); NULL then stands for the stream
    if not torch.cuda.is_available():
        return C.c_void_p(None)
    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _dtype_code(dt):
    if dt == torch.bfloat16:
        return MF_BF16
    if dt == torch.float32:
        return MF_F32
    raise ValueError(f"unsupported dtype {dt}")


def _workspace(nbytes, device):
    buf = torch.empty(int(nbytes) + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    return buf, buf.data_ptr() + off


@dataclass
class Context:
    """A packed varlen sender context and its attention settings."""

    cu_seqlens: torch.Tensor        # int32 [nseq+1] on the device
    cu_seqlens_host: np.ndarray     # int32 [nseq+1]
    Hs: int
    d: int
    B: int
    band_bias: float
    band_width: int
    dtype: torch.dtype

    @classmethod
    def make(cls, lengths, Hs, d, B, band_bias, band_width, dtype, device="cuda"):
        cu = np.zeros(len(lengths) + 1, dtype=np.int32)
        cu[1:] = np.cumsum(np.asarray(lengths, dtype=np.int64))
        return cls(torch.from_numpy(cu).to(device), cu, Hs, d, B, float(band_bias),
                   int(band_width), dtype)

    @property
    def nseq(self):
        return len(self.cu_seqlens_host) - 1

    @property
    def ntok(self):
        return int(self.cu_seqlens_host[-1])

    def desc(self) -> AttnDesc:
        self._host = np.ascontiguousarray(self.cu_seqlens_host, dtype=np.int32)
        return AttnDesc(self.nseq, self.cu_seqlens.data_ptr(),
                        self._host.ctypes.data, self.Hs, self.d, self.B,
                        self.band_bias, self.band_width, _dtype_code(self.dtype))

    def layout_sizes(self):
        return layout_sizes(self.cu_seqlens_host, self.B)

    def range_blocks(self, qb_begin, qb_end):
        """Causal blocks of the global query blocks [qb_begin, qb_end): the
        CSR capacity a cache of that range can never overflow."""
        n = 0
        q0 = 0
        for L in np.diff(self.cu_seqlens_host):
            nq = (int(L) + self.B - 1) // self.B
            a, b = max(qb_begin - q0, 0), min(qb_end - q0, nq)
            if a < b:
                n += b * (b + 1) // 2 - a * (a + 1) // 2
            q0 += nq
        return n


def layout_sizes(cu_seqlens_host, B):
    """(nqb_total, nblocks_total) of a context."""
    L = load_library()
    cu = np.ascontiguousarray(cu_seqlens_host, dtype=np.int32)
    a, b = C.c_int64(), C.c_int64()
    _check(L.mf_layout_sizes(len(cu) - 1, cu.ctypes.data, B, C.byref(a), C.byref(b)))
    return a.value, b.value


def block_stats(ctx: Context, Q, K, lse=None, mass=None, qb_range=None):
    """Stage 1: lse [Hs, ntok] float32 and block masses [nblocks] float32.
    `qb_range` = (begin, end) restricts the call to those global query
    blocks: only their lse rows and block masses are written."""
    L = load_library()
    d = ctx.desc()
    _, nblocks = ctx.layout_sizes()
    dev = Q.device
    if lse is None:
        lse = torch.empty((ctx.Hs, ctx.ntok), dtype=torch.float32, device=dev)
    if mass is None:
        mass = torch.empty((max(nblocks, 1),), dtype=torch.float32, device=dev)
    nbytes = L.mf_block_stats_workspace(C.byref(d))
    if nbytes == 0:
        _check(MF_ERR_INVALID_ARG)
    ws, wsp = _workspace(nbytes, dev)
    if qb_range is None:
        _check(L.mf_block_stats(C.byref(d), _ptr(Q), _ptr(K), _ptr(lse), _ptr(mass),
                                C.c_void_p(wsp), nbytes, _stream()))
    else:
        _check(L.mf_block_stats_range(C.byref(d), _ptr(Q), _ptr(K), _ptr(lse), _ptr(mass),
                                      int(qb_range[0]), int(qb_range[1]), C.c_void_p(wsp),
                                      nbytes, _stream()))
    ctx._stats_ws = ws  # keep the workspace alive until the stream has used it
    return lse, mass


class Cache:
    """Caller-owned buffers of one CSR block cache (device memory, or pinned
    host memory for the host tier)."""

    def __init__(self, ctx: Context, capacity=None, device="cuda", pin=False):
        nqb, nblocks = ctx.layout_sizes()
        cap = nblocks if capacity is None else int(capacity)
        self.ctx = ctx
        self.nqb = nqb
        self.capacity = cap
        self.row_ptr = torch.empty(nqb + 1, dtype=torch.int64, device=device)
        self.col_idx = torch.empty(max(cap, 1), dtype=torch.int32, device=device)
        self.qb_seq = torch.empty(max(nqb, 1), dtype=torch.int32, device=device)
        self.qb_idx = torch.empty(max(nqb, 1), dtype=torch.int32, device=device)
        nvals = max(cap, 1) * ctx.B * ctx.B * ctx.Hs
        self.values = torch.empty(nvals, dtype=ctx.dtype, device=device)
        if pin:
            for name in ("row_ptr", "col_idx", "qb_seq", "qb_idx", "values"):
                setattr(self, name, getattr(self, name).pin_memory())

    def struct(self) -> CsrCache:
        return CsrCache(self.nqb, self.capacity, self.row_ptr.data_ptr(),
                        self.col_idx.data_ptr(), self.qb_seq.data_ptr(),
                        self.qb_idx.data_ptr(), self.values.data_ptr(), self.ctx.Hs,
                        self.ctx.B, _dtype_code(self.ctx.dtype), self.ctx.nseq,
                        self.ctx.cu_seqlens.data_ptr())

    @property
    def nnz(self):
        return int(self.row_ptr[-1].item())

    def values_view(self):
        """values in stored order [capacity, B/16 key groups, B/8 row slices, 2 halves,
        Hs, 8 chunks, 8] (see the C header for the chunk permutation)."""
        B, Hs = self.ctx.B, self.ctx.Hs
        return self.values[: self.capacity * B * B * Hs].view(
            self.capacity, B // 16, B // 8, 2, Hs, 8, 8)


def select_extract(ctx: Context, Q, K, lse, mass, tau, cache: Cache | None = None,
                   qb_range=None):
    """Stage 2: kept blocks per query block (CSR) and their probability blocks.
    `qb_range` = (begin, end) restricts the call to those global query blocks;
    the CSR rows of every other query block are empty."""
    L = load_library()
    d = ctx.desc()
    if cache is None:
        cache = Cache(ctx, device=Q.device)
    cs = cache.struct()
    nbytes = L.mf_select_extract_workspace(C.byref(d))
    if nbytes == 0:
        _check(MF_ERR_INVALID_ARG)
    ws, wsp = _workspace(nbytes, Q.device)
    if qb_range is None:
        _check(L.mf_select_extract(C.byref(d), _ptr(Q), _ptr(K), _ptr(lse), _ptr(mass),
                                   float(tau), C.byref(cs), C.c_void_p(wsp), nbytes, _stream()))
    else:
        _check(L.mf_select_extract_range(C.byref(d), _ptr(Q), _ptr(K), _ptr(lse), _ptr(mass),
                                         float(tau), C.byref(cs), int(qb_range[0]),
                                         int(qb_range[1]), C.c_void_p(wsp), nbytes,
                                         _stream()))
    cache._ws = ws  # keep the workspace alive until the stream has used it
    return cache


def extract(ctx: Context, Q, K, lse, cache: Cache):
    """Probability blocks of every entry of a filled CSR (this layer's Q, K, lse)."""
    L = load_library()
    d = ctx.desc()
    nbytes = L.mf_extract_workspace(C.byref(d))
    if nbytes == 0:
        _check(MF_ERR_INVALID_ARG)
    ws, wsp = _workspace(nbytes, Q.device)
    cs = cache.struct()
    _check(L.mf_extract(C.byref(d), _ptr(Q), _ptr(K), _ptr(lse), C.byref(cs), C.c_void_p(wsp),
                        nbytes, _stream()))
    cache._ws = ws
    return cache


def select_rounds(ctx: Context, mass, round_starts, tau, cache: Cache | None = None):
    """Round-level selection from the watershed layer's block masses: the CSR
    of every query block (values are written by `extract`, per layer).
    round_starts: packed token offsets of the rounds, 0 .. ntok."""
    L = load_library()
    d = ctx.desc()
    st = np.ascontiguousarray(round_starts, dtype=np.int32)
    nr = len(st) - 1
    dev = mass.device
    st_dev = torch.from_numpy(st).to(dev)
    if cache is None:
        cache = Cache(ctx, device=dev)
    nbytes = L.mf_select_rounds_workspace(C.byref(d), nr, st.ctypes.data)
    if nbytes == 0:
        _check(L.mf_select_rounds(C.byref(d), _ptr(mass), nr, _ptr(st_dev), st.ctypes.data,
                                  float(tau), None, None, 0, _stream()))
        _check(MF_ERR_INVALID_ARG)
    ws, wsp = _workspace(nbytes, dev)
    cs = cache.struct()
    _check(L.mf_select_rounds(C.byref(d), _ptr(mass), nr, _ptr(st_dev), st.ctypes.data,
                              float(tau), C.byref(cs), C.c_void_p(wsp), nbytes, _stream()))
    cache._round_ws = (ws, st_dev)
    return cache


def cache_offload(dev_cache: Cache, host_cache: Cache):
    """Copy a device cache into a (pinned) host cache of the same layout."""
    _check(load_library().mf_cache_offload(C.byref(dev_cache.struct()),
                                           C.byref(host_cache.struct()), _stream()))
    return host_cache


def cache_fetch(host_cache: Cache, dev_cache: Cache, qb_range):
    """Enqueue the copies of a range of rows of a host cache into a device
    cache on the current stream."""
    _check(load_library().mf_cache_fetch(C.byref(host_cache.struct()),
                                         C.byref(dev_cache.struct()), int(qb_range[0]),
                                         int(qb_range[1]), _stream()))
    return dev_cache


def mapped_av(cache: Cache, Hr, W, V, Hkv, page_table=None, page_size=16, O=None,
              workspace=None, qb_range=None):
    """Stage 3: O [ntok, Hr, d] = (W-mixed kept map) x V (fused).

    `workspace` may be a uint8 device tensor reused across calls (grown when
    too small); by default one is allocated per call.  `qb_range` =
    (begin, end) restricts the call to those global query blocks (chunked
    prefill, prefix reuse): only their rows of O are written."""
    L = load_library()
    ctx = cache.ctx
    d = ctx.desc()
    if O is None:
        O = torch.empty((ctx.ntok, Hr, ctx.d), dtype=ctx.dtype, device=W.device)
    maxp = 0 if page_table is None else int(page_table.shape[1])
    npages = 0 if page_table is None else int(V.shape[0])
    vd = VDesc(V.data_ptr(), 0 if page_table is None else page_table.data_ptr(),
               page_size, maxp, npages, Hkv, ctx.d)
    cs = cache.struct()
    nbytes = L.mf_mapped_av_workspace(C.byref(cs), C.byref(d), int(Hr), C.byref(vd))
    if nbytes == 0:
        _check(MF_ERR_INVALID_ARG)
    if workspace is not None and workspace.numel() >= nbytes + 256:
        ws = workspace
        wsp = ws.data_ptr() + (-ws.data_ptr()) % 256
    else:
        ws, wsp = _workspace(nbytes, W.device)
    if qb_range is None:
        _check(L.mf_mapped_av(C.byref(cs), C.byref(d), int(Hr), _ptr(W), C.byref(vd), _ptr(O),
                              C.c_void_p(wsp), nbytes, _stream()))
    else:
        _check(L.mf_mapped_av_range(C.byref(cs), C.byref(d), int(Hr), _ptr(W), C.byref(vd),
                                    _ptr(O), int(qb_range[0]), int(qb_range[1]),
                                    C.c_void_p(wsp), nbytes, _stream()))
    cache._av_ws = ws  # keep the workspace alive until the stream has used it
    return O


# ---- the receiver's own tokens: rotary positions, paged keys and values, and
# the attention of one new token over them

_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}


def _refuse(msg):
    raise MapflowError(MF_ERR_INVALID_ARG, msg)


def _require(ok, msg):
    if not ok:
        _refuse(msg)


# The decode calls are made by _fast (csrc_py/marshal.cpp), which checks its arguments,
# makes the call on their device and returns None where it refuses one; the checks
# below then say what is wrong, and make no call.

def _load_fast():
    global _fast
    L = load_library()
    why = ("_marshal.so is missing or does not fit this torch: build it with "
           "`python -m cross_model_attention_block_b200.build --force`")
    try:
        from . import _marshal
    except ImportError as e:
        raise RuntimeError(why) from e
    if getattr(_marshal, "built_for", None) != marshal_key():
        raise RuntimeError(why)
    _marshal.bind(*(C.cast(getattr(L, n), C.c_void_p).value for n in (
        "mf_rope", "mf_kv_append", "mf_paged_attn", "mf_paged_attn_workspace")))
    _fast = _marshal
    return _fast


def _made(r):
    """The result of a call that _fast made: its outputs, unless it is a status."""
    if type(r) is int:
        _check(r)
    return r


def _rows(name, t, ntok, H, d, dtype):
    """Checks a [ntok, H, d] tensor whose heads are d apart."""
    if t.shape != (ntok, H, d):
        _refuse(f"{name} must be [{ntok}, {H}, {d}], got {tuple(t.shape)}")
    if t.dtype != dtype:
        _refuse(f"{name} must be {dtype}, got {t.dtype}")
    _, head, dim = t.stride()
    if dim != 1 or (head != d and H != 1):
        _refuse(f"{name}'s heads must be {d} elements apart")


def _index(name, t, n):
    if t.dtype != torch.int32 or t.shape != (n,) or not t.is_contiguous():
        _refuse(f"{name} must be a contiguous int32 tensor of {n} entries")


def _refuse_the_rest(*tensors):
    """The last refusals of a call: tensors apart, or arguments that are none."""
    given = [t for t in tensors if t is not None]
    if any(not t.is_cuda or t.device != given[0].device for t in given):
        _refuse("every tensor must be on one CUDA device")
    _refuse("an argument is not of a kind that the call takes")


def rope_freqs(rot_dim, base=10000.0, scaling="none", factor=1.0, original_length=0.0, low=1.0,
               high=32.0):
    """Inverse frequencies float64 [rot_dim/2] (host); scalings as mf_rope_scaling in
    the C header: "none", "linear", "ntk" or "parts"."""
    _require(scaling in _SCALINGS, f"scaling must be one of {sorted(_SCALINGS)}")
    out = np.zeros(max(int(rot_dim) // 2, 1), dtype=np.float64)
    _check(load_library().mf_rope_freqs(int(rot_dim), base, _SCALINGS[scaling], factor,
                                        original_length, low, high, out.ctypes.data))
    return out


class Rope:
    """Rotary positions: the phases of rot_dim/2 pairs (int64 tensor on the device,
    the bits of mf_rope_phases), their layout and their scale."""

    def __init__(self, phases, interleaved=False, scale=1.0):
        _require(phases.dtype == torch.int64 and phases.dim() == 1 and phases.is_contiguous(),
                 "phases must be a contiguous int64 tensor [rot_dim / 2]")
        self._args = phases, bool(interleaved), float(scale)
        self._desc = RopeDesc(2 * phases.shape[0], int(self.interleaved), phases.data_ptr(),
                              self.scale)
        self._addr = C.addressof(self._desc)

    # what _desc was made of: not to be set, and a copy makes its own
    phases = property(lambda self: self._args[0])
    interleaved = property(lambda self: self._args[1])
    scale = property(lambda self: self._args[2])

    def __reduce__(self):
        return type(self), self._args

    @classmethod
    def from_freqs(cls, inv_freq, interleaved=False, scale=1.0, device="cuda"):
        """From host inverse frequencies (radians per position)."""
        f = np.ascontiguousarray(inv_freq, dtype=np.float64)
        ph = np.zeros(len(f), dtype=np.uint64)
        _check(load_library().mf_rope_phases(f.ctypes.data, len(f), ph.ctypes.data))
        return cls(torch.from_numpy(ph.view(np.int64)).to(device), interleaved, scale)

    @classmethod
    def make(cls, rot_dim, base=10000.0, interleaved=False, scale=1.0, scaling="none",
             factor=1.0, original_length=0.0, low=1.0, high=32.0, device="cuda"):
        return cls.from_freqs(rope_freqs(rot_dim, base, scaling, factor, original_length, low,
                                         high), interleaved, scale, device)


def _batch(ntok, start, cu_seqlens):
    nseq = ntok
    if cu_seqlens is not None:
        nseq = max(cu_seqlens.numel(), 1) - 1
        _index("cu_seqlens", cu_seqlens, nseq + 1)
    if start is not None:
        _index("start", start, nseq)


def rope(rp: Rope, Q, K=None, start=None, cu_seqlens=None, Q_out=None, K_out=None,
         backward=False):
    """Rotates Q [ntok, Hq, d] and, if given, K [ntok, Hk, d]: Q_out, or (Q_out, K_out).

    Token t of sequence s (cu_seqlens [nseq + 1], int32 on the device) has position
    start[s] + t - cu_seqlens[s], and the rows of tokens past cu_seqlens[nseq] are left as
    they were; without cu_seqlens, start [ntok] holds every token's own position.
    backward=True takes gradients of the outputs to those of the inputs; the call does not
    record itself for autograd.
    Q_out may be Q, and K_out may be K."""
    f = _fast or _load_fast()
    r = f.rope(rp._addr, rp._args[0], Q, K, start, cu_seqlens, Q_out, K_out, backward)
    if r is not None:
        return _made(r)
    _require(start is not None or cu_seqlens is not None, "start or cu_seqlens must be given")
    _require(Q.dim() == 3, "Q must be [ntok, Hq, d]")
    ntok, Hq, d = Q.shape
    _dtype_code(Q.dtype)
    _batch(ntok, start, cu_seqlens)
    for name, t in (("Q", Q), ("Q_out", Q_out)):
        if t is not None:
            _rows(name, t, ntok, Hq, d, Q.dtype)
    if K is not None:
        _require(K.dim() == 3 and K.shape[1] > 0, "K must be [ntok, Hk, d]")
        for name, t in (("K", K), ("K_out", K_out)):
            if t is not None:
                _rows(name, t, ntok, K.shape[1], d, Q.dtype)
    else:
        _require(K_out is None, "K_out without K")
    _refuse_the_rest(Q, K, start, cu_seqlens, Q_out, K_out, rp.phases)


class KVCache:
    """A receiver's paged keys and values: pools [npages, page_size, Hkv, d] and the page
    table int32 [nseq, max_pages_per_seq], all owned by the caller, who may change what
    they hold but not where they lie.  `V` with `page_table` is what mapped_av reads."""

    def __init__(self, K, V, page_table):
        r = (_fast or _load_fast()).kv_cache(K, V, page_table)
        if r is None:
            if (K.dim() != 4 or K.shape != V.shape or K.dtype != V.dtype
                    or not K.is_contiguous() or not V.is_contiguous()):
                _refuse("K and V must be contiguous pools [npages, page_size, Hkv, d] of one "
                        "dtype")
            if (page_table.dtype != torch.int32 or page_table.dim() != 2
                    or not page_table.is_contiguous()):
                _refuse("page_table must be a contiguous int32 tensor "
                        "[nseq, max_pages_per_seq]")
            _dtype_code(K.dtype)
            _refuse("a size of the pools or of the page table is past 32 bits")
        self._args = K, V, page_table
        (self.npages, self.page_size, self.Hkv, self.d, self.nseq, self.max_pages,
         self._device, self._bytes, self._addr) = r

    # what _bytes was made of: not to be set, and a copy makes its own
    K = property(lambda self: self._args[0])
    V = property(lambda self: self._args[1])
    page_table = property(lambda self: self._args[2])

    def __reduce__(self):
        return type(self), self._args

    @property
    def _desc(self):
        return KvCacheDesc.from_buffer_copy(self._bytes)

    @classmethod
    def make(cls, npages, page_size, Hkv, d, dtype, page_table):
        """New pools (uninitialised) beside a page table."""
        shape, dev = (int(npages), int(page_size), int(Hkv), int(d)), page_table.device
        return cls(torch.empty(shape, dtype=dtype, device=dev),
                   torch.empty(shape, dtype=dtype, device=dev), page_table)


def kv_append(cache: KVCache, K, V, lens=None, rope=None, Q=None, Q_out=None, cu_seqlens=None):
    """Writes new keys (rotated by `rope`, a Rope, if given) and values [ntok, Hkv, d] into
    their pages, behind the lens[s] tokens (int32 on the device; None: 0) that sequence s
    holds; rotates the same tokens' queries Q [ntok, Hq, d] and returns them (None
    without Q).  cu_seqlens [nseq + 1]: the new tokens of every sequence; None: one each.
    The rows of a padding sequence, marked by a negative length, and of tokens past
    cu_seqlens[nseq] are left as they were.  A token without a page is not written and is
    reported by sync_status.  `lens` itself is not changed."""
    f = _fast or _load_fast()
    r = f.kv_append(cache._addr, cache._device, K, V, lens, None if rope is None else rope._addr,
                    None if rope is None else rope._args[0], Q, Q_out, cu_seqlens)
    if r is not None:
        return None if r is True else _made(r)
    _require(K.dim() == 3, "K must be [ntok, Hkv, d]")
    ntok, dt, d = K.shape[0], cache.K.dtype, cache.d
    _batch(ntok, lens, cu_seqlens)
    _rows("K", K, ntok, cache.Hkv, d, dt)
    _rows("V", V, ntok, cache.Hkv, d, dt)
    if Q is not None:
        _require(Q.dim() == 3 and Q.shape[1] > 0, "Q must be [ntok, Hq, d]")
        for name, t in (("Q", Q), ("Q_out", Q_out)):
            if t is not None:
                _rows(name, t, ntok, Q.shape[1], d, dt)
    else:
        _require(Q_out is None, "Q_out without Q")
    _refuse_the_rest(*cache._args, K, V, lens, Q, Q_out, cu_seqlens,
                     None if rope is None else rope.phases)


def paged_attn(cache: KVCache, Q, lens, len_add=0, scale=None, band_bias=0.0, band_width=0,
               window=0, O=None, lse=None, workspace=None):
    """Attention of one new token per sequence, Q [nseq, Hq, d], over the lens[s] + len_add
    tokens (int32 on the device) that sequence s holds in `cache`, the new one among them:
    O [nseq, Hq, d] and the log-sum-exp [Hq, nseq] float32.

    scale: 1/sqrt(d) by default; band_bias within band_width tokens, as the sender's
    logits; window: keys more than window - 1 tokens back are masked (0: none).
    `workspace` may be a uint8 device tensor reused across calls (one per call in flight), of
    256 bytes more than mf_paged_attn_workspace; with less, or without, the call allocates.
    Several new tokens of a sequence: a cache whose page table repeats the sequence's row once
    a token, and each token's own length."""
    if scale is None:
        scale = cache.d ** -0.5
    f = _fast or _load_fast()
    r = f.paged_attn(cache._addr, cache._device, Q, lens, O, lse, workspace, len_add, scale,
                     band_bias, band_width, window)
    if r is not None:
        return _made(r)
    nseq, d, dt = cache.nseq, cache.d, cache.K.dtype
    for name, x in (("len_add", len_add), ("band_width", band_width), ("window", window)):
        _require(-2 ** 31 <= x < 2 ** 31, f"{name} must fit in 32 bits")
    _require(Q.dim() == 3, "Q must be [nseq, Hq, d]")
    Hq = Q.shape[1]
    _rows("Q", Q, nseq, Hq, d, dt)
    _index("lens", lens, nseq)
    if O is not None:
        _rows("O", O, nseq, Hq, d, dt)
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (Hq, nseq)
                            or not lse.is_contiguous()):
        _refuse("lse must be a contiguous float32 tensor [Hq, nseq]")
    L, c = load_library(), cache._desc
    a = PagedAttnDesc(Hq, scale, band_bias, band_width, window, len_add)
    if L.mf_paged_attn_workspace(C.byref(c), C.byref(a)) == 0:  # says what is wrong, as the call
        _check(L.mf_paged_attn(C.byref(c), C.byref(a), None, None, 0, None, 0, None, None, 0, None))
    if workspace is not None:
        _require(workspace.dtype == torch.uint8 and workspace.is_contiguous(),
                 "workspace must be a contiguous uint8 tensor")
    _refuse_the_rest(*cache._args, Q, lens, O, lse, workspace)


def mapped_av_plan(Hs, Hr, Hkv):
    """The fused kernel's shared-memory plan for a shape (host only): dict."""
    out = np.zeros(8, dtype=np.int32)
    _check(load_library().mf_mapped_av_plan(int(Hs), int(Hr), int(Hkv), out.ctypes.data))
    keys = ("groups_per_stage", "map_stages", "v_stages", "smem_bytes", "off_map", "off_mt",
            "off_w", "off_bar")
    return dict(zip(keys, (int(v) for v in out)))


MF_PATH_STATS_TC, MF_PATH_EXTRACT_TC, MF_PATH_AV_TC = 1, 2, 4


def path_info(ctx: Context, Hr=None, Hkv=None):
    """Which kernels the three calls run for a shape (host only): dict of
    bools for the statistics, extraction and fused stages."""
    d = ctx.desc()
    vd = None
    if Hr is not None:
        vd = VDesc(0, 0, 16, 0, 0, int(Hkv), ctx.d)
    f = C.c_uint32()
    _check(load_library().mf_path_info(C.byref(d), int(Hr or 0),
                                       None if vd is None else C.byref(vd), C.byref(f)))
    return {"stats_tc": bool(f.value & MF_PATH_STATS_TC),
            "extract_tc": bool(f.value & MF_PATH_EXTRACT_TC),
            "mapped_av_tc": bool(f.value & MF_PATH_AV_TC)}


def exp2_fma_eval(x):
    """2^x by the statistics kernel's FMA-pipe exponential (float32 CUDA tensor)."""
    L = load_library()
    if x.dtype != torch.float32 or not x.is_cuda:
        _check(MF_ERR_INVALID_ARG)
    x = x.contiguous()
    y = torch.empty_like(x)
    _check(L.mf_exp2_fma_eval(_ptr(x), _ptr(y), x.numel(), _stream()))
    return y


def selftest_timeout(limit_ms=20):
    """Make one bounded device wait give up (nothing completes its barrier)."""
    _check(load_library().mf_selftest_timeout(int(limit_ms), _stream()))


def sync_status():
    """Wait for the current stream; raise on a device-side status."""
    _check(load_library().mf_sync_status(_stream()))


def prefix_hash(tokens, B, seed=0):
    """Chained 128-bit per-block prefix hashes, uint64 [ceil(n/B), 2]."""
    L = load_library()
    t = np.ascontiguousarray(tokens, dtype=np.int32)
    nb = (len(t) + B - 1) // B
    out = np.zeros((max(nb, 1), 2), dtype=np.uint64)
    _check(L.mf_prefix_hash(t.ctypes.data if len(t) else None, len(t), B, C.c_uint64(seed),
                            out.ctypes.data))
    return out[:nb]


class PrefixIndex:
    """Host prefix-hash index of cache descriptors (C ABI object)."""

    def __init__(self):
        self._L = load_library()
        h = C.c_void_p()
        _check(self._L.mf_index_create(C.byref(h)))
        self._h = h

    def close(self):
        if self._h:
            self._L.mf_index_destroy(self._h)
            self._h = None

    __del__ = close

    def __len__(self):
        return int(self._L.mf_index_size(self._h))

    def insert(self, hashes, sender_layer, seq, cache_struct: CsrCache):
        h = np.ascontiguousarray(hashes, dtype=np.uint64)
        _check(self._L.mf_index_insert(self._h, h.ctypes.data, len(h), sender_layer, seq,
                                       C.byref(cache_struct)))

    def lookup(self, hashes, sender_layer):
        """(CsrCache, seq, matched_blocks) or None when nothing matches."""
        h = np.ascontiguousarray(hashes, dtype=np.uint64)
        out = CsrCache()
        seq, matched = C.c_int32(), C.c_int64()
        st = self._L.mf_index_lookup(self._h, h.ctypes.data if len(h) else None, len(h),
                                     sender_layer, C.byref(out), C.byref(seq),
                                     C.byref(matched))
        if st == MF_ERR_NOT_FOUND:
            return None
        _check(st)
        return out, seq.value, matched.value
