"""Thin Python binding of libhyb (include/hyb.h): argument marshalling only.

Every step of the product runs in the CUDA library; PyTorch provides device
memory and the current stream.  Function names follow the C ABI without the
``hyb_`` prefix.  bf16 tensors cross as their raw 16-bit patterns.

If ``libhyb.so`` is missing the first call raises; there is no fallback.

The 8-bit operators (quant_fp8, matmul_fp8, cache_append, cache_attention) are
also bound in C++ (``_hyb_torch.so``), which serves their ordinary calls -- a
workspace given, the current device and stream -- in a third of the time; other
calls, and those with an argument at fault, take the Python code below.
"""
import contextlib
import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhyb.so")

HYB_OK = 0
HYB_ERR_INVALID_ARG = -1
HYB_ERR_UNSUPPORTED = -2
HYB_ERR_ALIGNMENT = -3
HYB_ERR_WORKSPACE = -4
HYB_ERR_CUDA = -5
HYB_ERR_DEVICE_CHECK = -6
HYB_ERR_TIMEOUT = -7

HYB_F32 = 0
HYB_BF16 = 1
HYB_E4M3 = 2
HYB_I8 = 3
LAUNCH_OVERLAP_PREV = 1  # HYB_LAUNCH_OVERLAP_PREV

STATUS_NAN = 1
STATUS_BAD_MAP = 2
STATUS_TIMEOUT = 4
STATUS_BAD_SEQ = 8

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_SZ = ctypes.c_size_t


class HybMatrix(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("b1", ctypes.c_int32), ("b2", ctypes.c_int32),
                ("num_tiles", ctypes.c_int64),
                ("tile_map", _P), ("vals", _P), ("meta", _P),
                ("val_off", _P), ("meta_off", _P),
                ("n_vals", ctypes.c_int64), ("n_meta_bytes", ctypes.c_int64),
                ("plan", _P), ("plan_ctas", ctypes.c_int32)]


class HybLowrank(ctypes.Structure):
    _fields_ = [("rank", ctypes.c_int32), ("U", _P), ("ldu", ctypes.c_int64),
                ("V", _P), ("ldv", ctypes.c_int64)]


class HybFp8Matrix(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("k", ctypes.c_int64), ("q", _P), ("ldq", ctypes.c_int64),
                ("scale", _P), ("lds", ctypes.c_int64)]


class HybCache(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P),
                ("type", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("stride_page", ctypes.c_int64),
                ("stride_head", ctypes.c_int64), ("stride_token", ctypes.c_int64)]


class HybSequences(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("lens", _P), ("off", _P), ("page_table", _P),
                ("max_pages", ctypes.c_int32), ("table_stride", ctypes.c_int64)]


class HybError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} ({status})")


_lib = None

EXPORTS = ["hyb_packed_sizes", "hyb_pack_workspace_bytes", "hyb_pack",
           "hyb_workspace_bytes", "hyb_workspace_init", "hyb_spmv",
           "hyb_spmm_skinny", "hyb_lowrank_workspace_bytes", "hyb_lowrank_add",
           "hyb_dense_workspace_bytes", "hyb_gemv_dense", "hyb_check_status",
           "hyb_status_string", "hyb_spmv_noalloc", "hyb_spmv_noalloc_max_scratch_bytes",
           "hyb_spmv_noalloc_check_status", "hyb_gate_up_workspace_bytes",
           "hyb_spmm_skinny_gate_up", "hyb_prefill_workspace_bytes", "hyb_spmm_prefill",
           "hyb_prefill_block_shape", "hyb_spmm_prefill_blocked", "hyb_shard_bands",
           "hyb_plan_entries", "hyb_make_plan", "hyb_selftest_wait_timeout",
           "hyb_spmm_skinny_ex", "hyb_gemv_dense_ex", "hyb_packed_sizes_nm",
           "hyb_pack_nm", "hyb_spmm_skinny_nm", "hyb_fp8_quant_workspace_bytes",
           "hyb_fp8_quant", "hyb_fp8_workspace_bytes", "hyb_fp8_matmul",
           "hyb_cache_append_workspace_bytes", "hyb_cache_append",
           "hyb_cache_attention_workspace_bytes", "hyb_cache_attention"]


def lib():
    """Load libhyb.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libhyb.so not built ({LIB_PATH}); run "
                           "`python -m sparse_weight_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    L.hyb_packed_sizes.argtypes = [_I64, _I64, _I, _I, _P, _P, _P]
    L.hyb_packed_sizes.restype = _I
    L.hyb_pack_workspace_bytes.argtypes = []
    L.hyb_pack_workspace_bytes.restype = _SZ
    L.hyb_pack.argtypes = [_I64, _I64, _I, _I, _P, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P]
    L.hyb_pack.restype = _I
    L.hyb_workspace_bytes.argtypes = [ctypes.POINTER(HybMatrix), _I, _I]
    L.hyb_workspace_bytes.restype = _SZ
    L.hyb_workspace_init.argtypes = [_P, _SZ, _P]
    L.hyb_workspace_init.restype = _I
    L.hyb_spmv.argtypes = [ctypes.POINTER(HybMatrix), _P, _I64, _P, _I64, _I,
                           ctypes.POINTER(HybLowrank), _P, _SZ, _P]
    L.hyb_spmv.restype = _I
    L.hyb_spmm_skinny.argtypes = [ctypes.POINTER(HybMatrix), _I, _P, _I64, _P, _I64, _I,
                                  ctypes.POINTER(HybLowrank), _P, _SZ, _P]
    L.hyb_spmm_skinny.restype = _I
    L.hyb_spmm_skinny_ex.argtypes = [ctypes.POINTER(HybMatrix), _I, _P, _I64, _P, _I64, _I,
                                     ctypes.POINTER(HybLowrank), ctypes.c_uint32, _P, _SZ, _P]
    L.hyb_spmm_skinny_ex.restype = _I
    L.hyb_gate_up_workspace_bytes.argtypes = [ctypes.POINTER(HybMatrix), ctypes.POINTER(HybMatrix),
                                              _I, _I]
    L.hyb_gate_up_workspace_bytes.restype = _SZ
    L.hyb_spmm_skinny_gate_up.argtypes = [ctypes.POINTER(HybMatrix), ctypes.POINTER(HybMatrix), _I,
                                          _P, _I64, _P, _I64, _P, _I64, _I,
                                          ctypes.POINTER(HybLowrank), _P, _I64, ctypes.c_uint32,
                                          _P, _SZ, _P]
    L.hyb_spmm_skinny_gate_up.restype = _I
    L.hyb_shard_bands.argtypes = [_I64, _I64, _I, _I, _P, _I, _I, ctypes.POINTER(ctypes.c_int64),
                                  ctypes.POINTER(ctypes.c_int64)]
    L.hyb_shard_bands.restype = _I
    L.hyb_prefill_workspace_bytes.argtypes = []
    L.hyb_prefill_workspace_bytes.restype = _SZ
    L.hyb_spmm_prefill.argtypes = [ctypes.POINTER(HybMatrix), _I64, _P, _I64, _P, _I64, _P, _SZ,
                                   _P]
    L.hyb_spmm_prefill.restype = _I
    L.hyb_prefill_block_shape.argtypes = [_I64, _I64, ctypes.POINTER(_I), ctypes.POINTER(_I)]
    L.hyb_prefill_block_shape.restype = _I
    L.hyb_spmm_prefill_blocked.argtypes = [ctypes.POINTER(HybMatrix), _I64, _P, _I64, _P, _I64,
                                           _I, _I, _P, _SZ, _P]
    L.hyb_spmm_prefill_blocked.restype = _I
    L.hyb_lowrank_workspace_bytes.argtypes = [_I64, _I, _I]
    L.hyb_lowrank_workspace_bytes.restype = _SZ
    L.hyb_lowrank_add.argtypes = [_I64, _I64, _I, ctypes.POINTER(HybLowrank), _P, _I64,
                                  _P, _I64, _P, _SZ, _P]
    L.hyb_lowrank_add.restype = _I
    L.hyb_dense_workspace_bytes.argtypes = [_I64, _I64, _I]
    L.hyb_dense_workspace_bytes.restype = _SZ
    L.hyb_gemv_dense.argtypes = [_I64, _I64, _I, _P, _I64, _P, _I64, _P, _I64, _I, _P,
                                 _SZ, _P]
    L.hyb_gemv_dense.restype = _I
    L.hyb_gemv_dense_ex.argtypes = [_I64, _I64, _I, _P, _I64, _P, _I64, _P, _I64, _I,
                                    ctypes.c_uint32, _P, _SZ, _P]
    L.hyb_gemv_dense_ex.restype = _I
    L.hyb_check_status.argtypes = [_P, _P, ctypes.POINTER(ctypes.c_uint32)]
    L.hyb_check_status.restype = _I
    L.hyb_selftest_wait_timeout.argtypes = [_P, _SZ, ctypes.c_uint32, _P]
    L.hyb_selftest_wait_timeout.restype = _I
    L.hyb_spmv_noalloc.argtypes = [ctypes.POINTER(HybMatrix), _P, _I64, _P, _I64, _I, _P]
    L.hyb_spmv_noalloc.restype = _I
    L.hyb_spmv_noalloc_max_scratch_bytes.argtypes = []
    L.hyb_spmv_noalloc_max_scratch_bytes.restype = _SZ
    L.hyb_spmv_noalloc_check_status.argtypes = [_P, ctypes.POINTER(ctypes.c_uint32)]
    L.hyb_spmv_noalloc_check_status.restype = _I
    L.hyb_plan_entries.argtypes = []
    L.hyb_plan_entries.restype = _SZ
    L.hyb_make_plan.argtypes = [ctypes.POINTER(HybMatrix), _P, _P, ctypes.POINTER(ctypes.c_int32),
                                _P]
    L.hyb_make_plan.restype = _I
    L.hyb_packed_sizes_nm.argtypes = [_I64, _I64, _I, _I, _I, _I, _P, _P, _P]
    L.hyb_packed_sizes_nm.restype = _I
    L.hyb_pack_nm.argtypes = [_I64, _I64, _I, _I, _I, _I, _P, _I64, _P, _P, _P, _P, _P, _P,
                              _SZ, _P]
    L.hyb_pack_nm.restype = _I
    L.hyb_spmm_skinny_nm.argtypes = [ctypes.POINTER(HybMatrix), _I, _I, _I, _P, _I64, _P,
                                     _I64, _I, _P, _SZ, _P]
    L.hyb_spmm_skinny_nm.restype = _I
    L.hyb_fp8_quant_workspace_bytes.argtypes = []
    L.hyb_fp8_quant_workspace_bytes.restype = _SZ
    L.hyb_fp8_quant.argtypes = [_I64, _I64, _P, _I64, _I, _I, _P, _I64, _P, _I64, _P, _SZ, _P]
    L.hyb_fp8_quant.restype = _I
    L.hyb_fp8_workspace_bytes.argtypes = [_I64, _I64, _I64]
    L.hyb_fp8_workspace_bytes.restype = _SZ
    L.hyb_fp8_matmul.argtypes = [ctypes.POINTER(HybFp8Matrix), _I64, _P, _I64, _I, _P, _I64, _P,
                                 _I64, _I, ctypes.c_uint32, _P, _SZ, _P]
    L.hyb_fp8_matmul.restype = _I
    L.hyb_cache_append_workspace_bytes.argtypes = []
    L.hyb_cache_append_workspace_bytes.restype = _SZ
    L.hyb_cache_append.argtypes = [ctypes.POINTER(HybCache), ctypes.POINTER(HybSequences), _P,
                                   _I64, _I64, _P, _I64, _I64, _P, _SZ, _P]
    L.hyb_cache_append.restype = _I
    L.hyb_cache_attention_workspace_bytes.argtypes = [ctypes.POINTER(HybCache), ctypes.c_int32,
                                                      ctypes.c_int32, ctypes.c_int32,
                                                      ctypes.c_int32]
    L.hyb_cache_attention_workspace_bytes.restype = _SZ
    L.hyb_cache_attention.argtypes = [ctypes.POINTER(HybCache), ctypes.POINTER(HybSequences), _P,
                                      _I64, _I64, _P, _I64, _I64, _P, _I64, ctypes.c_int32,
                                      ctypes.c_float, ctypes.c_int32, ctypes.c_int32, _P, _SZ,
                                      _P]
    L.hyb_cache_attention.restype = _I
    L.hyb_status_string.argtypes = [_I]
    L.hyb_status_string.restype = ctypes.c_char_p
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().hyb_status_string(int(status)).decode()


def _check(fn, rc):
    if rc != HYB_OK:
        raise HybError(fn, rc)


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _bits(t: torch.Tensor) -> torch.Tensor:
    """View a bf16 (or int16/uint16) tensor as its 16-bit patterns."""
    if t.dtype == torch.bfloat16:
        return t.view(torch.int16)
    if t.dtype in (torch.int16, torch.uint16):
        return t
    raise TypeError(f"expected bf16 data, got {t.dtype}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# ---------------------------------------------------------------------------
# format
# ---------------------------------------------------------------------------

def packed_sizes(n: int, k: int, b1: int, b2: int, tile_map) -> tuple:
    """(n_vals, n_meta_bytes) for a host tile map (numpy/torch CPU uint8)."""
    m = np.ascontiguousarray(np.asarray(tile_map.cpu() if torch.is_tensor(tile_map)
                                        else tile_map, dtype=np.uint8).reshape(-1))
    nv, nm = _I64(), _I64()
    _check("hyb_packed_sizes", lib().hyb_packed_sizes(
        n, k, b1, b2, m.ctypes.data_as(_P), ctypes.byref(nv), ctypes.byref(nm)))
    return nv.value, nm.value


@dataclass
class Packed:
    """A packed tile-hybrid matrix on the device (tensors own the memory)."""
    n: int
    k: int
    b1: int
    b2: int
    tile_map: torch.Tensor   # uint8 [T], device
    vals: torch.Tensor       # int16 [n_vals] (bf16 bits), device
    meta: torch.Tensor       # uint8 [max(n_meta, 1)], device
    val_off: torch.Tensor    # int64 [T+1], device
    meta_off: torch.Tensor   # int64 [T+1], device
    n_vals: int
    n_meta: int
    plan: Optional[torch.Tensor] = None  # int64 work split (hyb_make_plan), host, optional
    plan_ctas: int = 0

    @property
    def num_tiles(self) -> int:
        return self.tile_map.numel()

    def struct(self) -> HybMatrix:
        return HybMatrix(self.n, self.k, self.b1, self.b2, self.num_tiles,
                         self.tile_map.data_ptr(), self.vals.data_ptr(),
                         self.meta.data_ptr(), self.val_off.data_ptr(),
                         self.meta_off.data_ptr(), self.n_vals, self.n_meta,
                         None if self.plan is None else self.plan.data_ptr(),
                         self.plan_ctas if self.plan is not None else 0)

    def nbytes(self) -> int:
        """Packed bytes the product streams (values + masks)."""
        return 2 * self.n_vals + self.n_meta

    def clone(self) -> "Packed":
        return Packed(self.n, self.k, self.b1, self.b2, self.tile_map.clone(),
                      self.vals.clone(), self.meta.clone(), self.val_off.clone(),
                      self.meta_off.clone(), self.n_vals, self.n_meta,
                      None if self.plan is None else self.plan.clone(), self.plan_ctas)


def shard_bands(n: int, k: int, b1: int, b2: int, tile_map, world: int, rank: int):
    """hyb_shard_bands: the tile-row bands [begin, end) rank `rank` of `world`
    holds (host only)."""
    tm = tile_map.cpu().numpy() if torch.is_tensor(tile_map) else np.asarray(tile_map)
    tm = np.ascontiguousarray(tm, dtype=np.uint8).reshape(-1)
    lo, hi = ctypes.c_int64(0), ctypes.c_int64(0)
    _check("hyb_shard_bands", lib().hyb_shard_bands(n, k, b1, b2, tm.ctypes.data, world, rank,
                                                    ctypes.byref(lo), ctypes.byref(hi)))
    return lo.value, hi.value


def shard(A: "Packed", rank: int, world: int, plan: bool = True) -> Optional["Packed"]:
    """The rows of A that rank `rank` of `world` holds (hyb_shard_bands): its
    bands' slice of A's packed buffers (views), offsets rebased to the slice,
    and (with ``plan``, on a GPU) its own work split.  None when the rank
    holds no band."""
    r0, r1 = shard_bands(A.n, A.k, A.b1, A.b2, A.tile_map, world, rank)
    if r1 <= r0:
        return None
    tpr = A.k // A.b2
    t0, t1 = r0 * tpr, r1 * tpr
    vo, mo = A.val_off[t0:t1 + 1], A.meta_off[t0:t1 + 1]
    v0, v1, m0, m1 = int(vo[0]), int(vo[-1]), int(mo[0]), int(mo[-1])
    # a shard without 2:4 tiles still passes a valid, aligned mask pointer
    meta = A.meta[m0:m1] if m1 > m0 else torch.zeros(16, dtype=torch.uint8, device=A.meta.device)
    S = Packed((r1 - r0) * A.b1, A.k, A.b1, A.b2, A.tile_map[t0:t1], A.vals[v0:v1], meta,
               vo - v0, mo - m0, v1 - v0, m1 - m0)
    if plan and S.val_off.is_cuda:
        S.plan, S.plan_ctas = make_plan(S)
    return S


def pack_workspace_bytes() -> int:
    return int(lib().hyb_pack_workspace_bytes())


def workspace_init(ws: torch.Tensor, stream=None):
    _check("hyb_workspace_init", lib().hyb_workspace_init(_ptr(ws), ws.numel(), _stream(stream)))


def new_workspace(nbytes: int, device) -> torch.Tensor:
    """Zeroed device workspace (uint8), 256-byte aligned by the allocator."""
    ws = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws


def make_plan(A: "Packed", stream=None):
    """hyb_make_plan: the product's work split for A on the current device;
    returns (host int64 plan tensor, CTA count).  Synchronises the stream."""
    entries = int(lib().hyb_plan_entries())
    scratch = torch.empty(entries, dtype=torch.int64, device=A.val_off.device)
    plan = torch.zeros(entries, dtype=torch.int64)
    s = A.struct()
    s.plan = None
    ctas = ctypes.c_int32(0)
    _check("hyb_make_plan", lib().hyb_make_plan(ctypes.byref(s), _ptr(scratch), _ptr(plan),
                                                ctypes.byref(ctas), _stream(stream)))
    return plan, ctas.value


def pack(W: torch.Tensor, tile_map, b1: int, b2: int, ws: torch.Tensor = None,
         stream=None, check: bool = True, plan: bool = True) -> Packed:
    """hyb_pack: dense bf16 W [n][k] (device) + tile map -> Packed.

    With ``check`` the call synchronises and raises HybError on a NaN weight or
    a bad map byte (the pack itself is complete either way).  With ``plan`` the
    product's work split is made once here (hyb_make_plan)."""
    Wb = _bits(W)
    assert Wb.is_cuda and Wb.dim() == 2
    n, k = Wb.shape
    tm_host = tile_map.cpu().numpy() if torch.is_tensor(tile_map) else np.asarray(tile_map)
    tm_host = np.ascontiguousarray(tm_host, dtype=np.uint8).reshape(-1)
    nv, nm = packed_sizes(n, k, b1, b2, tm_host)
    dev = Wb.device
    tm = torch.from_numpy(tm_host).to(dev)
    T = tm.numel()
    vals = torch.empty(nv, dtype=torch.int16, device=dev)
    meta = torch.empty(max(nm, 1), dtype=torch.uint8, device=dev)
    vo = torch.empty(T + 1, dtype=torch.int64, device=dev)
    mo = torch.empty(T + 1, dtype=torch.int64, device=dev)
    own_ws = ws is None
    if own_ws:
        ws = new_workspace(pack_workspace_bytes(), dev)
    _check("hyb_pack", lib().hyb_pack(n, k, b1, b2, _ptr(Wb), Wb.stride(0), _ptr(tm),
                                      _ptr(vals), _ptr(meta), _ptr(vo), _ptr(mo),
                                      _ptr(ws), ws.numel(), _stream(stream)))
    if check:
        check_status(ws, stream)
    P = Packed(n, k, b1, b2, tm, vals, meta, vo, mo, nv, nm)
    if plan:
        P.plan, P.plan_ctas = make_plan(P, stream)
    return P


def packed_sizes_nm(n: int, k: int, b1: int, b2: int, nk: int, m: int, tile_map) -> tuple:
    """(n_vals, n_meta_bytes) of nk:m tiles for a host tile map."""
    mp = np.ascontiguousarray(np.asarray(tile_map.cpu() if torch.is_tensor(tile_map)
                                         else tile_map, dtype=np.uint8).reshape(-1))
    nv, nmb = _I64(), _I64()
    _check("hyb_packed_sizes_nm", lib().hyb_packed_sizes_nm(
        n, k, b1, b2, nk, m, mp.ctypes.data_as(_P), ctypes.byref(nv), ctypes.byref(nmb)))
    return nv.value, nmb.value


def pack_nm(W: torch.Tensor, tile_map, b1: int, b2: int, nk: int, m: int,
            ws: torch.Tensor = None, stream=None, check: bool = True,
            plan: bool = True) -> Packed:
    """hyb_pack_nm: dense bf16 W [n][k] (device) + tile map -> Packed with
    nk:m sparse tiles.  With ``plan``, 2:4 and 4:8 matrices (whose products run
    the streaming kernel) get their work split made once here."""
    Wb = _bits(W)
    assert Wb.is_cuda and Wb.dim() == 2
    n, k = Wb.shape
    tm_host = tile_map.cpu().numpy() if torch.is_tensor(tile_map) else np.asarray(tile_map)
    tm_host = np.ascontiguousarray(tm_host, dtype=np.uint8).reshape(-1)
    nv, nmb = packed_sizes_nm(n, k, b1, b2, nk, m, tm_host)
    dev = Wb.device
    tm = torch.from_numpy(tm_host).to(dev)
    T = tm.numel()
    vals = torch.empty(nv, dtype=torch.int16, device=dev)
    meta = torch.empty(max(nmb, 1), dtype=torch.uint8, device=dev)
    vo = torch.empty(T + 1, dtype=torch.int64, device=dev)
    mo = torch.empty(T + 1, dtype=torch.int64, device=dev)
    if ws is None:
        ws = new_workspace(pack_workspace_bytes(), dev)
    _check("hyb_pack_nm", lib().hyb_pack_nm(n, k, b1, b2, nk, m, _ptr(Wb), Wb.stride(0),
                                            _ptr(tm), _ptr(vals), _ptr(meta), _ptr(vo),
                                            _ptr(mo), _ptr(ws), ws.numel(), _stream(stream)))
    if check:
        check_status(ws, stream)
    P = Packed(n, k, b1, b2, tm, vals, meta, vo, mo, nv, nmb)
    if plan and (nk, m) in ((2, 4), (4, 8)):
        P.plan, P.plan_ctas = make_plan(P, stream)
    return P


def spmm_skinny_nm(A: Packed, X: torch.Tensor, nk: int, m: int, Y: torch.Tensor = None,
                   ydt: int = HYB_F32, ws: torch.Tensor = None, stream=None) -> torch.Tensor:
    """hyb_spmm_skinny_nm: Y[batch][n] = W_hat X for nk:m tiles; X bf16 [batch][k]."""
    Xb = _bits(X)
    if Xb.dim() == 1:
        Xb = Xb.view(1, -1)
    batch = Xb.shape[0]
    Y = _out(A.n, batch, ydt, Xb.device, Y)
    if ws is None:
        ws = new_workspace(workspace_bytes(A, batch), Xb.device)
    s = A.struct()
    _check("hyb_spmm_skinny_nm", lib().hyb_spmm_skinny_nm(
        ctypes.byref(s), nk, m, batch, _ptr(Xb), Xb.stride(0), _ptr(Y), Y.stride(0), ydt,
        _ptr(ws), ws.numel(), _stream(stream)))
    return Y


def selftest_wait_timeout(ws: torch.Tensor, wait_limit: int = 2000, stream=None):
    """hyb_selftest_wait_timeout: launch the failure-path self test (a bounded
    wait that can never complete); the next check_status reports the timeout."""
    _check("hyb_selftest_wait_timeout",
           lib().hyb_selftest_wait_timeout(_ptr(ws), ws.numel(), wait_limit, _stream(stream)))


def check_status(ws: torch.Tensor, stream=None) -> int:
    """hyb_check_status: sync, read + clear the status word; raise on a flag."""
    flags = ctypes.c_uint32(0)
    rc = lib().hyb_check_status(_ptr(ws), _stream(stream), ctypes.byref(flags))
    if rc != HYB_OK:
        err = HybError("hyb_check_status", rc)
        err.flags = flags.value
        raise err
    return flags.value


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

def workspace_bytes(A: Packed, batch: int = 1, rank: int = 0) -> int:
    s = A.struct()
    nbytes = int(lib().hyb_workspace_bytes(ctypes.byref(s), batch, rank))
    if nbytes == 0:
        raise HybError("hyb_workspace_bytes", HYB_ERR_INVALID_ARG)
    return nbytes


def _lowrank_struct(lowrank):
    if lowrank is None:
        return None, None
    U, V = (_bits(t) for t in lowrank)
    lr = HybLowrank(U.shape[1], U.data_ptr(), U.stride(0), V.data_ptr(), V.stride(0))
    return lr, (U, V)


def _out(n, batch, ydt, device, Y):
    if Y is not None:
        return Y
    dt = torch.float32 if ydt == HYB_F32 else torch.bfloat16
    return torch.empty(batch, n, dtype=dt, device=device)


def spmm_skinny(A: Packed, X: torch.Tensor, Y: torch.Tensor = None, ydt: int = HYB_F32,
                lowrank=None, ws: torch.Tensor = None, stream=None,
                flags: int = 0) -> torch.Tensor:
    """hyb_spmm_skinny_ex: Y[batch][n] = W_hat X (+ U (V^T X)); X bf16 [batch][k].
    flags: LAUNCH_OVERLAP_PREV lets the kernel start streaming A before the
    kernel queued ahead of it on the stream has finished (A must not be
    written by that kernel)."""
    Xb = _bits(X)
    if Xb.dim() == 1:
        Xb = Xb.view(1, -1)
    batch = Xb.shape[0]
    Y = _out(A.n, batch, ydt, Xb.device, Y)
    lr, keep = _lowrank_struct(lowrank)
    if ws is None:
        ws = new_workspace(workspace_bytes(A, batch, lr.rank if lr else 0), Xb.device)
    s = A.struct()
    _check("hyb_spmm_skinny_ex", lib().hyb_spmm_skinny_ex(
        ctypes.byref(s), batch, _ptr(Xb), Xb.stride(0), _ptr(Y), Y.stride(0), ydt,
        ctypes.byref(lr) if lr else None, flags, _ptr(ws), ws.numel(), _stream(stream)))
    return Y


def spmm_prefill(A: Packed, X: torch.Tensor, Y: torch.Tensor = None, ws: torch.Tensor = None,
                 stream=None, block=None) -> torch.Tensor:
    """hyb_spmm_prefill: Y[m][n] = W_hat X for m tokens (tensor cores); X bf16
    [m][k], Y fp32 [m][n].  block = (rows, tokens) calls
    hyb_spmm_prefill_blocked with that CTA shape."""
    Xb = _bits(X)
    m = Xb.shape[0]
    if Y is None:
        Y = torch.empty(m, A.n, dtype=torch.float32, device=Xb.device)
    if ws is None:
        ws = new_workspace(int(lib().hyb_prefill_workspace_bytes()), Xb.device)
    s = A.struct()
    if block is None:
        _check("hyb_spmm_prefill", lib().hyb_spmm_prefill(
            ctypes.byref(s), m, _ptr(Xb), Xb.stride(0), _ptr(Y), Y.stride(0), _ptr(ws),
            ws.numel(), _stream(stream)))
    else:
        _check("hyb_spmm_prefill_blocked", lib().hyb_spmm_prefill_blocked(
            ctypes.byref(s), m, _ptr(Xb), Xb.stride(0), _ptr(Y), Y.stride(0), block[0], block[1],
            _ptr(ws), ws.numel(), _stream(stream)))
    return Y


PREFILL_SHAPES = ((128, 128), (128, 256), (256, 240), (256, 208))


def prefill_block_shape(n: int, m: int):
    """hyb_prefill_block_shape: the (rows, tokens) CTA shape hyb_spmm_prefill takes."""
    r, t = ctypes.c_int(0), ctypes.c_int(0)
    _check("hyb_prefill_block_shape",
           lib().hyb_prefill_block_shape(n, m, ctypes.byref(r), ctypes.byref(t)))
    return r.value, t.value


def gate_up_workspace_bytes(Ag: Packed, Au: Packed, batch: int, rank: int) -> int:
    sg, su = Ag.struct(), Au.struct()
    return int(lib().hyb_gate_up_workspace_bytes(ctypes.byref(sg), ctypes.byref(su), batch, rank))


def spmm_skinny_gate_up(Ag: Packed, Au: Packed, X: torch.Tensor, Ug: torch.Tensor,
                        Uu: torch.Tensor, V: torch.Tensor, ydt: int = HYB_F32,
                        ws: torch.Tensor = None, stream=None, flags: int = 0):
    """hyb_spmm_skinny_gate_up: (Yg, Yu) = (Ag X + Ug (V^T X), Au X + Uu (V^T X))
    with V^T X computed once; X bf16 [batch][k]."""
    Xb = _bits(X)
    if Xb.dim() == 1:
        Xb = Xb.view(1, -1)
    batch = Xb.shape[0]
    Yg = _out(Ag.n, batch, ydt, Xb.device, None)
    Yu = _out(Au.n, batch, ydt, Xb.device, None)
    lr, keep = _lowrank_struct((Ug, V))
    Uub = _bits(Uu)
    if ws is None:
        ws = new_workspace(gate_up_workspace_bytes(Ag, Au, batch, lr.rank), Xb.device)
    sg, su = Ag.struct(), Au.struct()
    _check("hyb_spmm_skinny_gate_up", lib().hyb_spmm_skinny_gate_up(
        ctypes.byref(sg), ctypes.byref(su), batch, _ptr(Xb), Xb.stride(0), _ptr(Yg),
        Yg.stride(0), _ptr(Yu), Yu.stride(0), ydt, ctypes.byref(lr), _ptr(Uub), Uub.stride(0),
        flags, _ptr(ws), ws.numel(), _stream(stream)))
    return Yg, Yu


def spmv(A: Packed, x: torch.Tensor, y: torch.Tensor = None, ydt: int = HYB_F32,
         lowrank=None, ws: torch.Tensor = None, stream=None) -> torch.Tensor:
    """hyb_spmv: y[1][n] = W_hat x (+ U (V^T x)); x bf16 [k] or [1][k]."""
    xb = _bits(x).reshape(1, -1)
    y = _out(A.n, 1, ydt, xb.device, y)
    lr, keep = _lowrank_struct(lowrank)
    if ws is None:
        ws = new_workspace(workspace_bytes(A, 1, lr.rank if lr else 0), xb.device)
    s = A.struct()
    _check("hyb_spmv", lib().hyb_spmv(
        ctypes.byref(s), _ptr(xb), xb.stride(0), _ptr(y), y.stride(0), ydt,
        ctypes.byref(lr) if lr else None, _ptr(ws), ws.numel(), _stream(stream)))
    return y


def lowrank_workspace_bytes(k: int, batch: int, rank: int) -> int:
    return int(lib().hyb_lowrank_workspace_bytes(k, batch, rank))


def lowrank_add(U: torch.Tensor, V: torch.Tensor, X: torch.Tensor, Y: torch.Tensor,
                ws: torch.Tensor = None, stream=None) -> torch.Tensor:
    """hyb_lowrank_add: Y (fp32 [batch][n]) += U (V^T X), in place."""
    Xb = _bits(X)
    if Xb.dim() == 1:
        Xb = Xb.view(1, -1)
    batch, k = Xb.shape
    n = Y.shape[-1]
    lr, keep = _lowrank_struct((U, V))
    if ws is None:
        ws = new_workspace(lowrank_workspace_bytes(k, batch, lr.rank), Xb.device)
    _check("hyb_lowrank_add", lib().hyb_lowrank_add(
        n, k, batch, ctypes.byref(lr), _ptr(Xb), Xb.stride(0), _ptr(Y), Y.stride(0),
        _ptr(ws), ws.numel(), _stream(stream)))
    return Y


def dense_workspace_bytes(n: int, k: int, batch: int = 1) -> int:
    return int(lib().hyb_dense_workspace_bytes(n, k, batch))


def gemv_dense(W: torch.Tensor, X: torch.Tensor, Y: torch.Tensor = None,
               ydt: int = HYB_F32, ws: torch.Tensor = None, stream=None,
               flags: int = 0) -> torch.Tensor:
    """hyb_gemv_dense_ex: Y[batch][n] = W X for a plain row-major bf16 W [n][k]
    (flags as for spmm_skinny)."""
    Wb = _bits(W)
    Xb = _bits(X)
    if Xb.dim() == 1:
        Xb = Xb.view(1, -1)
    n, k = Wb.shape
    batch = Xb.shape[0]
    Y = _out(n, batch, ydt, Xb.device, Y)
    if ws is None:
        ws = new_workspace(dense_workspace_bytes(n, k, batch), Xb.device)
    _check("hyb_gemv_dense_ex", lib().hyb_gemv_dense_ex(
        n, k, batch, _ptr(Wb), Wb.stride(0), _ptr(Xb), Xb.stride(0), _ptr(Y), Y.stride(0),
        ydt, flags, _ptr(ws), ws.numel(), _stream(stream)))
    return Y


def spmv_noalloc(A: Packed, x: torch.Tensor, y: torch.Tensor = None, ydt: int = HYB_F32,
                 stream=None) -> torch.Tensor:
    """hyb_spmv_noalloc: hyb_spmv (batch 1, no low-rank term) without a caller
    workspace; the library's own static device array holds the scratch, so the
    call allocates nothing (``y`` may be passed in to avoid the output
    allocation here too).  Make the first call on a device outside any stream
    capture, and do not let two calls overlap on the GPU."""
    xb = _bits(x).reshape(1, -1)
    y = _out(A.n, 1, ydt, xb.device, y)
    s = A.struct()
    _check("hyb_spmv_noalloc", lib().hyb_spmv_noalloc(
        ctypes.byref(s), _ptr(xb), xb.stride(0), _ptr(y), y.stride(0), ydt, _stream(stream)))
    return y


def spmv_noalloc_max_scratch_bytes() -> int:
    return int(lib().hyb_spmv_noalloc_max_scratch_bytes())


def spmv_noalloc_check_status(stream=None) -> int:
    """hyb_spmv_noalloc_check_status: sync, read + clear the status word of the
    static array behind hyb_spmv_noalloc; raise on a flag."""
    flags = ctypes.c_uint32(0)
    rc = lib().hyb_spmv_noalloc_check_status(_stream(stream), ctypes.byref(flags))
    if rc != HYB_OK:
        err = HybError("hyb_spmv_noalloc_check_status", rc)
        err.flags = flags.value
        raise err
    return flags.value


# ---------------------------------------------------------------------------
# 8-bit floating-point weights
# ---------------------------------------------------------------------------

_NO_SCOPE = contextlib.nullcontext()
# the current stream's handle without a Stream object around it (3 us less per call)
_raw_stream = torch._C._cuda_getCurrentRawStream


def _scope(index, stream):
    """Make device ``index`` current and ``stream`` (or the device's current
    stream) the one that new tensors belong to; returns (stream handle,
    context).  Outputs and workspaces made inside a call are then allocated in
    the order of the stream that uses them."""
    if stream is not None:
        if stream.device_index != index:
            raise ValueError(f"stream of device {stream.device_index}, tensors on device {index}")
        return stream.cuda_stream, torch.cuda.stream(stream)
    if index == torch._C._cuda_getDevice():
        return _raw_stream(index), _NO_SCOPE
    return _raw_stream(index), torch.cuda.device(index)


def _device_of(fn, first, *tensors):
    """The index of the CUDA device that every tensor lives on."""
    index = first.get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"{fn}: tensors on {first.device} and {t.device}")
    if index < 0:
        raise ValueError(f"{fn}: tensors must live on a CUDA device")
    return index


def _want(fn, ok, what):
    if not ok:
        raise ValueError(f"{fn}: {what}")


def _int32(fn, names, *values):
    """Refuse what a 32-bit field would cut off without a word."""
    if min(values) < -1 << 31 or max(values) >= 1 << 31:
        raise ValueError(f"{fn}: one of {names} = {values} does not fit 32 bits")


_native = None


def _load_native():
    """The C++ binding of the 8-bit operators (raises if it has not been built)."""
    global _native
    lib()
    path = os.path.join(_HERE, "_hyb_torch.so")
    if not os.path.exists(path):
        raise RuntimeError(f"_hyb_torch.so not built ({path}); run "
                           "`python -m sparse_weight_b200.build`")
    from . import _hyb_torch
    _native = _hyb_torch
    return _native


@dataclass(frozen=True)
class Fp8Matrix:
    """An e4m3 weight with one fp32 scale per 128 x 128 block, on the device.
    (Moving or cloning q packs its rows: where k is no multiple of 16 the copy
    has to be given padded rows again.)"""
    n: int
    k: int
    q: torch.Tensor      # float8_e4m3fn [n][k], rows a multiple of 16 bytes apart
    scale: torch.Tensor  # fp32 [ceil(n / 128)][ceil(k / 128)]

    def __post_init__(self):
        self.struct()
        # what the C++ binding reads, on every call anew
        object.__setattr__(self, "_at", (self.q, self.scale, self.n, self.k))

    def struct(self) -> HybFp8Matrix:
        """The C struct, from the tensors as they are now: a tensor keeps its
        identity when its storage is replaced (``.data``, a module moved)."""
        f, q, s, n, k = "Fp8Matrix", self.q, self.scale, self.n, self.k
        nb, kb = -(-n // 128), -(-k // 128)
        _want(f, q.dtype in (torch.float8_e4m3fn, torch.uint8), "q must be float8_e4m3fn")
        _want(f, s.dtype == torch.float32, "scale must be fp32")
        _want(f, q.shape == (n, k), "q must be [n][k]")
        _want(f, s.shape == (nb, kb), "scale must be [ceil(n / 128)][ceil(k / 128)]")
        (ldq, one), (lds, sone) = q.stride(), s.stride()
        _want(f, (k == 1 or one == 1) and (kb == 1 or sone == 1),
              "rows of q and scale must be contiguous")
        _want(f, (n == 1 or ldq >= k) and (nb == 1 or lds >= kb),
              "rows of q and scale must not overlap (an expanded tensor has to be copied)")
        # (a single row's stride says nothing: at least the row's length)
        return HybFp8Matrix(n, k, q.data_ptr(), ldq if n > 1 else -(-k // 16) * 16,
                            s.data_ptr(), max(lds, kb))

    _index = None  # (for the binding: its tensors' own device)

    def nbytes(self) -> int:
        """Bytes the product streams (values + scales)."""
        return self.n * self.k + 4 * self.scale.numel()


def fp8_quant_workspace_bytes() -> int:
    return int(lib().hyb_fp8_quant_workspace_bytes())


def quant_fp8(X: torch.Tensor, block_rows: int = 1, ws: torch.Tensor = None, stream=None):
    """hyb_fp8_quant: bf16 or fp32 X [rows][cols] -> (q float8_e4m3fn [rows][cols],
    scale fp32 [ceil(rows / block_rows)][ceil(cols / 128)]).  The rows of q lie a
    multiple of 16 bytes apart, as the products need them."""
    if ws is not None and stream is None:
        r = (_native or _load_native()).quant_fp8(X, block_rows, ws)
        if r is not None:
            if type(r) is int:
                raise HybError("hyb_fp8_quant", r)
            return r
    f = "quant_fp8"
    xdt = _QUANT_TYPES.get(X.dtype)
    if xdt is None or X.dim() != 2:
        raise ValueError(f"{f}: X must be bf16 or fp32 [rows][cols]")
    rows, cols = X.shape
    ldx, one = X.stride()
    if rows < 1 or cols < 1 or (one != 1 and cols > 1):
        raise ValueError(f"{f}: X must not be empty and its rows must be contiguous")
    if rows == 1:
        ldx = cols  # a single row's stride says nothing
    elif ldx < cols:
        raise ValueError(f"{f}: rows of X must not overlap "
                         "(an expanded tensor has to be copied)")
    if block_rows != 1 and block_rows != 128:
        raise ValueError(f"{f}: block_rows must be 1 or 128")
    index = _device_of(f, X, ws)
    handle, scope = _scope(index, stream)
    ld, cb = -(-cols // 16) * 16, -(-cols // 128)
    dev = X.device
    with scope:
        # (empty_strided: 1 us less per tensor than empty)
        q = torch.empty_strided((rows, cols), (ld, 1), dtype=torch.float8_e4m3fn, device=dev)
        s = torch.empty_strided((-(-rows // block_rows), cb), (cb, 1), dtype=torch.float32,
                                device=dev)
        if ws is None:
            ws = new_workspace(fp8_quant_workspace_bytes(), dev)
        rc = lib().hyb_fp8_quant(rows, cols, X.data_ptr(), ldx, xdt, block_rows,
                                 q.data_ptr(), ld, s.data_ptr(), cb, ws.data_ptr(),
                                 ws.numel(), handle)
    if rc:
        raise HybError("hyb_fp8_quant", rc)
    return q, s


_QUANT_TYPES = {torch.bfloat16: HYB_BF16, torch.float32: HYB_F32}


def pack_fp8(W: torch.Tensor, ws: torch.Tensor = None, stream=None,
             check: bool = True) -> Fp8Matrix:
    """A bf16 or fp32 weight W [n][k] as an Fp8Matrix (hyb_fp8_quant with
    128 x 128 blocks).  With ``check`` the call synchronises and raises HybError
    on a NaN or infinite weight."""
    if ws is None:
        with _scope(_device_of("pack_fp8", W), stream)[1]:
            ws = new_workspace(fp8_quant_workspace_bytes(), W.device)
    q, s = quant_fp8(W, 128, ws, stream)
    if check:
        check_status(ws, stream)
    return Fp8Matrix(W.shape[0], W.shape[1], q, s)


def fp8_workspace_bytes(m: int, n: int, k: int) -> int:
    nbytes = int(lib().hyb_fp8_workspace_bytes(m, n, k))
    if nbytes == 0:
        raise HybError("hyb_fp8_workspace_bytes", HYB_ERR_INVALID_ARG)
    return nbytes


def matmul_fp8(A: Fp8Matrix, X: torch.Tensor, xs: torch.Tensor = None, Y: torch.Tensor = None,
               ydt: int = HYB_F32, ws: torch.Tensor = None, stream=None,
               flags: int = 0) -> torch.Tensor:
    """hyb_fp8_matmul: Y[m][n] = W X for an e4m3 weight and any number of tokens.
    X is bf16 [m][k] (or [k]), quantised inside the call, or float8_e4m3fn with
    its scales xs (quant_fp8).  flags as for spmm_skinny."""
    if ws is not None and stream is None:
        r = (_native or _load_native()).matmul_fp8(A._at, A._index, X, xs, Y, ydt, flags, ws)
        if r is not None:
            if type(r) is int:
                raise HybError("hyb_fp8_matmul", r)
            return r
    f = "matmul_fp8"
    if X.dim() == 1:
        X = X.view(1, -1)
    n, k, a = A.n, A.k, A.struct()
    if X.dim() != 2 or X.shape[1] != k or X.shape[0] < 1:
        raise ValueError(f"{f}: X must be [m][k]")
    m = X.shape[0]
    ldx, one = X.stride()
    if one != 1 and k > 1:
        raise ValueError(f"{f}: rows of X must be contiguous")
    if xs is None:
        if X.dtype != torch.bfloat16:
            raise ValueError(f"{f}: X must be bf16, or e4m3 with xs")
        xdt, sp, lds = HYB_BF16, None, 0
    else:
        kb = -(-k // 128)
        if X.dtype != torch.float8_e4m3fn:
            raise ValueError(f"{f}: X with xs must be float8_e4m3fn")
        if xs.dtype != torch.float32 or xs.shape != (m, kb) or (xs.stride(1) != 1 and kb > 1):
            raise ValueError(f"{f}: xs must be fp32 [m][ceil(k / 128)]")
        xdt, sp, lds = HYB_E4M3, xs.data_ptr(), xs.stride(0) if m > 1 else kb
        if lds < kb:
            raise ValueError(f"{f}: rows of xs must not overlap "
                             "(an expanded tensor has to be copied)")
    if not 0 <= flags < 1 << 32:
        raise ValueError(f"{f}: flags = {flags} does not fit 32 bits")
    ytype = _OUT_TYPES.get(ydt)
    if ytype is None:
        raise ValueError(f"{f}: ydt must be HYB_F32 or HYB_BF16")
    if Y is not None and (Y.shape != (m, n) or (Y.stride(1) != 1 and n > 1) or Y.dtype != ytype):
        raise ValueError(f"{f}: Y must be [m][n] in ydt")
    index = _device_of(f, X, A.q, A.scale, xs, Y, ws)
    handle, scope = _scope(index, stream)
    with scope:
        if Y is None:
            Y = torch.empty_strided((m, n), (n, 1), dtype=ytype, device=X.device)
        if ws is None:
            ws = new_workspace(fp8_workspace_bytes(m, n, k), X.device)
        # a single row's stride says nothing
        rc = lib().hyb_fp8_matmul(ctypes.byref(a), m, X.data_ptr(), ldx if m > 1 else -(-k // 16) * 16, xdt,
                                  sp, lds, Y.data_ptr(), Y.stride(0) if m > 1 else n, ydt, flags,
                                  ws.data_ptr(), ws.numel(), handle)
    if rc:
        raise HybError("hyb_fp8_matmul", rc)
    return Y


_OUT_TYPES = {HYB_F32: torch.float32, HYB_BF16: torch.bfloat16}


# ---------------------------------------------------------------------------
# 8-bit key / value cache
# ---------------------------------------------------------------------------

@dataclass(frozen=True)
class Cache:
    """Keys and values in pages of 8-bit values with one scale per page and
    head (hyb_cache).  k, v: [num_pages][kv_heads][page_size][head_dim], any
    strides (multiples of 16) with head_dim contiguous."""
    k: torch.Tensor        # float8_e4m3fn or int8
    v: torch.Tensor
    k_scale: torch.Tensor  # fp32 [num_pages][kv_heads]
    v_scale: torch.Tensor

    def __post_init__(self):
        self.struct()
        # what the C++ binding reads, on every call anew
        object.__setattr__(self, "_at", (self.k, self.v, self.k_scale, self.v_scale))

    def struct(self) -> HybCache:
        """The C struct, from the tensors as they are now (see Fp8Matrix.struct)."""
        f, k, v, ks, vs = "Cache", self.k, self.v, self.k_scale, self.v_scale
        _want(f, k.dtype in (torch.float8_e4m3fn, torch.int8) and v.dtype == k.dtype,
              "k and v must both be float8_e4m3fn or both int8")
        shape, strides = k.shape, k.stride()
        _want(f, len(shape) == 4 and v.shape == shape and v.stride() == strides
              and strides[3] == 1,
              "k and v must be [pages][heads][tokens][dim] of the same strides, dim contiguous")
        pages, heads, size, dim = shape
        sp, sh, st, _ = strides
        _int32(f, "pages, heads, tokens, dim", *shape)
        _want(f, ks.dtype == vs.dtype == torch.float32 and ks.shape == vs.shape == (pages, heads)
              and ks.is_contiguous() and vs.is_contiguous(),
              "scales must be contiguous fp32 [pages][heads]")
        _want(f, k.get_device() == v.get_device() == ks.get_device() == vs.get_device(),
              "all tensors must live on one device")
        return HybCache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(),
                        HYB_I8 if k.dtype == torch.int8 else HYB_E4M3, pages, heads, size, dim,
                        sp, sh, st)

    _index = None  # (for the binding: its tensors' own device)

    @property
    def page_size(self) -> int:
        return self.k.shape[2]


def new_cache(num_pages: int, kv_heads: int, page_size: int, head_dim: int,
              dtype=torch.float8_e4m3fn, device="cuda") -> Cache:
    """An empty cache (zeros)."""
    kv = [torch.zeros(num_pages, kv_heads, page_size, head_dim, dtype=torch.uint8,
                      device=device).view(dtype) for _ in range(2)]
    sc = [torch.zeros(num_pages, kv_heads, device=device) for _ in range(2)]
    return Cache(kv[0], kv[1], sc[0], sc[1])


def _sequences(f, rows, page_table, lens, off, max_new):
    if page_table.dtype != torch.int32 or page_table.dim() != 2:
        raise ValueError(f"{f}: page_table must be int32 [batch][pages]")
    batch, pages = page_table.shape
    stride, one = page_table.stride()
    if one != 1 and pages > 1:
        raise ValueError(f"{f}: rows of page_table must be contiguous")
    if batch <= 1:
        stride = pages  # a single row's stride says nothing
    elif stride < pages:
        raise ValueError(f"{f}: rows of page_table must not overlap "
                         "(an expanded tensor has to be copied)")
    if lens.dtype != torch.int32 or lens.shape != (batch,) or not lens.is_contiguous():
        raise ValueError(f"{f}: lens must be int32 [batch]")
    at = None
    if off is None:
        if max_new is None and batch and rows % batch == 0:
            max_new = rows // batch
        if max_new is None or rows != batch * max_new:
            raise ValueError(f"{f}: without off every sequence has max_new rows")
    else:
        if off.dtype != torch.int32 or off.shape != (batch + 1,) or not off.is_contiguous():
            raise ValueError(f"{f}: off must be int32 [batch + 1]")
        if max_new is None:
            raise ValueError(f"{f}: off needs max_new")
        at = off.data_ptr()
    _int32(f, "batch, max_new, pages", batch, max_new, pages)
    return HybSequences(batch, max_new, rows, lens.data_ptr(), at, page_table.data_ptr(), pages,
                        stride)


def _heads(f, x, heads, dim, what):
    """(rows, heads, row stride, head stride) of bf16 rows [rows][heads][dim]."""
    if x.dtype == torch.bfloat16 and x.dim() == 3:
        rows, h, d = x.shape
        ld, hs, one = x.stride()
        if d == dim and (heads is None or h == heads) and one == 1:
            return rows, h, ld if rows > 1 else max(dim, h * dim), hs if h > 1 else dim
    raise ValueError(f"{f}: {what} must be bf16 [rows][heads][head_dim] with head_dim contiguous")


def cache_append_workspace_bytes() -> int:
    return int(lib().hyb_cache_append_workspace_bytes())


def cache_append(C: Cache, K: torch.Tensor, V: torch.Tensor, page_table: torch.Tensor,
                 lens: torch.Tensor, off: torch.Tensor = None, max_new: int = None,
                 ws: torch.Tensor = None, stream=None) -> None:
    """hyb_cache_append: store new keys and values (bf16 [rows][kv_heads][head_dim])
    as the last tokens of sequences whose lengths are ``lens`` with them.  off
    [batch + 1]: the sequences' rows (None: max_new rows each)."""
    if ws is not None and stream is None:
        r = (_native or _load_native()).cache_append(C._at, C._index, K, V, page_table, lens, off,
                                                     max_new, ws)
        if r is not None:
            if type(r) is int:
                raise HybError("hyb_cache_append", r)
            return
    f = "cache_append"
    c = C.struct()
    heads, dim = c.kv_heads, c.head_dim
    rows, _, ldk, hsk = _heads(f, K, heads, dim, "K")
    rows_v, _, ldv, hsv = _heads(f, V, heads, dim, "V")
    if rows != rows_v:
        raise ValueError(f"{f}: K and V must have the same rows")
    seq = _sequences(f, rows, page_table, lens, off, max_new)
    index = _device_of(f, C.k, K, V, page_table, lens, off, ws)
    if rows == 0:
        return
    handle, scope = _scope(index, stream)
    with scope:
        if ws is None:
            ws = new_workspace(cache_append_workspace_bytes(), C.k.device)
        rc = lib().hyb_cache_append(ctypes.byref(c), ctypes.byref(seq), K.data_ptr(), ldk, hsk,
                                    V.data_ptr(), ldv, hsv, ws.data_ptr(), ws.numel(), handle)
    if rc:
        raise HybError("hyb_cache_append", rc)


def cache_attention_workspace_bytes(C: Cache, batch: int, heads: int, max_new: int,
                                    max_len: int) -> int:
    """For sequences of up to max_len tokens (the page table's width times the
    page size) and max_new new ones."""
    c = C.struct()
    pages = -(-max_len // c.page_size)
    _int32("cache_attention_workspace_bytes", "batch, max_new, pages, heads", batch, max_new, pages,
           heads)
    n = int(lib().hyb_cache_attention_workspace_bytes(ctypes.byref(c), batch, max_new, pages, heads))
    if n == 0:
        raise HybError("hyb_cache_attention_workspace_bytes", HYB_ERR_INVALID_ARG)
    return n


def cache_attention(C: Cache, Q: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
                    off: torch.Tensor = None, max_new: int = None, scale: float = None,
                    window: int = 0, sinks: int = 0, out: torch.Tensor = None,
                    return_lse: bool = False, ws: torch.Tensor = None, stream=None):
    """hyb_cache_attention: the new tokens' queries (bf16 [rows][heads][head_dim])
    over the cache; causal, with a sliding window and first tokens that stay
    visible (sinks) where window > 0.  scale defaults to 1 / sqrt(head_dim).
    Returns O (bf16, as Q), with return_lse also the fp32 log-sum-exp
    [rows][heads]."""
    if ws is not None and stream is None:
        r = (_native or _load_native()).cache_attention(C._at, C._index, Q, page_table, lens, off,
                                                        max_new, scale, window, sinks, out,
                                                        return_lse, ws)
        if r is not None:
            if type(r) is int:
                raise HybError("hyb_cache_attention", r)
            return r
    f = "cache_attention"
    c = C.struct()
    dim = c.head_dim
    rows, heads, ldq, hsq = _heads(f, Q, None, dim, "Q")
    _int32(f, "heads, window, sinks", heads, window, sinks)
    seq = _sequences(f, rows, page_table, lens, off, max_new)
    index = _device_of(f, C.k, Q, page_table, lens, off, out, ws)
    if out is not None:
        out_rows, _, ldo, hso = _heads(f, out, heads, dim, "out")
        if out_rows != rows:
            raise ValueError(f"{f}: out must have Q's shape")
    else:
        ldo, hso = heads * dim, dim
    handle, scope = _scope(index, stream)
    dev = Q.device
    with scope:
        if out is None:
            out = torch.empty_strided((rows, heads, dim), (ldo, dim, 1), dtype=torch.bfloat16,
                                      device=dev)
        lse = torch.empty_strided((rows, heads), (heads, 1), dtype=torch.float32,
                                  device=dev) if return_lse else None
        rc = HYB_OK
        if rows:
            if ws is None:
                ws = new_workspace(cache_attention_workspace_bytes(
                    C, seq.batch, heads, seq.max_new, seq.max_pages * c.page_size), dev)
            rc = lib().hyb_cache_attention(
                ctypes.byref(c), ctypes.byref(seq), Q.data_ptr(), ldq, hsq, out.data_ptr(), ldo, hso,
                lse.data_ptr() if return_lse else None, heads, heads,
                dim ** -0.5 if scale is None else scale, window, sinks, ws.data_ptr(), ws.numel(),
                handle)
    if rc:
        raise HybError("hyb_cache_attention", rc)
    return (out, lse) if return_lse else out
