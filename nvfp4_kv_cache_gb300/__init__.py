"""Python binding of libmsa.so: the MSA decode step over a paged NVFP4 cache on GB300.

Argument marshalling only: every function forwards torch tensors' device pointers and the
current CUDA stream to the C ABI of the same name (include/msa.h), and raises MsaError on a
non-OK status. All arithmetic runs in the library's CUDA kernels. There is no fallback:
importing this package fails if libmsa.so has not been built (``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libmsa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libmsa.so is not built ({LIB_PATH}); run `python -c 'import __graft_entry__ as g; g.build()'`")

_lib = ctypes.CDLL(LIB_PATH)

MSA_OK = 0
MSA_ERR_INVALID_ARG = 1
MSA_ERR_UNSUPPORTED = 2
MSA_ERR_CUDA = 3
MSA_ERR_TIMEOUT = 4
MSA_ERR_DEVICE_FAULT = 5
MSA_INDEX_NVFP4 = 0
MSA_INDEX_FP8 = 1
MSA_HOST_STEP_DIRECT_OUT = 1
MSA_ROPE_HALF = 0
MSA_ROPE_INTERLEAVED = 1
MSA_ROPE_PLAIN = 0
MSA_ROPE_LINEAR = 1
MSA_ROPE_BY_PARTS = 2
MSA_ROPE_BY_TURNS = 3
MSA_F32 = 0
MSA_BF16 = 1
MSA_F16 = 2

HEAD_DIM = 128
GROUPS = 4
Q_HEADS = 64
BLOCK = 128
K_SEL = 16
INDEX_PAGE_BYTES = {MSA_INDEX_NVFP4: 9216, MSA_INDEX_FP8: 16384}
KV_PAGE_BYTES = 73728


class msa_geometry(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_q_heads", "num_kv_heads", "head_dim", "index_dim",
                                               "block_size", "topk", "local_blocks", "init_blocks")]


class msa_batch(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("query_start_loc", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("max_blocks_per_seq", ctypes.c_int32), ("max_q_len", ctypes.c_int32)]


class msa_cache(ctypes.Structure):
    _fields_ = [("kv_pages", ctypes.c_void_p), ("index_pages", ctypes.c_void_p), ("index_dtype", ctypes.c_int32),
                ("num_pages", ctypes.c_int32)]


class msa_host_step_io(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("query_start_loc", "seq_lens", "block_table", "q", "index_q", "out")]


class msa_rope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class msa_kv_rows(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("ik", ctypes.c_void_p), ("dtype", ctypes.c_int32)] + [
        (n, ctypes.c_int64) for n in ("k_token_stride", "k_head_stride", "v_token_stride", "v_head_stride",
                                      "ik_token_stride")]


GEOMETRY = msa_geometry(64, 4, 128, 128, 128, 16, 1, 0)
_GEO_REF = ctypes.byref(GEOMETRY)

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_GP = ctypes.POINTER(msa_geometry)
_BP = ctypes.POINTER(msa_batch)
_CP = ctypes.POINTER(msa_cache)
_HP = ctypes.POINTER(msa_host_step_io)
_RP = ctypes.POINTER(msa_rope)
_F32 = ctypes.c_float
_F64 = ctypes.c_double

_SIGS = {
    "msa_status_string": (ctypes.c_char_p, [_I32]),
    "msa_abi_version": (_I32, []),
    "msa_quantize_nvfp4": (_I32, [_P, _I64, _I32, _P, _I64, _P, _I64, _P]),
    "msa_quantize_fp8": (_I32, [_P, _I64, _P, _P]),
    "msa_dequant_nvfp4": (_I32, [_P, _I64, _P, _I64, _I64, _I32, _P, _P]),
    "msa_kv_insert": (_I32, [_P, _P, _P, _I64, _P, _P, _P, _I32, _I32, _P, _P]),
    "msa_rope_inv_freq": (_I32, [_I32, _F64, _I32, _F64, _F64, _F64, _F64, _P, _P]),
    "msa_rope_fp8": (_I32, [_P, _I32, _I32, _I32, _I64, _I64, _P, _RP, _P, _F32, _P, _P]),
    "msa_rope_kv_insert": (_I32, [ctypes.POINTER(msa_kv_rows), _I64, _P, _P, _RP, _P, _P, _F32, _P, _P, _I32, _I32,
                                  _P, _P]),
    "msa_kv_read": (_I32, [_P, _I64, _P, _P, _I32, _I32, _P, _P, _P, _P, _P]),
    "msa_dense_attn_workspace_size": (_SZ, [_GP, _I32, _I32, _I32]),
    "msa_dense_attn": (_I32, [_GP, _BP, _CP, _P, _F32, _P, _SZ, _P, _P, _P, _P]),
    "msa_indexer_decode": (_I32, [_GP, _BP, _CP, _P, _P, _P, _P]),
    "msa_topk_blocks": (_I32, [_GP, _BP, _P, _P, _P, _P]),
    "msa_indexer_decode_range": (_I32, [_GP, _BP, _CP, _P, _I32, _I32, _P, _P, _P]),
    "msa_indexer_decode_exact": (_I32, [_GP, _BP, _CP, _P, _P, _P, _P]),
    "msa_indexer_prefill": (_I32, [_GP, _BP, _CP, _P, _P, _P, _P]),
    "msa_topk_prefill": (_I32, [_GP, _BP, _P, _P, _P, _P]),
    "msa_prefill_workspace_size": (_SZ, [_GP, _I32, _I32, _I32]),
    "msa_prefill_attn": (_I32, [_GP, _BP, _CP, _P, _P, ctypes.c_float, _P, _SZ, _P, _P, _P]),
    "msa_topk_candidates": (_I32, [_GP, _BP, _P, _I32, _I32, _P, _P, _P]),
    "msa_topk_merge": (_I32, [_GP, _BP, _P, _I32, _P, _P, _P]),
    "msa_topk_candidates_host": (_I32, [_P, _I64, _I32, _P, _I32, _I32, _P]),
    "msa_topk_merge_host": (_I32, [_P, _I32, _I64, _P, _P]),
    "msa_kv_gather_map": (_I32, [_GP, _BP, _P, _P, _P, _P, _P, _P]),
    "msa_kv_gather_pages": (_I32, [_GP, _BP, _CP, _P, _P, _I32, _I32, _P, _I32, _P, _P]),
    "msa_kv_gather_map_host": (_I32, [_I32, _I32, _P, _P, _I32, _P, _P, _P]),
    "msa_kv_gather_pages_host": (_I32, [_I32, _I32, _P, _P, _I32, _P, _P, _I32, _I32, _P, _I32]),
    "msa_attn_workspace_size": (_SZ, [_GP, _I32, _I32, _I32]),
    "msa_sparse_attn_decode": (_I32, [_GP, _BP, _CP, _P, _P, ctypes.c_float, _I32, _P, _SZ, _P, _P, _P]),
    "msa_sparse_attn_decode_noalloc": (_I32, [_GP, _BP, _CP, _P, _P, ctypes.c_float, _I32, _P, _P, _P]),
    "msa_noalloc_scratch_bytes": (_SZ, []),
    "msa_decode_workspace_size": (_SZ, [_GP, _I32, _I32, _I32]),
    "msa_decode_step": (_I32, [_GP, _BP, _CP, _P, _P, ctypes.c_float, _P, _P, _P, _SZ, _P, _P]),
    "msa_decode_step_host": (_I32, [_GP, _BP, _CP, _HP, _P, _P, ctypes.c_float, _P, _SZ, _P, _I32, _P, _P]),
    "msa_read_device_status": (_I32, [_P, _P]),
    "msa_selftest_wait_timeout": (_I32, [_P, _I64, _P]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class MsaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {_lib.msa_status_string(code).decode()}")


def _check(code: int, where: str) -> None:
    if code != MSA_OK:
        raise MsaError(code, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream] = None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t: torch.Tensor, dtype, name: str) -> None:
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")


# The checks of the calls below: a few attribute reads a tensor, since a small call's host time is
# mostly theirs (bare ctypes call and launch: 3 us).
_ROW_DTYPES = {torch.float32: MSA_F32, torch.bfloat16: MSA_BF16, torch.float16: MSA_F16}
_U8, _INT32, _INT64, _FLOAT32 = torch.uint8, torch.int32, torch.int64, torch.float32
# torch's own bindings where it has them: current_stream().cuda_stream makes an object, 3 us more. A torch without
# CUDA has neither; the host-only entry points work there.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _at(t: Optional[torch.Tensor], dtype, numel: int, device: int, name: str):
    """The address of a contiguous `dtype` tensor of at least numel elements on the current device (None: null)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() < numel or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor of at least {numel} elements")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the call on cuda:{device}")
    return t.data_ptr()


def _one_device(*tensors: torch.Tensor) -> int:
    """The device that all of them are on, or -1."""
    devices = {t.get_device() for t in tensors}
    return devices.pop() if len(devices) == 1 else -1


def _status_at(t: Optional[torch.Tensor], device: int):
    """The address of a 32-bit status word on the current device (None: null)."""
    if t is None:
        return None
    if t.get_device() != device or t.element_size() != 4 or t.numel() < 1:
        raise ValueError(f"status must be a 32-bit tensor on cuda:{device}")
    return t.data_ptr()


def _rows_at(t: torch.Tensor, dims: int, device: int, name: str):
    """Address, type, shape and strides of projected rows: fp32, bf16 or fp16, 128 contiguous elements each, any
    other strides."""
    dt, shape, strides = _ROW_DTYPES.get(t.dtype), t.shape, t.stride()
    if dt is None or len(shape) != dims or shape[-1] != HEAD_DIM or strides[-1] != 1:
        raise ValueError(f"{name} must be a {dims}-d CUDA tensor of {HEAD_DIM}-element fp32, bf16 or fp16 rows")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the call on cuda:{device}")
    return t.data_ptr(), dt, shape, strides


# ------------------------------------------------------------------ descriptors ----------
class Batch:
    """Decode batch: device int32 tensors + the msa_batch struct (keeps the tensors alive)."""

    def __init__(self, query_start_loc: torch.Tensor, seq_lens: torch.Tensor, block_table: torch.Tensor,
                 max_q_len: int, T: Optional[int] = None):
        for n, t in (("query_start_loc", query_start_loc), ("seq_lens", seq_lens), ("block_table", block_table)):
            _need(t, torch.int32, n)
        self.query_start_loc, self.seq_lens, self.block_table = query_start_loc, seq_lens, block_table
        self.B = int(seq_lens.numel())
        self.T = int(T) if T is not None else int(query_start_loc[-1].item())
        self.max_blocks = int(block_table.shape[1]) if block_table.dim() == 2 else 1
        self.max_q_len = int(max_q_len)
        self.c = msa_batch(self.B, self.T, query_start_loc.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(),
                           self.max_blocks, self.max_q_len)
        self.ref = ctypes.byref(self.c)
        self.device = _one_device(query_start_loc, seq_lens, block_table)


class Cache:
    """One layer's paged caches (uint8 device tensors) + the msa_cache struct."""

    def __init__(self, kv_pages: torch.Tensor, index_pages: torch.Tensor, index_dtype: int, num_pages: int):
        _need(kv_pages, torch.uint8, "kv_pages")
        _need(index_pages, torch.uint8, "index_pages")
        self.kv_pages, self.index_pages = kv_pages, index_pages
        self.index_dtype, self.num_pages = int(index_dtype), int(num_pages)
        self.kv_at, self.index_at = kv_pages.data_ptr(), index_pages.data_ptr()
        self.c = msa_cache(self.kv_at, self.index_at, self.index_dtype, self.num_pages)
        self.ref = ctypes.byref(self.c)
        self.device = _one_device(kv_pages, index_pages)

    @staticmethod
    def empty(num_pages: int, index_dtype: int, device="cuda") -> "Cache":
        kv = torch.zeros(num_pages * KV_PAGE_BYTES, dtype=torch.uint8, device=device)
        ix = torch.zeros(num_pages * INDEX_PAGE_BYTES[index_dtype], dtype=torch.uint8, device=device)
        return Cache(kv, ix, index_dtype, num_pages)


class Rope:
    """Rotary positions: inv_freq (float64 CUDA tensor, rot_dim / 2 radians a position; None for no
    rotation) + the msa_rope struct (keeps the tensor alive). `frequencies` makes one of the
    usual scalings."""

    def __init__(self, inv_freq: Optional[torch.Tensor], layout: int = MSA_ROPE_HALF, scale: float = 1.0):
        if inv_freq is not None:
            _need(inv_freq, torch.float64, "inv_freq")
        self.inv_freq = inv_freq
        self.c = msa_rope(None if inv_freq is None else inv_freq.data_ptr(),
                          0 if inv_freq is None else 2 * inv_freq.numel(), int(layout), float(scale))
        self.ref = ctypes.byref(self.c)
        self.device = None if inv_freq is None else inv_freq.get_device()

    @staticmethod
    def frequencies(rot_dim: int, theta: float, kind: int = MSA_ROPE_PLAIN, factor: float = 1.0,
                    original_len: float = 0.0, slow: float = 1.0, fast: float = 32.0, layout: int = MSA_ROPE_HALF,
                    device="cuda") -> "Rope":
        freq, scale = msa_rope_inv_freq(rot_dim, theta, kind, factor, original_len, slow, fast)
        return Rope(torch.from_numpy(freq).to(device), layout, scale)


# ------------------------------------------------------------------ the C ABI ------------
def msa_abi_version() -> int:
    return int(_lib.msa_abi_version())


def msa_status_string(code: int) -> str:
    return _lib.msa_status_string(code).decode()


def msa_quantize_nvfp4(x: torch.Tensor, vals: torch.Tensor, scales: torch.Tensor,
                       vals_row_stride: Optional[int] = None, scales_row_stride: Optional[int] = None) -> None:
    _need(x, torch.float32, "x")
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    _check(_lib.msa_quantize_nvfp4(_ptr(x), rows, cols, _ptr(vals), vals_row_stride or cols // 2, _ptr(scales),
                                   scales_row_stride or cols // 16, _stream()), "msa_quantize_nvfp4")


def msa_quantize_fp8(x: torch.Tensor, out: torch.Tensor) -> None:
    _need(x, torch.float32, "x")
    _check(_lib.msa_quantize_fp8(_ptr(x), x.numel(), _ptr(out), _stream()), "msa_quantize_fp8")


def msa_dequant_nvfp4(vals: torch.Tensor, scales: torch.Tensor, out: torch.Tensor) -> None:
    cols = vals.shape[-1] * 2
    rows = vals.numel() // vals.shape[-1]
    _check(_lib.msa_dequant_nvfp4(_ptr(vals), cols // 2, _ptr(scales), cols // 16, rows, cols, _ptr(out), _stream()),
           "msa_dequant_nvfp4")


def msa_kv_insert(k: torch.Tensor, v: torch.Tensor, ik: Optional[torch.Tensor], slots: torch.Tensor, cache: Cache,
                  status: Optional[torch.Tensor] = None) -> None:
    _need(k, torch.float32, "k")
    _need(v, torch.float32, "v")
    _need(slots, torch.int64, "slots")
    n = int(slots.numel())
    _check(_lib.msa_kv_insert(_ptr(k), _ptr(v), _ptr(ik), n, _ptr(slots), _ptr(cache.kv_pages),
                              _ptr(cache.index_pages), cache.index_dtype, cache.num_pages, _ptr(status), _stream()),
           "msa_kv_insert")


def msa_rope_inv_freq(rot_dim: int, theta: float, kind: int = MSA_ROPE_PLAIN, factor: float = 1.0,
                      original_len: float = 0.0, slow: float = 1.0, fast: float = 32.0):
    """Host arithmetic: (inv_freq float64 [rot_dim / 2], the factor on cos and sin)."""
    freq = np.zeros(max(int(rot_dim), 0) // 2, dtype=np.float64)
    scale = np.zeros(1, dtype=np.float32)
    _check(_lib.msa_rope_inv_freq(int(rot_dim), float(theta), int(kind), float(factor), float(original_len),
                                  float(slow), float(fast), freq.ctypes.data, scale.ctypes.data), "msa_rope_inv_freq")
    return freq, float(scale[0])


def msa_rope_fp8(x: torch.Tensor, positions: Optional[torch.Tensor], rope: Rope, out: torch.Tensor,
                 norm_weight: Optional[torch.Tensor] = None, eps: float = 1e-6) -> None:
    """x [T, heads, 128] (fp32, bf16 or fp16, any token and head strides) -> E4M3 bytes out [T, heads, 128]."""
    dev = _current_device()
    px, dt, (T, heads, _), (st, sh, _) = _rows_at(x, 3, dev, "x")
    if rope.device != dev and rope.device is not None:
        raise ValueError(f"rope's frequencies are on cuda:{rope.device}, the call on cuda:{dev}")
    code = _lib.msa_rope_fp8(px, dt, T, heads, st, sh, _at(positions, _INT32, T, dev, "positions"), rope.ref,
                             _at(norm_weight, _FLOAT32, HEAD_DIM, dev, "norm_weight"), eps,
                             _at(out, _U8, T * heads * HEAD_DIM, dev, "out"), _raw_stream(dev))
    if code:
        raise MsaError(code, "msa_rope_fp8")


def msa_rope_kv_insert(k: torch.Tensor, v: torch.Tensor, ik: Optional[torch.Tensor],
                       positions: Optional[torch.Tensor], slots: torch.Tensor, rope: Rope, cache: Cache,
                       k_norm: Optional[torch.Tensor] = None, ik_norm: Optional[torch.Tensor] = None,
                       eps: float = 1e-6, status: Optional[torch.Tensor] = None) -> None:
    """msa_kv_insert of projected rows: k, v [n, 4, 128] and ik [n, 128] of one type (fp32, bf16 or
    fp16, any token and head strides), K and the index key normalised and rotated on the way."""
    dev = _current_device()
    n = slots.numel()
    pk, dt, (kn, kg, _), (kt, kh, _) = _rows_at(k, 3, dev, "k")
    pv, dv, (vn, vg, _), (vt, vh, _) = _rows_at(v, 3, dev, "v")
    pi, di, (im, _), (it, _) = (None, dt, (n, 0), (0, 0)) if ik is None else _rows_at(ik, 2, dev, "ik")
    if dv != dt or di != dt:
        raise ValueError("k, v and ik must have one type")
    if kn < n or vn < n or im < n or kg != GROUPS or vg != GROUPS:
        raise ValueError(f"k and v must hold [{n}, {GROUPS}, {HEAD_DIM}], ik [{n}, {HEAD_DIM}]")
    if rope.device != dev and rope.device is not None:
        raise ValueError(f"rope's frequencies are on cuda:{rope.device}, the call on cuda:{dev}")
    if cache.device != dev:
        raise ValueError(f"the cache must be on cuda:{dev}")
    rows = msa_kv_rows(pk, pv, pi, dt, kt, kh, vt, vh, it)
    code = _lib.msa_rope_kv_insert(ctypes.byref(rows), n, _at(positions, _INT32, n, dev, "positions"),
                                   _at(slots, _INT64, n, dev, "slots"), rope.ref,
                                   _at(k_norm, _FLOAT32, HEAD_DIM, dev, "k_norm"),
                                   _at(ik_norm, _FLOAT32, HEAD_DIM, dev, "ik_norm"), eps,
                                   cache.kv_at, cache.index_at, cache.index_dtype, cache.num_pages, _status_at(status, dev), _raw_stream(dev))
    if code:
        raise MsaError(code, "msa_rope_kv_insert")


def msa_kv_read(slots: torch.Tensor, cache: Cache, k: Optional[torch.Tensor], v: Optional[torch.Tensor],
                ik: Optional[torch.Tensor], status: Optional[torch.Tensor] = None) -> None:
    """The cached rows at `slots` as E4M3 bytes: k, v [n, 4, 128], ik [n, 128] (uint8, None to skip)."""
    dev = _current_device()
    n = slots.numel()
    if cache.device != dev:
        raise ValueError(f"the cache must be on cuda:{dev}")
    code = _lib.msa_kv_read(_at(slots, _INT64, n, dev, "slots"), n, cache.kv_at, cache.index_at, cache.index_dtype,
                            cache.num_pages, _at(k, _U8, n * GROUPS * HEAD_DIM, dev, "k"), _at(v, _U8, n * GROUPS * HEAD_DIM, dev, "v"),
                            _at(ik, _U8, n * HEAD_DIM, dev, "ik"), _status_at(status, dev), _raw_stream(dev))
    if code:
        raise MsaError(code, "msa_kv_read")


def msa_indexer_decode(batch: Batch, cache: Cache, index_q: torch.Tensor, block_scores: torch.Tensor,
                       status: Optional[torch.Tensor] = None) -> None:
    _check(_lib.msa_indexer_decode(ctypes.byref(GEOMETRY), ctypes.byref(batch.c), ctypes.byref(cache.c),
                                   _ptr(index_q), _ptr(block_scores), _ptr(status), _stream()),
           "msa_indexer_decode")


def msa_topk_blocks(batch: Batch, block_scores: torch.Tensor, sel: torch.Tensor,
                    status: Optional[torch.Tensor] = None) -> None:
    _check(_lib.msa_topk_blocks(ctypes.byref(GEOMETRY), ctypes.byref(batch.c), _ptr(block_scores), _ptr(sel),
                                _ptr(status), _stream()), "msa_topk_blocks")


def msa_indexer_decode_range(batch: Batch, cache: Cache, index_q: torch.Tensor, block_begin: int, block_end: int,
                             block_scores: torch.Tensor, status: Optional[torch.Tensor] = None) -> None:
    """The indexer over one context shard: blocks block_begin <= k < block_end of every sequence."""
    _check(_lib.msa_indexer_decode_range(ctypes.byref(GEOMETRY), ctypes.byref(batch.c), ctypes.byref(cache.c),
                                         _ptr(index_q), int(block_begin), int(block_end), _ptr(block_scores),
                                         _ptr(status), _stream()), "msa_indexer_decode_range")


def msa_indexer_decode_exact(batch: Batch, cache: Cache, index_q: torch.Tensor, block_scores: torch.Tensor,
                             status: Optional[torch.Tensor] = None) -> None:
    """The exact-score indexer: NVFP4 index keys as E2M1 x E4M3 exactly (f16 score MMA)."""
    _check(_lib.msa_indexer_decode_exact(ctypes.byref(GEOMETRY), ctypes.byref(batch.c), ctypes.byref(cache.c),
                                         _ptr(index_q), _ptr(block_scores), _ptr(status), _stream()),
           "msa_indexer_decode_exact")


def msa_prefill_workspace_size(B: int, T: int, max_blocks_per_seq: int) -> int:
    return int(_lib.msa_prefill_workspace_size(ctypes.byref(GEOMETRY), B, T, max_blocks_per_seq))


def msa_indexer_prefill(batch: Batch, cache: Cache, index_q: torch.Tensor, block_scores: torch.Tensor,
                        status: Optional[torch.Tensor] = None) -> None:
    """The indexer for a prefill batch (any number of query tokens per sequence)."""
    _check(_lib.msa_indexer_prefill(ctypes.byref(GEOMETRY), ctypes.byref(batch.c), ctypes.byref(cache.c),
                                    _ptr(index_q), _ptr(block_scores), _ptr(status), _stream()),
           "msa_indexer_prefill")


def msa_topk_prefill(batch: Batch, block_scores: torch.Tensor, sel: torch.Tensor,
                     status: Optional[torch.Tensor] = None) -> None:
    """The block selection for a prefill batch (any number of query tokens per sequence)."""
    _check(_lib.msa_topk_prefill(ctypes.byref(GEOMETRY), ctypes.byref(batch.c), _ptr(block_scores), _ptr(sel),
                                 _ptr(status), _stream()), "msa_topk_prefill")


def msa_prefill_attn(batch: Batch, cache: Cache, q: torch.Tensor, sel: torch.Tensor, softmax_scale: float,
                     out: torch.Tensor, workspace: torch.Tensor, status: Optional[torch.Tensor] = None) -> None:
    """Block-major sparse attention for any number of query tokens per sequence."""
    _check(_lib.msa_prefill_attn(ctypes.byref(GEOMETRY), ctypes.byref(batch.c), ctypes.byref(cache.c), _ptr(q),
                                 _ptr(sel), ctypes.c_float(softmax_scale), _ptr(workspace),
                                 ctypes.c_size_t(workspace.numel() * workspace.element_size()), _ptr(out),
                                 _ptr(status), _stream()), "msa_prefill_attn")


def msa_dense_attn_workspace_size(B: int, T: int, max_q_len: int) -> int:
    return int(_lib.msa_dense_attn_workspace_size(ctypes.byref(GEOMETRY), B, T, max_q_len))


def msa_dense_attn(batch: Batch, cache: Cache, q: torch.Tensor, softmax_scale: float, out: torch.Tensor,
                   workspace: torch.Tensor, lse: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None) -> None:
    """Causal attention of q [T, 64, 128] (E4M3 bytes) over the whole cache; out [T, 64, 128] bf16 bits,
    lse [T, 64] fp32 (natural logarithm) if given. Shards of a context join by lse if each call has one query
    token a sequence."""
    dev = _current_device()
    n = batch.T * Q_HEADS
    if out.element_size() != 2 or not out.is_contiguous() or out.numel() < n * HEAD_DIM or out.get_device() != dev:
        raise ValueError(f"out must be a contiguous tensor of at least {n * HEAD_DIM} 16-bit elements on cuda:{dev}")
    if cache.device != dev or batch.device != dev:
        raise ValueError(f"the cache and the batch must be on cuda:{dev}")
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    code = _lib.msa_dense_attn(_GEO_REF, batch.ref, cache.ref, _at(q, _U8, n * HEAD_DIM, dev, "q"), softmax_scale,
                               workspace.data_ptr(), workspace.numel() * workspace.element_size(), out.data_ptr(),
                               _at(lse, _FLOAT32, n, dev, "lse"), _status_at(status, dev), _raw_stream(dev))
    if code:
        raise MsaError(code, "msa_dense_attn")


def msa_topk_candidates(batch: Batch, block_scores: torch.Tensor, block_begin: int, block_end: int,
                        cand: torch.Tensor, status: Optional[torch.Tensor] = None) -> None:
    """A context shard's 15 best non-local blocks per (t, g) as 64-bit keys (int64 tensor [T, 4, 15])."""
    _check(_lib.msa_topk_candidates(ctypes.byref(GEOMETRY), ctypes.byref(batch.c), _ptr(block_scores),
                                    int(block_begin), int(block_end), _ptr(cand), _ptr(status), _stream()),
           "msa_topk_candidates")


def msa_topk_merge(batch: Batch, cand: torch.Tensor, n_shards: int, sel: torch.Tensor,
                   status: Optional[torch.Tensor] = None) -> None:
    """The owner's merge of n_shards candidate lists ([n_shards, T, 4, 15]) into sel [T, 4, 16]."""
    _check(_lib.msa_topk_merge(ctypes.byref(GEOMETRY), ctypes.byref(batch.c), _ptr(cand), int(n_shards), _ptr(sel),
                               _ptr(status), _stream()), "msa_topk_merge")


def msa_topk_candidates_host(block_scores: np.ndarray, local: np.ndarray, block_begin: int,
                             block_end: int) -> np.ndarray:
    """Host version of msa_topk_candidates: block_scores float32 [rows, maxb], local int32 [rows]."""
    sc = np.ascontiguousarray(block_scores, dtype=np.float32)
    lc = np.ascontiguousarray(local, dtype=np.int32)
    out = np.zeros((sc.shape[0], 15), dtype=np.uint64)
    _check(_lib.msa_topk_candidates_host(sc.ctypes.data, sc.shape[0], sc.shape[1], lc.ctypes.data, int(block_begin),
                                         int(block_end), out.ctypes.data), "msa_topk_candidates_host")
    return out


def msa_topk_merge_host(cand: np.ndarray, local: np.ndarray) -> np.ndarray:
    """Host version of msa_topk_merge: cand uint64 [n_shards, rows, 15], local int32 [rows]."""
    cd = np.ascontiguousarray(cand, dtype=np.uint64)
    lc = np.ascontiguousarray(local, dtype=np.int32)
    out = np.zeros((cd.shape[1], 16), dtype=np.int32)
    _check(_lib.msa_topk_merge_host(cd.ctypes.data, cd.shape[0], cd.shape[1], lc.ctypes.data, out.ctypes.data),
           "msa_topk_merge_host")
    return out


def msa_kv_gather_map(batch: Batch, sel: torch.Tensor, map_out: torch.Tensor, masks: torch.Tensor,
                      num_gathered: torch.Tensor, status: Optional[torch.Tensor] = None) -> None:
    """map_out int32 [B, max_blocks], masks uint8 [B, max_blocks], num_gathered int32 [1] (device)."""
    _check(_lib.msa_kv_gather_map(ctypes.byref(GEOMETRY), ctypes.byref(batch.c), _ptr(sel), _ptr(map_out),
                                  _ptr(masks), _ptr(num_gathered), _ptr(status), _stream()), "msa_kv_gather_map")


def msa_kv_gather_pages(batch: Batch, cache: Cache, map_in: torch.Tensor, masks: torch.Tensor, block_begin: int,
                        block_end: int, gathered_kv: torch.Tensor, max_gathered: int,
                        status: Optional[torch.Tensor] = None) -> None:
    """Copy the selected K/V regions this shard holds (blocks [block_begin, block_end)) into the
    gathered pool gathered_kv (uint8, max_gathered x 73,728 B, device)."""
    _check(_lib.msa_kv_gather_pages(ctypes.byref(GEOMETRY), ctypes.byref(batch.c), ctypes.byref(cache.c), _ptr(map_in),
                                    _ptr(masks), int(block_begin), int(block_end), _ptr(gathered_kv),
                                    int(max_gathered), _ptr(status), _stream()), "msa_kv_gather_pages")


def msa_kv_gather_map_host(query_start_loc: np.ndarray, seq_lens: np.ndarray, max_blocks: int,
                           sel: np.ndarray):
    """Host version of msa_kv_gather_map: returns (map int32 [B, max_blocks], masks uint8, count)."""
    qsl = np.ascontiguousarray(query_start_loc, dtype=np.int32)
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    sl_ = np.ascontiguousarray(sel, dtype=np.int32)
    B = sl.shape[0]
    mp = np.zeros((B, max_blocks), dtype=np.int32)
    mk = np.zeros((B, max_blocks), dtype=np.uint8)
    n = int(_lib.msa_kv_gather_map_host(B, int(qsl[-1]), qsl.ctypes.data, sl.ctypes.data, int(max_blocks),
                                        sl_.ctypes.data, mp.ctypes.data, mk.ctypes.data))
    if n < 0:
        raise MsaError(MSA_ERR_INVALID_ARG, "msa_kv_gather_map_host")
    return mp, mk, n


def msa_kv_gather_pages_host(block_table: np.ndarray, kv_pages: np.ndarray, num_pages: int, map_in: np.ndarray,
                             masks: np.ndarray, block_begin: int, block_end: int, gathered_kv: np.ndarray) -> None:
    """Host version of msa_kv_gather_pages (numpy arrays; gathered_kv uint8 [n, 73,728] is filled)."""
    bt = np.ascontiguousarray(block_table, dtype=np.int32)
    kv = np.ascontiguousarray(kv_pages, dtype=np.uint8)
    mp = np.ascontiguousarray(map_in, dtype=np.int32)
    mk = np.ascontiguousarray(masks, dtype=np.uint8)
    assert gathered_kv.dtype == np.uint8 and gathered_kv.flags.c_contiguous
    _check(_lib.msa_kv_gather_pages_host(bt.shape[0], bt.shape[1], bt.ctypes.data, kv.ctypes.data, int(num_pages),
                                         mp.ctypes.data, mk.ctypes.data, int(block_begin), int(block_end),
                                         gathered_kv.ctypes.data, gathered_kv.size // KV_PAGE_BYTES),
           "msa_kv_gather_pages_host")


def msa_attn_workspace_size(B: int, T: int, num_splits: int = 0) -> int:
    return int(_lib.msa_attn_workspace_size(ctypes.byref(GEOMETRY), B, T, num_splits))


def msa_sparse_attn_decode(batch: Batch, cache: Cache, q: torch.Tensor, sel: torch.Tensor, softmax_scale: float,
                           out: torch.Tensor, num_splits: int = 0, workspace: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.msa_sparse_attn_decode(ctypes.byref(GEOMETRY), ctypes.byref(batch.c), ctypes.byref(cache.c), _ptr(q),
                                       _ptr(sel), float(softmax_scale), num_splits, _ptr(workspace), ws_bytes,
                                       _ptr(out), _ptr(status), _stream()), "msa_sparse_attn_decode")


def msa_sparse_attn_decode_noalloc(batch: Batch, cache: Cache, q: torch.Tensor, sel: torch.Tensor,
                                   softmax_scale: float, out: torch.Tensor, num_splits: int = 0,
                                   status: Optional[torch.Tensor] = None) -> None:
    """msa_sparse_attn_decode for callers that cannot allocate: split partials go to the
    library's own device array (msa_noalloc_scratch_bytes() bytes); calls must not overlap."""
    _check(_lib.msa_sparse_attn_decode_noalloc(ctypes.byref(GEOMETRY), ctypes.byref(batch.c), ctypes.byref(cache.c),
                                               _ptr(q), _ptr(sel), float(softmax_scale), num_splits, _ptr(out),
                                               _ptr(status), _stream()), "msa_sparse_attn_decode_noalloc")


def msa_noalloc_scratch_bytes() -> int:
    return int(_lib.msa_noalloc_scratch_bytes())


def msa_decode_workspace_size(B: int, T: int, max_blocks_per_seq: int) -> int:
    return int(_lib.msa_decode_workspace_size(ctypes.byref(GEOMETRY), B, T, max_blocks_per_seq))


def msa_decode_step(batch: Batch, cache: Cache, q: torch.Tensor, index_q: torch.Tensor, softmax_scale: float,
                    workspace: torch.Tensor, out: torch.Tensor, dbg_block_scores: Optional[torch.Tensor] = None,
                    dbg_sel: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(_lib.msa_decode_step(ctypes.byref(GEOMETRY), ctypes.byref(batch.c), ctypes.byref(cache.c), _ptr(q),
                                _ptr(index_q), float(softmax_scale), _ptr(dbg_block_scores), _ptr(dbg_sel),
                                _ptr(workspace), ws_bytes, _ptr(out), _stream(stream)), "msa_decode_step")


def msa_decode_step_host(batch: Batch, cache: Cache, host_qsl: torch.Tensor, host_seq_lens: torch.Tensor,
                         host_block_table: torch.Tensor, host_q: torch.Tensor, host_index_q: torch.Tensor,
                         host_out: torch.Tensor, q: torch.Tensor, index_q: torch.Tensor, softmax_scale: float,
                         workspace: torch.Tensor, out: Optional[torch.Tensor], copy_stream: torch.cuda.Stream,
                         direct_out: bool = False, stream: Optional[torch.cuda.Stream] = None) -> None:
    """msa_decode_step from page-locked host tensors: `batch`'s device arrays, q and index_q are
    filled from the host ones and host_out receives the output (copied back from `out`, or with
    direct_out stored there by the attention itself), the copies on copy_stream and `stream`
    overlapping the kernels (include/msa.h). host_out is complete once `stream` has passed the
    call."""
    for n, t in (("host_qsl", host_qsl), ("host_seq_lens", host_seq_lens), ("host_block_table", host_block_table),
                 ("host_q", host_q), ("host_index_q", host_index_q), ("host_out", host_out)):
        if t.is_cuda or not t.is_pinned() or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous page-locked host tensor")
    io = msa_host_step_io(host_qsl.data_ptr(), host_seq_lens.data_ptr(), host_block_table.data_ptr(),
                          host_q.data_ptr(), host_index_q.data_ptr(), host_out.data_ptr())
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(_lib.msa_decode_step_host(ctypes.byref(GEOMETRY), ctypes.byref(batch.c), ctypes.byref(cache.c),
                                     ctypes.byref(io), _ptr(q), _ptr(index_q), float(softmax_scale), _ptr(workspace),
                                     ws_bytes, _ptr(out), MSA_HOST_STEP_DIRECT_OUT if direct_out else 0,
                                     _stream(stream), _stream(copy_stream)),
           "msa_decode_step_host")


def msa_read_device_status(workspace: torch.Tensor) -> int:
    return int(_lib.msa_read_device_status(_ptr(workspace), _stream()))


def msa_selftest_wait_timeout(status: torch.Tensor, limit_ns: int) -> None:
    _check(_lib.msa_selftest_wait_timeout(_ptr(status), int(limit_ns), _stream()), "msa_selftest_wait_timeout")


def status_bits(status: torch.Tensor) -> int:
    """Bits of a device status word (1 << msa_status code)."""
    return int(status.view(torch.int32)[0].item()) & 0xFFFFFFFF
