"""Python binding of libmlora.so, the MI355X heterogeneous multi-LoRA linear.

Argument marshalling only: every step of the layer runs in the HIP kernels
behind include/mlora.h.  torch is used for device memory (tensors give
pointers) and streams (the current stream is passed to every call).  There
is no CPU fallback: if the library is missing, every call raises.

Typical use::

    pool = Pool(din, dout, n_proj, max_adapters, max_rank, n_pages)
    pool.load(adapter_id, rank, scale, down_bits, up_bits)   # host bf16 bits
    seg = build_segments(pool, row_adapter)                  # device int32 [n]
    Y = apply(pool, proj, X, W0, seg)                        # device bf16

and, for the attention between a layer's projections (these calls and those
below want their tensors on the current device)::

    cache = KVCache(n_layers, n_blocks, kv_heads, dim, block)          # paged 8-bit keys and values
    batch = KVBatch(table, kv_len, row_off, n_rows, max_new=max_new)   # device int32 tensors
    kv_append(cache, layer, k, v, batch)
    O = kv_attention(cache, layer, q, batch)                           # device bf16

with a base weight in 4 bits, norms and rotation of the heads, and the next tokens::

    w4 = q4_quantize(W0)
    Y = q4_apply(pool, proj, X, w4, seg)                               # as apply, with w4 for W0
    q, k = qk_norm_rotary(q, k, batch, Rotary(dim), q_weight=qw, k_weight=kw)
    tokens = sample(logits, u, temperature=t, top_k=k, top_p=p, min_p=m)
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import numpy as np

__all__ = [
    "MloraError", "lib", "Pool", "build_segments", "segments_header", "segments_status", "read_segments",
    "base_gemm", "shrink", "shrink_max_chunks", "expand", "fused", "shrink_rows", "gemm_lora", "new_work", "rows_t", "apply", "forward", "plan", "work_bytes",
    "forward_static", "STATIC_SCRATCH_BYTES", "merge", "hbm_copy", "hbm_read", "hbm_read_lds", "timing_arm", "timing_read", "VARIANTS", "ITEM_ROWS", "TILE_ROWS", "MAX_ROWS", "MAX_RANK", "SEG", "EXPORTS", "LIB_PATH",
    "KVCache", "KVBatch", "kv_append", "kv_read", "kv_attention", "kv_work_bytes", "new_kv_work",
    "Q4Weight", "q4_quantize", "q4_dequantize", "q4_gemm", "q4_apply", "q4_work_bytes", "new_q4_work",
    "Rotary", "qk_norm_rotary", "sample", "sample_work_bytes", "new_sample_work",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmlora.so")

OK, EINVAL, ENOSPC, EEXIST, ENOENT, EHIP = range(6)
VARIANTS = {"auto": 0, "split": 1, "fused": 2, "rows": 3}
ITEM_ROWS = 4
TILE_ROWS = 64
MAX_ROWS = 16384
MAX_RANK = 128
SEG = dict(nseg=0, n_act=1, n_none=2, n_bad=3, status=4, n_items=5, n_rows=6, max_adapters=7, n_tiles=8)
SEG_HEADER = 16
SEG_BAD_ID, SEG_NOT_RESIDENT = 1, 2  # bits of the status word

_c_void_p, _i32, _i64, _f32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_pi32, _pi64, _pf32 = ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_float)


class _PoolDesc(ctypes.Structure):
    _fields_ = [("din", _i32), ("dout", _i32), ("n_proj", _i32), ("max_adapters", _i32), ("max_rank", _i32),
                ("reserved", _i32), ("n_down_pages", _i64), ("n_up_pages", _i64), ("down_pages", _c_void_p),
                ("up_pages", _c_void_p), ("meta", _c_void_p)]


class _KVCacheDesc(ctypes.Structure):
    _fields_ = [("n_layers", _i32), ("kv_heads", _i32), ("dim", _i32), ("block", _i32), ("n_blocks", _i64),
                ("k", _c_void_p), ("v", _c_void_p), ("k_scale", _c_void_p), ("v_scale", _c_void_p)]


class _KVBatchDesc(ctypes.Structure):
    _fields_ = [("table", _c_void_p), ("kv_len", _c_void_p), ("row_off", _c_void_p), ("n_seq", _i32), ("width", _i32),
                ("table_stride", _i32), ("n_rows", _i32), ("max_new", _i32)]


class _Q4Desc(ctypes.Structure):
    _fields_ = [("codes", _c_void_p), ("scales", _c_void_p), ("din", _i32), ("dout", _i32)]


class _RotaryDesc(ctypes.Structure):
    _fields_ = [("freq", _c_void_p), ("rot", _i32), ("interleaved", _i32), ("factor", _f32)]


# name -> (restype, argtypes); every symbol include/mlora.h declares
EXPORTS = {
    "mlora_version": (ctypes.c_char_p, []),
    "mlora_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "mlora_last_error": (ctypes.c_char_p, []),
    "mlora_pool_meta_bytes": (_sz, [_i32, _i32, _i32]),
    "mlora_pool_create": (ctypes.c_int, [ctypes.POINTER(_PoolDesc), _c_void_p, ctypes.POINTER(_c_void_p)]),
    "mlora_pool_destroy": (ctypes.c_int, [_c_void_p]),
    "mlora_pool_load": (ctypes.c_int, [_c_void_p, _i32, _i32, _f32, _c_void_p, _c_void_p, _c_void_p]),
    "mlora_pool_unload": (ctypes.c_int, [_c_void_p, _i32, _c_void_p]),
    "mlora_pool_ready": (ctypes.c_int, [_c_void_p, _i32, _c_void_p]),
    "mlora_pool_query": (ctypes.c_int, [_c_void_p, _i32, _pi32, _pf32]),
    "mlora_pool_free_pages": (ctypes.c_int, [_c_void_p, _pi64, _pi64, _pi32]),
    "mlora_pool_fail_next_load": (ctypes.c_int, [_c_void_p, _i32]),
    "mlora_segments_bytes": (_sz, [_i32]),
    "mlora_build_segments": (ctypes.c_int, [_c_void_p, _c_void_p, _i32, _c_void_p, _c_void_p]),
    "mlora_segments_header": (ctypes.c_int, [_c_void_p, _pi32, _c_void_p]),
    "mlora_segments_status": (ctypes.c_int, [_c_void_p, _pi32, _c_void_p]),
    "mlora_base_gemm": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _i32, _i32, _i32, _c_void_p]),
    "mlora_shrink_max_chunks": (_i32, [_i32]),
    "mlora_shrink": (ctypes.c_int, [_c_void_p, _i32, _c_void_p, _c_void_p, _i32, _c_void_p, _i32, _c_void_p]),
    "mlora_expand": (ctypes.c_int, [_c_void_p, _i32, _c_void_p, _i32, _c_void_p, _c_void_p, _i32, _c_void_p]),
    "mlora_fused": (ctypes.c_int, [_c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p, _i32, _c_void_p]),
    "mlora_work_bytes": (_sz, [_c_void_p, _i32]),
    "mlora_shrink_rows": (ctypes.c_int, [_c_void_p, _i32, _c_void_p, _c_void_p, _i32, _c_void_p, _sz, _c_void_p]),
    "mlora_gemm_lora": (ctypes.c_int, [_c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p,
                                       _i32, _c_void_p]),
    "mlora_plan": (ctypes.c_int, [_c_void_p, _i32, _i32, _pi32, _pi32]),
    "mlora_apply": (ctypes.c_int, [_c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32, _c_void_p,
                                   _sz, _i32, _c_void_p]),
    "mlora_forward": (ctypes.c_int, [_c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32,
                                     _c_void_p, _sz, _i32, _c_void_p]),
    "mlora_forward_static": (ctypes.c_int, [_c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                            _i32, _i32, _c_void_p]),
    "mlora_merge": (ctypes.c_int, [_c_void_p, _i32, _i32, _c_void_p, _f32, _c_void_p]),
    "mlora_kv_append": (ctypes.c_int, [_c_void_p, _i32, _c_void_p, _c_void_p, _i64, _i64, _c_void_p, _c_void_p]),
    "mlora_kv_read": (ctypes.c_int, [_c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "mlora_kv_work_bytes": (_sz, [_c_void_p, _c_void_p, _i32]),
    "mlora_kv_attention": (ctypes.c_int, [_c_void_p, _i32, _c_void_p, _i64, _i64, _i32, _c_void_p, _i32, _i32, _f32,
                                          _c_void_p, _c_void_p, _sz, _c_void_p]),
    "mlora_q4_quantize": (ctypes.c_int, [_c_void_p, _i32, _i32, _c_void_p, _c_void_p, _c_void_p]),
    "mlora_q4_dequantize": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p]),
    "mlora_q4_work_bytes": (_sz, [_c_void_p, _c_void_p, _i32]),
    "mlora_q4_gemm": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _i32, _c_void_p, _sz, _c_void_p]),
    "mlora_q4_apply": (ctypes.c_int, [_c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32, _c_void_p,
                                      _sz, _c_void_p]),
    "mlora_qk_norm_rotary": (ctypes.c_int, [_c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p, _f32, _c_void_p]),
    "mlora_sample_work_bytes": (_sz, [_i32, _i32]),
    "mlora_sample": (ctypes.c_int, [_c_void_p, _i32, _i64, _i32, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                    _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "mlora_hbm_copy": (ctypes.c_int, [_c_void_p, _c_void_p, _sz, _c_void_p]),
    "mlora_hbm_read": (ctypes.c_int, [_c_void_p, _sz, _c_void_p, _c_void_p]),
    "mlora_hbm_read_lds": (ctypes.c_int, [_c_void_p, _sz, _c_void_p, _c_void_p]),
    "mlora_timing_arm": (ctypes.c_int, [ctypes.c_int32]),
    "mlora_timing_read": (ctypes.c_int, [ctypes.POINTER(ctypes.c_float), ctypes.c_int32,
                                         ctypes.POINTER(ctypes.c_int32)]),
    "mlora_timing_name": (ctypes.c_char_p, [ctypes.c_int32]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (loaded on first use).  Raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run `python -m lora_serving_mlora_amd.build` "
                               "(the multi-LoRA path has no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


class MloraError(RuntimeError):
    def __init__(self, status: int, where: str):
        L = lib()
        self.status = status
        msg = L.mlora_status_string(status).decode()
        detail = L.mlora_last_error().decode()
        super().__init__(f"{where}: {msg}" + (f" ({detail})" if detail else ""))


def _check(status: int, where: str) -> None:
    if status != OK:
        raise MloraError(status, where)


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream():
    return ctypes.c_void_p(_torch().cuda.current_stream().cuda_stream)


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr() if t is not None else 0)


def _bf16_dev(t, name: str):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous bfloat16 CUDA tensor")
    return t


def _host_bits(a, shape, name: str) -> np.ndarray:
    """bf16 data on the host as a C-contiguous uint16 array of `shape`."""
    torch = _torch()
    if isinstance(a, torch.Tensor):
        a = a.detach().cpu()
        if a.dtype == torch.bfloat16:
            a = a.view(torch.int16)
        a = a.numpy()
    a = np.asarray(a)
    if a.dtype not in (np.int16, np.uint16):
        raise TypeError(f"{name} must hold bf16 bit patterns (uint16/int16 array or bfloat16 tensor)")
    a = np.ascontiguousarray(a).view(np.uint16)
    if tuple(a.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(a.shape)}, expected {tuple(shape)}")
    return a


class Pool:
    """A rank-stacked paged adapter pool on the current device.

    One page is one rank row of one adapter for one projection (Down rows of
    din, Up^T rows of dout).  n_pages pages are allocated in each arena."""

    def __init__(self, din: int, dout: int, n_proj: int, max_adapters: int, max_rank: int,
                 n_pages: int, n_up_pages: Optional[int] = None):
        torch = _torch()
        L = lib()
        self.din, self.dout, self.n_proj = din, dout, n_proj
        self.max_adapters, self.max_rank = max_adapters, max_rank
        n_up = n_pages if n_up_pages is None else n_up_pages
        dev = torch.device("cuda", torch.cuda.current_device())
        self.down_pages = torch.zeros((max(n_pages, 1), din), dtype=torch.bfloat16, device=dev)
        self.up_pages = torch.zeros((max(n_up, 1), dout), dtype=torch.bfloat16, device=dev)
        mb = L.mlora_pool_meta_bytes(max_adapters, n_proj, max_rank)
        self.meta = torch.empty(max(mb, 256), dtype=torch.uint8, device=dev)
        d = _PoolDesc(din, dout, n_proj, max_adapters, max_rank, 0, n_pages, n_up,
                      self.down_pages.data_ptr(), self.up_pages.data_ptr(), self.meta.data_ptr())
        h = ctypes.c_void_p()
        _check(L.mlora_pool_create(ctypes.byref(d), _stream(), ctypes.byref(h)), "mlora_pool_create")
        self._h = h

    @property
    def handle(self) -> ctypes.c_void_p:
        if self._h is None:
            raise RuntimeError("pool is closed")
        return self._h

    def load(self, adapter_id: int, rank: int, scale: float, down, up) -> None:
        """down: bf16 bits [n_proj][rank][din]; up: bf16 bits [n_proj][dout][rank]."""
        d = _host_bits(down, (self.n_proj, rank, self.din), "down")
        u = _host_bits(up, (self.n_proj, self.dout, rank), "up")
        _check(lib().mlora_pool_load(self.handle, adapter_id, rank, ctypes.c_float(scale),
                                     d.ctypes.data_as(ctypes.c_void_p), u.ctypes.data_as(ctypes.c_void_p), _stream()),
               f"mlora_pool_load({adapter_id})")

    def unload(self, adapter_id: int) -> None:
        _check(lib().mlora_pool_unload(self.handle, adapter_id, _stream()), f"mlora_pool_unload({adapter_id})")

    def ready(self, adapter_id: int) -> None:
        """Makes the current stream wait (on the device) for the adapter's
        latest load, which may have been issued on another stream."""
        _check(lib().mlora_pool_ready(self.handle, adapter_id, _stream()), f"mlora_pool_ready({adapter_id})")

    def query(self, adapter_id: int):
        r, s = ctypes.c_int32(), ctypes.c_float()
        st = lib().mlora_pool_query(self.handle, adapter_id, ctypes.byref(r), ctypes.byref(s))
        if st == ENOENT:
            return None
        _check(st, "mlora_pool_query")
        return r.value, s.value

    def free_pages(self):
        fd, fu, nr = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int32()
        _check(lib().mlora_pool_free_pages(self.handle, ctypes.byref(fd), ctypes.byref(fu), ctypes.byref(nr)),
               "mlora_pool_free_pages")
        return fd.value, fu.value, nr.value

    def fail_next_load(self, step: int) -> None:
        """Testing aid: the next load on this pool fails at `step` (1: before
        its last staging flush, 2: after its metadata copies; 0: off)."""
        _check(lib().mlora_pool_fail_next_load(self.handle, step), "mlora_pool_fail_next_load")

    def close(self) -> None:
        if getattr(self, "_h", None) is not None:
            _check(lib().mlora_pool_destroy(self._h), "mlora_pool_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def segments_bytes(n: int) -> int:
    return int(lib().mlora_segments_bytes(n))


def build_segments(pool: Pool, row_adapter, seg_ws=None):
    """row_adapter: int32 CUDA tensor [n].  Returns the seg_ws tensor."""
    torch = _torch()
    if row_adapter.dtype != torch.int32 or not row_adapter.is_cuda or not row_adapter.is_contiguous():
        raise TypeError("row_adapter must be a contiguous int32 CUDA tensor")
    n = row_adapter.shape[0]
    nb = segments_bytes(n)
    if seg_ws is None:
        seg_ws = torch.empty(nb // 4, dtype=torch.int32, device=row_adapter.device)
    elif seg_ws.numel() * seg_ws.element_size() < nb:
        raise ValueError("seg_ws too small")
    _check(lib().mlora_build_segments(pool.handle, _ptr(row_adapter), n, _ptr(seg_ws), _stream()),
           "mlora_build_segments")
    return seg_ws


def segments_header(seg_ws) -> dict:
    """The header words of seg_ws (synchronises the stream)."""
    h = (ctypes.c_int32 * SEG_HEADER)()
    _check(lib().mlora_segments_header(_ptr(seg_ws), h, _stream()), "mlora_segments_header")
    return {k: int(h[i]) for k, i in SEG.items()}


def segments_status(seg_ws) -> int:
    """The batch's status word (SEG_BAD_ID | SEG_NOT_RESIDENT bits; synchronises the stream)."""
    st = ctypes.c_int32(0)
    _check(lib().mlora_segments_status(_ptr(seg_ws), ctypes.byref(st), _stream()), "mlora_segments_status")
    return int(st.value)


def read_segments(seg_ws, n: int) -> dict:
    """Copies seg_ws to the host and splits it by the documented layout."""
    w = seg_ws.cpu().numpy()
    hdr = {k: int(w[i]) for k, i in SEG.items()}
    nseg = hdr["nseg"]
    perm0, inv0, ad0, off0 = SEG_HEADER, SEG_HEADER + n, SEG_HEADER + 2 * n, SEG_HEADER + 3 * n
    items0 = (SEG_HEADER + 4 * n + 2) & ~1
    out = dict(hdr)
    max_items = n + (n + ITEM_ROWS - 1) // ITEM_ROWS + 1
    rk0 = items0 + 2 * max_items
    out["row_key"] = w[rk0:rk0 + n].copy()
    tl0 = rk0 + n
    out["tiles"] = w[tl0:tl0 + 2 * hdr["n_tiles"]].reshape(-1, 2).copy()
    out.update(perm=w[perm0:perm0 + n].copy(), inv=w[inv0:inv0 + n].copy(),
               seg_adapter=w[ad0:ad0 + nseg].copy(), seg_off=w[off0:off0 + nseg + 1].copy(),
               items=w[items0:items0 + 2 * hdr["n_items"]].reshape(-1, 2).copy())
    return out


def base_gemm(X, W0, Y=None):
    torch = _torch()
    _bf16_dev(X, "X"), _bf16_dev(W0, "W0")
    n, din = X.shape
    dout = W0.shape[0]
    if W0.shape[1] != din:
        raise ValueError("X and W0 disagree on din")
    if Y is None:
        Y = torch.empty((n, dout), dtype=torch.bfloat16, device=X.device)
    _bf16_dev(Y, "Y")
    if tuple(Y.shape) != (n, dout):
        raise ValueError("Y has the wrong shape")
    _check(lib().mlora_base_gemm(_ptr(X), _ptr(W0), _ptr(Y), n, din, dout, _stream()), "mlora_base_gemm")
    return Y


def shrink_max_chunks(din: int) -> int:
    return int(lib().mlora_shrink_max_chunks(din))


def _rows_check(pool: Pool, X, n: int):
    _bf16_dev(X, "X")
    if tuple(X.shape) != (n, pool.din):
        raise ValueError(f"X must be [{n}][{pool.din}]")


def shrink(pool: Pool, proj: int, X, seg_ws, n_chunks: int = 1, T=None):
    """Returns T, fp32 [n_chunks][n][max_rank] partial t in sorted-row order."""
    torch = _torch()
    n = X.shape[0]
    _rows_check(pool, X, n)
    if T is None:
        T = torch.zeros((n_chunks, n, pool.max_rank), dtype=torch.float32, device=X.device)
    _check(lib().mlora_shrink(pool.handle, proj, _ptr(X), _ptr(seg_ws), n, _ptr(T), n_chunks, _stream()),
           "mlora_shrink")
    return T


def expand(pool: Pool, proj: int, T, seg_ws, Y):
    """Y[perm[j]] += s * Up t_j (in place), t_j summed over T's chunks."""
    torch = _torch()
    _bf16_dev(Y, "Y")
    n = Y.shape[0]
    if T.dtype != torch.float32 or T.dim() != 3 or tuple(T.shape[1:]) != (n, pool.max_rank) or not T.is_contiguous():
        raise ValueError(f"T must be contiguous fp32 [chunks][{n}][{pool.max_rank}]")
    _check(lib().mlora_expand(pool.handle, proj, _ptr(T), T.shape[0], _ptr(seg_ws), _ptr(Y), n, _stream()),
           "mlora_expand")
    return Y


def fused(pool: Pool, proj: int, X, seg_ws, Y):
    n = X.shape[0]
    _rows_check(pool, X, n)
    _bf16_dev(Y, "Y")
    _check(lib().mlora_fused(pool.handle, proj, _ptr(X), _ptr(seg_ws), _ptr(Y), n, _stream()), "mlora_fused")
    return Y


def new_work(pool: Pool, n: int, device=None):
    """A zeroed work buffer for apply / the per-row path (mlora_work_bytes)."""
    torch = _torch()
    return torch.zeros(max(work_bytes(pool, n), 256), dtype=torch.uint8,
                       device=device if device is not None else torch.device("cuda", torch.cuda.current_device()))


def rows_t(pool: Pool, work, n: int):
    """The T region of a per-row work buffer: fp32 [n][max_rank] view."""
    torch = _torch()
    return work[: n * pool.max_rank * 4].view(torch.float32).view(n, pool.max_rank)


def shrink_rows(pool: Pool, proj: int, X, seg_ws, work=None):
    """Per-row shrink; returns the work buffer (T = rows_t(pool, work, n))."""
    n = X.shape[0]
    _rows_check(pool, X, n)
    if work is None:
        work = new_work(pool, n, X.device)
    _check(lib().mlora_shrink_rows(pool.handle, proj, _ptr(X), _ptr(seg_ws), n, _ptr(work),
                                   work.numel() * work.element_size(), _stream()), "mlora_shrink_rows")
    return work


def gemm_lora(pool: Pool, proj: int, X, W0, seg_ws, work, Y=None):
    """Y = X W0^T + per-row s * Up t, t from shrink_rows in `work`."""
    torch = _torch()
    n = X.shape[0]
    _rows_check(pool, X, n)
    _bf16_dev(W0, "W0")
    if Y is None:
        Y = torch.empty((n, pool.dout), dtype=torch.bfloat16, device=X.device)
    _bf16_dev(Y, "Y")
    _check(lib().mlora_gemm_lora(pool.handle, proj, _ptr(X), _ptr(W0), _ptr(seg_ws), _ptr(work),
                                 work.numel() * work.element_size(), _ptr(Y), n, _stream()), "mlora_gemm_lora")
    return Y


def work_bytes(pool: Pool, n: int) -> int:
    return int(lib().mlora_work_bytes(pool.handle, n))


def plan(pool: Pool, n: int, variant: str = "auto"):
    """(variant name, shrink slices) that apply() runs for a batch of n rows."""
    v, c = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().mlora_plan(pool.handle, n, VARIANTS[variant], ctypes.byref(v), ctypes.byref(c)), "mlora_plan")
    return {0: "auto", 1: "split", 2: "fused", 3: "rows"}[v.value], c.value


def apply(pool: Pool, proj: int, X, W0, seg_ws, Y=None, work=None, variant: str = "auto"):
    """The whole layer for one projection: Y = X W0^T + each row's delta."""
    torch = _torch()
    n = X.shape[0]
    _rows_check(pool, X, n)
    _bf16_dev(W0, "W0")
    if tuple(W0.shape) != (pool.dout, pool.din):
        raise ValueError(f"W0 must be [{pool.dout}][{pool.din}]")
    if Y is None:
        Y = torch.empty((n, pool.dout), dtype=torch.bfloat16, device=X.device)
    _bf16_dev(Y, "Y")
    if work is None:
        work = new_work(pool, n, X.device)
    _check(lib().mlora_apply(pool.handle, proj, _ptr(X), _ptr(W0), _ptr(seg_ws), _ptr(Y), n, _ptr(work),
                             work.numel() * work.element_size(), VARIANTS[variant], _stream()), "mlora_apply")
    return Y


def forward(pool: Pool, proj: int, X, W0, row_adapter, seg_ws=None, Y=None, work=None, variant: str = "auto"):
    """Segment build and the layer for one projection in one call (the
    results of build_segments followed by apply).  Returns (Y, seg_ws); seg_ws
    serves apply on the batch's other projections."""
    torch = _torch()
    n = X.shape[0]
    _rows_check(pool, X, n)
    _bf16_dev(W0, "W0")
    if tuple(W0.shape) != (pool.dout, pool.din):
        raise ValueError(f"W0 must be [{pool.dout}][{pool.din}]")
    if row_adapter.dtype != torch.int32 or not row_adapter.is_cuda or not row_adapter.is_contiguous():
        raise TypeError("row_adapter must be a contiguous int32 CUDA tensor")
    if row_adapter.shape[0] != n:
        raise ValueError("row_adapter must have one id per row of X")
    nb = segments_bytes(n)
    if seg_ws is None:
        seg_ws = torch.empty(nb // 4, dtype=torch.int32, device=X.device)
    elif seg_ws.numel() * seg_ws.element_size() < nb:
        raise ValueError("seg_ws too small")
    if Y is None:
        Y = torch.empty((n, pool.dout), dtype=torch.bfloat16, device=X.device)
    _bf16_dev(Y, "Y")
    if work is None:
        work = new_work(pool, n, X.device)
    _check(lib().mlora_forward(pool.handle, proj, _ptr(X), _ptr(W0), _ptr(row_adapter), _ptr(seg_ws), _ptr(Y), n,
                               _ptr(work), work.numel() * work.element_size(), VARIANTS[variant], _stream()),
           "mlora_forward")
    return Y, seg_ws


def forward_static(pool: Pool, proj: int, X, W0, row_adapter, seg_ws=None, Y=None, variant: str = "auto"):
    """forward() with the library's static scratch in place of a work buffer
    (the call allocates no device memory).  Returns (Y, seg_ws)."""
    torch = _torch()
    n = X.shape[0]
    _rows_check(pool, X, n)
    _bf16_dev(W0, "W0")
    if tuple(W0.shape) != (pool.dout, pool.din):
        raise ValueError(f"W0 must be [{pool.dout}][{pool.din}]")
    if row_adapter.dtype != torch.int32 or not row_adapter.is_cuda or not row_adapter.is_contiguous():
        raise TypeError("row_adapter must be a contiguous int32 CUDA tensor")
    if row_adapter.shape[0] != n:
        raise ValueError("row_adapter must have one id per row of X")
    nb = segments_bytes(n)
    if seg_ws is None:
        seg_ws = torch.empty(nb // 4, dtype=torch.int32, device=X.device)
    elif seg_ws.numel() * seg_ws.element_size() < nb:
        raise ValueError("seg_ws too small")
    if Y is None:
        Y = torch.empty((n, pool.dout), dtype=torch.bfloat16, device=X.device)
    _bf16_dev(Y, "Y")
    _check(lib().mlora_forward_static(pool.handle, proj, _ptr(X), _ptr(W0), _ptr(row_adapter), _ptr(seg_ws), _ptr(Y),
                                      n, VARIANTS[variant], _stream()), "mlora_forward_static")
    return Y, seg_ws


STATIC_SCRATCH_BYTES = 20 << 20


def merge(pool: Pool, adapter_id: int, proj: int, W0, sign: float = 1.0):
    """W0 (device bf16 [dout][din], in place) += sign * s_a * Up_a Down_a."""
    torch = _torch()
    if W0.dtype != torch.bfloat16 or not W0.is_cuda or not W0.is_contiguous() or W0.dim() != 2:
        raise ValueError("W0 must be a contiguous CUDA bfloat16 matrix")
    if tuple(W0.shape) != (pool.dout, pool.din):
        raise ValueError(f"W0 must be [{pool.dout}][{pool.din}], got {tuple(W0.shape)}")
    _check(lib().mlora_merge(pool.handle, adapter_id, proj, _ptr(W0), ctypes.c_float(sign), _stream()),
           f"mlora_merge({adapter_id})")
    return W0


class KVCache:
    """Pages of an 8-bit key/value cache on the current device: e4m3 codes
    with a power-of-two scale for each page, head and side (layouts and
    limits: include/mlora.h).

    storage: (k, v, k_scale, v_scale) of the documented shapes to use in
    place of newly allocated, zeroed buffers."""

    def __init__(self, n_layers: int, n_blocks: int, kv_heads: int, dim: int, block: int = 16, storage=None):
        torch = _torch()
        self.n_layers, self.n_blocks, self.kv_heads, self.dim, self.block = n_layers, n_blocks, kv_heads, dim, block
        if min(n_layers, n_blocks, kv_heads, dim, block) < 1 or block % 16 != 0:
            raise ValueError("KVCache sizes must be positive and block a multiple of 16")
        shapes = ((n_layers, n_blocks, kv_heads, block, dim), (n_layers, n_blocks, kv_heads, block // 16, dim, 16),
                  (n_layers, n_blocks, kv_heads), (n_layers, n_blocks, kv_heads))
        dtypes = (torch.uint8, torch.uint8, torch.float32, torch.float32)
        if storage is None:
            dev = torch.device("cuda", torch.cuda.current_device())
            storage = tuple(torch.zeros(s, dtype=t, device=dev) for s, t in zip(shapes, dtypes))
        if len(storage) != 4:
            raise ValueError("storage must be (k, v, k_scale, v_scale)")
        for name, x, shape, dt in zip(("k", "v", "k_scale", "v_scale"), storage, shapes, dtypes):
            if not isinstance(x, torch.Tensor) or x.dtype != dt or not x.is_cuda or not x.is_contiguous():
                raise TypeError(f"storage: {name} must be a contiguous {dt} CUDA tensor")
            if tuple(x.shape) != shape:
                raise ValueError(f"storage: {name} has shape {tuple(x.shape)}, expected {shape}")
            if x.get_device() != storage[0].get_device():
                raise ValueError(f"storage: {name} is on another device than k")
        self.k, self.v, self.k_scale, self.v_scale = storage
        self.device_index = self.k.get_device()
        self._d = _KVCacheDesc(n_layers, kv_heads, dim, block, n_blocks, *(x.data_ptr() for x in storage))
        self._ref = ctypes.addressof(self._d)


class KVBatch:
    """Sequences of one batch and their new rows, all device int32: table
    [n_seq][width] of page ids, kv_len [n_seq] tokens with the new ones,
    row_off [n_seq + 1] offsets of each sequence's rows.  The tensors are kept,
    not copied: a program that updates them in place (as a captured graph
    does) keeps the object.  max_new bounds the rows of one sequence (n_rows
    where it is not given)."""

    def __init__(self, table, kv_len, row_off, n_rows: int, max_new: Optional[int] = None):
        torch = _torch()
        for name, x, nd in (("table", table, 2), ("kv_len", kv_len, 1), ("row_off", row_off, 1)):
            if not isinstance(x, torch.Tensor) or x.dtype != torch.int32 or not x.is_cuda or x.dim() != nd:
                raise TypeError(f"{name} must be an int32 CUDA tensor of {nd} dimension(s)")
            if x.shape[-1] > 1 and x.stride(-1) != 1:
                raise TypeError(f"{name} must be dense in its last dimension")
            if x.get_device() != table.get_device():
                raise ValueError(f"{name} is on another device than table")
        n_seq = kv_len.shape[0]
        if table.shape[0] != n_seq or row_off.shape[0] != n_seq + 1:
            raise ValueError(f"table must have {n_seq} rows and row_off {n_seq + 1} entries, as kv_len has {n_seq}")
        self.table, self.kv_len, self.row_off, self.n_rows, self.n_seq = table, kv_len, row_off, n_rows, n_seq
        self.max_new = n_rows if max_new is None else max_new
        self.device_index = table.get_device()
        width = table.shape[1]
        self._d = _KVBatchDesc(table.data_ptr(), kv_len.data_ptr(), row_off.data_ptr(), n_seq, width,
                               table.stride(0) if n_seq > 1 else width, n_rows, self.max_new)
        self._ref = ctypes.addressof(self._d)


def _kv_rows(x, name: str, cache: KVCache, batch: KVBatch, heads: int):
    """Checks bf16 rows [n_rows][heads][dim] and where they and the batch are;
    strides in elements."""
    device = cache.device_index
    if x.dtype is not _torch().bfloat16 or x.get_device() != device:
        raise TypeError(f"{name} must be a bfloat16 tensor on cuda:{device}, as the cache is")
    if batch.device_index != device:
        raise ValueError(f"the batch must be on cuda:{device}, as the cache is")
    shape = x.shape
    if len(shape) != 3 or shape[0] != batch.n_rows or shape[2] != cache.dim or (heads and shape[1] != heads):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected [{batch.n_rows}][{heads or 'heads'}][{cache.dim}]")
    st = x.stride()
    if st[2] != 1:
        raise TypeError(f"{name} must be dense in its channels")
    return st


def _raw_stream(device: int) -> int:
    """The current stream of cuda:`device`, which has to be the current device:
    a launch goes to that one, and to its default stream where the handle is
    that of a default stream."""
    C = _torch()._C
    if C._cuda_getDevice() != device:
        raise ValueError(f"the tensors are on cuda:{device}, the current device is cuda:{C._cuda_getDevice()}")
    # the handle alone: building a Stream object costs as much as a small launch
    return C._cuda_getCurrentRawStream(device)


def _kv_stream(cache: KVCache) -> int:
    return _raw_stream(cache.device_index)


def kv_append(cache: KVCache, layer: int, k, v, batch: KVBatch) -> None:
    """Quantises the batch's new rows, bf16 [n_rows][kv_heads][dim] (slices
    of a joint projection's output serve as they are), into the cache."""
    st = _kv_rows(k, "k", cache, batch, cache.kv_heads)
    if _kv_rows(v, "v", cache, batch, cache.kv_heads) != st:
        k, v = k.contiguous(), v.contiguous()
        st = k.stride()
    status = lib().mlora_kv_append(cache._ref, layer, k.data_ptr(), v.data_ptr(), st[0], st[1], batch._ref,
                                   _kv_stream(cache))
    if status != OK:
        raise MloraError(status, "mlora_kv_append")


def kv_read(cache: KVCache, layer: int, batch: KVBatch):
    """The batch's rows of the cache as bf16: (k, v), [n_rows][kv_heads][dim]."""
    torch = _torch()
    if batch.device_index != cache.device_index:
        raise ValueError(f"the batch must be on cuda:{cache.device_index}, as the cache is")
    shape, dev = (batch.n_rows, cache.kv_heads, cache.dim), cache.k.device
    k = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    v = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    status = lib().mlora_kv_read(cache._ref, layer, batch._ref, k.data_ptr(), v.data_ptr(), _kv_stream(cache))
    if status != OK:
        raise MloraError(status, "mlora_kv_read")
    return k, v


def kv_work_bytes(cache: KVCache, batch: KVBatch, heads: int) -> int:
    return int(lib().mlora_kv_work_bytes(cache._ref, batch._ref, heads))


def new_kv_work(cache: KVCache, batch: KVBatch, heads: int):
    """A work buffer for kv_attention with `heads` query heads; it serves
    every layer, and every batch that needs no more bytes (kv_work_bytes)."""
    torch = _torch()
    return torch.empty(max(kv_work_bytes(cache, batch, heads), 256), dtype=torch.uint8, device=cache.k.device)


def kv_attention(cache: KVCache, layer: int, q, batch: KVBatch, causal: bool = True, window: int = 0,
                 scale: Optional[float] = None, work=None, out=None):
    """Attention of q, bf16 [n_rows][heads][dim], over the batch's sequences;
    scale defaults to dim ** -0.5.  Returns bf16 [n_rows][heads][dim]."""
    torch = _torch()
    rs, hs, _ = _kv_rows(q, "q", cache, batch, 0)
    shape = (batch.n_rows, q.shape[1], cache.dim)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=cache.k.device)
    elif tuple(_bf16_dev(out, "out").shape) != shape or out.get_device() != cache.device_index:
        raise ValueError(f"out must be {list(shape)} on cuda:{cache.device_index}, as the cache is")
    if work is None:
        work = new_kv_work(cache, batch, shape[1])
    elif not isinstance(work, torch.Tensor) or work.get_device() != cache.device_index or not work.is_contiguous():
        raise TypeError(f"work must be a contiguous tensor on cuda:{cache.device_index}, as the cache is")
    status = lib().mlora_kv_attention(cache._ref, layer, q.data_ptr(), rs, hs, shape[1], batch._ref, causal, window,
                                      cache.dim ** -0.5 if scale is None else scale, out.data_ptr(), work.data_ptr(),
                                      work.nbytes, _kv_stream(cache))
    if status != OK:
        raise MloraError(status, "mlora_kv_attention")
    return out


def _on_device(t, name: str, dtype, device: int, shape=None):
    """Checks a contiguous tensor of `dtype` on cuda:`device`."""
    if (not isinstance(t, _torch().Tensor) or t.dtype is not dtype or t.get_device() != device
            or not t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous {dtype} tensor on cuda:{device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _work(work, device: int):
    if not isinstance(work, _torch().Tensor) or work.get_device() != device or not work.is_contiguous():
        raise TypeError(f"work must be a contiguous tensor on cuda:{device}")
    return work


class Q4Weight:
    """A weight [dout][din] in 4 bits: codes uint8 [dout][din / 2], two e2m1
    codes a byte with the lower half first, and scales uint8 [dout][din / 32],
    byte b standing for 2^(b - 127) (include/mlora.h).  The tensors are kept,
    not copied."""

    def __init__(self, codes, scales):
        torch = _torch()
        for name, t in (("codes", codes), ("scales", scales)):
            if (not isinstance(t, torch.Tensor) or t.dtype is not torch.uint8 or not t.is_cuda or t.dim() != 2
                    or not t.is_contiguous()):
                raise TypeError(f"{name} must be a contiguous uint8 CUDA matrix")
        self.dout, self.din = codes.shape[0], 2 * codes.shape[1]
        if self.din < 32 or self.din % 32 or tuple(scales.shape) != (self.dout, self.din // 32):
            raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} are not "
                             "[dout][din / 2] and [dout][din / 32]")
        if scales.get_device() != codes.get_device():
            raise ValueError("scales is on another device than codes")
        self._hold(codes, scales)

    def _hold(self, codes, scales):
        self.codes, self.scales = codes, scales
        self.device_index = codes.get_device()
        self._d = _Q4Desc(codes.data_ptr(), scales.data_ptr(), self.din, self.dout)
        self._ref = ctypes.addressof(self._d)


def q4_quantize(W) -> Q4Weight:
    """W, device bf16 [dout][din] with din a multiple of 32, in 4 bits."""
    torch = _torch()
    if _bf16_dev(W, "W").dim() != 2 or W.shape[1] < 32 or W.shape[1] % 32:
        raise ValueError(f"W has shape {tuple(W.shape)}, expected [dout][din], din a multiple of 32")
    w = Q4Weight.__new__(Q4Weight)
    w.dout, w.din = W.shape
    w._hold(W.new_empty((w.dout, w.din // 2), dtype=torch.uint8), W.new_empty((w.dout, w.din // 32), dtype=torch.uint8))
    _check(lib().mlora_q4_quantize(W.data_ptr(), w.dout, w.din, w._d.codes, w._d.scales, _raw_stream(w.device_index)),
           "mlora_q4_quantize")
    return w


def q4_dequantize(w: Q4Weight, out=None):
    """The weight as bf16 [dout][din] (every 4-bit weight is a bf16 value)."""
    torch = _torch()
    if out is None:
        out = w.codes.new_empty((w.dout, w.din), dtype=torch.bfloat16)
    _on_device(out, "out", torch.bfloat16, w.device_index, (w.dout, w.din))
    _check(lib().mlora_q4_dequantize(w._ref, out.data_ptr(), _raw_stream(w.device_index)), "mlora_q4_dequantize")
    return out


def _pool_handle(pool: Optional[Pool], w: Q4Weight):
    if pool is None:
        return None
    if (pool.dout, pool.din) != (w.dout, w.din):
        raise ValueError(f"the weight is [{w.dout}][{w.din}], the pool's projections are [{pool.dout}][{pool.din}]")
    if pool.meta.get_device() != w.device_index:
        raise ValueError(f"the pool must be on cuda:{w.device_index}, as the weight is")
    return pool.handle


def q4_work_bytes(w: Q4Weight, n: int, pool: Optional[Pool] = None) -> int:
    return int(lib().mlora_q4_work_bytes(w._ref, _pool_handle(pool, w), n))


def new_q4_work(w: Q4Weight, n: int, pool: Optional[Pool] = None):
    """A work buffer for q4_gemm of n rows, or with `pool` for q4_apply."""
    torch = _torch()
    return torch.empty(max(q4_work_bytes(w, n, pool), 256), dtype=torch.uint8, device=w.codes.device)


def _q4_rows(X, w: Q4Weight, Y):
    torch = _torch()
    _on_device(X, "X", torch.bfloat16, w.device_index)
    if X.dim() != 2 or X.shape[1] != w.din:
        raise ValueError(f"X has shape {tuple(X.shape)}, expected [n][{w.din}]")
    shape = (X.shape[0], w.dout)
    if Y is None:
        return X.new_empty(shape)
    return _on_device(Y, "Y", torch.bfloat16, w.device_index, shape)


def q4_gemm(X, w: Q4Weight, Y=None, work=None):
    """Y = X W^T, X device bf16 [n][din]."""
    Y = _q4_rows(X, w, Y)
    n = X.shape[0]
    work = new_q4_work(w, n) if work is None else _work(work, w.device_index)
    status = lib().mlora_q4_gemm(w._ref, X.data_ptr(), Y.data_ptr(), n, work.data_ptr(), work.nbytes,
                                 _raw_stream(w.device_index))
    if status != OK:
        raise MloraError(status, "mlora_q4_gemm")
    return Y


def q4_apply(pool: Pool, proj: int, X, w: Q4Weight, seg_ws, Y=None, work=None):
    """apply() with the base weight in 4 bits: Y = X W^T + each row's delta."""
    h = _pool_handle(pool, w)
    Y = _q4_rows(X, w, Y)
    n = X.shape[0]
    _on_device(seg_ws, "seg_ws", _torch().int32, w.device_index)
    if seg_ws.nbytes < segments_bytes(n):
        raise ValueError("seg_ws too small")
    work = new_q4_work(w, n, pool) if work is None else _work(work, w.device_index)
    status = lib().mlora_q4_apply(h, proj, X.data_ptr(), w._ref, seg_ws.data_ptr(), Y.data_ptr(), n, work.data_ptr(),
                                  work.nbytes, _raw_stream(w.device_index))
    if status != OK:
        raise MloraError(status, "mlora_q4_apply")
    return Y


class Rotary:
    """Frequencies of a rotation of the first `dim` channels of a head, on the
    current device.  Pair i turns by position * freqs[i] radians; freqs
    defaults to base^(-2i / dim).  A pair is made of channels i and
    i + dim / 2, or 2i and 2i + 1 (interleaved); the rotated pairs are
    multiplied by `factor`."""

    def __init__(self, dim: int, base: float = 10000.0, freqs=None, interleaved: bool = False, factor: float = 1.0):
        torch = _torch()
        if dim < 8 or dim % 8:
            raise ValueError(f"Rotary: dim {dim} is not a positive multiple of 8")
        if freqs is None:
            freqs = base ** (-2.0 * np.arange(dim // 2) / dim)
        elif isinstance(freqs, torch.Tensor):
            freqs = freqs.detach().cpu().double().numpy()
        freqs = np.asarray(freqs, np.float64)
        if freqs.shape != (dim // 2,) or not np.isfinite(freqs).all():
            raise ValueError(f"Rotary: freqs must be {dim // 2} finite numbers")
        turns = freqs / (2 * np.pi)
        # revolutions modulo 1 in 64-bit fixed point (a float64 fraction has at most 53 significant bits)
        fixed = [int(t * 2.0 ** 64) % (1 << 64) for t in (turns - np.floor(turns)).tolist()]
        self.dim, self.interleaved, self.factor = dim, bool(interleaved), float(factor)
        self.freq = torch.from_numpy(np.array(fixed, np.uint64).view(np.int64)).to(
            torch.device("cuda", torch.cuda.current_device()))
        self.device_index = self.freq.get_device()
        self._d = _RotaryDesc(self.freq.data_ptr(), dim, int(self.interleaved), self.factor)
        self._ref = ctypes.addressof(self._d)


# mlora_head_rows as bytes: building one costs a third of filling a ctypes structure
_head_rows = struct.Struct("<QQqqqqQi4x").pack


def _qk_rows(x, name: str, shape, weight, out, device: int):
    """Checks one side of qk_norm_rotary; its output and its descriptor."""
    torch = _torch()
    if x.dtype is not torch.bfloat16 or x.get_device() != device:
        raise TypeError(f"{name} must be a bfloat16 tensor on cuda:{device}, as the batch is")
    if len(shape) != 3:
        raise ValueError(f"{name} must be [n_rows][heads][dim]")
    if out is None:  # (empty_like takes a third of the time of empty)
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    elif out.dtype is not torch.bfloat16 or out.get_device() != device:
        raise TypeError(f"{name}_out must be a bfloat16 tensor on cuda:{device}, as the batch is")
    elif out.shape != shape:
        raise ValueError(f"{name}_out has shape {tuple(out.shape)}, expected {tuple(shape)}")
    rs, hs, cs = x.stride()
    ors, ohs, ocs = out.stride()
    if cs != 1 or ocs != 1:
        raise TypeError(f"{name} and {name}_out must be dense in their channels")
    w = 0 if weight is None else _on_device(weight, name + "_weight", torch.bfloat16, device, shape[2:]).data_ptr()
    return out, _head_rows(x.data_ptr(), out.data_ptr(), rs, hs, ors, ohs, w, shape[1])


def qk_norm_rotary(q, k, batch: KVBatch, rotary: Rotary, q_weight=None, k_weight=None, eps: float = 1e-6,
                   q_out=None, k_out=None):
    """The norm of each head of q and k, bf16 [n_rows][heads][dim] (slices of a
    joint projection's output serve as they are), with weights bf16 [dim]
    (None: no norm), then the rotation by each row's position in `batch`.  k
    may be None.  q_out=q and k_out=k work in place; otherwise the outputs are
    new.  Rows past the last sequence are left as they are.  Returns (q, k)."""
    device, shape = batch.device_index, q.shape
    if rotary.device_index != device:
        raise ValueError(f"rotary must be on cuda:{device}, as the batch is")
    q_out, qs = _qk_rows(q, "q", shape, q_weight, q_out, device)
    n, _, dim = shape
    ks = None
    if k is not None:
        kshape = k.shape
        k_out, ks = _qk_rows(k, "k", kshape, k_weight, k_out, device)
        if kshape[0] != n or kshape[2] != dim:
            raise ValueError(f"k has shape {tuple(kshape)}, expected [{n}][heads][{dim}]")
    elif k_weight is not None or k_out is not None:
        raise ValueError("k_weight and k_out need k")
    if n != batch.n_rows:
        raise ValueError(f"q has {n} rows, the batch {batch.n_rows}")
    status = lib().mlora_qk_norm_rotary(batch._ref, dim, rotary._ref, qs, ks, eps, _raw_stream(device))
    if status != OK:
        raise MloraError(status, "mlora_qk_norm_rotary")
    return q_out, k_out


def sample_work_bytes(n: int, vocab: int) -> int:
    """0: sample() needs no work buffer (the argument is reserved)."""
    return int(lib().mlora_sample_work_bytes(n, vocab))


def new_sample_work(n: int, vocab: int, device=None):
    """A work buffer for sample() of n rows of `vocab` logits: an empty one."""
    torch = _torch()
    return torch.empty(sample_work_bytes(n, vocab), dtype=torch.uint8,
                       device=device if device is not None else torch.device("cuda", torch.cuda.current_device()))


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, out=None, work=None):
    """One token a row of logits, device bf16 or fp32 [n][vocab], drawn with the
    random numbers u, fp32 [n] in [0, 1).  temperature, top_p, min_p (fp32
    [n]) and top_k (int32 [n]) are each row's own; None leaves that out.
    Returns int32 [n] (-1 for a row without any logit above -infinity); the
    definition is in include/mlora.h."""
    torch = _torch()
    if not isinstance(logits, torch.Tensor) or logits.dtype not in (torch.bfloat16, torch.float32) or not logits.is_cuda:
        raise TypeError("logits must be a bfloat16 or float32 CUDA tensor")
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise TypeError("logits must be [n][vocab], dense in the vocabulary")
    (n, vocab), device = logits.shape, logits.get_device()
    _on_device(u, "u", torch.float32, device, (n,))
    ptr = []
    for name, t, dt in (("temperature", temperature, torch.float32), ("top_k", top_k, torch.int32),
                        ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32)):
        ptr.append(None if t is None else _on_device(t, name, dt, device, (n,)).data_ptr())
    if out is None:
        out = torch.empty_like(u, dtype=torch.int32)
    else:
        _on_device(out, "out", torch.int32, device, (n,))
    wp = wn = 0
    if work is not None:
        wp, wn = _work(work, device).data_ptr(), work.nbytes
    status = lib().mlora_sample(logits.data_ptr(), logits.dtype is torch.float32, logits.stride(0) if n > 1 else vocab,
                                n, vocab, u.data_ptr(), *ptr, out.data_ptr(), wp, wn, _raw_stream(device))
    if status != OK:
        raise MloraError(status, "mlora_sample")
    return out


def hbm_copy(dst, src, nbytes: Optional[int] = None):
    nb = src.numel() * src.element_size() if nbytes is None else nbytes
    _check(lib().mlora_hbm_copy(_ptr(dst), _ptr(src), nb, _stream()), "mlora_hbm_copy")
    return dst


def hbm_read(src, out, nbytes: Optional[int] = None):
    """Streams src and XORs its 32-bit words into out[0] (device int32)."""
    nb = src.numel() * src.element_size() if nbytes is None else nbytes
    _check(lib().mlora_hbm_read(_ptr(src), nb, _ptr(out), _stream()), "mlora_hbm_read")
    return out


def hbm_read_lds(src, out, nbytes: Optional[int] = None):
    """Streams src through LDS DMA in 1 KiB pieces (mlora_hbm_read_lds)."""
    nb = src.numel() * src.element_size() if nbytes is None else nbytes
    _check(lib().mlora_hbm_read_lds(_ptr(src), nb, _ptr(out), _stream()), "mlora_hbm_read_lds")
    return out


_timing_armed = [0]


def timing_arm(n_launches: int):
    """Arms kernel start/end events on the library's next n_launches kernel
    launches (a measurement aid)."""
    _check(lib().mlora_timing_arm(n_launches), "mlora_timing_arm")
    _timing_armed[0] = n_launches


def timing_read() -> list:
    """Waits for the armed events: [(kernel name, milliseconds)] per marked
    launch, in launch order."""
    cap = max(_timing_armed[0], 1)
    ms = (ctypes.c_float * cap)()
    n = ctypes.c_int32(0)
    _check(lib().mlora_timing_read(ms, cap, ctypes.byref(n)), "mlora_timing_read")
    return [(lib().mlora_timing_name(i).decode(), float(ms[i])) for i in range(n.value)]
