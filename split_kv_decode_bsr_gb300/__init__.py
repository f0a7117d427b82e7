"""Python binding of libsta (masked MHA over a two-level BSR + bitmap mask, split-KV decode).

Thin ctypes marshalling over the C ABI in ``include/sta.h``: every function of the
same name calls the CUDA library, on the current torch stream, with device memory
held in torch tensors. There is no fallback: when ``libsta.so`` has not been built
(``python -m split_kv_decode_bsr_gb300.build`` or ``__graft_entry__.build()``) every
call raises.

Operations (sources):
  * ``sta_encode_mask`` -- STOF's two-level storage format ("Accelerating Sparse
    Transformer Inference on GPU", 手法 / 2 段階ストレージ形式).
  * ``sta_mha_fwd`` -- masked MHA forward with the row-wise / block-wise kernels and
    the analytic selector (same page, デュアルカーネル戦略 / カーネル選択).
  * ``sta_decode_splitkv`` / ``sta_merge_lse`` -- Cleave's Split operator on the KV
    reduction of GQA decode with a log-sum-exp merge ("Cleave: Scaling Tensor
    Program Optimization ...", Split演算子によるSplit-Kの対応).
  * ``sta_rope``, ``sta_rope_append_paged``, ``sta_chunk_fwd_paged``, ``sta_pages_*`` --
    serving over the paged KV cache of the paged decode: rotary positions, the write of new
    tokens, the attention of chunks of new tokens, and the bookkeeping of pages.
"""

from __future__ import annotations

import contextlib
import ctypes as C
import functools
import math
import os
import threading
from dataclasses import dataclass
from typing import List, Optional, Sequence

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsta.so")

STA_OK, STA_ERR_INVALID_ARG, STA_ERR_UNSUPPORTED, STA_ERR_WORKSPACE, STA_ERR_CUDA = 0, 1, 2, 3, 4
STA_BF16, STA_F32 = 0, 1
STA_MASK_PATTERN, STA_MASK_DENSE_U8, STA_MASK_DENSE_BITS = 0, 1, 2
STA_KERNEL_AUTO, STA_KERNEL_BLOCK, STA_KERNEL_ROW, STA_KERNEL_MIXED = 0, 1, 2, 3
STA_O_BHLD, STA_O_BLHD = 0, 1
STA_ROPE_HALF, STA_ROPE_INTERLEAVED = 0, 1
STA_ROPE_SCALE_NONE, STA_ROPE_SCALE_LINEAR, STA_ROPE_SCALE_BLEND = 0, 1, 2
_KERNELS = {"auto": STA_KERNEL_AUTO, "block": STA_KERNEL_BLOCK, "row": STA_KERNEL_ROW}

EXPORTED = ("sta_encode_mask", "sta_tile_lists_bytes", "sta_mha_fwd", "sta_mha_fwd_splitkv", "sta_mha_fwd_layout",
            "sta_bias_residual_layernorm", "sta_validate_mask", "sta_mla_decode", "sta_mha_select_kernel", "sta_decode_splitkv",
            "sta_decode_splitkv_noalloc", "sta_decode_splitkv_paged", "sta_merge_lse", "sta_status_string", "sta_device_error",
            "sta_check_bounded_wait", "sta_last_cuda_error", "sta_last_cuda_error_string", "sta_rope",
            "sta_rope_append_paged", "sta_chunk_fwd_paged", "sta_pages_copy", "sta_pages_grow", "sta_pages_fork",
            "sta_pages_free", "sta_pages_compact")

BIG = 1 << 40


class StaError(RuntimeError):
    """A library call returned a status other than STA_OK (.status holds it)."""
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = f"{fn} failed: {status_string(status)} ({status})"
        if status == STA_ERR_CUDA:
            msg += f": {lib().sta_last_cuda_error_string().decode()} ({lib().sta_last_cuda_error()})"
        super().__init__(msg)


class _MaskSrc(C.Structure):
    _fields_ = [("kind", C.c_int32), ("causal", C.c_int32), ("win_lo", C.c_int64), ("win_hi", C.c_int64),
                ("n_global_cols", C.c_int64), ("data", C.c_void_p)]


class _BsrMask(C.Structure):
    _fields_ = [("n_mask_heads", C.c_int32), ("Lq", C.c_int32), ("Lk", C.c_int32), ("ot_rows", C.c_int32),
                ("ot_cols", C.c_int32), ("full_row_ptr", C.c_void_p), ("full_col_idx", C.c_void_p),
                ("part_row_ptr", C.c_void_p), ("part_col_idx", C.c_void_p), ("part_bitmap", C.c_void_p),
                ("n_full", C.c_int64), ("n_part", C.c_int64), ("n_valid", C.c_int64),
                ("head_tiles", C.c_void_p), ("tile_lists", C.c_void_p), ("head_valid", C.c_void_p)]


class _RopeParams(C.Structure):
    _fields_ = [("rot_dim", C.c_int32), ("layout", C.c_int32), ("scaling", C.c_int32), ("mscale", C.c_float),
                ("base", C.c_double), ("factor", C.c_double), ("orig_len", C.c_double), ("low_turns", C.c_double),
                ("high_turns", C.c_double), ("freqs", C.c_void_p)]


_lock = threading.Lock()
_lib_handle = None


def lib():
    """The loaded libsta.so (raises if it has not been built)."""
    global _lib_handle
    with _lock:
        if _lib_handle is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libsta.so not built at {LIB_PATH}; run split_kv_decode_bsr_gb300.build.build()")
            h = C.CDLL(LIB_PATH)
            P, i32, f32, sz = C.c_void_p, C.c_int, C.c_float, C.POINTER(C.c_size_t)
            h.sta_encode_mask.argtypes = [P, i32, i32, i32, C.POINTER(_BsrMask), P, sz, P]
            h.sta_tile_lists_bytes.argtypes = [i32, i32, i32]
            h.sta_tile_lists_bytes.restype = C.c_size_t
            h.sta_mha_fwd.argtypes = [P, P, P, P, P, C.POINTER(_BsrMask), P, i32, i32, i32, i32, i32, i32, f32, i32, P]
            h.sta_mha_fwd_splitkv.argtypes = [P, P, P, P, P, C.POINTER(_BsrMask), P, i32, i32, i32, i32, i32, i32, f32,
                                              i32, i32, P, sz, P]
            h.sta_mha_fwd_layout.argtypes = [P, P, P, P, P, C.POINTER(_BsrMask), P, i32, i32, i32, i32, i32, i32, f32,
                                             i32, i32, i32, P, sz, P]
            h.sta_bias_residual_layernorm.argtypes = [P, P, P, P, P, P, P, C.c_int64, i32, f32, i32, P]
            h.sta_validate_mask.argtypes = [C.POINTER(_BsrMask), C.POINTER(C.c_int)]
            h.sta_mla_decode.argtypes = [P, P, P, P, i32, i32, f32, i32, P, P, P, sz, P]
            h.sta_mha_select_kernel.argtypes = [C.POINTER(_BsrMask), i32, i32, i32, i32, i32, i32]
            h.sta_decode_splitkv.argtypes = [P, P, P, P, P, i32, i32, i32, i32, i32, f32, i32, P, P, P, sz, P]
            h.sta_decode_splitkv_paged.argtypes = [P, P, P, i32, i32, P, P, P, P, i32, i32, i32, i32, i32, f32, i32,
                                                   P, P, P, sz, P]
            h.sta_decode_splitkv_noalloc.argtypes = [P, P, P, P, P, i32, i32, i32, i32, i32, f32, i32, P, P, P]
            h.sta_merge_lse.argtypes = [P, P, i32, i32, i32, P, i32, P, P]
            i64, R = C.c_int64, C.POINTER(_RopeParams)
            h.sta_rope.argtypes = [P, P, P, R, i64, i32, i32, i64, i64, i32, i32, P]
            h.sta_rope_append_paged.argtypes = [P, P, P, i64, i64, i64, P, P, P, i32, i32, P, P, P, P, P, R, i64, i32,
                                                i32, i32, i32, i32, P]
            h.sta_chunk_fwd_paged.argtypes = [P, i64, P, P, i32, i32, P, P, P, P, P, P, i32, i32, i32, i32, i32, f32,
                                              C.POINTER(_MaskSrc), i32, P, P, P, sz, P]
            h.sta_pages_copy.argtypes = [P, i32, C.c_size_t, i32, P, P, i32, P]
            h.sta_pages_grow.argtypes = [P, i32, P, P, P, P, i32, i32, P, P, sz, P]
            h.sta_pages_fork.argtypes = [P, i32, C.c_size_t, P, i32, P, P, P, i32, i32, P, P, i32, P, P, sz, P]
            h.sta_pages_free.argtypes = [P, i32, P, P, P, i32, i32, P, i32, P]
            h.sta_pages_compact.argtypes = [P, i32, C.c_size_t, P, i32, P, P, P, i32, i32, P, P, P, sz, P]
            h.sta_status_string.argtypes = [i32]
            h.sta_status_string.restype = C.c_char_p
            h.sta_device_error.argtypes = [C.POINTER(C.c_int), i32]
            h.sta_check_bounded_wait.argtypes = [C.c_int64, P, P]
            h.sta_last_cuda_error.argtypes = []
            h.sta_last_cuda_error_string.argtypes = []
            h.sta_last_cuda_error_string.restype = C.c_char_p
            for n in EXPORTED:
                if n not in ("sta_status_string", "sta_last_cuda_error_string", "sta_tile_lists_bytes"):
                    getattr(h, n).restype = C.c_int
            _lib_handle = h
    return _lib_handle


def status_string(status: int) -> str:
    """The library's message for a status code."""
    return lib().sta_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != STA_OK:
        raise StaError(fn, status)


def _stream(stream) -> C.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return STA_BF16
    if dt == torch.float32:
        return STA_F32
    raise TypeError(f"unsupported dtype {dt}")


# ---------------------------------------------------------------------------
# mask sources and the encoded mask


@dataclass
class MaskSource:
    """One [Lq, Lk] mask head: a pattern, or dense uint8 / bit-packed device data.

    Pattern: valid(i, j) = (not causal or j <= i) and
                           (win_lo <= j - i <= win_hi or j < n_global_cols).
    Bits: int64/uint64 tensor [Lq, ceil(Lk/64)], element (i, j) at word j >> 6, bit j & 63.
    """
    kind: int
    causal: int = 0
    win_lo: int = -BIG
    win_hi: int = BIG
    n_global_cols: int = 0
    data: Optional[torch.Tensor] = None

    @staticmethod
    def pattern(causal=False, win_lo=-BIG, win_hi=BIG, n_global_cols=0) -> "MaskSource":
        return MaskSource(STA_MASK_PATTERN, int(bool(causal)), int(win_lo), int(win_hi), int(n_global_cols))

    @staticmethod
    def dense_u8(t: torch.Tensor) -> "MaskSource":
        assert t.is_cuda and t.dtype == torch.uint8 and t.dim() == 2 and t.is_contiguous()
        return MaskSource(STA_MASK_DENSE_U8, data=t)

    @staticmethod
    def dense_bits(t: torch.Tensor) -> "MaskSource":
        assert t.is_cuda and t.dtype in (torch.int64, torch.uint64) and t.dim() == 2 and t.is_contiguous()
        return MaskSource(STA_MASK_DENSE_BITS, data=t)


class BsrMask:
    """Encoded two-level mask: device tensors plus host counts (mirrors sta_bsr_mask)."""

    def __init__(self, Hm, Lq, Lk, full_row_ptr, full_col_idx, part_row_ptr, part_col_idx, part_bitmap,
                 n_full, n_part, n_valid):
        self.Hm, self.Lq, self.Lk = Hm, Lq, Lk
        self.ot_rows, self.ot_cols = (Lq + 63) // 64, (Lk + 63) // 64
        self.full_row_ptr, self.full_col_idx = full_row_ptr, full_col_idx
        self.part_row_ptr, self.part_col_idx = part_row_ptr, part_col_idx
        self.part_bitmap = part_bitmap
        self.n_full, self.n_part, self.n_valid = n_full, n_part, n_valid
        self.head_tiles = None  # ctypes int64 array [Hm] when known
        self.head_valid = None  # ctypes int64 array [Hm] when known (with head_tiles: per-head kernel choice)
        self.tile_lists = None  # uint8 device tensor of the block kernel's column lists, when encoded

    def struct(self) -> _BsrMask:
        s = _BsrMask()
        s.n_mask_heads, s.Lq, s.Lk, s.ot_rows, s.ot_cols = self.Hm, self.Lq, self.Lk, self.ot_rows, self.ot_cols
        s.full_row_ptr = self.full_row_ptr.data_ptr()
        s.full_col_idx = self.full_col_idx.data_ptr() if self.n_full else None
        s.part_row_ptr = self.part_row_ptr.data_ptr()
        s.part_col_idx = self.part_col_idx.data_ptr() if self.n_part else None
        s.part_bitmap = self.part_bitmap.data_ptr() if self.n_part else None
        s.n_full, s.n_part, s.n_valid = self.n_full, self.n_part, self.n_valid
        s.head_tiles = C.cast(self.head_tiles, C.c_void_p) if self.head_tiles is not None else None
        s.tile_lists = self.tile_lists.data_ptr() if self.tile_lists is not None else None
        s.head_valid = C.cast(self.head_valid, C.c_void_p) if self.head_valid is not None else None
        return s

    def refill(self, stream=None):
        """Run the encoder's fill call again into this mask's arrays (asynchronous on the stream;
        the same sources, workspace and capacities as the original encode)."""
        arr, out, ws, ws_bytes, _ = self._fill
        _check("sta_encode_mask", lib().sta_encode_mask(arr, self.Hm, self.Lq, self.Lk, C.byref(out), _ptr(ws),
                                                        C.byref(ws_bytes), _stream(stream)))

    def host_arrays(self) -> dict:
        return dict(full_row_ptr=self.full_row_ptr.cpu().numpy(), full_col_idx=self.full_col_idx.cpu().numpy(),
                    part_row_ptr=self.part_row_ptr.cpu().numpy(), part_col_idx=self.part_col_idx.cpu().numpy(),
                    part_bitmap=self.part_bitmap.cpu().numpy().view("uint64").reshape(-1, 64),
                    n_full=self.n_full, n_part=self.n_part, n_valid=self.n_valid)

    def validate(self) -> None:
        """Copy the arrays to the host and run sta_validate_mask on them; raises StaError
        (with .failed_check, the header's check number) when the mask is malformed."""
        a = self.host_arrays()
        tl = self.tile_lists.cpu().numpy() if self.tile_lists is not None else None
        validate_mask_host(a, self.Hm, self.Lq, self.Lk, tile_lists=tl)


def validate_mask_host(arrays: dict, Hm: int, Lq: int, Lk: int, tile_lists=None) -> None:
    """sta_validate_mask on host numpy arrays (keys as BsrMask.host_arrays(); n_valid may be -1
    to skip that check). Raises StaError with .failed_check set when a check fails."""
    import numpy as np

    keep = {k: np.ascontiguousarray(arrays[k], dtype=dt) for k, dt in
            (("full_row_ptr", np.int32), ("full_col_idx", np.int32), ("part_row_ptr", np.int32),
             ("part_col_idx", np.int32), ("part_bitmap", np.uint64))}
    s = _BsrMask()
    s.n_mask_heads, s.Lq, s.Lk = Hm, Lq, Lk
    s.ot_rows, s.ot_cols = (Lq + 63) // 64, (Lk + 63) // 64
    for k, v in keep.items():
        setattr(s, k, v.ctypes.data if v.size else None)
    s.full_row_ptr, s.part_row_ptr = keep["full_row_ptr"].ctypes.data, keep["part_row_ptr"].ctypes.data
    s.n_full, s.n_part, s.n_valid = int(arrays["n_full"]), int(arrays["n_part"]), int(arrays.get("n_valid", -1))
    tl = None if tile_lists is None else np.ascontiguousarray(tile_lists, dtype=np.uint8)
    s.tile_lists = tl.ctypes.data if tl is not None else None
    code = C.c_int(0)
    st = lib().sta_validate_mask(C.byref(s), C.byref(code))
    if st != STA_OK:
        err = StaError("sta_validate_mask", st)
        err.failed_check = code.value
        raise err


def _src_array(srcs: Sequence[MaskSource]):
    arr = (_MaskSrc * len(srcs))()
    for i, s in enumerate(srcs):
        arr[i].kind, arr[i].causal, arr[i].win_lo, arr[i].win_hi = s.kind, s.causal, s.win_lo, s.win_hi
        arr[i].n_global_cols = s.n_global_cols
        arr[i].data = s.data.data_ptr() if s.data is not None else None
    return arr


def tile_lists_bytes(Hm: int, Lq: int, Lk: int) -> int:
    """Size of the block kernel's per-query-tile column lists (0 when Lk > 65536)."""
    return int(lib().sta_tile_lists_bytes(Hm, Lq, Lk))


def sta_encode_mask(srcs: Sequence[MaskSource], Lq: int, Lk: int, device=None, stream=None,
                    tile_lists: bool = True) -> BsrMask:
    """Encode Hm = len(srcs) mask heads (size query, then fill). Synchronises once.

    tile_lists: also write the block kernel's per-query-tile column lists (when
    the mask is narrow enough for them), which the MHA calls then copy instead of
    building each tile's column union themselves.
    """
    h = lib()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    Hm = len(srcs)
    arr = _src_array(srcs)
    ws_bytes = C.c_size_t(0)
    out = _BsrMask()
    _check("sta_encode_mask", h.sta_encode_mask(arr, Hm, Lq, Lk, C.byref(out), None, C.byref(ws_bytes), None))
    ws = torch.empty(max(int(ws_bytes.value), 256), dtype=torch.uint8, device=dev)
    R = (Lq + 63) // 64
    frp = torch.empty(Hm * R + 1, dtype=torch.int32, device=dev)
    prp = torch.empty(Hm * R + 1, dtype=torch.int32, device=dev)
    out.full_row_ptr, out.part_row_ptr = frp.data_ptr(), prp.data_ptr()
    head_tiles = (C.c_int64 * Hm)()
    out.head_tiles = C.cast(head_tiles, C.c_void_p)
    head_valid = (C.c_int64 * Hm)()
    out.head_valid = C.cast(head_valid, C.c_void_p)
    st = _stream(stream)
    _check("sta_encode_mask", h.sta_encode_mask(arr, Hm, Lq, Lk, C.byref(out), _ptr(ws), C.byref(ws_bytes), st))
    nf, npart, nv = int(out.n_full), int(out.n_part), int(out.n_valid)
    fci = torch.empty(max(nf, 1), dtype=torch.int32, device=dev)
    pci = torch.empty(max(npart, 1), dtype=torch.int32, device=dev)
    pbm = torch.empty(max(npart, 1) * 64, dtype=torch.int64, device=dev)
    out.full_col_idx, out.part_col_idx, out.part_bitmap = fci.data_ptr(), pci.data_ptr(), pbm.data_ptr()
    tl_bytes = int(h.sta_tile_lists_bytes(Hm, Lq, Lk)) if tile_lists else 0
    tl = torch.empty(tl_bytes, dtype=torch.uint8, device=dev) if tl_bytes else None
    out.tile_lists = tl.data_ptr() if tl is not None else None
    _check("sta_encode_mask", h.sta_encode_mask(arr, Hm, Lq, Lk, C.byref(out), _ptr(ws), C.byref(ws_bytes), st))
    m = BsrMask(Hm, Lq, Lk, frp, fci[:nf], prp, pci[:npart], pbm[:npart * 64], nf, npart, nv)
    m.head_tiles = head_tiles
    m.head_valid = head_valid
    m.tile_lists = tl
    m._fill = (arr, out, ws, ws_bytes, srcs)  # keeps the sources alive for refill()
    return m


# ---------------------------------------------------------------------------
# masked MHA


def sta_mha_select_kernel(mask: BsrMask, B: int, H: int, d: int, dtype=torch.bfloat16) -> str:
    """Which kernel sta_mha_fwd would run under kernel="auto": "block", "row", or "mixed" when the
    per-mask-head choice (mask.head_tiles and mask.head_valid known) picks both (host only)."""
    s = mask.struct()
    r = lib().sta_mha_select_kernel(C.byref(s), B, H, mask.Lq, mask.Lk, d, _dtype_code(dtype))
    if r < 0:
        raise StaError("sta_mha_select_kernel", -r)
    return {STA_KERNEL_BLOCK: "block", STA_KERNEL_ROW: "row", STA_KERNEL_MIXED: "mixed"}[r]


def sta_mha_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, mask: BsrMask, head_map=None, scale=None,
                kernel: str = "auto", o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                stream=None):
    """O = softmax(Q K^T * scale + mask) V and LSE; q [B,H,Lq,d], k/v [B,H,Lk,d] (bf16 or fp32)."""
    B, H, Lq, d = q.shape
    Lk = k.shape[2]
    assert q.is_contiguous() and k.is_contiguous() and v.is_contiguous()
    assert k.shape == (B, H, Lk, d) and v.shape == k.shape and q.dtype == k.dtype == v.dtype
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Lq), dtype=torch.float32, device=q.device)
    hm = None
    if head_map is not None:
        hm = (C.c_int32 * H)(*[int(x) for x in head_map])
    s = mask.struct()
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    st = lib().sta_mha_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), C.byref(s), hm, B, H, Lq, Lk, d,
                           _dtype_code(q.dtype), scale, _KERNELS[kernel], _stream(stream))
    _check("sta_mha_fwd", st)
    return o, lse


def _mha_common(q, k, v, o, lse, head_map):
    B, H, Lq, d = q.shape
    Lk = k.shape[2]
    assert q.is_contiguous() and k.is_contiguous() and v.is_contiguous()
    assert k.shape == (B, H, Lk, d) and v.shape == k.shape and q.dtype == k.dtype == v.dtype
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Lq), dtype=torch.float32, device=q.device)
    hm = None if head_map is None else (C.c_int32 * H)(*[int(x) for x in head_map])
    return B, H, Lq, Lk, d, o, lse, hm


def mha_splitkv_workspace_bytes(mask: BsrMask, B: int, H: int, d: int, dtype=torch.bfloat16, head_map=None,
                                kernel: str = "auto", num_splits: int = 0) -> int:
    """Workspace size sta_mha_fwd_splitkv needs for these arguments (never 0)."""
    hm = None if head_map is None else (C.c_int32 * H)(*[int(x) for x in head_map])
    s = mask.struct()
    n = C.c_size_t(0)
    _check("sta_mha_fwd_splitkv", lib().sta_mha_fwd_splitkv(None, None, None, None, None, C.byref(s), hm, B, H,
                                                            mask.Lq, mask.Lk, d, _dtype_code(dtype),
                                                            1.0 / math.sqrt(d), _KERNELS[kernel], num_splits, None,
                                                            C.byref(n), None))
    return int(n.value)


def sta_mha_fwd_splitkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, mask: BsrMask, head_map=None, scale=None,
                        kernel: str = "auto", num_splits: int = 0, o: Optional[torch.Tensor] = None,
                        lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None,
                        o_layout: str = "bhld"):
    """sta_mha_fwd with the block kernel's key-tile loop split into chunks merged by log-sum-exp.

    num_splits 0 lets the library choose per head (from mask.head_tiles); s > 0 cuts
    every head's key-tile list into s chunks. workspace: a uint8 device tensor of at
    least mha_splitkv_workspace_bytes(...) bytes (allocated here when None).
    o_layout "bhld": O is [B, H, Lq, d]; "blhd": O is [B, Lq, H, d] (the heads of each
    token side by side, written by the same epilogue store; sta_mha_fwd_layout).
    """
    layout = {"bhld": STA_O_BHLD, "blhd": STA_O_BLHD}[o_layout]
    if o is None and layout == STA_O_BLHD:
        B_, H_, Lq_, d_ = q.shape
        o = torch.empty((B_, Lq_, H_, d_), dtype=q.dtype, device=q.device)
    if o is not None:
        assert o.is_contiguous() and o.dtype == q.dtype and o.numel() == q.numel()
    B, H, Lq, Lk, d, o, lse, hm = _mha_common(q, k, v, o, lse, head_map)
    s = mask.struct()
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    h = lib()
    need = C.c_size_t(0)
    args = (C.byref(s), hm, B, H, Lq, Lk, d, _dtype_code(q.dtype), scale, _KERNELS[kernel], num_splits, layout)
    _check("sta_mha_fwd_layout", h.sta_mha_fwd_layout(None, None, None, None, None, *args, None, C.byref(need), None))
    if workspace is None or workspace.numel() < need.value:
        workspace = torch.empty(int(need.value), dtype=torch.uint8, device=q.device)
    have = C.c_size_t(workspace.numel())
    _check("sta_mha_fwd_layout", h.sta_mha_fwd_layout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), *args,
                                                      _ptr(workspace), C.byref(have), _stream(stream)))
    return o, lse


def mla_workspace_bytes(kv_indptr, n_req: int, Hq: int, chunk_tokens: int = 0) -> int:
    """Workspace size sta_mla_decode needs for these requests (host only, never 0)."""
    n = C.c_size_t(0)
    _check("sta_mla_decode", lib().sta_mla_decode(None, None, None, _indptr_host(kv_indptr), n_req, Hq, 1.0,
                                                   chunk_tokens, None, None, None, C.byref(n), None))
    return int(n.value)


def sta_mla_decode(q: torch.Tensor, kv: torch.Tensor, kv_indptr_dev: torch.Tensor, kv_indptr_host, scale=None,
                   chunk_tokens: int = 0, o=None, lse=None, workspace=None, stream=None):
    """Decode against a shared latent KV cache: q [n_req, Hq, 576], kv [T, 576] bf16 (a 512-entry
    latent then a 64-entry rotary part per row), kv_indptr int32 [n_req + 1]; returns
    O [n_req, Hq, 512] bf16 and LSE [n_req, Hq] float32."""
    n_req, Hq, dqk = q.shape
    assert dqk == 576 and kv.dim() == 2 and kv.shape[1] == 576 and q.dtype == kv.dtype == torch.bfloat16
    assert q.is_contiguous() and kv.is_contiguous()
    scale = 1.0 / math.sqrt(192.0) if scale is None else float(scale)
    if o is None:
        o = torch.empty((n_req, Hq, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((n_req, Hq), dtype=torch.float32, device=q.device)
    ind = _indptr_host(kv_indptr_host)
    need = mla_workspace_bytes(kv_indptr_host, n_req, Hq, chunk_tokens)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    have = C.c_size_t(workspace.numel())
    _check("sta_mla_decode", lib().sta_mla_decode(_ptr(q), _ptr(kv), _ptr(kv_indptr_dev), ind, n_req, Hq, scale,
                                                   chunk_tokens, _ptr(o), _ptr(lse), _ptr(workspace), C.byref(have),
                                                   _stream(stream)))
    return o, lse


# ---------------------------------------------------------------------------
# fused epilogue of the output projection


def sta_bias_residual_layernorm(x: torch.Tensor, bias=None, residual=None, gamma=None, beta=None, eps: float = 1e-5,
                                y: Optional[torch.Tensor] = None, h_out=None, return_sum: bool = False, stream=None):
    """y = LayerNorm((x + bias) + residual) * gamma + beta over the last dimension, one kernel.

    x, residual [..., n] bf16; bias [n] bf16; gamma, beta [n] float32; any of bias,
    residual, gamma, beta may be None. return_sum also returns the pre-norm sum
    (bf16, written by the same kernel into h_out when given).
    """
    assert x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous()
    n = x.shape[-1]
    rows = x.numel() // n
    for t, shape, dt in ((bias, (n,), torch.bfloat16), (residual, tuple(x.shape), torch.bfloat16),
                         (gamma, (n,), torch.float32), (beta, (n,), torch.float32)):
        if t is not None:
            assert t.is_contiguous() and tuple(t.shape) == shape and t.dtype == dt and t.device == x.device
    y = torch.empty_like(x) if y is None else y
    if return_sum and h_out is None:
        h_out = torch.empty_like(x)
    _check("sta_bias_residual_layernorm",
           lib().sta_bias_residual_layernorm(_ptr(x), _ptr(bias), _ptr(residual), _ptr(gamma), _ptr(beta), _ptr(y),
                                             _ptr(h_out), rows, n, float(eps), STA_BF16, _stream(stream)))
    return (y, h_out) if return_sum else y


# ---------------------------------------------------------------------------
# split-KV decode and merge


def _indptr_host(kv_indptr) -> "C.Array":
    vals = kv_indptr.tolist() if hasattr(kv_indptr, "tolist") else list(kv_indptr)
    return (C.c_int32 * len(vals))(*[int(x) for x in vals])


def decode_workspace_bytes(kv_indptr, n_req, Hq, Hkv, d, num_splits=0, page_size=0) -> int:
    """Workspace size sta_decode_splitkv (page_size 0) or sta_decode_splitkv_paged needs for these
    requests (host only)."""
    n = C.c_size_t(0)
    ind = _indptr_host(kv_indptr)
    if page_size:
        _check("sta_decode_splitkv_paged",
               lib().sta_decode_splitkv_paged(None, None, None, page_size, 0, None, None, None, ind, n_req, Hq, Hkv, d,
                                              STA_BF16, 1.0, num_splits, None, None, None, C.byref(n), None))
    else:
        _check("sta_decode_splitkv", lib().sta_decode_splitkv(None, None, None, None, ind, n_req, Hq, Hkv, d, STA_BF16,
                                                               1.0, num_splits, None, None, None, C.byref(n), None))
    return int(n.value)


def sta_decode_splitkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kv_indptr_dev: torch.Tensor, kv_indptr_host,
                       scale=None, num_splits: int = 0, o=None, lse=None, workspace=None, stream=None):
    """GQA decode: q [n_req, Hq, d], k/v [T, Hkv, d] bf16, kv_indptr int32 [n_req + 1]."""
    n_req, Hq, d = q.shape
    T, Hkv, dk = k.shape
    assert dk == d and v.shape == k.shape and kv_indptr_dev.dtype == torch.int32
    ind = _indptr_host(kv_indptr_host)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((n_req, Hq), dtype=torch.float32, device=q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    need = C.c_size_t(0)
    h = lib()
    _check("sta_decode_splitkv", h.sta_decode_splitkv(None, None, None, None, ind, n_req, Hq, Hkv, d,
                                                       _dtype_code(q.dtype), scale, num_splits, None, None, None,
                                                       C.byref(need), None))
    if workspace is None or workspace.numel() < need.value:
        workspace = torch.empty(max(int(need.value), 256), dtype=torch.uint8, device=q.device)
    have = C.c_size_t(workspace.numel())
    _check("sta_decode_splitkv", h.sta_decode_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(kv_indptr_dev), ind, n_req, Hq,
                                                       Hkv, d, _dtype_code(q.dtype), scale, num_splits, _ptr(o),
                                                       _ptr(lse), _ptr(workspace), C.byref(have), _stream(stream)))
    return o, lse


def sta_decode_splitkv_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                             page_indptr_dev: torch.Tensor, page_indices_dev: torch.Tensor, kv_indptr_dev: torch.Tensor,
                             kv_indptr_host, scale=None, num_splits: int = 0, o=None, lse=None, workspace=None,
                             stream=None):
    """GQA decode over a paged KV cache: k_pages/v_pages [n_pages, page_size, Hkv, d] bf16,
    page_indptr int32 [n_req + 1] and page_indices int32 (device), kv_indptr int32 [n_req + 1]
    token prefix sums (device and host)."""
    n_req, Hq, d = q.shape
    n_pages, page_size, Hkv, dk = k_pages.shape
    assert dk == d and v_pages.shape == k_pages.shape and kv_indptr_dev.dtype == torch.int32
    assert page_indptr_dev.dtype == torch.int32 and page_indices_dev.dtype == torch.int32
    ind = _indptr_host(kv_indptr_host)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((n_req, Hq), dtype=torch.float32, device=q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    h = lib()
    args = lambda ws, nb, st: (_ptr(q), _ptr(k_pages), _ptr(v_pages), page_size, n_pages, _ptr(page_indptr_dev),
                               _ptr(page_indices_dev), _ptr(kv_indptr_dev), ind, n_req, Hq, Hkv, d,
                               _dtype_code(q.dtype), scale, num_splits, _ptr(o), _ptr(lse), ws, nb, st)
    need = C.c_size_t(0)
    _check("sta_decode_splitkv_paged", h.sta_decode_splitkv_paged(*args(None, C.byref(need), None)))
    if workspace is None or workspace.numel() < need.value:
        workspace = torch.empty(max(int(need.value), 256), dtype=torch.uint8, device=q.device)
    have = C.c_size_t(workspace.numel())
    _check("sta_decode_splitkv_paged",
           h.sta_decode_splitkv_paged(*args(_ptr(workspace), C.byref(have), _stream(stream))))
    return o, lse


def sta_decode_splitkv_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kv_indptr_dev: torch.Tensor,
                               kv_indptr_host, o: torch.Tensor, lse: Optional[torch.Tensor] = None, scale=None,
                               num_splits: int = 0, stream=None):
    """Split-KV decode that allocates nothing: partials go to the library's fixed 16 MiB device array.

    For callers that cannot allocate device memory (see include/sta.h). The caller
    passes the outputs o [n_req, Hq, d] (and optionally lse [n_req, Hq]); calls that
    overlap on the GPU share that array and must not be issued.
    """
    n_req, Hq, d = q.shape
    T, Hkv, dk = k.shape
    assert dk == d and v.shape == k.shape and kv_indptr_dev.dtype == torch.int32
    assert o.shape == q.shape and o.dtype == q.dtype
    ind = _indptr_host(kv_indptr_host)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    _check("sta_decode_splitkv_noalloc",
           lib().sta_decode_splitkv_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(kv_indptr_dev), ind, n_req, Hq, Hkv, d,
                                            _dtype_code(q.dtype), scale, num_splits, _ptr(o), _ptr(lse),
                                            _stream(stream)))
    return o, lse


def sta_merge_lse(part_o: torch.Tensor, part_lse: torch.Tensor, o_dtype=torch.bfloat16, o=None, lse=None,
                  stream=None):
    """Merge partials: part_o [n_rows, s, d] fp32, part_lse [n_rows, s] fp32 -> o [n_rows, d], lse [n_rows]."""
    n_rows, s, d = part_o.shape
    assert part_o.dtype == torch.float32 and part_lse.shape == (n_rows, s) and part_lse.dtype == torch.float32
    if o is None:
        o = torch.empty((n_rows, d), dtype=o_dtype, device=part_o.device)
    if lse is None:
        lse = torch.empty((n_rows,), dtype=torch.float32, device=part_o.device)
    _check("sta_merge_lse", lib().sta_merge_lse(_ptr(part_o.contiguous()), _ptr(part_lse.contiguous()), n_rows, s, d,
                                                _ptr(o), _dtype_code(o.dtype), _ptr(lse), _stream(stream)))
    return o, lse


# ---------------------------------------------------------------------------
# serving over a paged KV cache


def _need(ok, what: str):
    if not ok:
        raise ValueError(what)


def _on(dev: torch.device, *tensors):
    """Every tensor given (None allowed) lies on CUDA device `dev`."""
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, not {dev}")
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError("tensors on different devices")


def _i32(dev: torch.device, **tensors):
    """The named index tensors: contiguous int32 on `dev`."""
    for name, t in tensors.items():
        if t.dtype is not torch.int32 or not t.is_contiguous() or t.device != dev:
            raise ValueError(f"{name}: contiguous int32 on {dev}")


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


class _Launch:
    """The device a call launches on, made current, and its stream, made torch's current one so that
    what the call allocates belongs to that stream; leave() puts back what was current."""

    def __init__(self, dev: torch.device, stream):
        self._outer = contextlib.ExitStack()
        with contextlib.ExitStack() as outer:
            outer.enter_context(torch.cuda.device(dev))
            if stream is None:
                stream = torch.cuda.current_stream(dev)
            else:
                if not isinstance(stream, torch.cuda.Stream):
                    stream = torch.cuda.ExternalStream(int(stream), device=dev) if int(stream) else torch.cuda.default_stream(dev)
                outer.enter_context(torch.cuda.stream(stream))
            self.handle = stream.cuda_stream
            self._outer = outer.pop_all()

    def leave(self):
        self._outer.close()


def _enter(dev: torch.device, stream):
    """The handle of the stream to launch on, and the _Launch to leave afterwards (None: the current
    device and stream, which the calls of a decoding loop use, need nothing changed)."""
    if stream is None and dev.index == torch._C._cuda_getDevice():
        return torch._C._cuda_getCurrentRawStream(dev.index), None
    ctx = _Launch(dev, stream)
    return ctx.handle, ctx


def _workspace(need: int, workspace: Optional[torch.Tensor], dev: torch.device) -> torch.Tensor:
    """The caller's scratch when it is large enough, else one of `need` bytes."""
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    _need(workspace.dtype == torch.uint8 and workspace.is_contiguous() and workspace.device == dev,
          f"workspace: contiguous uint8 on {dev}")
    _need(workspace.numel() >= need, f"workspace: {need} bytes needed, {workspace.numel()} given")
    return workspace


def _host_i32(x, n: int, what: str):
    """Host int32 values: their address, the last one, and the object that keeps them alive."""
    if isinstance(x, torch.Tensor) and x.dtype is torch.int32 and x.device.type == "cpu" and x.is_contiguous():
        at, shape = x.data_ptr(), x.shape
    else:
        x = np.ascontiguousarray(x, dtype=np.int32)
        at, shape = x.__array_interface__["data"][0], x.shape
    if n < 1 or len(shape) != 1 or shape[0] != n:
        raise ValueError(f"{what}: {n} values, at least one")
    return at, C.c_int32.from_address(at + 4 * (n - 1)).value, x


_ROPE_SCALINGS = {"none": STA_ROPE_SCALE_NONE, "linear": STA_ROPE_SCALE_LINEAR, "blend": STA_ROPE_SCALE_BLEND}


class Rope:
    """Rotary positions of a model's heads (sta_rope_params).

    The leading rot_dim elements of each head turn, in pairs (p, p + rot_dim / 2) or, interleaved,
    (2p, 2p + 1), pair p by base^(-2p / rot_dim) radians a token. scaling "linear" divides the
    speeds by factor; "blend" does so only for pairs that turn less than low_turns times within
    orig_len tokens, and by a blend up to high_turns. mscale multiplies cosine and sine. freqs:
    rot_dim / 2 speeds in radians a token, in place of base and scaling.
    """

    def __init__(self, rot_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, orig_len: float = 0.0, low_turns: float = 1.0, high_turns: float = 32.0,
                 mscale: float = 1.0, freqs: Optional[Sequence[float]] = None):
        kind = _ROPE_SCALINGS.get(scaling)
        if kind is None:
            raise ValueError(f"scaling: one of {sorted(_ROPE_SCALINGS)}")
        self._freqs = None
        if freqs is not None:
            if len(freqs) != rot_dim // 2:
                raise ValueError("freqs: rot_dim / 2 values")
            self._freqs = (C.c_double * len(freqs))(*[float(f) for f in freqs])
        self.rot_dim = int(rot_dim)
        self.struct = _RopeParams(int(rot_dim), STA_ROPE_INTERLEAVED if interleaved else STA_ROPE_HALF, kind,
                                  float(mscale), float(base), float(factor), float(orig_len), float(low_turns),
                                  float(high_turns), C.cast(self._freqs, C.c_void_p) if self._freqs else None)


def _heads_view(t: torch.Tensor, what: str):
    """[n, H, d] with contiguous heads: the token stride."""
    if t.dim() != 3:
        raise ValueError(f"{what}: [tokens, heads, d]")
    n, H, d = t.shape
    if t.is_contiguous():
        return H * d
    if not (n == 0 or ((d == 1 or t.stride(2) == 1) and (H == 1 or t.stride(1) == d))):
        raise ValueError(f"{what}: a token's heads must be contiguous")
    return t.stride(0) if n > 1 else H * d


def sta_rope(x: torch.Tensor, positions: torch.Tensor, rope: Rope, transpose: bool = False,
             y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rotary positions: x [n, H, d] bf16 or float32 (any token stride), positions int32 [n].

    transpose turns the other way: the gradient of the input from the gradient of the result.
    y may be x (in place); otherwise a new [n, H, d] tensor is returned.
    """
    xs = _heads_view(x, "x")
    n, H, d = x.shape
    dev = x.device
    _on(dev, y)
    _i32(dev, positions=positions)
    if positions.shape != (n,):
        raise ValueError("positions: one a token")
    code = _dtype_code(x.dtype)
    st, ctx = _enter(dev, stream)
    try:
        if y is None:
            y, ys = torch.empty((n, H, d), dtype=x.dtype, device=dev), H * d
        else:
            if not (y.shape == x.shape and y.dtype == x.dtype):
                raise ValueError("y: x's shape and dtype")
            ys = _heads_view(y, "y")
        _check("sta_rope", (_lib_handle or lib()).sta_rope(
            _addr(x), _addr(y), _addr(positions), C.byref(rope.struct), n, H, d, xs, ys, int(bool(transpose)),
            code, st))
    finally:
        if ctx is not None:
            ctx.leave()
    return y


def sta_rope_append_paged(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor,
                          v_pages: torch.Tensor, page_indptr_dev: torch.Tensor, page_indices_dev: torch.Tensor,
                          q_indptr_dev: torch.Tensor, kv_indptr_dev: torch.Tensor, rope: Optional[Rope] = None,
                          positions: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None, stream=None):
    """Turns q [n, Hq, d] and k [n, Hkv, d] of a step's new tokens (any token strides, bf16) and
    writes k and v to their places in k_pages / v_pages [n_pages, page_size, Hkv, d].

    Request r's new tokens are rows q_indptr[r] .. q_indptr[r+1]-1, the last ones of its sequence of
    kv_indptr[r+1] - kv_indptr[r] tokens (both int32, device). rope None: nothing turns. q None: keys
    and values only. Returns the turned q [n, Hq, d] (rows of a padded batch's padding unwritten).
    """
    dev = k.device
    _on(dev, q, v, k_pages, v_pages, q_out)
    n_pages, page_size, Hkv, d = k_pages.shape
    n = k.shape[0]
    if not (v_pages.shape == k_pages.shape and k_pages.is_contiguous() and v_pages.is_contiguous()):
        raise ValueError("k_pages, v_pages: contiguous [n_pages, page_size, Hkv, d]")
    if not (k.shape == (n, Hkv, d) and v.shape == k.shape):
        raise ValueError("k, v: [n, Hkv, d]")
    ks, vs = _heads_view(k, "k"), _heads_view(v, "v")
    Hq, qs = 0, 0
    if q is not None:
        qs = _heads_view(q, "q")
        Hq = q.shape[1]
        if not (q.shape == (n, Hq, d)):
            raise ValueError("q: [n, Hq, d]")
    for t in (q, k, v, k_pages, v_pages, q_out):
        if not (t is None or t.dtype == torch.bfloat16):
            raise ValueError("bf16 only")
    _i32(dev, page_indptr=page_indptr_dev, page_indices=page_indices_dev, q_indptr=q_indptr_dev, kv_indptr=kv_indptr_dev)
    n_req = q_indptr_dev.numel() - 1
    if not (kv_indptr_dev.numel() == n_req + 1 and page_indptr_dev.numel() == n_req + 1):
        raise ValueError("indptr: n_req + 1 values each")
    if positions is not None:
        _i32(dev, positions=positions)
        if positions.shape != (n,):
            raise ValueError("positions: one a token")
    st, ctx = _enter(dev, stream)
    try:
        if q_out is None:
            q_out = None if q is None else torch.empty((n, Hq, d), dtype=q.dtype, device=dev)
        elif not (q is not None and q_out.shape == q.shape and q_out.is_contiguous()):
            raise ValueError("q_out: contiguous, q's shape")
        _check("sta_rope_append_paged", (_lib_handle or lib()).sta_rope_append_paged(
            _addr(q), _addr(k), _addr(v), qs, ks, vs, _addr(q_out), _addr(k_pages), _addr(v_pages), page_size, n_pages,
            _addr(page_indptr_dev), _addr(page_indices_dev), _addr(q_indptr_dev), _addr(kv_indptr_dev), _addr(positions),
            C.byref(rope.struct) if rope is not None else None, n, n_req, Hq, Hkv, d, STA_BF16, st))
    finally:
        if ctx is not None:
            ctx.leave()
    return q_out


def sta_chunk_fwd_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_indptr_dev: torch.Tensor,
                        page_indices_dev: torch.Tensor, q_indptr_dev: torch.Tensor, q_indptr_host,
                        kv_indptr_dev: torch.Tensor, kv_indptr_host, scale=None, pattern: Optional[MaskSource] = None,
                        num_splits: int = 0, o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of each request's new tokens over its sequence in the paged cache.

    q [n, Hq, d] bf16 (any token stride that is a multiple of 8), request r's rows q_indptr[r] ..
    q_indptr[r+1]-1 being the last tokens of its sequence of kv_indptr[r+1] - kv_indptr[r] tokens;
    indptr int32 [n_req + 1], device and host. pattern: None (causal) or a MaskSource.pattern over
    positions. Rows past q_indptr[n_req] are left as they are. Returns O [n, Hq, d] and LSE
    [n, Hq] float32 (-inf for a token that sees no key).
    """
    qs = _heads_view(q, "q")
    n, Hq, d = q.shape
    dev = q.device
    _on(dev, k_pages, v_pages, o, lse)
    n_pages, page_size, Hkv, dk = k_pages.shape
    if not (dk == d and v_pages.shape == k_pages.shape and k_pages.is_contiguous() and v_pages.is_contiguous()):
        raise ValueError("k_pages, v_pages: contiguous [n_pages, page_size, Hkv, d]")
    if not (q.dtype == k_pages.dtype == v_pages.dtype):
        raise ValueError("q, k_pages, v_pages: one dtype")
    _i32(dev, page_indptr=page_indptr_dev, page_indices=page_indices_dev, q_indptr=q_indptr_dev, kv_indptr=kv_indptr_dev)
    n_req = q_indptr_dev.numel() - 1
    if not (kv_indptr_dev.numel() == n_req + 1 and page_indptr_dev.numel() == n_req + 1):
        raise ValueError("indptr: n_req + 1 values each")
    qh, rows, keep_q = _host_i32(q_indptr_host, n_req + 1, "q_indptr_host")
    kh, keys, keep_k = _host_i32(kv_indptr_host, n_req + 1, "kv_indptr_host")
    if not 0 <= rows <= n:
        raise ValueError("q_indptr: past q's rows")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    pat = None if pattern is None else _src_array([pattern])
    h = _lib_handle or lib()
    st, ctx = _enter(dev, stream)
    try:
        if o is None:
            o = torch.empty((n, Hq, d), dtype=q.dtype, device=dev)
        elif not (o.shape == q.shape and o.dtype == q.dtype and o.is_contiguous()):
            raise ValueError("o: contiguous, q's shape and dtype")
        if lse is None:
            lse = torch.empty((n, Hq), dtype=torch.float32, device=dev)
        elif not (lse.shape == (n, Hq) and lse.dtype == torch.float32 and lse.is_contiguous()):
            raise ValueError("lse: contiguous float32 [n, Hq]")
        args = (q.data_ptr(), qs, k_pages.data_ptr(), v_pages.data_ptr(), page_size, n_pages, page_indptr_dev.data_ptr(),
                page_indices_dev.data_ptr() or None, q_indptr_dev.data_ptr(), qh, kv_indptr_dev.data_ptr(), kh, n_req, Hq, Hkv, d,
                _dtype_code(q.dtype), scale, pat, num_splits, o.data_ptr(), lse.data_ptr())
        # Most calls cut nothing: they need the least size there is and use none of it. Few new tokens over many
        # cached ones are mostly cut, into no more than 32 pieces (64 single tokens: 48 us of host time a call,
        # 56 when it first asks). A call that needs more says how much.
        at, size = 256, C.c_size_t(256)
        if workspace is not None or (rows <= 8 * n_req and keys >= 8192):
            guess = 256 if workspace is not None else max(256, min(32 * rows * Hq * (d + 2) * 4, 1 << 26))
            ws = _workspace(guess, workspace, dev)
            at, size.value = ws.data_ptr(), ws.numel()
        status = h.sta_chunk_fwd_paged(*args, at, C.byref(size), st)
        if status == STA_ERR_WORKSPACE:
            ws = _workspace(size.value, workspace, dev)
            status = h.sta_chunk_fwd_paged(*args, ws.data_ptr(), C.byref(size), st)
        _check("sta_chunk_fwd_paged", status)
    finally:
        if ctx is not None:
            ctx.leave()
    return o, lse


def chunk_workspace_bytes(q_indptr, kv_indptr, n_req: int, Hq: int, Hkv: int, d: int, page_size: int = 16,
                          pattern: Optional[MaskSource] = None, num_splits: int = 0) -> int:
    """Workspace size sta_chunk_fwd_paged needs for these requests (host only, never 0)."""
    n = C.c_size_t(0)
    qh, _, keep_q = _host_i32(q_indptr, n_req + 1, "q_indptr")
    kh, _, keep_k = _host_i32(kv_indptr, n_req + 1, "kv_indptr")
    _check("sta_chunk_fwd_paged", (_lib_handle or lib()).sta_chunk_fwd_paged(
        None, 0, None, None, page_size, 1, None, None, None, qh, None, kh, n_req, Hq, Hkv, d, STA_BF16, 1.0,
        None if pattern is None else _src_array([pattern]), num_splits, None, None, None, C.byref(n), None))
    return int(n.value)


@functools.lru_cache(maxsize=1024)
def _pages_ws(fn: str, n_pages: int, n_req: int, n_forks: int) -> int:
    """Workspace size of a page call (it depends on these alone)."""
    n = C.c_size_t(0)
    h = lib()
    if fn == "sta_pages_grow":
        st = h.sta_pages_grow(None, n_pages, None, None, None, None, n_req, 1, None, None, C.byref(n), None)
    elif fn == "sta_pages_fork":
        st = h.sta_pages_fork(None, 0, 0, None, n_pages, None, None, None, n_req, 1, None, None, n_forks, None, None,
                              C.byref(n), None)
    else:
        st = h.sta_pages_compact(None, 0, 0, None, n_pages, None, None, None, n_req, 1, None, None, None, C.byref(n), None)
    _check(fn, st)
    return int(n.value)


def _buf_array(bufs: Sequence[torch.Tensor], dev: torch.device, n_pages: Optional[int] = None):
    """[n_pages, ...] buffers of one page size: their addresses, number, bytes a page and n_pages."""
    bufs = list(bufs)
    page_bytes, shape, dtype = 0, None, None
    for b in bufs:
        if not (b.is_contiguous() and b.device == dev and b.dim() >= 1):
            raise ValueError(f"buffers: contiguous on {dev}")
        if b.dtype is dtype and b.shape == shape:
            continue  # as the one before: a cache's buffers are alike
        shape, dtype = b.shape, b.dtype
        n_pages = shape[0] if n_pages is None else n_pages
        if not (shape[0] == n_pages and n_pages > 0):
            raise ValueError("buffers: [n_pages, ...] each")
        nb = b.numel() // n_pages * b.element_size()
        if page_bytes not in (0, nb):
            raise ValueError("buffers: the same bytes a page")
        page_bytes = nb
    return (C.c_void_p * max(len(bufs), 1))(*[b.data_ptr() for b in bufs]), len(bufs), page_bytes, n_pages


def _lists(ref, page_indptr, page_indices, kv_indptr):
    dev = ref.device
    _on(dev)
    _i32(dev, ref=ref, page_indptr=page_indptr, page_indices=page_indices, kv_indptr=kv_indptr)
    n_req = kv_indptr.numel() - 1
    if not (page_indptr.numel() == n_req + 1):
        raise ValueError("page_indptr, kv_indptr: n_req + 1 values each")
    return dev, n_req


def sta_pages_copy(bufs: Sequence[torch.Tensor], src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """Page src[i] onto page dst[i] of every buffer [n_pages, ...] (int32, device; negative: no copy).
    Pages of dst must be distinct and not among src."""
    bufs = list(bufs)
    if not bufs:
        raise ValueError("at least one buffer")
    dev = bufs[0].device
    _on(dev)
    _i32(dev, src=src, dst=dst)
    if not (src.dim() == 1 and src.shape == dst.shape):
        raise ValueError("src, dst: [n] each")
    arr, nb, page_bytes, n_pages = _buf_array(bufs, dev)
    st, ctx = _enter(dev, stream)
    try:
        _check("sta_pages_copy", (_lib_handle or lib()).sta_pages_copy(
            arr, nb, page_bytes, n_pages, _addr(src), _addr(dst), src.numel(), st))
    finally:
        if ctx is not None:
            ctx.leave()


def sta_pages_grow(ref: torch.Tensor, page_indptr: torch.Tensor, page_indices: torch.Tensor, kv_indptr: torch.Tensor,
                   new_kv_indptr: torch.Tensor, page_size: int, stream=None) -> torch.Tensor:
    """Gives each request the free pages (lowest first) it needs to go from kv_indptr's lengths to
    new_kv_indptr's; updates ref and page_indices, returns status int32 [2] {taken, missing}."""
    dev, n_req = _lists(ref, page_indptr, page_indices, kv_indptr)
    _i32(dev, new_kv_indptr=new_kv_indptr)
    if not (new_kv_indptr.numel() == n_req + 1):
        raise ValueError("new_kv_indptr: n_req + 1 values")
    st, ctx = _enter(dev, stream)
    try:
        status = torch.empty(2, dtype=torch.int32, device=dev)
        args = (_addr(ref), ref.numel(), _addr(page_indptr), _addr(page_indices), _addr(kv_indptr), _addr(new_kv_indptr), n_req,
                page_size, _addr(status))
        ws = torch.empty(_pages_ws("sta_pages_grow", ref.numel(), n_req, 0), dtype=torch.uint8, device=dev)
        _check("sta_pages_grow", (_lib_handle or lib()).sta_pages_grow(
            *args, ws.data_ptr(), C.byref(C.c_size_t(ws.numel())), st))
    finally:
        if ctx is not None:
            ctx.leave()
    return status


def sta_pages_fork(bufs: Sequence[torch.Tensor], ref: torch.Tensor, page_indptr: torch.Tensor,
                   page_indices: torch.Tensor, kv_indptr: torch.Tensor, parent: torch.Tensor, child: torch.Tensor,
                   page_size: int, stream=None) -> torch.Tensor:
    """Request child[i] becomes a copy of request parent[i]: whole pages shared, a last, partly filled
    page copied onto a free one in every buffer. A child must hold nothing. Updates ref and
    page_indices, returns status int32 [2] {pages taken, missing}."""
    dev, n_req = _lists(ref, page_indptr, page_indices, kv_indptr)
    _i32(dev, parent=parent, child=child)
    if not (parent.dim() == 1 and parent.shape == child.shape):
        raise ValueError("parent, child: [n_forks] each")
    arr, nb, page_bytes, _ = _buf_array(bufs, dev, ref.numel())
    st, ctx = _enter(dev, stream)
    try:
        status = torch.empty(2, dtype=torch.int32, device=dev)
        args = (arr, nb, page_bytes, _addr(ref), ref.numel(), _addr(page_indptr), _addr(page_indices), _addr(kv_indptr), n_req,
                page_size, _addr(parent), _addr(child), parent.numel(), _addr(status))
        ws = torch.empty(_pages_ws("sta_pages_fork", ref.numel(), n_req, parent.numel()), dtype=torch.uint8, device=dev)
        _check("sta_pages_fork", (_lib_handle or lib()).sta_pages_fork(
            *args, ws.data_ptr(), C.byref(C.c_size_t(ws.numel())), st))
    finally:
        if ctx is not None:
            ctx.leave()
    return status


def sta_pages_free(ref: torch.Tensor, page_indptr: torch.Tensor, page_indices: torch.Tensor, kv_indptr: torch.Tensor,
                   reqs: torch.Tensor, page_size: int, stream=None) -> None:
    """The listed requests (int32, device) let go of the pages they hold; their entries become -1."""
    dev, n_req = _lists(ref, page_indptr, page_indices, kv_indptr)
    _i32(dev, reqs=reqs)
    st, ctx = _enter(dev, stream)
    try:
        _check("sta_pages_free", (_lib_handle or lib()).sta_pages_free(
            _addr(ref), ref.numel(), _addr(page_indptr), _addr(page_indices), _addr(kv_indptr), n_req, page_size, _addr(reqs),
            reqs.numel(), st))
    finally:
        if ctx is not None:
            ctx.leave()


def sta_pages_compact(bufs: Sequence[torch.Tensor], ref: torch.Tensor, page_indptr: torch.Tensor,
                      page_indices: torch.Tensor, kv_indptr: torch.Tensor, page_size: int, stream=None):
    """Moves the used pages to the lowest numbers: page data in every buffer, ref and the lists.
    Returns page_map int32 [n_pages] (each used page's new number, -1: free) and status int32 [2]
    {pages in use, pages moved}."""
    dev, n_req = _lists(ref, page_indptr, page_indices, kv_indptr)
    arr, nb, page_bytes, _ = _buf_array(bufs, dev, ref.numel())
    st, ctx = _enter(dev, stream)
    try:
        page_map = torch.empty(ref.numel(), dtype=torch.int32, device=dev)
        status = torch.empty(2, dtype=torch.int32, device=dev)
        args = (arr, nb, page_bytes, _addr(ref), ref.numel(), _addr(page_indptr), _addr(page_indices), _addr(kv_indptr), n_req,
                page_size, _addr(page_map), _addr(status))
        ws = torch.empty(_pages_ws("sta_pages_compact", ref.numel(), n_req, 0), dtype=torch.uint8, device=dev)
        _check("sta_pages_compact", (_lib_handle or lib()).sta_pages_compact(
            *args, ws.data_ptr(), C.byref(C.c_size_t(ws.numel())), st))
    finally:
        if ctx is not None:
            ctx.leave()
    return page_map, status


# ---------------------------------------------------------------------------
# failure detection


def sta_check_bounded_wait(limit_ns: int, stream=None) -> int:
    """Run the failure-detection check (a bounded wait on a barrier nothing completes, limit
    limit_ns); returns the kernel's outcome (0: the wait gave up, as it must). The device
    error word then holds 0x7f1 unless an earlier code is there."""
    out = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    _check("sta_check_bounded_wait", lib().sta_check_bounded_wait(int(limit_ns), _ptr(out), _stream(stream)))
    return int(out.item())


def sta_device_error(reset: bool = True) -> int:
    """The device error word (nonzero: a kernel's bounded wait gave up, or a damaged input was
    met); synchronises, and clears the word when reset."""
    code = C.c_int(0)
    _check("sta_device_error", lib().sta_device_error(C.byref(code), int(reset)))
    return int(code.value)
