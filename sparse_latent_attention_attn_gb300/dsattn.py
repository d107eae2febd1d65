"""Python binding of libdsattn (include/dsattn.h): argument marshalling only.

Every function here takes torch tensors that already live on the current CUDA device, checks
dtypes and shapes, and passes raw pointers, sizes and the current stream to the C ABI of the
same name.  All computation happens in the library's CUDA kernels; there is no fallback of any
kind: importing this module fails when ``libdsattn.so`` is missing.

Sources, by page title and section: "DeepSeek V4.1", attention/attend (get_window_topk_idxs,
sparse_attn_kernel, sparse_attn wrapper); attention/query-latent (Attention.__init__ ring buffer,
Attention.forward concatenation); "Module attn" (act_quant_inplace, pow2_ceil, FP8_BLOCK,
sparse_attn, window_topk_idxs, the ring-cache and Precision paragraphs).
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdsattn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m sparse_latent_attention_attn_gb300.build`"
                      " (or __graft_entry__.build())")

_lib = ctypes.CDLL(LIB_PATH)

DS_OK = 0
DS_EINVAL = -1
DS_EUNSUPPORTED = -2
DS_EWORKSPACE = -3
DS_ECUDA = -4
DS_EDEVICE = -5
DS_DEV_TIMEOUT = 1
DS_DEV_BAD_INDEX = 2
DS_DEV_BAD_VALUE = 4

_P = ctypes.c_void_p
_i32, _i64, _f32, _sz = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t

_lib.ds_window_topk_idxs.argtypes = [_P, _i64, _i32, _i32, _i64, _i32, ctypes.POINTER(_i32), _P]
_lib.ds_window_topk_idxs.restype = _i32
_lib.ds_kv_quant_ring_write.argtypes = [_P, _i64, _P, _i64, _i32, _i32, _i32, _i64, _i32, _P]
_lib.ds_kv_quant_ring_write.restype = _i32
_lib.ds_sparse_attn_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32]
_lib.ds_sparse_attn_workspace_bytes.restype = _sz
_lib.ds_sparse_attn.argtypes = [_P, _P, _i64, _P, _P, _i32, _f32, _P, _i32, _i32, _i32, _i32, _P, _sz, _P]
_lib.ds_sparse_attn.restype = _i32
_lib.ds_sparse_attn_prefill_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32]
_lib.ds_sparse_attn_prefill_workspace_bytes.restype = _sz
_lib.ds_sparse_attn_prefill.argtypes = [_P, _P, _i64, _P, _P, _i32, _f32, _P, _i32, _i32, _i32, _i32, _P, _sz, _P]
_lib.ds_sparse_attn_prefill.restype = _i32
_lib.ds_sparse_attn_rope.argtypes = [_P, _P, _i64, _P, _P, _i32, _f32, _P, _i32, _i32, _i32, _i32, _P, _sz, _i32, _P,
                                    _i64, _i64, _P]
_lib.ds_sparse_attn_rope.restype = _i32
_lib.ds_apply_rotary.argtypes = [_P, _i64, _i32, _i32, _i64, _i64, _i64, _P, _i64, _i32, _P]
_lib.ds_apply_rotary.restype = _i32
_lib.ds_kv_rope_quant_ring_write.argtypes = [_P, _i64, _P, _i64, _i32, _i32, _i32, _i64, _i32, _i32, _P, _i64, _P]
_lib.ds_kv_rope_quant_ring_write.restype = _i32
_lib.ds_kv_quantize_fp8.argtypes = [_P, _i64, _i32, _P, _P, _P]
_lib.ds_kv_quantize_fp8.restype = _i32
_lib.ds_kv_quant_ring_write_fp8.argtypes = [_P, _i64, _P, _P, _i64, _i32, _i32, _i32, _i64, _i32, _P]
_lib.ds_kv_quant_ring_write_fp8.restype = _i32
_lib.ds_sparse_attn_fp8kv.argtypes = [_P, _P, _P, _i64, _P, _P, _i32, _f32, _P, _i32, _i32, _i32, _i32, _P, _sz, _P]
_lib.ds_sparse_attn_fp8kv.restype = _i32
_lib.ds_device_status.argtypes = [_P, ctypes.POINTER(ctypes.c_uint)]
_lib.ds_device_status.restype = _i32
_lib.ds_indexer_workspace_bytes.argtypes = [_i32, _i32, _i64, _i32]
_lib.ds_indexer_workspace_bytes.restype = _sz
_lib.ds_indexer_scores.argtypes = [_P, _P, _P, _i32, _i32, _i32, _i32, _i64, _i64, _i32, _P, _i64, _P]
_lib.ds_indexer_scores.restype = _i32
_lib.ds_indexer_select.argtypes = [_P, _i64, _i32, _i32, _i64, _i32, _i32, _i64, _P, _P]
_lib.ds_indexer_select.restype = _i32
_lib.ds_indexer_topk.argtypes = [_P, _P, _P, _i32, _i32, _i32, _i32, _i64, _i64, _i32, _i32, _i64, _P, _P, _sz, _P]
_lib.ds_indexer_topk.restype = _i32
_lib.ds_norm_rotary.argtypes = [_P, _i64, _i64, _P, _i32, _i32, _i32, _i32, _P, _f32, _i32, _P, _i64, _P, _P, _P]
_lib.ds_norm_rotary.restype = _i32
_lib.ds_kv_append_fp4_paged.argtypes = [_P, _i64, _i64, _P, _i32, _i32, _i32, _P, _f32, _i32, _P, _i64, _P, _P, _i32,
                                        _i32, _i32, _P, _P, _i64, _i32, _P, _i32, _P]
_lib.ds_kv_append_fp4_paged.restype = _i32
_lib.ds_kv_append_fp8_paged.argtypes = _lib.ds_kv_append_fp4_paged.argtypes
_lib.ds_kv_append_fp8_paged.restype = _i32
_lib.ds_kv_read_fp8_paged.argtypes = [_P, _P, _i64, _i32, _P, _i32, _P, _P, _P, _P, _i32, _i32, _i32, _P]
_lib.ds_kv_read_fp8_paged.restype = _i32
_lib.ds_kv_read_fp4_paged.argtypes = _lib.ds_kv_read_fp8_paged.argtypes
_lib.ds_kv_read_fp4_paged.restype = _i32
_lib.ds_chunk_attn_fp8_paged_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32]
_lib.ds_chunk_attn_fp8_paged_workspace_bytes.restype = _sz
_lib.ds_chunk_attn_fp8_paged.argtypes = [_P, _P, _P, _i64, _i32, _P, _i32, _P, _f32, _P, _i32, _i32, _i32, _i32, _P, _P,
                                         _i32, _i32, _i32, _i32, _P, _sz, _i32, _P, _i64, _P]
_lib.ds_chunk_attn_fp8_paged.restype = _i32
_lib.ds_sparse_attn_fp4_paged_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32]
_lib.ds_sparse_attn_fp4_paged_workspace_bytes.restype = _sz
_lib.ds_sparse_attn_fp4_paged.argtypes = [_P, _P, _P, _i64, _i32, _P, _i32, _P, _P, _i32, _f32, _P, _i32, _i32, _i32,
                                          _i32, _P, _sz, _i32, _P, _i64, _P, _P]
_lib.ds_sparse_attn_fp4_paged.restype = _i32
_lib.ds_sparse_attn_fp4_paged_ragged.argtypes = [*_lib.ds_sparse_attn_fp4_paged.argtypes[:-1], _P, _P]
_lib.ds_sparse_attn_fp4_paged_ragged.restype = _i32
_lib.ds_test_set_stall.argtypes = [_i32]
_lib.ds_test_set_stall.restype = None
_lib.ds_test_set_kernel.argtypes = [_i32]
_lib.ds_test_set_kernel.restype = _i32
_lib.ds_sparse_attn_launches.argtypes = [_i32, _i32, _i32, _i32, _i32, ctypes.POINTER(_i32),
                                         ctypes.POINTER(ctypes.c_size_t)]
_lib.ds_sparse_attn_launches.restype = _i32
_lib.ds_status_string.argtypes = [_i32]
_lib.ds_status_string.restype = ctypes.c_char_p


class DsError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {_lib.ds_status_string(status).decode()} ({status})")
        self.status = status


def _check(fn: str, status: int) -> None:
    if status != DS_OK:
        raise DsError(fn, status)


# The current device, and its current stream's raw handle: torch.cuda.current_stream() builds an object around that
# (3 us against 0.2).  A torch without these two (one built without CUDA, say) has the public functions.
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _stream(stream) -> int:
    return _raw_stream(torch.cuda.current_device()) if stream is None else stream.cuda_stream


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, dtype, name: str) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")


def window_topk_idxs(idx: torch.Tensor, b: int, s: int, start_pos: int, window: int, stream=None) -> int:
    """Write window index rows into ``idx`` (int32, last dim = row stride ``ld``); returns cols.

    ``idx`` is viewed as rows of length ``idx.shape[-1]``: row (bi, q) is ``idx.view(-1, ld)[bi*rows+q]``.
    """
    _need(idx, torch.int32, "idx")
    ld = idx.shape[-1]
    if idx.stride(-1) != 1 or not idx.is_contiguous():
        raise ValueError("idx must be contiguous")
    cols = _i32(0)
    _check("ds_window_topk_idxs",
           _lib.ds_window_topk_idxs(_ptr(idx), ld, b, s, start_pos, window, ctypes.byref(cols), _stream(stream)))
    return cols.value


def kv_quant_ring_write(kv: torch.Tensor, ring: torch.Tensor | None, start_pos: int, window: int,
                        stream=None) -> None:
    """fp8 round trip of ``kv`` [b][s][d] (bf16, rows contiguous) in place, then the ring store.

    ``ring`` is a bf16 view [b][>=window][d] whose rows are contiguous (it may be the leading
    ``window`` rows of a larger per-sequence kv tensor).
    """
    _need(kv, torch.bfloat16, "kv")
    b, s, d = kv.shape
    if kv.stride(2) != 1 or kv.stride(1) != d:
        raise ValueError("kv rows must be contiguous")
    ring_bstride = 0
    if ring is not None:
        _need(ring, torch.bfloat16, "ring")
        if ring.shape[0] != b or ring.shape[2] != d or ring.shape[1] < window or ring.stride(2) != 1 \
                or ring.stride(1) != d:
            raise ValueError("ring must be [b][>=window][d] with contiguous rows")
        ring_bstride = ring.stride(0)
    _check("ds_kv_quant_ring_write",
           _lib.ds_kv_quant_ring_write(_ptr(kv), kv.stride(0), _ptr(ring), ring_bstride, b, s, d, start_pos, window,
                                       _stream(stream)))


def sparse_attn_workspace_bytes(b: int, m: int, h: int, d: int, topk: int) -> int:
    return int(_lib.ds_sparse_attn_workspace_bytes(b, m, h, d, topk))


def sparse_attn(q: torch.Tensor, kv: torch.Tensor, sink: torch.Tensor, idx: torch.Tensor, scale: float,
                o: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """o[b][m][h][d] = sparse_attn(q[b][m][h][d], kv[b][n][d], sink[h], idx[b][m][topk], scale)."""
    _need(q, torch.bfloat16, "q")
    _need(kv, torch.bfloat16, "kv")
    _need(sink, torch.float32, "sink")
    _need(idx, torch.int32, "idx")
    b, m, h, d = q.shape
    n = kv.shape[1]
    topk = idx.shape[2]
    if kv.shape != (b, n, d) or idx.shape[:2] != (b, m) or sink.shape != (h,):
        raise ValueError("shape mismatch")
    for t, name in ((q, "q"), (kv, "kv"), (idx, "idx"), (sink, "sink")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if o is None:
        o = torch.empty_like(q)
    elif o.shape != q.shape or o.dtype != torch.bfloat16 or not o.is_contiguous():
        raise ValueError("o must be a contiguous bf16 tensor shaped like q")
    need = sparse_attn_workspace_bytes(b, m, h, d, topk)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("ds_sparse_attn",
           _lib.ds_sparse_attn(_ptr(q), _ptr(kv), n, _ptr(sink), _ptr(idx), topk, float(scale), _ptr(o), b, m, h, d,
                               _ptr(workspace), ws_bytes, _stream(stream)))
    return o


def sparse_attn_prefill_workspace_bytes(b: int, m: int, h: int, d: int, topk: int) -> int:
    return int(_lib.ds_sparse_attn_prefill_workspace_bytes(b, m, h, d, topk))


def sparse_attn_prefill(q: torch.Tensor, kv: torch.Tensor, sink: torch.Tensor, idx: torch.Tensor, scale: float,
                        o: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """``sparse_attn`` for a prefill chunk, queries 2j and 2j + 1 sharing one gather of the union
    of their index rows (valid entries of a row must be distinct)."""
    _need(q, torch.bfloat16, "q")
    _need(kv, torch.bfloat16, "kv")
    _need(sink, torch.float32, "sink")
    _need(idx, torch.int32, "idx")
    b, m, h, d = q.shape
    n = kv.shape[1]
    topk = idx.shape[2]
    if kv.shape != (b, n, d) or idx.shape[:2] != (b, m) or sink.shape != (h,):
        raise ValueError("shape mismatch")
    for t, name in ((q, "q"), (kv, "kv"), (idx, "idx"), (sink, "sink")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if o is None:
        o = torch.empty_like(q)
    elif o.shape != q.shape or o.dtype != torch.bfloat16 or not o.is_contiguous():
        raise ValueError("o must be a contiguous bf16 tensor shaped like q")
    need = sparse_attn_prefill_workspace_bytes(b, m, h, d, topk)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("ds_sparse_attn_prefill",
           _lib.ds_sparse_attn_prefill(_ptr(q), _ptr(kv), n, _ptr(sink), _ptr(idx), topk, float(scale), _ptr(o), b, m,
                                       h, d, _ptr(workspace), ws_bytes, _stream(stream)))
    return o


def sparse_attn_rope(q: torch.Tensor, kv: torch.Tensor, sink: torch.Tensor, idx: torch.Tensor, scale: float, rd: int,
                     table: torch.Tensor, start_pos: int, o: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``sparse_attn`` with the inverse RoPE of the output's last ``rd`` values fused in: token t of
    every sequence is rotated back by the angle of position ``start_pos + t`` (``table`` as for
    ``apply_rotary``).  Bit-identical to ``sparse_attn`` then ``apply_rotary(o, ..., inverse=True)``."""
    _need(q, torch.bfloat16, "q")
    _need(kv, torch.bfloat16, "kv")
    _need(sink, torch.float32, "sink")
    _need(idx, torch.int32, "idx")
    _check_table(table, rd)
    b, m, h, d = q.shape
    n = kv.shape[1]
    topk = idx.shape[2]
    if kv.shape != (b, n, d) or idx.shape[:2] != (b, m) or sink.shape != (h,):
        raise ValueError("shape mismatch")
    for t, name in ((q, "q"), (kv, "kv"), (idx, "idx"), (sink, "sink")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if o is None:
        o = torch.empty_like(q)
    elif o.shape != q.shape or o.dtype != torch.bfloat16 or not o.is_contiguous():
        raise ValueError("o must be a contiguous bf16 tensor shaped like q")
    need = sparse_attn_workspace_bytes(b, m, h, d, topk)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("ds_sparse_attn_rope",
           _lib.ds_sparse_attn_rope(_ptr(q), _ptr(kv), n, _ptr(sink), _ptr(idx), topk, float(scale), _ptr(o), b, m,
                                    h, d, _ptr(workspace), ws_bytes, rd, _ptr(table), table.shape[0], start_pos,
                                    _stream(stream)))
    return o


def _check_table(table: torch.Tensor, rd: int) -> None:
    _need(table, torch.float32, "table")
    if table.dim() != 3 or table.shape[1] * 2 != rd or table.shape[2] != 2 or not table.is_contiguous():
        raise ValueError("table must be a contiguous f32 [positions][rd/2][2] of (cos, sin)")


def apply_rotary(x: torch.Tensor, rd: int, table: torch.Tensor, start_pos: int, rows_per_pos: int,
                 positions_per_seq: int, inverse: bool = False, stream=None) -> torch.Tensor:
    """Rotate the last ``rd`` values of every row of ``x [..., row_len]`` (bf16, contiguous) in place;
    row r is at position start_pos + (r // rows_per_pos) % positions_per_seq.  For q or o
    ``[b][m][h][d]``: rows_per_pos = h, positions_per_seq = m."""
    _need(x, torch.bfloat16, "x")
    _check_table(table, rd)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    row_len = x.shape[-1]
    _check("ds_apply_rotary",
           _lib.ds_apply_rotary(_ptr(x), x.numel() // row_len if row_len else 0, row_len, rd, rows_per_pos,
                                positions_per_seq, start_pos, _ptr(table), table.shape[0], 1 if inverse else 0,
                                _stream(stream)))
    return x


def kv_rope_quant_ring_write(kv: torch.Tensor, ring: torch.Tensor | None, start_pos: int, window: int, rd: int,
                             table: torch.Tensor, stream=None) -> None:
    """RoPE on the last ``rd`` values of ``kv`` [b][s][d] (row t at start_pos + t), then the fp8
    round trip in place and the ring store (see ``kv_quant_ring_write``)."""
    _need(kv, torch.bfloat16, "kv")
    _check_table(table, rd)
    b, s, d = kv.shape
    if kv.stride(2) != 1 or kv.stride(1) != d:
        raise ValueError("kv rows must be contiguous")
    ring_bstride = 0
    if ring is not None:
        _need(ring, torch.bfloat16, "ring")
        if ring.shape[0] != b or ring.shape[2] != d or ring.shape[1] < window or ring.stride(2) != 1 \
                or ring.stride(1) != d:
            raise ValueError("ring must be [b][>=window][d] with contiguous rows")
        ring_bstride = ring.stride(0)
    _check("ds_kv_rope_quant_ring_write",
           _lib.ds_kv_rope_quant_ring_write(_ptr(kv), kv.stride(0), _ptr(ring), ring_bstride, b, s, d, start_pos,
                                            window, rd, _ptr(table), table.shape[0], _stream(stream)))


def kv_quantize_fp8(x: torch.Tensor, codes: torch.Tensor | None = None, exps: torch.Tensor | None = None,
                    stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """fp8 row store of bf16 rows ``x [..., d]`` (contiguous): e4m3fn codes ``[..., d]`` uint8 and
    per-32 scale exponents ``[..., d / 32]`` int8 (scale = 2^k)."""
    _need(x, torch.bfloat16, "x")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    d = x.shape[-1]
    if d % 32:
        raise ValueError("the last dimension must be a multiple of 32")
    if codes is None:
        codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if exps is None:
        exps = torch.empty(x.shape[:-1] + (d // 32,), dtype=torch.int8, device=x.device)
    _need(codes, torch.uint8, "codes")
    _need(exps, torch.int8, "exps")
    if codes.shape != x.shape or exps.shape != x.shape[:-1] + (d // 32,) or not codes.is_contiguous() \
            or not exps.is_contiguous():
        raise ValueError("codes must be shaped like x and exps like x with d / 32 columns, both contiguous")
    _check("ds_kv_quantize_fp8",
           _lib.ds_kv_quantize_fp8(_ptr(x), x.numel() // d if d else 0, d, _ptr(codes), _ptr(exps), _stream(stream)))
    return codes, exps


def kv_quant_ring_write_fp8(kv: torch.Tensor, ring_codes: torch.Tensor, ring_exps: torch.Tensor, start_pos: int,
                            window: int, stream=None) -> None:
    """fp8 round trip of ``kv`` [b][s][d] in place; the ring is an fp8 row store ``ring_codes``
    [b][R][d] uint8, ``ring_exps`` [b][R][d/32] int8 (R >= window; it may be the leading rows of
    the store ``sparse_attn_fp8kv`` reads)."""
    _need(kv, torch.bfloat16, "kv")
    _need(ring_codes, torch.uint8, "ring_codes")
    _need(ring_exps, torch.int8, "ring_exps")
    b, s, d = kv.shape
    if kv.stride(2) != 1 or kv.stride(1) != d:
        raise ValueError("kv rows must be contiguous")
    R = ring_codes.shape[1]
    if ring_codes.shape != (b, R, d) or ring_exps.shape != (b, R, d // 32) or not ring_codes.is_contiguous() \
            or not ring_exps.is_contiguous() or R < window:
        raise ValueError("the ring must be contiguous [b][>=window][d] codes and [b][>=window][d/32] exps")
    _check("ds_kv_quant_ring_write_fp8",
           _lib.ds_kv_quant_ring_write_fp8(_ptr(kv), kv.stride(0), _ptr(ring_codes), _ptr(ring_exps), R, b, s, d,
                                           start_pos, window, _stream(stream)))


def sparse_attn_fp8kv(q: torch.Tensor, kv_codes: torch.Tensor, kv_exps: torch.Tensor, sink: torch.Tensor,
                      idx: torch.Tensor, scale: float, o: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``sparse_attn`` with the rows read from an fp8 row store: kv_codes [b][n][d] uint8,
    kv_exps [b][n][d/32] int8.  Bit-identical to ``sparse_attn`` on the decoded rows."""
    _need(q, torch.bfloat16, "q")
    _need(kv_codes, torch.uint8, "kv_codes")
    _need(kv_exps, torch.int8, "kv_exps")
    _need(sink, torch.float32, "sink")
    _need(idx, torch.int32, "idx")
    b, m, h, d = q.shape
    n = kv_codes.shape[1]
    topk = idx.shape[2]
    if kv_codes.shape != (b, n, d) or kv_exps.shape != (b, n, d // 32) or idx.shape[:2] != (b, m) \
            or sink.shape != (h,):
        raise ValueError("shape mismatch")
    for t, name in ((q, "q"), (kv_codes, "kv_codes"), (kv_exps, "kv_exps"), (idx, "idx"), (sink, "sink")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if o is None:
        o = torch.empty_like(q)
    elif o.shape != q.shape or o.dtype != torch.bfloat16 or not o.is_contiguous():
        raise ValueError("o must be a contiguous bf16 tensor shaped like q")
    need = sparse_attn_workspace_bytes(b, m, h, d, topk)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("ds_sparse_attn_fp8kv",
           _lib.ds_sparse_attn_fp8kv(_ptr(q), _ptr(kv_codes), _ptr(kv_exps), n, _ptr(sink), _ptr(idx), topk,
                                     float(scale), _ptr(o), b, m, h, d, _ptr(workspace), ws_bytes,
                                     _stream(stream)))
    return o


# ---- the paged row stores: calls of a few microseconds, so their checks are single comparisons on the
# ---- way in, and only a refused call goes back over them to say what is wrong

_BF16, _F32, _I32, _U8, _I8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.int8


def _on(stream):
    """Tensors made inside belong to the stream of the call, not to the current one."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _fits(t: torch.Tensor, dtype, shape: tuple, dev: int) -> bool:
    return t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev


def _row_fits(t: torch.Tensor, dtype, n: int, dev: int) -> bool:
    return t.dtype is dtype and t.dim() == 1 and t.numel() == n and t.is_contiguous() and t.get_device() == dev


def _refuse(**tensors) -> None:
    """Raise for the first tensor (name=(tensor, dtype, shape or None)) that is not as it has to be."""
    cur = torch.cuda.current_device() if torch.cuda.is_available() else -1
    for name, (t, dtype, shape) in tensors.items():
        if t is None:
            raise ValueError(f"{name} is missing")
        _need(t, dtype, name)
        if t.get_device() != cur:
            raise ValueError(f"{name}: must be on the current CUDA device")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
        if shape is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    raise ValueError("the tensors do not fit together")


def _refuse_wide(fn: str, *sizes: int) -> None:
    """Raise for a number that the C call's int would not hold (ctypes would take its low 32 bits)."""
    if any(not -1 << 31 <= v < 1 << 31 for v in sizes):
        raise DsError(fn, DS_EUNSUPPORTED)


def _table_shape(rd: int, table: torch.Tensor | None) -> tuple:
    return (table.shape[0] if table is not None and table.dim() == 3 else 0, rd // 2, 2)


def norm_rotary(x: torch.Tensor, eps: float, rd: int, table: torch.Tensor | None, first: torch.Tensor,
                weight: torch.Tensor | None = None, lens: torch.Tensor | None = None, y: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """RMS norm of every row of ``x [b][s][h][d]`` (bf16, the h * d values of a token contiguous; tokens may
    lie in a wider tensor) and the rotation of its last ``rd`` values to position ``first[b] + t``, in
    one pass.  ``y``: bf16 [b][s][h][d] contiguous (``x`` itself when laid out so); tokens at or behind
    ``lens[b]`` leave it as it was (zeros in a new one).  So do tokens outside the table, which the device status
    names; in a new ``y`` without ``lens`` they hold nothing defined."""
    if x.dim() != 4:
        raise ValueError("x must be [b][s][h][d]")
    b, s, h, d = x.shape
    xb, xt, xh, xd = x.stride()
    dev = x.get_device()
    tab = _table_shape(rd, table) if rd else None
    if not (x.dtype is _BF16 and dev >= 0 and dev == _device() and _row_fits(first, _I32, b, dev)
            and (lens is None or _row_fits(lens, _I32, b, dev)) and (weight is None or _row_fits(weight, _F32, d, dev))
            and (rd == 0 or (table is not None and _fits(table, _F32, tab, dev)))
            and (y is None or _fits(y, _BF16, (b, s, h, d), dev))):
        given = {"lens": (lens, _I32, (b,)), "weight": (weight, _F32, (d,)), "y": (y, _BF16, x.shape)}
        _refuse(x=(x, _BF16, None), first=(first, _I32, (b,)), **{k: v for k, v in given.items() if v[0] is not None},
                **({"table": (table, _F32, tab)} if rd else {}))
    if x.numel() and (xd != 1 or (h > 1 and xh != d)):
        raise ValueError("the heads of a token must be contiguous")
    if (b * s * h | rd) >> 31:
        _refuse_wide("ds_norm_rotary", b * s * h, rd)
    if y is None:
        with _on(stream):
            y = (torch.empty if lens is None else torch.zeros)((b, s, h, d), dtype=_BF16, device=x.device)
    st = _lib.ds_norm_rotary(x.data_ptr(), xb if b > 1 else 0, xt if s > 1 else 0, y.data_ptr(), b, s, h, d,
                             None if weight is None else weight.data_ptr(), eps, rd, table.data_ptr() if rd else None,
                             tab[0] if rd else 0, first.data_ptr(), None if lens is None else lens.data_ptr(),
                             _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _check("ds_norm_rotary", st)
    return y


def kv_append_fp4_paged(x: torch.Tensor, codes: torch.Tensor, exps: torch.Tensor, block_table: torch.Tensor,
                        first: torch.Tensor, rd: int = 0, table: torch.Tensor | None = None, eps: float = 0.0,
                        weight: torch.Tensor | None = None, lens: torch.Tensor | None = None, pos_step: int = 1,
                        base: int = 0, window: int = 0, y: torch.Tensor | None = None, stream=None) -> None:
    """Rows ``x [b][s][d]`` (bf16), normalised (``eps`` > 0) and rotated (``rd`` > 0), into the paged 4-bit
    row store ``codes [pages][page][d/2]``, ``exps [pages][page][d/32]``: row ``i = first[b] + t`` goes to
    logical row ``base + i % window`` (``window`` > 0, the last ``window`` tokens) or ``base + i``, rotated
    to position ``i * pos_step``.  ``y``: bf16 [b][s][d] contiguous, receives the stored values."""
    _kv_append("ds_kv_append_fp4_paged", _lib.ds_kv_append_fp4_paged, 4, x, codes, exps, block_table, first, rd, table, eps,
               weight, lens, pos_step, base, window, y, stream)


def kv_append_fp8_paged(x: torch.Tensor, codes: torch.Tensor, exps: torch.Tensor, block_table: torch.Tensor,
                        first: torch.Tensor, rd: int = 0, table: torch.Tensor | None = None, eps: float = 0.0,
                        weight: torch.Tensor | None = None, lens: torch.Tensor | None = None, pos_step: int = 1,
                        base: int = 0, window: int = 0, y: torch.Tensor | None = None, stream=None) -> None:
    """``kv_append_fp4_paged`` into the paged 8-bit row store: ``codes [pages][page][d]`` of e4m3 codes."""
    _kv_append("ds_kv_append_fp8_paged", _lib.ds_kv_append_fp8_paged, 8, x, codes, exps, block_table, first, rd, table, eps,
               weight, lens, pos_step, base, window, y, stream)


_ROW = {4: "d/2", 8: "d"}     # bytes of a row's codes


def _kv_append(name, call, bits, x, codes, exps, block_table, first, rd, table, eps, weight, lens, pos_step, base, window, y,
               stream):
    if x.dim() != 3 or codes.dim() != 3 or block_table.dim() != 2:
        raise ValueError(f"x must be [b][s][d], codes [pages][page][{_ROW[bits]}] and block_table [b][max_pages]")
    b, s, d = x.shape
    xb, xt, xd = x.stride()
    pages, page, row = codes.shape
    tables, max_pages = block_table.shape
    dev = x.get_device()
    tab = _table_shape(rd, table) if rd else None
    if not (x.dtype is _BF16 and dev >= 0 and dev == _device()
            and codes.dtype is _U8 and row == d * bits // 8 and codes.is_contiguous() and codes.get_device() == dev
            and _fits(exps, _I8, (pages, page, d // 32), dev) and block_table.dtype is _I32 and tables == b
            and block_table.is_contiguous() and block_table.get_device() == dev and _row_fits(first, _I32, b, dev)
            and (lens is None or _row_fits(lens, _I32, b, dev)) and (weight is None or _row_fits(weight, _F32, d, dev))
            and (rd == 0 or (table is not None and _fits(table, _F32, tab, dev)))
            and (y is None or _fits(y, _BF16, (b, s, d), dev))):
        given = {"lens": (lens, _I32, (b,)), "weight": (weight, _F32, (d,)), "y": (y, _BF16, x.shape)}
        _refuse(x=(x, _BF16, None), codes=(codes, _U8, (pages, page, d * bits // 8)), exps=(exps, _I8, (pages, page, d // 32)),
                block_table=(block_table, _I32, (b, max_pages)), first=(first, _I32, (b,)),
                **{k: v for k, v in given.items() if v[0] is not None}, **({"table": (table, _F32, tab)} if rd else {}))
    if x.numel() and xd != 1:
        raise ValueError("the values of a row must be contiguous")
    if (b * s | page | max_pages | pos_step | base | window | rd) >> 31:
        _refuse_wide(name, b * s, page, max_pages, pos_step, base, window, rd)
    if 0.0 < eps < 2.0 ** -100:            # as a float it could be 0, which is no norm
        raise DsError(name, DS_EINVAL)
    st = call(x.data_ptr(), xb if b > 1 else 0, xt if s > 1 else 0, None if y is None else y.data_ptr(), b, s, d,
              None if weight is None else weight.data_ptr(), eps, rd, table.data_ptr() if rd else None, tab[0] if rd else 0,
              first.data_ptr(), None if lens is None else lens.data_ptr(), pos_step, base, window, codes.data_ptr(),
              exps.data_ptr(), pages, page, block_table.data_ptr(), max_pages,
              _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _check(name, st)


def kv_read_fp8_paged(codes: torch.Tensor, exps: torch.Tensor, block_table: torch.Tensor, n: int,
                      first: torch.Tensor | None = None, idx: torch.Tensor | None = None,
                      lens: torch.Tensor | None = None, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``n`` rows of every sequence of the paged 8-bit row store as bf16 ``y [b][n][d]``: logical rows
    ``idx [b][n]`` (entries < 0: zeros), or rows ``first[b] + i`` (``first`` missing: from row 0).  Rows at or behind
    ``lens[b]`` leave ``y`` as it was (zeros in a new one)."""
    return _kv_read("ds_kv_read_fp8_paged", _lib.ds_kv_read_fp8_paged, 8, codes, exps, block_table, n, first, idx, lens, y,
                    stream)


def kv_read_fp4_paged(codes: torch.Tensor, exps: torch.Tensor, block_table: torch.Tensor, n: int,
                      first: torch.Tensor | None = None, idx: torch.Tensor | None = None,
                      lens: torch.Tensor | None = None, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``kv_read_fp8_paged`` of the paged 4-bit row store (``codes [pages][page][d/2]``)."""
    return _kv_read("ds_kv_read_fp4_paged", _lib.ds_kv_read_fp4_paged, 4, codes, exps, block_table, n, first, idx, lens, y,
                    stream)


def _kv_read(name, call, bits, codes, exps, block_table, n, first, idx, lens, y, stream):
    if codes.dim() != 3 or block_table.dim() != 2:
        raise ValueError(f"codes must be [pages][page][{_ROW[bits]}] and block_table [b][max_pages]")
    pages, page, row = codes.shape
    d = row * 8 // bits
    b, max_pages = block_table.shape
    dev = codes.get_device()
    if not (codes.dtype is _U8 and codes.is_contiguous() and dev >= 0 and dev == _device()
            and _fits(exps, _I8, (pages, page, d // 32), dev) and _fits(block_table, _I32, (b, max_pages), dev)
            and (first is None or _row_fits(first, _I32, b, dev)) and (idx is None or _fits(idx, _I32, (b, n), dev))
            and (lens is None or _row_fits(lens, _I32, b, dev)) and (y is None or _fits(y, _BF16, (b, n, d), dev))):
        given = {"first": (first, _I32, (b,)), "idx": (idx, _I32, (b, n)), "lens": (lens, _I32, (b,)), "y": (y, _BF16, (b, n, d))}
        _refuse(codes=(codes, _U8, codes.shape), exps=(exps, _I8, (pages, page, d // 32)),
                block_table=(block_table, _I32, (b, max_pages)), **{k: v for k, v in given.items() if v[0] is not None})
    if idx is not None and first is not None:
        raise ValueError("rows are listed by idx or follow first, not both")
    if n < 0 or (b * n | page | max_pages) >> 31:
        _refuse_wide(name, b * n, page, max_pages)
        raise DsError(name, DS_EINVAL)
    if y is None:
        with _on(stream):
            y = (torch.empty if lens is None else torch.zeros)((b, n, d), dtype=_BF16, device=codes.device)
    st = call(codes.data_ptr(), exps.data_ptr(), pages, page, block_table.data_ptr(), max_pages,
              None if idx is None else idx.data_ptr(), None if first is None else first.data_ptr(),
              None if lens is None else lens.data_ptr(), y.data_ptr(), b, n, d,
              _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        _check(name, st)
    return y


def chunk_attn_fp8_paged_workspace_bytes(b: int, m: int, h: int, d: int, window: int, ratio: int, page: int,
                                         max_pages: int) -> int:
    return int(_lib.ds_chunk_attn_fp8_paged_workspace_bytes(b, m, h, d, window, ratio, page, max_pages))


@functools.lru_cache(maxsize=64)
def _chunk_workspace_bytes(dev: int, *args: int) -> int:
    return chunk_attn_fp8_paged_workspace_bytes(*args)


def chunk_attn_fp8_paged(q: torch.Tensor, codes: torch.Tensor, exps: torch.Tensor, block_table: torch.Tensor,
                         first: torch.Tensor, sink: torch.Tensor, scale: float, window: int, ring: int = 0, ratio: int = 0,
                         base: int = 0, lens: torch.Tensor | None = None, rd: int = 0, table: torch.Tensor | None = None,
                         o: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of a chunk of new tokens ``q [b][m][h][512]`` over the paged 8-bit row store.  Token t of a sequence is at
    position ``p = first[b] + t`` and sees the rows of its last ``window`` positions (0: all; position i is logical row
    ``i % ring``, or i without a ring) and compressed rows 0 .. (p + 1) // ratio - 1 (``ratio`` 0: none), logical
    rows ``base + j``; with ``rd`` > 0 the last ``rd`` values of its output are rotated back.  Tokens at or behind
    ``lens[b]`` leave ``o`` as it was (zeros in a new one).  Workspace and form go by ``block_table``'s columns: one much
    wider than the sequences are long is better given as a copy of its first columns."""
    if q.dim() != 4 or codes.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q must be [b][m][h][d], codes [pages][page][d] and block_table [b][max_pages]")
    b, m, h, d = q.shape
    pages, page, row = codes.shape
    tables, max_pages = block_table.shape
    dev = q.get_device()
    tab = _table_shape(rd, table) if rd else None
    if not (q.dtype is _BF16 and q.is_contiguous() and dev >= 0 and dev == _device()
            and codes.dtype is _U8 and row == d and codes.is_contiguous() and codes.get_device() == dev
            and _fits(exps, _I8, (pages, page, d // 32), dev) and block_table.dtype is _I32 and tables == b
            and block_table.is_contiguous() and block_table.get_device() == dev and _row_fits(sink, _F32, h, dev)
            and _row_fits(first, _I32, b, dev) and (lens is None or _row_fits(lens, _I32, b, dev))
            and (o is None or _fits(o, _BF16, (b, m, h, d), dev))
            and (rd == 0 or (table is not None and _fits(table, _F32, tab, dev)))
            and (workspace is None or (workspace.get_device() == dev and workspace.is_contiguous()))):
        given = {"lens": (lens, _I32, (b,)), "o": (o, _BF16, q.shape),
                 "workspace": (workspace, None if workspace is None else workspace.dtype, None if workspace is None else workspace.shape)}
        _refuse(q=(q, _BF16, q.shape), codes=(codes, _U8, (pages, page, d)), exps=(exps, _I8, (pages, page, d // 32)),
                block_table=(block_table, _I32, (b, max_pages)), first=(first, _I32, (b,)), sink=(sink, _F32, (h,)),
                **{k: v for k, v in given.items() if v[0] is not None}, **({"table": (table, _F32, tab)} if rd else {}))
    if (b * m * h | page | max_pages | window | ring | ratio | base | rd) >> 31:
        _refuse_wide("ds_chunk_attn_fp8_paged", b * m * h, page, max_pages, window, ring, ratio, base, rd)
    if o is None:
        with _on(stream):
            o = torch.empty_like(q) if lens is None else torch.zeros_like(q)
    ws, ws_bytes = None, 0
    if workspace is not None:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    else:
        need = _chunk_workspace_bytes(dev, b, m, h, d, window, ratio, page, max_pages)
        if need:
            with _on(stream):
                workspace = torch.empty(need, dtype=_U8, device=q.device)
            ws, ws_bytes = workspace.data_ptr(), need
    st = _lib.ds_chunk_attn_fp8_paged(q.data_ptr(), codes.data_ptr(), exps.data_ptr(), pages, page, block_table.data_ptr(),
                                      max_pages, sink.data_ptr(), scale, o.data_ptr(), b, m, h, d, first.data_ptr(),
                                      None if lens is None else lens.data_ptr(), window, ring, ratio, base, ws, ws_bytes,
                                      rd, table.data_ptr() if rd else None, tab[0] if rd else 0,
                                      _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        # the size kept for this shape may be the 0 of a query that failed: the next call asks anew
        _chunk_workspace_bytes.cache_clear()
        _check("ds_chunk_attn_fp8_paged", st)
    return o


def sparse_attn_fp4_paged_workspace_bytes(b: int, m: int, h: int, d: int, topk: int) -> int:
    return int(_lib.ds_sparse_attn_fp4_paged_workspace_bytes(b, m, h, d, topk))


@functools.lru_cache(maxsize=64)
def _fp4_workspace_bytes(dev: int, b: int, m: int, h: int, d: int, topk: int) -> int:
    return sparse_attn_fp4_paged_workspace_bytes(b, m, h, d, topk)


def sparse_attn_fp4_paged(q: torch.Tensor, codes: torch.Tensor, exps: torch.Tensor, block_table: torch.Tensor,
                          sink: torch.Tensor, idx: torch.Tensor, scale: float, rd: int = 0,
                          table: torch.Tensor | None = None, first: torch.Tensor | None = None,
                          o: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                          stream=None, lens: torch.Tensor | None = None) -> torch.Tensor:
    """``sparse_attn`` over the paged 4-bit row store (``idx`` lists logical rows of each sequence); with
    ``rd`` > 0 the last ``rd`` values of token t's output are rotated back by position ``first[b] + t``.
    Tokens at or behind ``lens[b]`` leave ``o`` as it was (zeros in a new one)."""
    if q.dim() != 4 or idx.dim() != 3 or codes.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q must be [b][m][h][d], idx [b][m][topk], codes [pages][page][d/2] and block_table [b][max_pages]")
    b, m, h, d = q.shape
    pages, page, half = codes.shape
    tables, max_pages = block_table.shape
    ib, im, topk = idx.shape
    dev = q.get_device()
    tab = _table_shape(rd, table) if rd else None
    if not (q.dtype is _BF16 and q.is_contiguous() and dev >= 0 and dev == _device()
            and codes.dtype is _U8 and half == d // 2 and codes.is_contiguous() and codes.get_device() == dev
            and _fits(exps, _I8, (pages, page, d // 32), dev) and block_table.dtype is _I32 and tables == b
            and block_table.is_contiguous() and block_table.get_device() == dev and _row_fits(sink, _F32, h, dev)
            and idx.dtype is _I32 and ib == b and im == m and idx.is_contiguous() and idx.get_device() == dev
            and (o is None or _fits(o, _BF16, (b, m, h, d), dev)) and (lens is None or _row_fits(lens, _I32, b, dev))
            and (rd == 0 or (table is not None and _fits(table, _F32, tab, dev) and first is not None
                             and _row_fits(first, _I32, b, dev)))
            and (workspace is None or (workspace.get_device() == dev and workspace.is_contiguous()))):
        _refuse(q=(q, _BF16, q.shape), codes=(codes, _U8, (pages, page, d // 2)), exps=(exps, _I8, (pages, page, d // 32)),
                block_table=(block_table, _I32, (b, max_pages)), sink=(sink, _F32, (h,)), idx=(idx, _I32, (b, m, topk)),
                **({"o": (o, _BF16, q.shape)} if o is not None else {}), **({"lens": (lens, _I32, (b,))} if lens is not None else {}),
                **({"table": (table, _F32, tab), "first": (first, _I32, (b,))} if rd else {}),
                **({"workspace": (workspace, workspace.dtype, workspace.shape)} if workspace is not None else {}))
    if (b * m | topk | page | max_pages | rd) >> 31:
        _refuse_wide("ds_sparse_attn_fp4_paged", b * m, topk, page, max_pages, rd)
    if o is None:
        if stream is None and lens is None:
            o = torch.empty_like(q)
        else:
            with _on(stream):
                o = torch.empty_like(q) if lens is None else torch.zeros_like(q)
    ws, ws_bytes = None, 0
    if workspace is not None:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    else:
        need = _fp4_workspace_bytes(dev, b, m, h, d, topk)
        if need:
            if stream is None:
                workspace = torch.empty(need, dtype=_U8, device=q.device)
            else:
                with _on(stream):
                    workspace = torch.empty(need, dtype=_U8, device=q.device)
            ws, ws_bytes = workspace.data_ptr(), need
    args = (q.data_ptr(), codes.data_ptr(), exps.data_ptr(), pages, page, block_table.data_ptr(), max_pages,
            sink.data_ptr(), idx.data_ptr(), topk, scale, o.data_ptr(), b, m, h, d, ws, ws_bytes, rd,
            table.data_ptr() if rd else None, tab[0] if rd else 0, first.data_ptr() if rd else None)
    on = _raw_stream(dev) if stream is None else stream.cuda_stream
    if lens is None:
        st = _lib.ds_sparse_attn_fp4_paged(*args, on)
    else:
        st = _lib.ds_sparse_attn_fp4_paged_ragged(*args, lens.data_ptr(), on)
    if st:
        # the size kept for this shape may be the 0 of a query that failed: the next call asks anew
        _fp4_workspace_bytes.cache_clear()
        _check("ds_sparse_attn_fp4_paged", st)
    return o


def device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status bits (0 = clean)."""
    bits = ctypes.c_uint(0)
    st = _lib.ds_device_status(_stream(stream), ctypes.byref(bits))
    if st not in (DS_OK, DS_EDEVICE):
        raise DsError("ds_device_status", st)
    return bits.value


def _indexer_inputs(q: torch.Tensor, k: torch.Tensor, w: torch.Tensor):
    _need(q, torch.bfloat16, "q")
    _need(k, torch.bfloat16, "k")
    _need(w, torch.float32, "w")
    b, s, H, D = q.shape
    T = k.shape[1]
    if k.shape != (b, T, D) or w.shape != (b, s, H):
        raise ValueError("shape mismatch: q [b][s][H][D], k [b][T][D], w [b][s][H]")
    for t, name in ((q, "q"), (k, "k"), (w, "w")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return b, s, H, D, T


def indexer_visible(s: int, start_pos: int, ratio: int) -> int:
    """Compressed positions scored for a step of s queries at start_pos: (start_pos + s) // ratio."""
    return (start_pos + s) // ratio


def indexer_scores(q: torch.Tensor, k: torch.Tensor, w: torch.Tensor, start_pos: int, ratio: int,
                   scores: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """f32 scores [b][s][Tv] of the Indexer (-inf where a position is not visible yet)."""
    b, s, H, D, T = _indexer_inputs(q, k, w)
    Tv = indexer_visible(s, start_pos, ratio)
    if scores is None:
        scores = torch.empty((b, s, Tv), dtype=torch.float32, device=q.device)
    _need(scores, torch.float32, "scores")
    if scores.shape[:2] != (b, s) or scores.shape[2] < Tv or scores.stride(2) != 1 or scores.stride(1) != scores.shape[2] \
            or scores.stride(0) != s * scores.shape[2]:
        raise ValueError("scores must be a contiguous f32 [b][s][>= Tv]")
    _check("ds_indexer_scores",
           _lib.ds_indexer_scores(_ptr(q), _ptr(k), _ptr(w), b, s, H, D, T, start_pos, ratio, _ptr(scores),
                                  scores.shape[2], _stream(stream)))
    return scores


def indexer_select(scores: torch.Tensor, start_pos: int, ratio: int, topk: int, offset: int = 0,
                   idx: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Top-k positions per query from scores [b][s][>= Tv] (contiguous f32): int32 [b][s][kk]."""
    _need(scores, torch.float32, "scores")
    if not scores.is_contiguous():
        raise ValueError("scores must be contiguous")
    b, s, ld = scores.shape
    kk = min(topk, indexer_visible(s, start_pos, ratio))
    if idx is None:
        idx = torch.empty((b, s, kk), dtype=torch.int32, device=scores.device)
    _need(idx, torch.int32, "idx")
    if idx.shape != (b, s, kk) or not idx.is_contiguous():
        raise ValueError("idx must be a contiguous int32 [b][s][kk]")
    _check("ds_indexer_select",
           _lib.ds_indexer_select(_ptr(scores), ld, b, s, start_pos, ratio, topk, offset, _ptr(idx), _stream(stream)))
    return idx


def indexer_workspace_bytes(b: int, s: int, start_pos: int, ratio: int) -> int:
    return int(_lib.ds_indexer_workspace_bytes(b, s, start_pos, ratio))


def indexer_topk(q: torch.Tensor, k: torch.Tensor, w: torch.Tensor, start_pos: int, ratio: int, topk: int,
                 offset: int = 0, idx: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """The Indexer's kept positions: int32 [b][s][min(topk, Tv)], ascending, + offset, -1 if unseen."""
    b, s, H, D, T = _indexer_inputs(q, k, w)
    kk = min(topk, indexer_visible(s, start_pos, ratio))
    if idx is None:
        idx = torch.empty((b, s, kk), dtype=torch.int32, device=q.device)
    _need(idx, torch.int32, "idx")
    if idx.shape != (b, s, kk) or not idx.is_contiguous():
        raise ValueError("idx must be a contiguous int32 [b][s][kk]")
    need = indexer_workspace_bytes(b, s, start_pos, ratio)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check("ds_indexer_topk",
           _lib.ds_indexer_topk(_ptr(q), _ptr(k), _ptr(w), b, s, H, D, T, start_pos, ratio, topk, offset, _ptr(idx),
                                _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return idx


def test_set_stall(on: bool) -> None:
    """Test hook: while on, every sparse_attn launch has a bounded wait run out (DS_DEV_TIMEOUT)."""
    _lib.ds_test_set_stall(1 if on else 0)


KERNEL_AUTO, KERNEL_CLUSTER, KERNEL_ONE_CTA = 0, 1, 2


def sparse_attn_launches(b: int, m: int, h: int, d: int, topk: int) -> tuple[int, int]:
    """(kernels a sparse_attn call of this shape launches, the attention kernel it runs:
    KERNEL_CLUSTER or KERNEL_ONE_CTA)."""
    n, which, _ = sparse_attn_plan(b, m, h, d, topk)
    return n, which


def sparse_attn_plan(b: int, m: int, h: int, d: int, topk: int) -> tuple[int, int, int]:
    """(kernels launched, attention kernel, workspace bytes that kernel needs) for a sparse_attn
    call of this shape."""
    which = ctypes.c_int(0)
    ws = ctypes.c_size_t(0)
    n = _lib.ds_sparse_attn_launches(b, m, h, d, topk, ctypes.byref(which), ctypes.byref(ws))
    if n < 0:
        raise DsError("ds_sparse_attn_launches", n)
    return n, which.value, ws.value


def test_set_kernel(which: int) -> None:
    """Test hook: the attention kernel ds_sparse_attn runs (KERNEL_AUTO, KERNEL_CLUSTER or
    KERNEL_ONE_CTA, the latter wherever it is built for the shape)."""
    _check("ds_test_set_kernel", _lib.ds_test_set_kernel(int(which)))


def status_string(status: int) -> str:
    return _lib.ds_status_string(status).decode()
