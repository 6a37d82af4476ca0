"""Python binding of the GB300 verify-attention library (``include/trtv.h``).

Argument marshalling only: each function takes torch CUDA tensors (or raw
device pointers), converts them to pointers and sizes, and calls the C entry
point of the same name in ``_lib/libtrtv.so``.  Every step of the path runs in
the library's CUDA kernels; there is no fallback.  Importing the package does
not need a GPU, but calling a compute function without the built library or
without a GPU raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

from . import _build

__all__ = [
    "TRTV_OK", "TRTV_BF16", "TRTV_FP8_E4M3", "TRTV_F32", "TRTV_FP4_E2M1", "TrtvError", "Geom", "load",
    "trtv_subpage_view", "trtv_workspace_bytes", "trtv_verify_dense", "trtv_msa_proxy_score",
    "trtv_msa_topk", "trtv_msa_sparse_attn", "trtv_get_device_error", "trtv_version",
    "trtv_verify_dense_noalloc", "trtv_stage_kv", "trtv_flatten_page_table",
    "trtv_page_table_from_flat", "trtv_workspace_bytes_flat", "trtv_verify_dense_flat",
    "trtv_draft_attn_p32", "trtv_msa_select", "trtv_msa_verify", "trtv_status_string",
    "trtv_test_withhold_pages", "trtv_norm_rope_stage", "trtv_workspace_bytes_rows", "trtv_prompt_attn",
    "trtv_verify_tree", "trtv_tree_commit", "trtv_read_kv", "trtv_workspace_bytes_pages",
    "trtv_pages_fork", "trtv_pages_compact", "NormRope", "geom_of", "EXPORTS",
]

TRTV_OK, TRTV_ERR_INVALID_ARG, TRTV_ERR_UNSUPPORTED, TRTV_ERR_CUDA, TRTV_ERR_WORKSPACE = range(5)
TRTV_BF16, TRTV_FP8_E4M3, TRTV_F32, TRTV_FP4_E2M1 = 0, 1, 2, 3
DEVERR_KV_LEN, DEVERR_PAGE_ID, DEVERR_BLOCK_IDX, DEVERR_TIMEOUT = 1, 2, 4, 8
DEVERR_INDPTR, DEVERR_POSITION, DEVERR_PATH = 16, 32, 64
DEVERR_SLOTS, DEVERR_REFS, DEVERR_PARENT, DEVERR_LOGITS = 128, 256, 512, 1024

# every function the C header declares
EXPORTS = ("trtv_status_string", "trtv_version", "trtv_subpage_view", "trtv_workspace_bytes",
           "trtv_verify_dense", "trtv_verify_dense_noalloc", "trtv_msa_proxy_score", "trtv_msa_topk",
           "trtv_msa_sparse_attn", "trtv_stage_kv", "trtv_flatten_page_table",
           "trtv_page_table_from_flat", "trtv_workspace_bytes_flat", "trtv_verify_dense_flat",
           "trtv_draft_attn_p32", "trtv_msa_select", "trtv_msa_verify", "trtv_test_withhold_pages",
           "trtv_get_device_error", "trtv_norm_rope_stage", "trtv_workspace_bytes_rows", "trtv_prompt_attn",
           "trtv_verify_tree", "trtv_tree_commit", "trtv_read_kv", "trtv_workspace_bytes_pages", "trtv_pages_fork",
           "trtv_pages_compact")


class TrtvError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {msg} (status {status})")
        self.status = status


class Geom(ctypes.Structure):
    """Mirror of ``trtv_geom``."""
    _fields_ = [("batch", ctypes.c_int32), ("qo_len", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("max_pages_per_req", ctypes.c_int32),
                ("num_slots", ctypes.c_int32), ("slot_stride", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("sm_scale", ctypes.c_float),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
                ("num_ctas", ctypes.c_int32)]


class NormRope(ctypes.Structure):
    """Mirror of ``trtv_norm_rope``."""
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("rope_table", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("table_len", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float)]


_NORM_ROPE = struct.Struct("=QQQqqqQQQQiiif")


_lib: Optional[ctypes.CDLL] = None


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load ``libtrtv.so`` (building it first when asked).  Raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if not os.path.exists(path):
        if not build_if_missing:
            raise ImportError(f"libtrtv.so is not built ({path}); run __graft_entry__.build() "
                              "or python -m speculative_decode_verify_kv_gb300._build")
        _build.build()
    h = ctypes.CDLL(path)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    G = ctypes.POINTER(Geom)
    h.trtv_status_string.restype = ctypes.c_char_p
    h.trtv_status_string.argtypes = [ctypes.c_int]
    h.trtv_version.restype = i32
    h.trtv_version.argtypes = []
    h.trtv_subpage_view.restype = ctypes.c_int
    h.trtv_subpage_view.argtypes = [G, vp, vp, vp, vp, vp]
    h.trtv_workspace_bytes.restype = sz
    h.trtv_workspace_bytes.argtypes = [G, i32]
    h.trtv_verify_dense.restype = ctypes.c_int
    h.trtv_verify_dense.argtypes = [G, vp, vp, vp, vp, vp, i32, vp, sz, vp]
    h.trtv_verify_dense_noalloc.restype = ctypes.c_int
    h.trtv_verify_dense_noalloc.argtypes = [G, vp, vp, vp, vp, vp, i32, vp]
    h.trtv_msa_proxy_score.restype = ctypes.c_int
    h.trtv_msa_proxy_score.argtypes = [G, vp, vp, vp, vp, vp, vp]
    h.trtv_msa_topk.restype = ctypes.c_int
    h.trtv_msa_topk.argtypes = [G, vp, vp, i32, vp, vp]
    h.trtv_msa_sparse_attn.restype = ctypes.c_int
    h.trtv_msa_sparse_attn.argtypes = [G, vp, vp, vp, vp, vp, i32, vp, i32, vp, sz, vp]
    h.trtv_stage_kv.restype = ctypes.c_int
    h.trtv_stage_kv.argtypes = [G, vp, vp, vp, vp, vp, vp]
    h.trtv_flatten_page_table.restype = ctypes.c_int
    h.trtv_flatten_page_table.argtypes = [G, vp, vp, vp, vp, vp]
    h.trtv_page_table_from_flat.restype = ctypes.c_int
    h.trtv_page_table_from_flat.argtypes = [G, vp, vp, vp, vp]
    h.trtv_workspace_bytes_flat.restype = sz
    h.trtv_workspace_bytes_flat.argtypes = [G]
    h.trtv_verify_dense_flat.restype = ctypes.c_int
    h.trtv_verify_dense_flat.argtypes = [G, vp, vp, vp, vp, vp, i32, vp, sz, vp]
    h.trtv_draft_attn_p32.restype = ctypes.c_int
    h.trtv_draft_attn_p32.argtypes = [G, vp, vp, vp, vp, vp, vp, i32, vp, sz, vp]
    h.trtv_msa_select.restype = ctypes.c_int
    h.trtv_msa_select.argtypes = [G, vp, vp, vp, vp, i32, vp, vp, vp, sz, vp]
    h.trtv_msa_verify.restype = ctypes.c_int
    h.trtv_msa_verify.argtypes = [G, vp, vp, vp, vp, i32, vp, vp, vp, i32, vp, sz, vp]
    h.trtv_get_device_error.restype = ctypes.c_int
    h.trtv_get_device_error.argtypes = [ctypes.POINTER(ctypes.c_int32), vp]
    h.trtv_test_withhold_pages.restype = ctypes.c_int
    h.trtv_test_withhold_pages.argtypes = [i32, ctypes.c_uint32]
    h.trtv_norm_rope_stage.restype = ctypes.c_int
    h.trtv_norm_rope_stage.argtypes = [G, ctypes.POINTER(NormRope), vp, i32, vp, vp, vp, vp, vp]
    h.trtv_workspace_bytes_rows.restype = sz
    h.trtv_workspace_bytes_rows.argtypes = [G]
    h.trtv_prompt_attn.restype = ctypes.c_int
    h.trtv_prompt_attn.argtypes = [G, vp, vp, vp, vp, vp, i32, vp, i32, vp, sz, vp]
    h.trtv_verify_tree.restype = ctypes.c_int
    h.trtv_verify_tree.argtypes = [G, vp, vp, vp, vp, vp, i32, vp, vp, i32, vp, sz, vp]
    h.trtv_tree_commit.restype = ctypes.c_int
    h.trtv_tree_commit.argtypes = [G, vp, vp, vp, vp, vp, vp, i32, vp, vp]
    h.trtv_read_kv.restype = ctypes.c_int
    h.trtv_read_kv.argtypes = [G, vp, vp, vp, vp, i32, vp, vp, vp]
    h.trtv_workspace_bytes_pages.restype = sz
    h.trtv_workspace_bytes_pages.argtypes = [G, i32]
    h.trtv_pages_fork.restype = ctypes.c_int
    h.trtv_pages_fork.argtypes = [G, vp, i32, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp]
    h.trtv_pages_compact.restype = ctypes.c_int
    h.trtv_pages_compact.argtypes = [G, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    _lib = h
    return h


def _ptr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not x.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return x.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return _begin(None)[1]
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, st: int) -> None:
    if st != TRTV_OK:
        raise TrtvError(fn, st, load().trtv_status_string(st).decode())


def geom_of(p, num_ctas: int = 0, **over) -> Geom:
    """Geom from a workloads.VerifyProblem-like object (fields overridable)."""
    f = dict(batch=p.batch, qo_len=p.qo_len, num_q_heads=p.num_q_heads,
             num_kv_heads=p.num_kv_heads, head_dim=p.head_dim,
             max_pages_per_req=p.max_pages_per_req, num_slots=p.num_slots,
             slot_stride=p.slot_stride,
             kv_dtype=TRTV_FP8_E4M3 if p.kv_dtype == "fp8_e4m3" else TRTV_BF16,
             sm_scale=p.sm_scale, k_scale=p.k_scale, v_scale=p.v_scale, num_ctas=num_ctas)
    f.update(over)
    return Geom(**f)


def trtv_version() -> int:
    return load().trtv_version()


def trtv_status_string(st: int) -> str:
    return load().trtv_status_string(st).decode()


def trtv_workspace_bytes(geom: Geom, topk: int = 0) -> int:
    return load().trtv_workspace_bytes(ctypes.byref(geom), topk)


def trtv_subpage_view(geom: Geom, page_table, kv_lens, k_sub, v_sub, stream=None) -> None:
    _check("trtv_subpage_view", load().trtv_subpage_view(
        ctypes.byref(geom), _ptr(page_table), _ptr(kv_lens), _ptr(k_sub), _ptr(v_sub),
        _stream(stream)))


def trtv_verify_dense(geom: Geom, q, kv_pool, page_table, kv_lens, out, out_dtype: int,
                      workspace, ws_bytes: int, stream=None) -> None:
    _check("trtv_verify_dense", load().trtv_verify_dense(
        ctypes.byref(geom), _ptr(q), _ptr(kv_pool), _ptr(page_table), _ptr(kv_lens), _ptr(out),
        out_dtype, _ptr(workspace), ws_bytes, _stream(stream)))


def trtv_verify_dense_noalloc(geom: Geom, q, kv_pool, page_table, kv_lens, out, out_dtype: int,
                              stream=None) -> None:
    """trtv_verify_dense with the library's static device scratch instead of a
    caller workspace (for callers that cannot allocate device memory)."""
    _check("trtv_verify_dense_noalloc", load().trtv_verify_dense_noalloc(
        ctypes.byref(geom), _ptr(q), _ptr(kv_pool), _ptr(page_table), _ptr(kv_lens), _ptr(out),
        out_dtype, _stream(stream)))


def trtv_msa_proxy_score(geom: Geom, q, kv_pool, page_table, kv_lens, scores, stream=None) -> None:
    _check("trtv_msa_proxy_score", load().trtv_msa_proxy_score(
        ctypes.byref(geom), _ptr(q), _ptr(kv_pool), _ptr(page_table), _ptr(kv_lens),
        _ptr(scores), _stream(stream)))


def trtv_msa_topk(geom: Geom, scores, kv_lens, topk: int, block_idx, stream=None) -> None:
    _check("trtv_msa_topk", load().trtv_msa_topk(
        ctypes.byref(geom), _ptr(scores), _ptr(kv_lens), topk, _ptr(block_idx), _stream(stream)))


def trtv_msa_select(geom: Geom, q, kv_pool, page_table, kv_lens, topk: int, scores, block_idx,
                    workspace, ws_bytes: int, stream=None) -> None:
    """Proxy scores and per-token top-k in one call (fused where the tcgen05
    proxy kernel applies)."""
    _check("trtv_msa_select", load().trtv_msa_select(
        ctypes.byref(geom), _ptr(q), _ptr(kv_pool), _ptr(page_table), _ptr(kv_lens), topk,
        _ptr(scores), _ptr(block_idx), _ptr(workspace), ws_bytes, _stream(stream)))


def trtv_msa_verify(geom: Geom, q, kv_pool, page_table, kv_lens, topk: int, scores, block_idx, out,
                    out_dtype: int, workspace, ws_bytes: int, stream=None) -> None:
    """Proxy scores, per-token top-k and sparse attention in one call (the
    fused select builds the sparse plan where it applies)."""
    _check("trtv_msa_verify", load().trtv_msa_verify(
        ctypes.byref(geom), _ptr(q), _ptr(kv_pool), _ptr(page_table), _ptr(kv_lens), topk,
        _ptr(scores), _ptr(block_idx), _ptr(out), out_dtype, _ptr(workspace), ws_bytes, _stream(stream)))


def trtv_msa_sparse_attn(geom: Geom, q, kv_pool, page_table, kv_lens, block_idx, topk: int, out,
                         out_dtype: int, workspace, ws_bytes: int, stream=None) -> None:
    _check("trtv_msa_sparse_attn", load().trtv_msa_sparse_attn(
        ctypes.byref(geom), _ptr(q), _ptr(kv_pool), _ptr(page_table), _ptr(kv_lens),
        _ptr(block_idx), topk, _ptr(out), out_dtype, _ptr(workspace), ws_bytes, _stream(stream)))


def trtv_stage_kv(geom: Geom, k_new, v_new, kv_pool, page_table, kv_lens, stream=None) -> None:
    _check("trtv_stage_kv", load().trtv_stage_kv(
        ctypes.byref(geom), _ptr(k_new), _ptr(v_new), _ptr(kv_pool), _ptr(page_table), _ptr(kv_lens),
        _stream(stream)))


def trtv_flatten_page_table(geom: Geom, page_table, kv_lens, flat, indptr=None, stream=None) -> None:
    """Restage the flat (CSR) page table from the padded one and the lengths."""
    _check("trtv_flatten_page_table", load().trtv_flatten_page_table(
        ctypes.byref(geom), _ptr(page_table), _ptr(kv_lens), _ptr(flat), _ptr(indptr),
        _stream(stream)))


def trtv_page_table_from_flat(geom: Geom, flat, kv_lens, page_table, stream=None) -> None:
    """Padded page table from a flat one whose row bases follow the lengths."""
    _check("trtv_page_table_from_flat", load().trtv_page_table_from_flat(
        ctypes.byref(geom), _ptr(flat), _ptr(kv_lens), _ptr(page_table), _stream(stream)))


def trtv_workspace_bytes_flat(geom: Geom) -> int:
    return load().trtv_workspace_bytes_flat(ctypes.byref(geom))


def trtv_verify_dense_flat(geom: Geom, q, kv_pool, flat, kv_lens, out, out_dtype: int, workspace,
                           ws_bytes: int, stream=None) -> None:
    _check("trtv_verify_dense_flat", load().trtv_verify_dense_flat(
        ctypes.byref(geom), _ptr(q), _ptr(kv_pool), _ptr(flat), _ptr(kv_lens), _ptr(out), out_dtype,
        _ptr(workspace), ws_bytes, _stream(stream)))


def trtv_draft_attn_p32(geom: Geom, q, kv_pool, k_sub, v_sub, kv_lens, out, out_dtype: int,
                        workspace, ws_bytes: int, stream=None) -> None:
    """Attention read through the P32 sub-page tables (the drafter's view)."""
    _check("trtv_draft_attn_p32", load().trtv_draft_attn_p32(
        ctypes.byref(geom), _ptr(q), _ptr(kv_pool), _ptr(k_sub), _ptr(v_sub), _ptr(kv_lens),
        _ptr(out), out_dtype, _ptr(workspace), ws_bytes, _stream(stream)))


def trtv_test_withhold_pages(pages: int, wait_us: int = 0) -> None:
    """Test hook of the bounded waits: K producers stop after ``pages`` pages
    and every wait gives up after ``wait_us``; ``pages < 0`` restores normal
    operation."""
    _check("trtv_test_withhold_pages", load().trtv_test_withhold_pages(pages, wait_us))


def trtv_get_device_error(stream=None) -> int:
    v = ctypes.c_int32(0)
    _check("trtv_get_device_error", load().trtv_get_device_error(ctypes.byref(v), _stream(stream)))
    return v.value


# -- packed token rows -------------------------------------------------------
# These calls know their tensors' shapes, so they check them (a buffer too small
# for the geometry would be read out of bounds on the device), in few steps: on a
# small step the host's time is the call's time.

_torch = None


def _begin(stream):
    """(current device, raw stream) of a call."""
    global _torch
    if _torch is None:
        import torch
        torch.cuda.init()
        _torch = torch
    dev = _torch._C._cuda_getDevice()
    if stream is None:
        return dev, _torch._C._cuda_getCurrentRawStream(dev)
    return dev, stream if isinstance(stream, int) else stream.cuda_stream


def _refuse(fn: str, name: str, x, dev: int, dtype, shape):
    have = f"{x.dtype} {tuple(x.shape)} on {x.device}" if hasattr(x, "dtype") else repr(x)
    raise ValueError(f"{fn}: {name} is {have}{'' if not hasattr(x, 'is_contiguous') or x.is_contiguous() else ', not contiguous'}; "
                     f"expected {dtype} {tuple('any' if w is None else w for w in shape)}, contiguous, on the current "
                     f"device cuda:{dev}")


def _arg(fn: str, name: str, x, dev: int, dtype, shape) -> int:
    """Pointer of a contiguous tensor of this dtype and shape on the current device (a raw pointer passes)."""
    if x.__class__ is int:
        return x
    try:
        if x.dtype is dtype and x.shape == shape and x.get_device() == dev and x.is_contiguous():
            return x.data_ptr()
    except AttributeError:
        pass
    _refuse(fn, name, x, dev, dtype, shape)


def _rows_arg(fn: str, name: str, x, dev: int, shape):
    """Pointer and row pitch of a bf16 [rows, heads, dim] tensor whose rows may lie apart."""
    rows, heads, dim = shape
    if x.dtype is not _torch.bfloat16 or x.shape != shape or x.get_device() != dev:
        _refuse(fn, name, x, dev, _torch.bfloat16, shape)
    pitch, head, one = x.stride()
    if one != 1 or (head != dim and heads > 1):
        raise ValueError(f"{fn}: {name}'s heads of one token are not contiguous (strides {x.stride()})")
    return x.data_ptr(), pitch if rows > 1 else heads * dim


def _pool_arg(fn: str, geom: Geom, x, dev: int) -> int:
    if x.__class__ is int:
        return x
    need = geom.num_slots * geom.slot_stride * 128 * geom.num_kv_heads * geom.head_dim
    types = (_torch.uint8, _torch.float8_e4m3fn) if geom.kv_dtype == TRTV_FP8_E4M3 else (_torch.bfloat16,)
    if geom.kv_dtype == TRTV_FP4_E2M1:   # bytes: 4-bit codes and a scale byte for each 16
        need, types = need * 9 // 16, (_torch.uint8,)
    if x.dtype not in types or x.numel() < need or x.get_device() != dev or not x.is_contiguous():
        _refuse(fn, "kv_pool", x, dev, " or ".join(map(str, types)), (f"{need} elements",))
    return x.data_ptr()


def _tables(fn: str, geom: Geom, page_table, kv_lens, qo_indptr, dev: int):
    i32, b = _torch.int32, geom.batch
    return (_arg(fn, "page_table", page_table, dev, i32, (b, geom.max_pages_per_req)),
            _arg(fn, "kv_lens", kv_lens, dev, i32, (b,)),
            0 if qo_indptr is None else _arg(fn, "qo_indptr", qo_indptr, dev, i32, (b + 1,)))


def trtv_norm_rope_stage(geom: Geom, q, k, v, q_weight, k_weight, eps: float, rope_table, rot_dim: int,
                         interleaved: bool, positions, qo_indptr, q_out, kv_pool, page_table, kv_lens,
                         stream=None) -> None:
    """Per-head norm of queries and keys, rotation, and K/V staging of packed token rows: q [rows, Hq, D],
    k, v [rows, Hk, D] bf16, each possibly a view of one projection; q_out [rows, Hq, D] bf16."""
    fn = "trtv_norm_rope_stage"
    dev, st = _begin(stream)
    bf16, d = _torch.bfloat16, geom.head_dim
    rows = q.shape[0]
    qs, ks = (rows, geom.num_q_heads, d), (rows, geom.num_kv_heads, d)
    qp, q_pitch = _rows_arg(fn, "q", q, dev, qs)
    kp, k_pitch = _rows_arg(fn, "k", k, dev, ks)
    vp, v_pitch = _rows_arg(fn, "v", v, dev, ks)
    table_len = 0 if rope_table is None else rope_table.shape[0]
    a = NormRope.from_buffer_copy(_NORM_ROPE.pack(   # (0.5 us less than naming the fields)
        qp, kp, vp, q_pitch, k_pitch, v_pitch,
        0 if q_weight is None else _arg(fn, "q_weight", q_weight, dev, bf16, (d,)),
        0 if k_weight is None else _arg(fn, "k_weight", k_weight, dev, bf16, (d,)),
        0 if rope_table is None else _arg(fn, "rope_table", rope_table, dev, _torch.float32, (table_len, rot_dim)),
        0 if positions is None else _arg(fn, "positions", positions, dev, _torch.int32, (rows,)),
        table_len, rot_dim, 1 if interleaved else 0, eps))
    pt, kl, ip = _tables(fn, geom, page_table, kv_lens, qo_indptr, dev)
    _check(fn, load().trtv_norm_rope_stage(ctypes.byref(geom), ctypes.byref(a), ip, rows,
                                           _arg(fn, "q_out", q_out, dev, bf16, qs), _pool_arg(fn, geom, kv_pool, dev),
                                           pt, kl, st))


def trtv_workspace_bytes_rows(geom: Geom) -> int:
    return load().trtv_workspace_bytes_rows(ctypes.byref(geom))


def _workspace_arg(fn: str, workspace, ws_bytes: int, dev: int) -> int:
    if workspace.__class__ is int:
        return workspace
    if workspace.get_device() != dev or workspace.nbytes < ws_bytes or not workspace.is_contiguous():
        _refuse(fn, "workspace", workspace, dev, "any type,", (f"{ws_bytes} bytes",))
    return workspace.data_ptr()


def _rows_attn(fn: str, geom: Geom, q, kv_pool, page_table, kv_lens, qo_indptr, tree_mask, out, out_dtype: int,
               workspace, ws_bytes: int, stream) -> None:
    dev, st = _begin(stream)
    rows = q.shape[0]
    shape = (rows, geom.num_q_heads, geom.head_dim)
    pt, kl, ip = _tables(fn, geom, page_table, kv_lens, qo_indptr, dev)
    args = [ctypes.byref(geom), _arg(fn, "q", q, dev, _torch.bfloat16, shape), _pool_arg(fn, geom, kv_pool, dev), pt, kl, ip,
            rows]
    if fn == "trtv_verify_tree":
        uint32 = getattr(_torch, "uint32", None)
        args.append(_arg(fn, "tree_mask", tree_mask, dev,
                         uint32 if uint32 is not None and getattr(tree_mask, "dtype", None) is uint32 else _torch.int32,
                         (rows, (geom.qo_len + 31) // 32)))
    args.append(_arg(fn, "out", out, dev, _torch.float32 if out_dtype == TRTV_F32 else _torch.bfloat16, shape))
    _check(fn, getattr(load(), fn)(*args, out_dtype, _workspace_arg(fn, workspace, ws_bytes, dev), ws_bytes, st))


def trtv_prompt_attn(geom: Geom, q, kv_pool, page_table, kv_lens, qo_indptr, out, out_dtype: int, workspace,
                     ws_bytes: int, stream=None) -> None:
    """Causal attention of packed prompts (q, out [rows, Hq, D]) over the paged cache."""
    _rows_attn("trtv_prompt_attn", geom, q, kv_pool, page_table, kv_lens, qo_indptr, None, out, out_dtype, workspace,
               ws_bytes, stream)


def trtv_verify_tree(geom: Geom, q, kv_pool, page_table, kv_lens, qo_indptr, tree_mask, out, out_dtype: int,
                     workspace, ws_bytes: int, stream=None) -> None:
    """Attention of drafted trees over the paged cache; tree_mask int32 [rows, ceil(qo_len / 32)]."""
    _rows_attn("trtv_verify_tree", geom, q, kv_pool, page_table, kv_lens, qo_indptr, tree_mask, out, out_dtype, workspace,
               ws_bytes, stream)


def trtv_tree_commit(geom: Geom, kv_pool, page_table, kv_lens, qo_indptr, path, path_len, new_kv_lens,
                     stream=None) -> None:
    """Accepted path's cache rows to the front of the tree's positions, and the new lengths."""
    fn = "trtv_tree_commit"
    dev, st = _begin(stream)
    i32, b = _torch.int32, geom.batch
    pt, kl, ip = _tables(fn, geom, page_table, kv_lens, qo_indptr, dev)
    width = path.shape[1]
    _check(fn, load().trtv_tree_commit(ctypes.byref(geom), _pool_arg(fn, geom, kv_pool, dev), pt, kl, ip,
                                       _arg(fn, "path", path, dev, i32, (b, width)),
                                       _arg(fn, "path_len", path_len, dev, i32, (b,)), width,
                                       _arg(fn, "new_kv_lens", new_kv_lens, dev, i32, (b,)), st))


def trtv_read_kv(geom: Geom, kv_pool, page_table, kv_lens, qo_indptr, k_out, v_out, stream=None) -> None:
    """The packed tokens' cache rows as bf16: k_out, v_out [rows, Hk, D], either may be None."""
    fn = "trtv_read_kv"
    dev, st = _begin(stream)
    if k_out is None and v_out is None:
        raise ValueError(f"{fn}: k_out and v_out are both None")
    rows = (v_out if k_out is None else k_out).shape[0]
    shape = (rows, geom.num_kv_heads, geom.head_dim)
    pt, kl, ip = _tables(fn, geom, page_table, kv_lens, qo_indptr, dev)
    _check(fn, load().trtv_read_kv(ctypes.byref(geom), _pool_arg(fn, geom, kv_pool, dev), pt, kl, ip, rows,
                                   0 if k_out is None else _arg(fn, "k_out", k_out, dev, _torch.bfloat16, shape),
                                   0 if v_out is None else _arg(fn, "v_out", v_out, dev, _torch.bfloat16, shape), st))


# -- pages under the tables ----------------------------------------------------

def trtv_workspace_bytes_pages(geom: Geom, new_batch: int = 0) -> int:
    return load().trtv_workspace_bytes_pages(ctypes.byref(geom), new_batch)


def trtv_pages_fork(geom: Geom, kv_pool, buffers: int, ref_count, page_table, kv_lens, num_pages, parent, new_tokens,
                    new_ref_count, new_page_table, new_kv_lens, new_num_pages, workspace, ws_bytes: int, stream=None) -> None:
    """The next step's requests from this one's: they share full pages, get copies of pages that they write to and
    fresh slots for new_tokens more tokens (None: none); num_pages None: the pages of kv_lens."""
    fn = "trtv_pages_fork"
    dev, st = _begin(stream)
    i32, b, mp, slots = _torch.int32, geom.batch, geom.max_pages_per_req, geom.num_slots
    n = parent.shape[0]
    _check(fn, load().trtv_pages_fork(
        ctypes.byref(geom), _pool_arg(fn, geom, kv_pool, dev), buffers, _arg(fn, "ref_count", ref_count, dev, i32, (slots,)),
        _arg(fn, "page_table", page_table, dev, i32, (b, mp)), _arg(fn, "kv_lens", kv_lens, dev, i32, (b,)),
        0 if num_pages is None else _arg(fn, "num_pages", num_pages, dev, i32, (b,)),
        _arg(fn, "parent", parent, dev, i32, (n,)),
        0 if new_tokens is None else _arg(fn, "new_tokens", new_tokens, dev, i32, (n,)), n,
        _arg(fn, "new_ref_count", new_ref_count, dev, i32, (slots,)),
        _arg(fn, "new_page_table", new_page_table, dev, i32, (n, mp)), _arg(fn, "new_kv_lens", new_kv_lens, dev, i32, (n,)),
        0 if new_num_pages is None else _arg(fn, "new_num_pages", new_num_pages, dev, i32, (n,)),
        _workspace_arg(fn, workspace, ws_bytes, dev), ws_bytes, st))


def trtv_pages_compact(geom: Geom, kv_pool, buffers: int, ref_count, page_table, num_pages, slot_map, num_used,
                       new_ref_count, new_page_table, workspace, ws_bytes: int, stream=None) -> None:
    """The used slots to the front of the pool; slot_map says where each went (-1: it was free)."""
    fn = "trtv_pages_compact"
    dev, st = _begin(stream)
    i32, b, mp, slots = _torch.int32, geom.batch, geom.max_pages_per_req, geom.num_slots
    _check(fn, load().trtv_pages_compact(
        ctypes.byref(geom), _pool_arg(fn, geom, kv_pool, dev), buffers, _arg(fn, "ref_count", ref_count, dev, i32, (slots,)),
        _arg(fn, "page_table", page_table, dev, i32, (b, mp)), _arg(fn, "num_pages", num_pages, dev, i32, (b,)),
        _arg(fn, "slot_map", slot_map, dev, i32, (slots,)), _arg(fn, "num_used", num_used, dev, i32, (1,)),
        _arg(fn, "new_ref_count", new_ref_count, dev, i32, (slots,)),
        _arg(fn, "new_page_table", new_page_table, dev, i32, (b, mp)), _workspace_arg(fn, workspace, ws_bytes, dev), ws_bytes, st))
