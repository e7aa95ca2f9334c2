"""Python binding of the sfm C-ABI (``include/sfm.h``).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``_build/libsfm.so``.  torch is used for device memory and streams.
There is no CPU path: if the library is missing or no CUDA device is present
the calls raise.

Two layers:

* ``sfm_metadata_size`` / ``sfm_workspace_size`` / ``sfm_metadata`` /
  ``sfm_forward`` / ``sfm_debug_attended`` / ``sfm_error_string`` -- the C
  entry points with the same names, taking ``SfmParams`` / ``SfmTensors``
  ctypes structs and raw device pointers;
* ``sparse_flash_mla_metadata`` / ``sparse_flash_mla`` -- the two-call torch
  API of the "sparse_flash_mla" doc (函数原型), building those structs from
  tensors and keyword attributes;
* ``rope_frequencies`` / ``apply_rope`` / ``store_kv`` / ``index_scores`` /
  ``select_topk`` -- the operators around the attention in the same form, over
  ``sfm_rope_frequencies`` / ``sfm_rope`` / ``sfm_kv_store`` /
  ``sfm_index_scores`` / ``sfm_topk_select``: rotary positions, the rows of the
  caches, and the sparse indices the attention reads;
* ``masked_attention`` / ``tree_attention`` / ``merge_attention`` / ``move_kv``
  -- attention of many queries over the same rows (``sfm_dense_forward``), the
  joining of results over separate keys (``sfm_merge``) and the moving of an
  accepted path's rows (``sfm_kv_move``).

None of the torch-level calls records a gradient.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import math
import os
import struct
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libsfm.so")

BSND, TND, PAGED = 0, 1, 2
BF16, FP16, E4M3 = 0, 1, 2
KV_PLAIN, KV_INT8_PACKED, KV_FP8_PACKED, KV_FP8_ROWS = 0, 1, 2, 3
ROPE_INTERLEAVED, ROPE_HALF = 0, 1
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
SPLIT_BATCH_INVARIANT, SPLIT_OCCUPANCY = 0, 1
_LAYOUTS = {"BSND": BSND, "TND": TND, "PAGED": PAGED, "PA_BBND": PAGED, "PA_BSND": PAGED, "PA_ND": PAGED}

STATUS_BAD_INDEX = 0x01
STATUS_BAD_BLOCK = 0x02
STATUS_BAD_LENGTH = 0x04
STATUS_METADATA_MISMATCH = 0x08
STATUS_WORKSPACE_OVERFLOW = 0x10
STATUS_PLAN_OVERFLOW = 0x20
STATUS_TIMEOUT = 0x40


class SfmParams(C.Structure):
    _fields_ = [(n, C.c_int32) for n in (
        "num_heads_q", "num_heads_kv", "head_dim", "rope_head_dim", "batch_size", "max_seqlen_q", "total_q",
        "max_seqlen_ori_kv", "max_seqlen_cmp_kv", "ori_topk", "cmp_topk", "cmp_ratio", "ori_mask_mode",
        "cmp_mask_mode", "ori_win_left", "ori_win_right", "layout_q", "layout_kv", "has_ori_kv", "has_cmp_kv",
        "dtype", "kv_format", "ori_block_size", "cmp_block_size", "return_lse", "kernel_hint", "sparse_block_size",
        "split_policy")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class SfmTensors(C.Structure):
    _fields_ = [
        ("q", C.c_void_p), ("ori_kv", C.c_void_p), ("ori_row_stride", C.c_int64), ("ori_rows", C.c_int64),
        ("cmp_kv", C.c_void_p), ("cmp_row_stride", C.c_int64), ("cmp_rows", C.c_int64),
        ("ori_sparse_indices", C.c_void_p), ("cmp_sparse_indices", C.c_void_p),
        ("ori_block_table", C.c_void_p), ("ori_block_table_stride", C.c_int32),
        ("cmp_block_table", C.c_void_p), ("cmp_block_table_stride", C.c_int32),
        ("cu_seqlens_q", C.c_void_p), ("cu_seqlens_ori_kv", C.c_void_p), ("cu_seqlens_cmp_kv", C.c_void_p),
        ("seqused_q", C.c_void_p), ("seqused_ori_kv", C.c_void_p), ("seqused_cmp_kv", C.c_void_p),
        ("cmp_residual_kv", C.c_void_p), ("sinks", C.c_void_p),
    ]


class _Params(C.Structure):
    """A struct whose fields are all given by name."""

    def __init__(self, **kw):
        super().__init__()
        names = {n for n, _ in self._fields_}
        if set(kw) - names:
            raise TypeError(f"unknown fields {sorted(set(kw) - names)}")
        for k, v in kw.items():
            setattr(self, k, v)


def _i32(*names):
    return [(n, C.c_int32) for n in names]


class SfmRopeSpec(_Params):
    _fields_ = _i32("rope_dim", "scaling") + [(n, C.c_double) for n in ("base", "factor", "beta_fast", "beta_slow")] + \
        _i32("original_max_position", "reserved")


class SfmRopeParams(_Params):
    _fields_ = _i32("tokens", "heads", "head_dim", "rope_dim", "rope_offset", "rope_layout", "inverse", "dtype") + \
        [("amplitude", C.c_float)] + _i32("reserved") + \
        [(n, C.c_int64) for n in ("x_token_stride", "x_head_stride", "y_token_stride", "y_head_stride")]


class SfmStoreParams(_Params):
    _fields_ = _i32("tokens", "heads", "head_dim", "dtype", "kv_format", "norm") + [("norm_eps", C.c_float)] + \
        _i32("rope_dim", "rope_offset", "rope_layout") + [("amplitude", C.c_float)] + _i32("reserved") + \
        [(n, C.c_int64) for n in ("x_token_stride", "x_head_stride", "row_stride", "rows")]


class SfmIndexParams(_Params):
    _fields_ = _i32("num_heads", "index_dim", "batch_size", "max_seqlen_q", "total_q", "max_seqlen_kv", "cmp_ratio",
                    "mask_mode", "layout_q", "layout_kv", "dtype", "block_size")


class SfmIndexTensors(_Params):
    _fields_ = [("q", C.c_void_p), ("k", C.c_void_p), ("k_row_stride", C.c_int64), ("k_rows", C.c_int64),
                ("k_scales", C.c_void_p), ("weights", C.c_void_p), ("block_table", C.c_void_p),
                ("block_table_stride", C.c_int32), ("cu_seqlens_q", C.c_void_p), ("cu_seqlens_kv", C.c_void_p),
                ("seqused_q", C.c_void_p), ("seqused_kv", C.c_void_p), ("cmp_residual_kv", C.c_void_p)]


class SfmTopkParams(_Params):
    _fields_ = _i32("rows", "n", "k", "block_size", "first_blocks", "last_blocks") + [("score_stride", C.c_int64)]


class SfmDenseParams(_Params):
    _fields_ = _i32("num_heads", "head_dim", "batch_size", "max_seqlen_q", "total_q", "max_seqlen_kv", "mask_mode",
                    "win_left", "win_right", "layout_q", "layout_kv", "dtype", "block_size", "tree_words", "split_keys",
                    "zero_rest") + [("softmax_scale", C.c_float), ("softcap", C.c_float)]


class SfmDenseTensors(_Params):
    _fields_ = [("q", C.c_void_p), ("kv", C.c_void_p), ("kv_row_stride", C.c_int64), ("kv_rows", C.c_int64),
                ("block_table", C.c_void_p), ("block_table_stride", C.c_int32)] + \
        [(n, C.c_void_p) for n in ("cu_seqlens_q", "cu_seqlens_kv", "seqused_q", "seqused_kv", "sinks", "bias_slopes",
                                   "prefix_lens", "key_begin", "key_end", "tree_mask", "positions")]


class SfmMergeParams(_Params):
    _fields_ = _i32("tokens", "heads", "head_dim", "parts", "dtype", "reserved")


class SfmMoveParams(_Params):
    _fields_ = _i32("batch_size", "max_path", "row_bytes", "block_size", "max_seqlen_kv", "block_table_stride") + \
        [("row_stride", C.c_int64), ("rows", C.c_int64)]


EXPORTS = ("sfm_metadata_size", "sfm_workspace_size", "sfm_metadata", "sfm_forward", "sfm_forward_noalloc",
           "sfm_debug_attended", "sfm_set_profile_events", "sfm_error_string", "sfm_abi_version",
           "sfm_rope_frequencies", "sfm_rope", "sfm_kv_store", "sfm_index_scores", "sfm_topk_select",
           "sfm_dense_workspace_size", "sfm_dense_forward", "sfm_merge", "sfm_kv_move")
MERGE_MAX_PARTS = 8
NOALLOC_WORKSPACE_BYTES = 32 << 20

_lib = None


def build(force: bool = False) -> str:
    from . import buildlib
    return buildlib.build(force=force)


def lib():
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"sfm CUDA library not built ({LIB_PATH}); run sparse_shared_kv_gb300.build()")
        l = C.CDLL(LIB_PATH)
        P, T = C.POINTER(SfmParams), C.POINTER(SfmTensors)
        l.sfm_metadata_size.argtypes = [P, C.POINTER(C.c_size_t)]
        l.sfm_workspace_size.argtypes = [P, C.POINTER(C.c_size_t)]
        l.sfm_metadata.argtypes = [P, T, C.c_void_p, C.c_size_t, C.c_void_p]
        l.sfm_forward.argtypes = [P, T, C.c_void_p, C.c_size_t, C.c_float, C.c_void_p, C.c_void_p, C.c_void_p,
                                  C.c_size_t, C.c_void_p, C.c_void_p]
        l.sfm_forward_noalloc.argtypes = [P, T, C.c_void_p, C.c_size_t, C.c_float, C.c_void_p, C.c_void_p,
                                          C.c_void_p, C.c_void_p]
        l.sfm_debug_attended.argtypes = [P, T, C.c_void_p, C.c_size_t, C.c_float, C.c_void_p, C.c_void_p,
                                         C.c_void_p, C.c_size_t, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p,
                                         C.c_void_p]
        l.sfm_set_profile_events.argtypes = [C.c_void_p, C.c_void_p]
        l.sfm_error_string.argtypes = [C.c_int]
        l.sfm_error_string.restype = C.c_char_p
        V = C.c_void_p
        l.sfm_rope_frequencies.argtypes = [C.POINTER(SfmRopeSpec), C.POINTER(C.c_double), C.POINTER(C.c_float)]
        # the structs of these come as ctypes structs or packed bytes
        l.sfm_rope.argtypes = [V] * 6
        l.sfm_kv_store.argtypes = [V] * 10
        l.sfm_index_scores.argtypes = [V, V, V, C.c_int64, V, V, V]
        l.sfm_topk_select.argtypes = [V] * 6
        l.sfm_dense_workspace_size.argtypes = [V, C.POINTER(C.c_size_t)]
        l.sfm_dense_forward.argtypes = [V, V, V, V, V, C.c_size_t, V, V]
        l.sfm_merge.argtypes = [V] * 7
        l.sfm_kv_move.argtypes = [V] * 7
        for n in ("sfm_metadata_size", "sfm_workspace_size", "sfm_metadata", "sfm_forward", "sfm_forward_noalloc",
                  "sfm_debug_attended", "sfm_set_profile_events", "sfm_abi_version", "sfm_rope_frequencies",
                  "sfm_rope", "sfm_kv_store", "sfm_index_scores", "sfm_topk_select", "sfm_dense_workspace_size",
                  "sfm_dense_forward", "sfm_merge", "sfm_kv_move"):
            getattr(l, n).restype = C.c_int
        _lib = l
    return _lib


class SfmError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed: {sfm_error_string(code)} ({code})")
        self.code = code


def _check(fn, code):
    if code != 0:
        raise SfmError(fn, code)


def _ptr(x: Optional[torch.Tensor]):
    if x is None:
        return None
    return x.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ---------------------------------------------------------------------------
# the C entry points
# ---------------------------------------------------------------------------
def sfm_set_profile_events(begin=None, end=None) -> None:
    """Record ``begin`` / ``end`` (torch.cuda.Event) around the main attention
    kernel of the following sfm_forward calls; ``None, None`` turns it off."""
    for ev in (begin, end):
        if ev is not None and ev.cuda_event == 0:
            ev.record()          # torch creates the underlying cudaEvent_t lazily
    b = begin.cuda_event if begin is not None else None
    e = end.cuda_event if end is not None else None
    _check("sfm_set_profile_events", lib().sfm_set_profile_events(b, e))


def sfm_error_string(code: int) -> str:
    return lib().sfm_error_string(code).decode()


def sfm_abi_version() -> int:
    return lib().sfm_abi_version()


def sfm_metadata_size(params: SfmParams) -> int:
    n = C.c_size_t(0)
    _check("sfm_metadata_size", lib().sfm_metadata_size(C.byref(params), C.byref(n)))
    return n.value


def sfm_workspace_size(params: SfmParams) -> int:
    n = C.c_size_t(0)
    _check("sfm_workspace_size", lib().sfm_workspace_size(C.byref(params), C.byref(n)))
    return n.value


def sfm_metadata(params: SfmParams, tensors: SfmTensors, metadata: torch.Tensor, stream=None) -> None:
    assert metadata.dtype == torch.int32 and metadata.is_cuda and metadata.is_contiguous()
    _check("sfm_metadata", lib().sfm_metadata(C.byref(params), C.byref(tensors), metadata.data_ptr(),
                                              metadata.numel(), _stream(stream)))


def sfm_forward(params: SfmParams, tensors: SfmTensors, metadata: torch.Tensor, softmax_scale: float,
                out: torch.Tensor, lse: Optional[torch.Tensor], workspace: Optional[torch.Tensor],
                status: Optional[torch.Tensor] = None, stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("sfm_forward", lib().sfm_forward(
        C.byref(params), C.byref(tensors), metadata.data_ptr(), metadata.numel(), C.c_float(softmax_scale),
        out.data_ptr(), _ptr(lse), _ptr(workspace), ws_bytes, _ptr(status), _stream(stream)))


def sfm_forward_noalloc(params: SfmParams, tensors: SfmTensors, metadata: torch.Tensor, softmax_scale: float,
                        out: torch.Tensor, lse: Optional[torch.Tensor], status: Optional[torch.Tensor] = None,
                        stream=None) -> None:
    """sfm_forward with the library's fixed device workspace (no allocation)."""
    _check("sfm_forward_noalloc", lib().sfm_forward_noalloc(
        C.byref(params), C.byref(tensors), metadata.data_ptr(), metadata.numel(), C.c_float(softmax_scale),
        out.data_ptr(), _ptr(lse), _ptr(status), _stream(stream)))


def sfm_debug_attended(params: SfmParams, tensors: SfmTensors, metadata: torch.Tensor, softmax_scale: float,
                       out: torch.Tensor, lse: Optional[torch.Tensor], workspace: Optional[torch.Tensor],
                       rows: torch.Tensor, cap: int, counts: torch.Tensor, status: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    """sfm_forward that also records the KV rows the attention kernel's
    resolver hands to its copy warps (rows[t * cap + k], see include/sfm.h)."""
    assert rows.dtype == torch.int32 and counts.dtype == torch.int32
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("sfm_debug_attended", lib().sfm_debug_attended(
        C.byref(params), C.byref(tensors), metadata.data_ptr(), metadata.numel(), C.c_float(softmax_scale),
        out.data_ptr(), _ptr(lse), _ptr(workspace), ws_bytes, rows.data_ptr(), cap, counts.data_ptr(),
        _ptr(status), _stream(stream)))


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
def _rows_of(kv: Optional[torch.Tensor], row_stride: int) -> int:
    if kv is None:
        return 0
    return kv.numel() * kv.element_size() // row_stride


def make_tensors(q, ori_kv, *, cmp_kv=None, ori_sparse_indices=None, cmp_sparse_indices=None,
                 ori_block_table=None, cmp_block_table=None, cu_seqlens_q=None, cu_seqlens_ori_kv=None,
                 cu_seqlens_cmp_kv=None, seqused_q=None, seqused_ori_kv=None, seqused_cmp_kv=None,
                 cmp_residual_kv=None, sinks=None, ori_row_stride=None, cmp_row_stride=None) -> SfmTensors:
    """SfmTensors from device tensors.  KV row strides default to the
    tensor's last-dim size in bytes (the stride of dim -3 for padded rows)."""
    t = SfmTensors()

    def stride_of(kv, given):
        if given is not None:
            return int(given)
        return kv.stride(-3) * kv.element_size() if kv.dim() >= 3 else kv.stride(0) * kv.element_size()

    for name in ("ori_sparse_indices", "cmp_sparse_indices", "ori_block_table", "cmp_block_table",
                 "cu_seqlens_q", "cu_seqlens_ori_kv", "cu_seqlens_cmp_kv", "seqused_q", "seqused_ori_kv",
                 "seqused_cmp_kv", "cmp_residual_kv"):
        x = locals()[name]
        if x is not None:
            assert x.dtype == torch.int32 and x.is_contiguous(), name
    t.q = _ptr(q)
    t.ori_kv = _ptr(ori_kv)
    t.ori_row_stride = stride_of(ori_kv, ori_row_stride)
    t.ori_rows = _rows_of(ori_kv, t.ori_row_stride)
    if cmp_kv is not None:
        t.cmp_kv = _ptr(cmp_kv)
        t.cmp_row_stride = stride_of(cmp_kv, cmp_row_stride)
        t.cmp_rows = _rows_of(cmp_kv, t.cmp_row_stride)
    t.ori_sparse_indices = _ptr(ori_sparse_indices)
    t.cmp_sparse_indices = _ptr(cmp_sparse_indices)
    t.ori_block_table = _ptr(ori_block_table)
    t.ori_block_table_stride = ori_block_table.shape[-1] if ori_block_table is not None else 0
    t.cmp_block_table = _ptr(cmp_block_table)
    t.cmp_block_table_stride = cmp_block_table.shape[-1] if cmp_block_table is not None else 0
    t.cu_seqlens_q = _ptr(cu_seqlens_q)
    t.cu_seqlens_ori_kv = _ptr(cu_seqlens_ori_kv)
    t.cu_seqlens_cmp_kv = _ptr(cu_seqlens_cmp_kv)
    t.seqused_q = _ptr(seqused_q)
    t.seqused_ori_kv = _ptr(seqused_ori_kv)
    t.seqused_cmp_kv = _ptr(seqused_cmp_kv)
    t.cmp_residual_kv = _ptr(cmp_residual_kv)
    t.sinks = _ptr(sinks)
    return t


def make_params(**kw) -> SfmParams:
    p = SfmParams()
    defaults = dict(num_heads_kv=1, head_dim=512, rope_head_dim=0, total_q=0, max_seqlen_cmp_kv=0, ori_topk=0,
                    cmp_topk=0, cmp_ratio=1, ori_mask_mode=4, cmp_mask_mode=3, ori_win_left=-1, ori_win_right=-1,
                    layout_q=BSND, layout_kv=BSND, has_ori_kv=1, has_cmp_kv=0, dtype=BF16, kv_format=KV_PLAIN,
                    ori_block_size=0, cmp_block_size=0, return_lse=0, kernel_hint=0, sparse_block_size=1,
                    split_policy=SPLIT_BATCH_INVARIANT)
    defaults.update(kw)
    for k, v in defaults.items():
        if k in ("layout_q", "layout_kv") and isinstance(v, str):
            v = _LAYOUTS[v]
        if k == "dtype" and isinstance(v, (str, torch.dtype)):
            v = BF16 if v in ("bf16", torch.bfloat16) else FP16
        setattr(p, k, int(v))
    return p


# ---------------------------------------------------------------------------
# the two-call torch API
# ---------------------------------------------------------------------------
@dataclass
class Metadata:
    """Device int32 plan plus the params it was built for."""
    tensor: torch.Tensor
    params: SfmParams


def sparse_flash_mla_metadata(num_heads_q: int, num_heads_kv: int, head_dim: int, *, cu_seqlens_q=None,
                              cu_seqlens_ori_kv=None, cu_seqlens_cmp_kv=None, seqused_q=None,
                              seqused_ori_kv=None, seqused_cmp_kv=None, cmp_residual_kv=None, batch_size=0,
                              max_seqlen_q=0, max_seqlen_ori_kv=0, max_seqlen_cmp_kv=0, total_q=0, ori_topk=0,
                              cmp_topk=0, cmp_ratio=1, ori_mask_mode=4, cmp_mask_mode=3, ori_win_left=-1,
                              ori_win_right=-1, layout_q="BSND", layout_kv="BSND", has_ori_kv=True,
                              has_cmp_kv=True, dtype=torch.bfloat16, kv_format=KV_PLAIN, rope_head_dim=0,
                              ori_block_size=0, cmp_block_size=0, return_softmax_lse=False,
                              sparse_block_size=1, batch_invariant=True, device=None,
                              stream=None) -> Metadata:
    """Enqueue the device planner and return its plan (two-call contract).

    ``batch_invariant=False`` selects the occupancy split policy: small
    batches are cut into more chunks so they fill the SMs, at the price of a
    row's rounding depending on the batch size."""
    if layout_q == "TND" and cu_seqlens_q is not None:
        batch_size = cu_seqlens_q.numel() - 1
    params = make_params(
        num_heads_q=num_heads_q, num_heads_kv=num_heads_kv, head_dim=head_dim, rope_head_dim=rope_head_dim,
        batch_size=batch_size, max_seqlen_q=max_seqlen_q, total_q=total_q, max_seqlen_ori_kv=max_seqlen_ori_kv,
        max_seqlen_cmp_kv=max_seqlen_cmp_kv, ori_topk=ori_topk, cmp_topk=cmp_topk, cmp_ratio=cmp_ratio,
        ori_mask_mode=ori_mask_mode, cmp_mask_mode=cmp_mask_mode, ori_win_left=ori_win_left,
        ori_win_right=ori_win_right, layout_q=layout_q, layout_kv=layout_kv, has_ori_kv=int(has_ori_kv),
        has_cmp_kv=int(has_cmp_kv), dtype=dtype, kv_format=kv_format, ori_block_size=ori_block_size,
        cmp_block_size=cmp_block_size, return_lse=int(return_softmax_lse), sparse_block_size=sparse_block_size,
        split_policy=SPLIT_BATCH_INVARIANT if batch_invariant else SPLIT_OCCUPANCY)
    lengths = make_tensors(None, None, cu_seqlens_q=cu_seqlens_q, cu_seqlens_ori_kv=cu_seqlens_ori_kv,
                           cu_seqlens_cmp_kv=cu_seqlens_cmp_kv, seqused_q=seqused_q, seqused_ori_kv=seqused_ori_kv,
                           seqused_cmp_kv=seqused_cmp_kv, cmp_residual_kv=cmp_residual_kv, ori_row_stride=0)
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    md = torch.empty(sfm_metadata_size(params), dtype=torch.int32, device=device)
    sfm_metadata(params, lengths, md, stream)
    return Metadata(md, params)


def sparse_flash_mla(q: torch.Tensor, *, metadata: Metadata, ori_kv=None, cmp_kv=None, ori_sparse_indices=None,
                     cmp_sparse_indices=None, ori_block_table=None, cmp_block_table=None, cu_seqlens_q=None,
                     cu_seqlens_ori_kv=None, cu_seqlens_cmp_kv=None, seqused_q=None, seqused_ori_kv=None,
                     seqused_cmp_kv=None, cmp_residual_kv=None, sinks=None, softmax_scale: float = 1.0,
                     ori_row_stride=None, cmp_row_stride=None, out=None, lse=None, workspace=None,
                     status=None, stream=None):
    """Attention output (q's layout, 512 dims per head) and LSE (fp32, or None
    when the plan was made without return_softmax_lse)."""
    params = metadata.params
    tensors = make_tensors(q, ori_kv, cmp_kv=cmp_kv, ori_sparse_indices=ori_sparse_indices,
                           cmp_sparse_indices=cmp_sparse_indices, ori_block_table=ori_block_table,
                           cmp_block_table=cmp_block_table, cu_seqlens_q=cu_seqlens_q,
                           cu_seqlens_ori_kv=cu_seqlens_ori_kv, cu_seqlens_cmp_kv=cu_seqlens_cmp_kv,
                           seqused_q=seqused_q, seqused_ori_kv=seqused_ori_kv, seqused_cmp_kv=seqused_cmp_kv,
                           cmp_residual_kv=cmp_residual_kv, sinks=sinks, ori_row_stride=ori_row_stride,
                           cmp_row_stride=cmp_row_stride)
    if out is None:
        out = torch.empty(q.shape[:-1] + (512,), dtype=q.dtype, device=q.device)
    if lse is None and params.return_lse:
        lse = torch.empty(q.shape[:-1].numel(), dtype=torch.float32, device=q.device)
    if workspace is None:
        nb = sfm_workspace_size(params)
        workspace = torch.empty(max(nb, 1), dtype=torch.uint8, device=q.device) if nb else None
    sfm_forward(params, tensors, metadata.tensor, softmax_scale, out, lse if params.return_lse else None,
                workspace, status, stream)
    return out, lse


# ---------------------------------------------------------------------------
# around the attention: rotary positions, cache rows, sparse indices
# ---------------------------------------------------------------------------
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_increment_version = torch.autograd.graph.increment_version
_forward_ad = torch.autograd.forward_ad
_I32, _F32, _F64 = torch.int32, torch.float32, torch.float64

# The structs of include/sfm.h as native-layout packers (the calls below build them every time; packing
# all fields at once costs a fraction of setting them one by one)
_ROPE_PARAMS = struct.Struct("@8ifi4q")
_STORE_PARAMS = struct.Struct("@6if3ifi4q")
_INDEX_PARAMS = struct.Struct("@12i")
_INDEX_TENSORS = struct.Struct("@PPqqPPPiPPPPP")
_TOPK_PARAMS = struct.Struct("@6iq")
_DENSE_PARAMS = struct.Struct("@16i2f")
_DENSE_TENSORS = struct.Struct("@PPqqPi11P")
_MERGE_PARAMS = struct.Struct("@6i")
_MOVE_PARAMS = struct.Struct("@6i2q")
_POINTERS = [struct.Struct(f"@{n}P") for n in range(MERGE_MAX_PARTS + 1)]
_SCORE_TYPES = {torch.float32: 0}
_SIXTEEN_BIT = {torch.bfloat16: BF16, torch.float16: FP16}
_INDEX_TYPES = {torch.bfloat16: BF16, torch.float16: FP16, torch.float8_e4m3fn: E4M3}


def _require(ok, what):
    if not ok:
        raise ValueError(what)


def _first(name, x, types):
    """Check a call's first tensor: its dtype's code and its device's index."""
    if not isinstance(x, torch.Tensor):
        raise ValueError(f"{name}: not a tensor")
    code = types.get(x.dtype)
    if code is None:
        raise ValueError(f"{name}: dtype {x.dtype}")
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"{name}: not on a CUDA device")
    return code, dev


def _refuse(name, x, dtype, dev, shape=None):
    """Say what is wrong with a tensor argument."""
    _require(isinstance(x, torch.Tensor), f"{name}: not a tensor")
    _require(x.dtype is dtype, f"{name}: dtype {x.dtype}, expected {dtype}")
    _require(x.get_device() >= 0, f"{name}: not on a CUDA device")
    _require(x.get_device() == dev, f"{name}: on {x.device}, expected cuda:{dev}")
    _require(shape is None or x.shape == shape, f"{name}: shape {tuple(x.shape)}, expected {shape and tuple(shape)}")
    raise ValueError(f"{name}: not contiguous")


def _address(name, x, dtype, dev, shape):
    """Device address of a contiguous tensor argument."""
    if (isinstance(x, torch.Tensor) and x.dtype is dtype and x.get_device() == dev and x.shape == shape
            and x.is_contiguous()):
        return x.data_ptr()
    _refuse(name, x, dtype, dev, shape)


def _tensor(name, x):
    if not isinstance(x, torch.Tensor):
        raise ValueError(f"{name}: not a tensor")
    return x


def _status_address(status, dev):
    if not (isinstance(status, torch.Tensor) and status.dtype is _I32 and status.get_device() == dev and status.numel() >= 1):
        raise ValueError(f"status: needs an int32 tensor on cuda:{dev}")
    return status.data_ptr()


def _on(dev, stream):
    """A context that makes the device and the stream (torch's, or a raw cudaStream_t) current, so that results
    are allocated on the stream that writes them."""
    ctx = contextlib.ExitStack()
    ctx.enter_context(torch.cuda.device(dev))
    if stream is not None:
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=dev)
        ctx.enter_context(torch.cuda.stream(stream))
    return ctx


def rope_frequencies(rope_dim: int, *, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_max_position: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """Angles per position (float64, rope_dim / 2) and the amplitude of rotary
    positions; ``scaling`` ("none", "linear", "ntk", "yarn") stretches them by
    ``factor`` for long contexts (see sfm_rope_frequencies in include/sfm.h)."""
    _require(scaling in ROPE_SCALINGS, f"scaling: {scaling!r}")
    spec = SfmRopeSpec(rope_dim=rope_dim, scaling=ROPE_SCALINGS[scaling], base=base, factor=factor, beta_fast=beta_fast,
                       beta_slow=beta_slow, original_max_position=original_max_position)
    freq = (C.c_double * max(rope_dim // 2, 1))()
    amplitude = C.c_float(1.0)
    _check("sfm_rope_frequencies", lib().sfm_rope_frequencies(C.byref(spec), freq, C.byref(amplitude)))
    return torch.tensor(list(freq), dtype=torch.float64, device=device), amplitude.value


def _heads(x, name):
    """(tokens, heads, dim, token stride, head stride) of a (..., heads, dim) tensor with contiguous values."""
    shape, strides = x.shape, x.stride()
    if len(shape) != 3:
        _require(len(shape) >= 2, f"{name}: needs (..., heads, values)")
        try:
            x = x.view(-1, shape[-2], shape[-1]) if x.numel() else x.reshape(shape[:-2].numel(), shape[-2], shape[-1])
        except RuntimeError:
            raise ValueError(f"{name}: the token dimensions do not flatten to one stride") from None
        shape, strides = x.shape, x.stride()
    tokens, heads, dim = shape
    if strides[2] != 1 and dim != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    # a dimension of one entry may report any stride: it gets that of dense rows
    head = strides[1] if heads > 1 else dim
    return tokens, heads, dim, strides[0] if tokens > 1 else max(head * heads, dim), head


def _rows(x, name):
    """(rows, bytes between them) of a (..., row) tensor with contiguous rows."""
    shape, strides = x.shape, x.stride()
    if len(shape) < 2 or (strides[-1] != 1 and shape[-1] != 1):
        raise ValueError(f"{name}: needs (..., row) with contiguous rows")
    rows, stride = shape[0], strides[0]
    if len(shape) != 2:
        rows, span = shape[:-1].numel(), None
        for i in range(len(shape) - 2, -1, -1):
            if shape[i] == 1 or not rows:
                continue        # a dimension of one entry may report any stride
            if span is None:
                stride = span = strides[i]
            elif strides[i] != span:
                raise ValueError(f"{name}: the row dimensions do not flatten to one stride")
            span *= shape[i]
    return rows, (stride if rows > 1 else shape[-1]) * x.element_size()


def apply_rope(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, *, amplitude: float = 1.0,
               rope_offset: int = 0, interleaved: bool = True, inverse: bool = False, out=None, stream=None):
    """Rotary positions of x (..., heads, head_dim), bf16 or fp16.

    The values [rope_offset, rope_offset + 2 len(inv_freq)) of every head are
    rotated by position * inv_freq as pairs (2i, 2i + 1), or (i, i + n / 2)
    with ``interleaved=False``, and multiplied by ``amplitude``.
    positions: int32, one per token.  ``inverse=True`` applies the transposed
    map: the gradient with respect to x, and the way back for amplitude 1.
    ``out``: None for a new tensor, x itself to rotate in place, or a tensor
    of x's shape that does not overlap it.  Views with strides are taken as they are.
    The call records no gradient of its own: where one would be lost (x or out
    requires it and grad mode is on) it raises, so a training step calls it inside
    its own torch.autograd.Function, with ``inverse=True`` in the backward pass."""
    code, dev = _first("x", x, _SIXTEEN_BIT)
    if x.requires_grad and torch.is_grad_enabled():
        raise ValueError("x: requires a gradient, which this call does not record (use no_grad, or an autograd.Function "
                         "with inverse=True as its backward pass)")
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return apply_rope(x, positions, inv_freq, amplitude=amplitude, rope_offset=rope_offset, interleaved=interleaved,
                              inverse=inverse, out=out)
    tokens, heads, dim, xt, xh = _heads(x, "x")
    pos = _address("positions", positions, _I32, dev, (tokens,) if _tensor("positions", positions).dim() == 1 else x.shape[:-2])
    n = _tensor("inv_freq", inv_freq).numel()
    freq = _address("inv_freq", inv_freq, _F64, dev, (n,))
    given = out is not None
    if not given:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        yt, yh = heads * dim, dim
    elif out is x:
        yt, yh = xt, xh
    else:
        if not (isinstance(out, torch.Tensor) and out.dtype is x.dtype and out.get_device() == dev and out.shape == x.shape):
            raise ValueError(f"out: needs {tuple(x.shape)} of {x.dtype} on cuda:{dev}")
        if out.requires_grad and torch.is_grad_enabled():
            raise ValueError("out: requires a gradient, which this call does not record")
        _, _, _, yt, yh = _heads(out, "out")
    params = _ROPE_PARAMS.pack(tokens if heads else 0, heads or 1, dim, 2 * n, rope_offset,
                               ROPE_INTERLEAVED if interleaved else ROPE_HALF, bool(inverse), code, amplitude, 0, xt, xh, yt, yh)
    rc = (_lib or lib()).sfm_rope(params, x.data_ptr(), pos, freq, out.data_ptr(), _raw_stream(dev))
    if rc:
        raise SfmError("sfm_rope", rc)
    if given and not out.is_inference():
        _increment_version(out)      # a graph that saved it for its backward pass must notice
    return out


def store_kv(x: torch.Tensor, cache: torch.Tensor, *, slot_mapping=None, kv_format: int = KV_PLAIN, norm_weight=None,
             norm_eps: Optional[float] = None, positions=None, inv_freq=None, amplitude: float = 1.0,
             rope_offset: Optional[int] = None, interleaved: bool = True, scales=None, status=None, stream=None):
    """Write the rows x (tokens, dim) or (tokens, heads, dim), bf16 or fp16,
    into ``cache`` as sfm_kv_store does: RMS norm (with ``norm_eps``; weight
    fp32 or ones), rotary positions (with ``positions`` and ``inv_freq``; the
    last 2 len(inv_freq) values unless ``rope_offset`` says otherwise), then
    the rounding of ``kv_format``.  Returns ``cache``.

    cache: (..., row) with dense rows: values of x's dtype (KV_PLAIN), bytes
    of packed rows, uint8 (KV_INT8_PACKED, KV_FP8_PACKED), or float8_e4m3fn values
    with fp32 ``scales``, one per row (KV_FP8_ROWS).  Rows may be padded apart.
    slot_mapping: int32, one per token: head h goes to row slot * heads + h;
    negative: not written; None: row t * heads + h."""
    code, dev = _first("x", x, _SIXTEEN_BIT)
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return store_kv(x, cache, slot_mapping=slot_mapping, kv_format=kv_format, norm_weight=norm_weight, norm_eps=norm_eps,
                            positions=positions, inv_freq=inv_freq, amplitude=amplitude, rope_offset=rope_offset,
                            interleaved=interleaved, scales=scales, status=status)
    if x.dim() == 2:
        tokens, dim = x.shape
        strides = x.stride()
        if strides[1] != 1 and dim != 1:
            raise ValueError("x: the last dimension must be contiguous")
        heads, xh, xt = 1, dim, strides[0] if tokens > 1 else dim
    elif x.dim() == 3:
        tokens, heads, dim, xt, xh = _heads(x, "x")
    else:
        raise ValueError("x: needs (tokens, dim) or (tokens, heads, dim)")
    if kv_format == KV_INT8_PACKED or kv_format == KV_FP8_PACKED:
        kind, width = torch.uint8, 512 + 2 * (dim - 512) + 16
    else:
        kind, width = torch.float8_e4m3fn if kv_format == KV_FP8_ROWS else x.dtype, dim
    if not (isinstance(cache, torch.Tensor) and cache.dtype is kind and cache.get_device() == dev):
        raise ValueError(f"cache: needs {kind} on cuda:{dev}")
    rows, row_stride = _rows(cache, "cache")
    if cache.shape[-1] != width:
        raise ValueError(f"cache: rows of {cache.shape[-1]}, expected {width}")
    if (scales is not None) != (kv_format == KV_FP8_ROWS):
        raise ValueError("scales: go with KV_FP8_ROWS rows")
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq go together")
    if norm_eps is None and norm_weight is not None:
        raise ValueError("norm_weight: needs norm_eps")
    rot = 0 if inv_freq is None else 2 * _tensor("inv_freq", inv_freq).numel()
    offset = 0 if not rot else dim - rot if rope_offset is None else rope_offset
    params = _STORE_PARAMS.pack(tokens if heads else 0, heads or 1, dim, code, kv_format, norm_eps is not None,
                                norm_eps or 0.0, rot, offset, ROPE_INTERLEAVED if interleaved else ROPE_HALF, amplitude, 0,
                                xt, xh, row_stride, rows)
    each = (tokens,)
    rc = (_lib or lib()).sfm_kv_store(
        params, x.data_ptr(), 0 if norm_weight is None else _address("norm_weight", norm_weight, _F32, dev, (min(dim, 512),)),
        0 if positions is None else _address("positions", positions, _I32, dev, each),
        0 if inv_freq is None else _address("inv_freq", inv_freq, _F64, dev, (rot // 2,)),
        0 if slot_mapping is None else _address("slot_mapping", slot_mapping, _I32, dev, each), cache.data_ptr(),
        0 if scales is None else _address("scales", scales, _F32, dev, (rows,) if _tensor("scales", scales).dim() == 1 else cache.shape[:-1]),
        0 if status is None else _status_address(status, dev), _raw_stream(dev))
    if rc:
        raise SfmError("sfm_kv_store", rc)
    return cache


def index_scores(q: torch.Tensor, index_k: torch.Tensor, weights: torch.Tensor, *, max_seqlen_kv: int, k_scales=None,
                 block_table=None, cu_seqlens_q=None, cu_seqlens_kv=None, seqused_q=None, seqused_kv=None,
                 cmp_residual_kv=None, max_seqlen_q: int = 0, cmp_ratio: int = 1, mask_mode: int = 3,
                 layout_q="BSND", layout_kv="BSND", out=None, visible=None, status=None, stream=None):
    """Scores of every query against the index keys of its sequence, and the
    number of keys each query may see (see sfm_index_scores).

    q: (b, q_s, heads, 128) or TND (tokens, heads, 128) in bf16, fp16 or
    float8_e4m3fn; index_k: (b, S, 128), (t, 128) or paged (blocks,
    block_size, 128) of the same dtype, rows may be padded apart; weights:
    fp32 (tokens, heads) in q's leading shape, and the scales of quantised
    queries (those of ``store_kv`` with KV_FP8_ROWS) belong multiplied into them;
    k_scales: fp32, one per row of index_k.  Returns (scores (tokens, max_seqlen_kv) fp32, its rows a
    multiple of four values apart, -inf where a key is not visible; visible
    (tokens) int32).  ``out`` may be a view with wider rows.

    Rows of a TND batch behind its last sequence are not written: a new
    ``visible`` is 0 there, so that ``select_topk(scores, k, lengths=visible)``
    selects nothing, while the new scores hold no particular values; in ``out``
    and ``visible`` of the caller's they stay as they were."""
    code, dev = _first("q", q, _INDEX_TYPES)
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return index_scores(q, index_k, weights, max_seqlen_kv=max_seqlen_kv, k_scales=k_scales, block_table=block_table,
                                cu_seqlens_q=cu_seqlens_q, cu_seqlens_kv=cu_seqlens_kv, seqused_q=seqused_q,
                                seqused_kv=seqused_kv, cmp_residual_kv=cmp_residual_kv, max_seqlen_q=max_seqlen_q,
                                cmp_ratio=cmp_ratio, mask_mode=mask_mode, layout_q=layout_q, layout_kv=layout_kv, out=out,
                                visible=visible, status=status)
    lq, lkv = _LAYOUTS[layout_q], _LAYOUTS[layout_kv]
    shape = q.shape
    if len(shape) != (4 if lq == BSND else 3):
        raise ValueError("q: BSND has 4 dimensions, TND 3")
    heads, dim = shape[-2], shape[-1]
    if lq == BSND:
        batch, max_seqlen_q = shape[0], shape[1]
        tokens = batch * max_seqlen_q
    elif cu_seqlens_q is None:
        raise ValueError("cu_seqlens_q: required for TND")
    else:
        batch, tokens = _tensor("cu_seqlens_q", cu_seqlens_q).numel() - 1, shape[0]
    if not (isinstance(index_k, torch.Tensor) and index_k.dtype is q.dtype and index_k.get_device() == dev):
        raise ValueError(f"index_k: needs {q.dtype} on cuda:{dev}")
    kshape = index_k.shape
    if len(kshape) != (2 if lkv == TND else 3) or kshape[-1] != dim:
        raise ValueError("index_k: needs (t, dim), (b, S, dim) or (blocks, block_size, dim) with q's dim")
    if lkv == BSND and (kshape[1] != max_seqlen_kv or kshape[0] != batch):
        raise ValueError("index_k: needs (b, max_seqlen_kv, dim)")
    rows, row_stride = _rows(index_k, "index_k")
    cols = table = 0
    each = (batch,)
    if block_table is not None:
        if _tensor("block_table", block_table).dim() != 2:
            raise ValueError("block_table: needs (b, blocks)")
        cols = block_table.shape[1]
        table = _address("block_table", block_table, _I32, dev, (batch, cols))
    params = _INDEX_PARAMS.pack(heads, dim, batch, max_seqlen_q, tokens, max_seqlen_kv, cmp_ratio, mask_mode, lq, lkv, code,
                                kshape[1] if lkv == PAGED else 0)
    tensors = _INDEX_TENSORS.pack(
        _address("q", q, q.dtype, dev, shape), index_k.data_ptr(), row_stride, rows,
        0 if k_scales is None else _address("k_scales", k_scales, _F32, dev, (rows,) if _tensor("k_scales", k_scales).dim() == 1 else kshape[:-1]),
        _address("weights", weights, _F32, dev, shape[:-1]), table, cols,
        0 if cu_seqlens_q is None else _address("cu_seqlens_q", cu_seqlens_q, _I32, dev, (batch + 1,)),
        0 if cu_seqlens_kv is None else _address("cu_seqlens_kv", cu_seqlens_kv, _I32, dev, (batch + 1,)),
        0 if seqused_q is None else _address("seqused_q", seqused_q, _I32, dev, each),
        0 if seqused_kv is None else _address("seqused_kv", seqused_kv, _I32, dev, each),
        0 if cmp_residual_kv is None else _address("cmp_residual_kv", cmp_residual_kv, _I32, dev, each))
    if out is None:
        stride = (max_seqlen_kv + 3) // 4 * 4     # rows on 16-byte boundaries, which the selection reads fastest
        out = torch.empty_strided((tokens, max(max_seqlen_kv, 0)), (max(stride, 1), 1), dtype=_F32, device=q.device)
    else:
        if not (isinstance(out, torch.Tensor) and out.dtype is _F32 and out.get_device() == dev
                and out.shape == (tokens, max_seqlen_kv) and (out.stride(1) == 1 or max_seqlen_kv == 1)):
            raise ValueError(f"out: needs fp32 ({tokens}, {max_seqlen_kv}) with contiguous rows on cuda:{dev}")
        stride = out.stride(0) if tokens > 1 else max_seqlen_kv
    if visible is None:
        # rows behind the last sequence (TND) are not written: they see nothing
        visible = (torch.empty if lq == BSND else torch.zeros)((tokens,), dtype=_I32, device=q.device)
        seen = visible.data_ptr()
    else:
        seen = _address("visible", visible, _I32, dev, (tokens,))
    rc = (_lib or lib()).sfm_index_scores(params, tensors, out.data_ptr(), stride, seen,
                                          0 if status is None else _status_address(status, dev), _raw_stream(dev))
    if rc:
        raise SfmError("sfm_index_scores", rc)
    return out, visible


def select_topk(scores: torch.Tensor, k: int, *, lengths=None, block_size: int = 1, first_blocks: int = 0,
                last_blocks: int = 0, out=None, status=None, stream=None):
    """Indices (rows, k) int32, ascending and padded with -1, of the k largest
    scores of every row of ``scores`` (rows, n) fp32, or with ``block_size``
    of the k blocks with the largest score in them, the row's ``first_blocks``
    and ``last_blocks`` always among them (see sfm_topk_select).  They are what
    sparse_flash_mla takes as cmp_sparse_indices / ori_sparse_indices.
    lengths: int32 (rows), scores a row really has (None: n)."""
    _, dev = _first("scores", scores, _SCORE_TYPES)
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return select_topk(scores, k, lengths=lengths, block_size=block_size, first_blocks=first_blocks,
                               last_blocks=last_blocks, out=out, status=status)
    if scores.dim() != 2:
        raise ValueError("scores: needs (rows, n)")
    rows, n = scores.shape
    strides = scores.stride()
    if strides[1] != 1 and n != 1:
        raise ValueError("scores: rows must be contiguous")
    if out is None:
        out = torch.empty((rows, max(k, 0)), dtype=_I32, device=scores.device)
        got = out.data_ptr()
    else:
        got = _address("out", out, _I32, dev, (rows, k))
    params = _TOPK_PARAMS.pack(rows, n, k, block_size, first_blocks, last_blocks, strides[0] if rows > 1 else n)
    rc = (_lib or lib()).sfm_topk_select(params, scores.data_ptr(),
                                         0 if lengths is None else _address("lengths", lengths, _I32, dev, (rows,)), got,
                                         0 if status is None else _status_address(status, dev), _raw_stream(dev))
    if rc:
        raise SfmError("sfm_topk_select", rc)
    return out


# ---------------------------------------------------------------------------
# many queries over the same rows: more kinds of scores and masks, drafted trees
# ---------------------------------------------------------------------------
_I64 = torch.int64
_dense_need = {}


def _no_gradient(name, x):
    if x.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name}: requires a gradient, which this call does not record (use no_grad)")


def _no_tangents(**inputs):
    """Inside forward_ad.dual_level: none of the inputs is a dual tensor."""
    for name, x in inputs.items():
        for y in x if isinstance(x, list) else [x]:
            if isinstance(y, torch.Tensor) and _forward_ad.unpack_dual(y).tangent is not None:
                raise ValueError(f"{name}: has a tangent, which this call does not carry on")


def _dense(q, kv, tree_mask, positions, softmax_scale, softcap, bias_slopes, sinks, mask_mode, win_left, win_right,
           prefix_lens, key_begin, key_end, block_table, cu_seqlens_q, cu_seqlens_kv, seqused_q, seqused_kv, max_seqlen_kv,
           layout_q, layout_kv, split_keys, out, lse, workspace, status, stream):
    code, dev = _first("q", q, _SIXTEEN_BIT)
    if _forward_ad._current_level >= 0:
        _no_tangents(q=q, kv=kv, sinks=sinks, bias_slopes=bias_slopes, out=out, lse=lse)
    if q.requires_grad:
        _no_gradient("q", q)
    if sinks is not None and _tensor("sinks", sinks).requires_grad:
        _no_gradient("sinks", sinks)
    if bias_slopes is not None and _tensor("bias_slopes", bias_slopes).requires_grad:
        _no_gradient("bias_slopes", bias_slopes)
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return _dense(q, kv, tree_mask, positions, softmax_scale, softcap, bias_slopes, sinks, mask_mode, win_left,
                          win_right, prefix_lens, key_begin, key_end, block_table, cu_seqlens_q, cu_seqlens_kv, seqused_q,
                          seqused_kv, max_seqlen_kv, layout_q, layout_kv, split_keys, out, lse, workspace, status, None)
    if layout_q not in ("BSND", "TND") or layout_kv not in _LAYOUTS:
        raise ValueError(f"layouts: {layout_q!r}, {layout_kv!r}")
    lq, lkv = _LAYOUTS[layout_q], _LAYOUTS[layout_kv]
    shape = q.shape
    if len(shape) != (4 if lq == BSND else 3):
        raise ValueError("q: BSND has 4 dimensions, TND 3")
    heads, dim, rows_shape = shape[-2], shape[-1], shape[:-1]
    if lq == BSND:
        batch, max_seqlen_q = shape[0], shape[1]
        tokens = batch * max_seqlen_q
    elif cu_seqlens_q is None:
        raise ValueError("cu_seqlens_q: required for TND")
    else:
        batch, max_seqlen_q, tokens = _tensor("cu_seqlens_q", cu_seqlens_q).numel() - 1, 0, shape[0]
        if batch < 0:
            raise ValueError("cu_seqlens_q: needs b + 1 offsets")
    if not (isinstance(kv, torch.Tensor) and kv.dtype is q.dtype and kv.get_device() == dev):
        raise ValueError(f"kv: needs {q.dtype} on cuda:{dev}")
    if kv.requires_grad:
        _no_gradient("kv", kv)
    kshape = kv.shape
    if len(kshape) == (3 if lkv == TND else 4) and kshape[-2] == 1:
        kv = kv.squeeze(-2)          # the one KV head
        kshape = kv.shape
    if len(kshape) != (2 if lkv == TND else 3) or kshape[-1] != dim:
        raise ValueError("kv: needs (t, dim), (b, S, dim) or (blocks, block_size, dim), a KV head of 1 before dim or not")
    if lkv == BSND:
        if kshape[0] != batch:
            raise ValueError("kv: needs (b, S, dim)")
        max_seqlen_kv = kshape[1]
    rows, row_stride = (kv.numel() // dim, 2 * dim) if dim and kv.is_contiguous() else _rows(kv, "kv")
    max_seqlen_kv = max_seqlen_kv or rows        # no sequence has more
    cols = table = words = tree = place = 0
    each, per_token = (batch,), shape[:-2]
    if block_table is not None:
        if _tensor("block_table", block_table).dim() != 2:
            raise ValueError("block_table: needs (b, blocks)")
        cols = block_table.shape[1]
        table = _address("block_table", block_table, _I32, dev, (batch, cols))
    if tree_mask is not None:
        words = tree_mask.shape[-1] if _tensor("tree_mask", tree_mask).dim() else 0
        tree = _address("tree_mask", tree_mask, _I64, dev, per_token + (words,))
        place = _address("positions", positions, _I32, dev, per_token)
        if not words:
            raise ValueError("tree_mask: needs a word per token")
    kind = q.dtype
    params = _DENSE_PARAMS.pack(heads, dim, batch or 1, max_seqlen_q, tokens, max_seqlen_kv, mask_mode, win_left, win_right, lq, lkv,
                                code, kshape[1] if lkv == PAGED else 0, words, split_keys,
                                (out is None) + 2 * (lse is None), softmax_scale, softcap)
    tensors = _DENSE_TENSORS.pack(
        _address("q", q, kind, dev, shape), kv.data_ptr(), row_stride, rows, table, cols,
        0 if cu_seqlens_q is None else _address("cu_seqlens_q", cu_seqlens_q, _I32, dev, (batch + 1,)),
        0 if cu_seqlens_kv is None else _address("cu_seqlens_kv", cu_seqlens_kv, _I32, dev, (batch + 1,)),
        0 if seqused_q is None else _address("seqused_q", seqused_q, _I32, dev, each),
        0 if seqused_kv is None else _address("seqused_kv", seqused_kv, _I32, dev, each),
        0 if sinks is None else _address("sinks", sinks, _F32, dev, (heads,)),
        0 if bias_slopes is None else _address("bias_slopes", bias_slopes, _F32, dev, (heads,)),
        0 if prefix_lens is None else _address("prefix_lens", prefix_lens, _I32, dev, each),
        0 if key_begin is None else _address("key_begin", key_begin, _I32, dev, per_token),
        0 if key_end is None else _address("key_end", key_end, _I32, dev, per_token), tree, place)
    given = ()
    if out is not None:
        given = (out,)
        to = _address("out", out, kind, dev, shape)
        _no_gradient("out", out)
    if lse is not None:
        given += (lse,)
        end = _address("lse", lse, _F32, dev, rows_shape)
        _no_gradient("lse", lse)
    # the workspace's size depends on the parameters and the device alone
    need = _dense_need.get((params, dev))
    if need is None:
        size = C.c_size_t(0)
        rc = lib().sfm_dense_workspace_size(params, size)
        if rc:
            raise SfmError("sfm_dense_workspace_size", rc)
        if len(_dense_need) >= 4096:
            _dense_need.clear()
        need = _dense_need[params, dev] = size.value
    if not batch:                # no sequence: all rows of q (there are some in TND only) lie behind the last one
        return torch.zeros_like(q) if out is None else out, q.new_full(rows_shape, -math.inf, dtype=_F32) if lse is None else lse
    room = 0
    if workspace is not None:
        if not (isinstance(workspace, torch.Tensor) and workspace.get_device() == dev and workspace.is_contiguous()):
            raise ValueError(f"workspace: needs a contiguous tensor on cuda:{dev}")
        room = workspace.numel() * workspace.element_size()
    elif need:
        workspace, room = torch.empty(need, dtype=torch.uint8, device=q.device), need
    if out is None:
        out = torch.empty_like(q)
        to = out.data_ptr()
    if lse is None:
        lse = torch.empty(rows_shape, dtype=_F32, device=q.device)
        end = lse.data_ptr()
    rc = _lib.sfm_dense_forward(params, tensors, to, end, workspace.data_ptr() if room else 0, room,
                                0 if status is None else _status_address(status, dev), _raw_stream(dev))
    if rc:
        raise SfmError("sfm_dense_forward", rc)
    for x in given:
        if not x.is_inference():
            _increment_version(x)
    return out, lse


def masked_attention(q: torch.Tensor, kv: torch.Tensor, *, softmax_scale: float = 1.0, softcap: float = 0.0, bias_slopes=None,
                     sinks=None, mask_mode: int = 3, win_left: int = -1, win_right: int = -1, prefix_lens=None, key_begin=None,
                     key_end=None, block_table=None, cu_seqlens_q=None, cu_seqlens_kv=None, seqused_q=None, seqused_kv=None,
                     max_seqlen_q: int = 0, max_seqlen_kv: int = 0, layout_q="BSND", layout_kv="BSND", split_keys: int = 0,
                     out=None, lse=None, workspace=None, status=None, stream=None):
    """Attention of q over the shared rows kv (K = V), all queries of a
    sequence over the same rows: prompts, and single tokens over a cache (see
    sfm_dense_forward).  Returns (out, q's shape; LSE, fp32, q's shape without
    its last dimension).

    q: (b, q_s, heads, 512) or TND (tokens, heads, 512), bf16 or fp16, dense;
    kv: (b, S, 512), (t, 512) or paged (blocks, block_size, 512) of the same
    dtype, with a KV head of 1 before the values or not, rows may be padded
    apart.  Contiguous kv may have no row (S or t of 0): every output is then 0 and every
    LSE -inf.  The scores are softmax_scale q.k, then ``softcap`` tanh(x / softcap)
    (0: none), then minus ``bias_slopes`` (fp32, heads) times the distance of
    query and key; ``sinks`` (fp32, heads) count in the denominator only.
    Query i of q_len sits at p = len - q_len + i, and sees key j if the mask
    mode allows it (0: all, 3: j <= p, 4: p - win_left <= j <= p + win_right,
    -1 for no bound) and ``key_begin`` <= j < ``key_end`` (int32, one per
    token: the bounds of the token's document), or if j < ``prefix_lens``
    (int32, one per sequence: keys that every token sees).

    ``split_keys``: 0 cuts long ranges of keys so that the GPU is filled; a
    multiple of 128 cuts them into as few even pieces of at most that many keys
    as there can be, so that a row's result does not depend on the other sequences
    of the batch.  ``max_seqlen_q`` may be given as to the other calls; nothing here
    needs it.  ``max_seqlen_kv`` (TND,
    paged): a bound on the keys of a sequence, which keeps the workspace small;
    longer sequences are cut.  ``workspace``: a
    uint8 tensor to use instead of a new one, sfm_dense_workspace_size bytes,
    for one call at a time.  Rows of a TND batch behind its last sequence are
    0 in a new output and -inf in a new LSE, and stay as they were in given ones.
    No gradient is recorded: inputs that require one (sinks and bias_slopes too)
    are refused in grad mode, and those that carry a tangent."""
    return _dense(q, kv, None, None, softmax_scale, softcap, bias_slopes, sinks, mask_mode, win_left, win_right, prefix_lens,
                  key_begin, key_end, block_table, cu_seqlens_q, cu_seqlens_kv, seqused_q, seqused_kv, max_seqlen_kv, layout_q,
                  layout_kv, split_keys, out, lse, workspace, status, stream)


def tree_attention(q: torch.Tensor, kv: torch.Tensor, tree_mask: torch.Tensor, positions: torch.Tensor, *,
                   softmax_scale: float = 1.0, softcap: float = 0.0, bias_slopes=None, sinks=None, mask_mode: int = 3,
                   win_left: int = -1, win_right: int = -1, block_table=None, cu_seqlens_q=None, cu_seqlens_kv=None,
                   seqused_q=None, seqused_kv=None, max_seqlen_q: int = 0, max_seqlen_kv: int = 0, layout_q="BSND",
                   layout_kv="BSND", split_keys: int = 0, out=None, lse=None, workspace=None, status=None, stream=None):
    """Attention of a tree of drafted tokens over a cache: as masked_attention,
    but the last q_len keys of a sequence are the drafted tokens' own rows
    (written before, in the queries' order), of which token i sees those whose
    bit is set in its row of ``tree_mask`` (int64, (tokens, words): bit k % 64
    of word k / 64 for drafted token k: the ancestors of i, and i itself).  It
    sees all keys before them, or with mask_mode 4 those inside the window.
    ``positions`` (int32, one per token) are the drafted tokens' places in the
    text (len - q_len + depth), which window and bias go by."""
    if tree_mask is None or positions is None:
        raise ValueError("tree_mask and positions are needed")
    return _dense(q, kv, tree_mask, positions, softmax_scale, softcap, bias_slopes, sinks, mask_mode, win_left, win_right, None,
                  None, None, block_table, cu_seqlens_q, cu_seqlens_kv, seqused_q, seqused_kv, max_seqlen_kv, layout_q,
                  layout_kv, split_keys, out, lse, workspace, status, stream)


def _rows_in_order(shape, lead):
    """Whether a shape lists the rows of `lead` (..., heads) in their order; dimensions of one entry do not count."""
    def plain(s):
        return [n for n in s if n != 1]
    rows, heads = lead.numel(), lead[-1]
    return plain(shape) in (plain(lead), plain((rows // heads if heads else 0, heads)), plain((rows,)))


def merge_attention(outs, lses, *, sinks=None, out=None, lse=None, stream=None):
    """Join attention results over separate sets of keys (see sfm_merge): outs
    (up to 8 of (..., heads, dim), bf16 or fp16, dense) with their LSEs (fp32,
    (..., heads), (tokens, heads) or flat, as sparse_flash_mla returns them) to
    (out, LSE) over all keys.  ``sinks`` (fp32,
    heads) count once, so the parts are computed without them.  ``out`` may be
    one of the parts.  Inputs that require a gradient are refused in grad mode."""
    outs, lses = list(outs), list(lses)
    if not outs or len(outs) != len(lses) or len(outs) > MERGE_MAX_PARTS:
        raise ValueError(f"outs and lses: need 1 to {MERGE_MAX_PARTS} each, as many of one as of the other")
    code, dev = _first("outs", outs[0], _SIXTEEN_BIT)
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return merge_attention(outs, lses, sinks=sinks, out=out, lse=lse)
    if _forward_ad._current_level >= 0:
        _no_tangents(outs=outs, lses=lses, sinks=sinks, out=out, lse=lse)
    x = outs[0]
    shape = x.shape
    if len(shape) < 2:
        raise ValueError("outs: need (..., heads, dim)")
    kind, lead, grad = x.dtype, shape[:-1], torch.is_grad_enabled()
    heads, dim, rows = lead[-1], shape[-1], lead.numel()
    parts, ends = [], []
    for o in outs:
        parts.append(_address("outs", o, kind, dev, shape))
        if grad and o.requires_grad:
            _no_gradient("outs", o)
    for l in lses:
        if _tensor("lses", l).numel() != rows:
            raise ValueError(f"lses: {l.numel()} values, expected {rows}")
        if l.shape != lead and not _rows_in_order(l.shape, lead):
            raise ValueError(f"lses: shape {tuple(l.shape)}, expected {tuple(lead)}, (tokens, heads) or flat")
        ends.append(_address("lses", l, _F32, dev, l.shape))
        if grad and l.requires_grad:
            _no_gradient("lses", l)
    if sinks is not None and _tensor("sinks", sinks).requires_grad:
        _no_gradient("sinks", sinks)
    given = ()
    if out is None:
        out = torch.empty_like(x)
        to = out.data_ptr()
    else:
        given = (out,)
        to = _address("out", out, kind, dev, shape)
        _no_gradient("out", out)
    if lse is None:
        lse = torch.empty(lead, dtype=_F32, device=x.device)
        end = lse.data_ptr()
    else:
        given += (lse,)
        end = _address("lse", lse, _F32, dev, lead)
        _no_gradient("lse", lse)
        if end in ends:
            raise ValueError("lse: must not be one of lses")
    n = len(parts)
    rc = (_lib or lib()).sfm_merge(_MERGE_PARAMS.pack(rows // heads if heads else 0, heads or 1, dim, n, code, 0),
                                   _POINTERS[n].pack(*parts), _POINTERS[n].pack(*ends),
                                   0 if sinks is None else _address("sinks", sinks, _F32, dev, (heads,)), to, end, _raw_stream(dev))
    if rc:
        raise SfmError("sfm_merge", rc)
    for y in given:
        if not y.is_inference():
            _increment_version(y)
    return out, lse


def move_kv(cache: torch.Tensor, path: torch.Tensor, first: torch.Tensor, *, block_table=None, status=None, stream=None):
    """Move the rows of the accepted path of every sequence to the front of
    its drafted rows (see sfm_kv_move): row first[b] + i becomes what row
    first[b] + path[b, i] was, up to the first negative entry.  path: int32
    (b, n), growing; first: int32 (b), the place of the first drafted row.
    cache: (blocks, block_size, row) with ``block_table`` (b, blocks) int32, or
    (b, S, row); any dtype, rows of a multiple of 16 bytes, a KV head of 1
    before the values or not.  Returns ``cache``."""
    if not isinstance(cache, torch.Tensor) or cache.get_device() < 0:
        raise ValueError("cache: not on a CUDA device" if isinstance(cache, torch.Tensor) else "cache: not a tensor")
    dev = cache.get_device()
    _no_gradient("cache", cache)
    if _forward_ad._current_level >= 0:
        _no_tangents(cache=cache)
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return move_kv(cache, path, first, block_table=block_table, status=status)
    kv = cache.squeeze(-2) if cache.dim() == 4 and cache.shape[-2] == 1 else cache
    if kv.dim() != 3:
        raise ValueError("cache: needs (blocks, block_size, row) or (b, S, row)")
    rows, row_stride = _rows(kv, "cache")
    if _tensor("path", path).dim() != 2:
        raise ValueError("path: needs (b, n)")
    batch, most = path.shape
    cols = table = 0
    if block_table is None:
        if kv.shape[0] != batch:
            raise ValueError("cache: needs (b, S, row) without a block table")
    else:
        if _tensor("block_table", block_table).dim() != 2:
            raise ValueError("block_table: needs (b, blocks)")
        cols = block_table.shape[1]
        table = _address("block_table", block_table, _I32, dev, (batch, cols))
    params = _MOVE_PARAMS.pack(batch, most, kv.shape[-1] * kv.element_size(), 0 if block_table is None else kv.shape[1], kv.shape[1],
                               cols, row_stride, rows)
    rc = (_lib or lib()).sfm_kv_move(params, _address("path", path, _I32, dev, (batch, most)),
                                     _address("first", first, _I32, dev, (batch,)), table, kv.data_ptr(),
                                     0 if status is None else _status_address(status, dev), _raw_stream(dev))
    if rc:
        raise SfmError("sfm_kv_move", rc)
    if not cache.is_inference():
        _increment_version(cache)
    return cache
