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
  caches, and the sparse indices the attention reads.
"""
from __future__ import annotations

import ctypes as C
import math
import os
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


EXPORTS = ("sfm_metadata_size", "sfm_workspace_size", "sfm_metadata", "sfm_forward", "sfm_forward_noalloc",
           "sfm_debug_attended", "sfm_set_profile_events", "sfm_error_string", "sfm_abi_version",
           "sfm_rope_frequencies", "sfm_rope", "sfm_kv_store", "sfm_index_scores", "sfm_topk_select")
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
        l.sfm_rope.argtypes = [C.POINTER(SfmRopeParams), V, V, V, V, V]
        l.sfm_kv_store.argtypes = [C.POINTER(SfmStoreParams), V, V, V, V, V, V, V, V, V]
        l.sfm_index_scores.argtypes = [C.POINTER(SfmIndexParams), C.POINTER(SfmIndexTensors), V, C.c_int64, V, V, V]
        l.sfm_topk_select.argtypes = [C.POINTER(SfmTopkParams), V, V, V, V, V]
        for n in ("sfm_metadata_size", "sfm_workspace_size", "sfm_metadata", "sfm_forward", "sfm_forward_noalloc",
                  "sfm_debug_attended", "sfm_set_profile_events", "sfm_abi_version", "sfm_rope_frequencies",
                  "sfm_rope", "sfm_kv_store", "sfm_index_scores", "sfm_topk_select"):
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
def _require(ok, what):
    if not ok:
        raise ValueError(what)


def _tensor(name, x, dtype=None, shape=None, device=None):
    """Check one tensor argument and return its device address (None for None)."""
    if x is None:
        return None
    _require(isinstance(x, torch.Tensor), f"{name}: not a tensor")
    if dtype is not None:
        _require(x.dtype in (dtype if isinstance(dtype, tuple) else (dtype,)), f"{name}: dtype {x.dtype}, expected {dtype}")
    if shape is not None:
        _require(tuple(x.shape) == tuple(shape), f"{name}: shape {tuple(x.shape)}, expected {tuple(shape)}")
        _require(x.is_contiguous(), f"{name}: not contiguous")
    _require(x.is_cuda, f"{name}: not on a CUDA device")
    if device is not None:
        _require(x.device == device, f"{name}: on {x.device}, expected {device}")
    return x.data_ptr()


class _Launch:
    """The device and stream of one call: makes the inputs' device current
    and allocates results on the stream that writes them."""

    def __init__(self, device, stream):
        self.device = torch.cuda.device(device)
        given = stream is not None and not hasattr(stream, "cuda_stream")
        self.given = torch.cuda.ExternalStream(int(stream), device=device) if given else stream
        self.stream = self.given

    def __enter__(self):
        self.device.__enter__()
        if self.given is None:
            self.stream = torch.cuda.current_stream()
            self.on = None
        else:
            self.on = torch.cuda.stream(self.given)
            self.on.__enter__()
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        if self.on is not None:
            self.on.__exit__(*exc)
        return self.device.__exit__(*exc)


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


def _dtype_code(x, name, fp8=False):
    codes = {torch.bfloat16: BF16, torch.float16: FP16}
    if fp8:
        codes[torch.float8_e4m3fn] = E4M3
    _require(x.dtype in codes, f"{name}: dtype {x.dtype}")
    return codes[x.dtype]


def _heads_view(x, name):
    """(tokens, heads, dim) of a (..., heads, dim) tensor, without a copy."""
    _require(isinstance(x, torch.Tensor) and x.dim() >= 2, f"{name}: needs (..., heads, values)")
    _require(x.stride(-1) == 1 or x.shape[-1] == 1, f"{name}: the last dimension must be contiguous")
    tokens = 1
    for n in x.shape[:-2]:
        tokens *= n
    try:
        return x.view(tokens, x.shape[-2], x.shape[-1])
    except RuntimeError:
        raise ValueError(f"{name}: the token dimensions do not flatten to one stride") from None


def _strides(v):
    """(token, head) strides of a (tokens, heads, dim) view; a dimension of one entry gets the stride of dense rows
    (torch may report any)."""
    head = v.stride(1) if v.shape[1] > 1 else v.shape[2]
    token = v.stride(0) if v.shape[0] > 1 else max(head * v.shape[1], v.shape[2])
    return token, head


def apply_rope(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, *, amplitude: float = 1.0,
               rope_offset: int = 0, interleaved: bool = True, inverse: bool = False, out=None, stream=None):
    """Rotary positions of x (..., heads, head_dim), bf16 or fp16.

    The values [rope_offset, rope_offset + 2 len(inv_freq)) of every head are
    rotated by position * inv_freq as pairs (2i, 2i + 1), or (i, i + n / 2)
    with ``interleaved=False``, and multiplied by ``amplitude``.
    positions: int32, one per token.  ``inverse=True`` applies the transposed
    map: the gradient with respect to x, and the way back for amplitude 1.
    ``out``: None for a new tensor, x itself to rotate in place, or a tensor
    of x's shape that does not overlap it.  Views with strides are taken as they are."""
    v = _heads_view(x, "x")
    dtype = _dtype_code(x, "x")
    _tensor("x", x)
    _require(inv_freq.dim() == 1 and inv_freq.numel() > 0, "inv_freq: needs one dimension")
    pos = _tensor("positions", positions, torch.int32, x.shape[:-2] if positions.dim() != 1 else (v.shape[0],), x.device)
    freq = _tensor("inv_freq", inv_freq, torch.float64, (inv_freq.numel(),), x.device)
    with _Launch(x.device, stream) as st:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        else:
            _tensor("out", out, x.dtype, None, x.device)
            _require(out.shape == x.shape, f"out: shape {tuple(out.shape)}, expected {tuple(x.shape)}")
        o = _heads_view(out, "out")
        (xt, xh), (yt, yh) = _strides(v), _strides(o)
        params = SfmRopeParams(tokens=v.shape[0], heads=max(v.shape[1], 1), head_dim=v.shape[2],
                               rope_dim=2 * inv_freq.numel(), rope_offset=rope_offset,
                               rope_layout=ROPE_INTERLEAVED if interleaved else ROPE_HALF, inverse=int(inverse),
                               dtype=dtype, amplitude=amplitude, x_token_stride=xt, x_head_stride=xh,
                               y_token_stride=yt, y_head_stride=yh)
        if v.shape[1] == 0:
            params.tokens = 0
        _check("sfm_rope", lib().sfm_rope(C.byref(params), v.data_ptr(), pos, freq, o.data_ptr(), st))
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
    _require(isinstance(x, torch.Tensor) and x.dim() in (2, 3), "x: needs (tokens, dim) or (tokens, heads, dim)")
    v = _heads_view(x.unsqueeze(1) if x.dim() == 2 else x, "x")
    dtype = _dtype_code(x, "x")
    T, H, D = v.shape
    _tensor("x", x)
    packed = kv_format in (KV_INT8_PACKED, KV_FP8_PACKED)
    kind = torch.uint8 if packed else torch.float8_e4m3fn if kv_format == KV_FP8_ROWS else x.dtype
    _tensor("cache", cache, kind, None, x.device)
    _require(cache.dim() >= 2 and (cache.stride(-1) == 1 or cache.shape[-1] == 1),
             "cache: needs (..., row) with contiguous rows")
    width = 512 + 2 * (D - 512) + 16 if packed else D
    _require(cache.shape[-1] == width, f"cache: rows of {cache.shape[-1]}, expected {width}")
    rows = 1
    for n in cache.shape[:-1]:
        rows *= n
    try:
        flat = cache.view(rows, width)
    except RuntimeError:
        raise ValueError("cache: the row dimensions do not flatten to one stride") from None
    _require((scales is not None) == (kv_format == KV_FP8_ROWS), "scales: go with KV_FP8_ROWS rows")
    _require((positions is None) == (inv_freq is None), "positions and inv_freq go together")
    _require(norm_eps is not None or norm_weight is None, "norm_weight: needs norm_eps")
    if scales is not None:
        _tensor("scales", scales, torch.float32, None, x.device)
        _require(scales.numel() == rows and scales.is_contiguous(), f"scales: {rows} contiguous values expected")
    if inv_freq is not None:
        _require(inv_freq.dim() == 1, "inv_freq: needs one dimension")
    rot = 2 * inv_freq.numel() if inv_freq is not None else 0
    xt, xh = _strides(v)
    params = SfmStoreParams(
        tokens=T if H else 0, heads=max(H, 1), head_dim=D, dtype=dtype, kv_format=kv_format,
        norm=int(norm_eps is not None), norm_eps=norm_eps if norm_eps is not None else 0.0, rope_dim=rot,
        rope_offset=(D - rot if rope_offset is None else rope_offset) if rot else 0,
        rope_layout=ROPE_INTERLEAVED if interleaved else ROPE_HALF, amplitude=amplitude, x_token_stride=xt,
        x_head_stride=xh, row_stride=(flat.stride(0) if rows > 1 else width) * cache.element_size(), rows=rows)
    args = (_tensor("norm_weight", norm_weight, torch.float32, (min(D, 512),), x.device),
            _tensor("positions", positions, torch.int32, (T,), x.device),
            _tensor("inv_freq", inv_freq, torch.float64, (rot // 2,), x.device),
            _tensor("slot_mapping", slot_mapping, torch.int32, (T,), x.device))
    _tensor("status", status, torch.int32, None, x.device)
    with _Launch(x.device, stream) as st:
        _check("sfm_kv_store", lib().sfm_kv_store(C.byref(params), v.data_ptr(), *args, flat.data_ptr(), _ptr(scales),
                                                  _ptr(status), st))
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
    fp32 (tokens, heads) in q's leading shape; k_scales: fp32, one per row of
    index_k.  Returns (scores (tokens, max_seqlen_kv) fp32, -inf where a key
    is not visible; visible (tokens) int32).  ``out`` may be a
    view with wider rows."""
    lq, lkv = _LAYOUTS[layout_q], _LAYOUTS[layout_kv]
    _require(isinstance(q, torch.Tensor) and q.dim() == (4 if lq == BSND else 3), "q: BSND has 4 dimensions, TND 3")
    dtype = _dtype_code(q, "q", fp8=True)
    tokens, heads = q.shape[:-2].numel(), q.shape[-2]
    _tensor("q", q, None, q.shape)
    dev = q.device
    _tensor("index_k", index_k, q.dtype, None, dev)
    _require(index_k.dim() == (2 if lkv == TND else 3) and index_k.shape[-1] == q.shape[-1] and index_k.stride(-1) == 1,
             "index_k: needs (t, dim), (b, S, dim) or (blocks, block_size, dim) with contiguous rows of q's dim")
    rows = index_k.shape[:-1].numel()
    try:
        flat = index_k.view(rows, index_k.shape[-1])
    except RuntimeError:
        raise ValueError("index_k: the row dimensions do not flatten to one stride") from None
    _tensor("weights", weights, torch.float32, q.shape[:-1], dev)
    if lkv == BSND:
        _require(index_k.shape[1] == max_seqlen_kv and index_k.shape[0] == q.shape[0], "index_k: needs (b, max_seqlen_kv, dim)")
    if lq == BSND:
        batch, max_seqlen_q = q.shape[0], q.shape[1]
    else:
        _require(cu_seqlens_q is not None, "cu_seqlens_q: required for TND")
        batch = cu_seqlens_q.numel() - 1
    if k_scales is not None:
        _tensor("k_scales", k_scales, torch.float32, None, dev)
        _require(k_scales.numel() == rows and k_scales.is_contiguous(), f"k_scales: {rows} contiguous values expected")
    if block_table is not None:
        _require(block_table.dim() == 2 and block_table.shape[0] == batch, "block_table: needs (b, blocks)")
    params = SfmIndexParams(
        num_heads=heads, index_dim=q.shape[-1], batch_size=batch, max_seqlen_q=max_seqlen_q, total_q=tokens,
        max_seqlen_kv=max_seqlen_kv, cmp_ratio=cmp_ratio, mask_mode=mask_mode, layout_q=lq, layout_kv=lkv, dtype=dtype,
        block_size=index_k.shape[1] if lkv == PAGED else 0)

    def ints(name, x, shape):
        return _tensor(name, x, torch.int32, shape, dev)

    tensors = SfmIndexTensors(
        q=q.data_ptr(), k=flat.data_ptr(),
        k_row_stride=(flat.stride(0) if rows > 1 else flat.shape[1]) * flat.element_size(), k_rows=rows,
        k_scales=_ptr(k_scales), weights=weights.data_ptr(),
        block_table=ints("block_table", block_table, block_table.shape if block_table is not None else None),
        block_table_stride=block_table.shape[1] if block_table is not None else 0,
        cu_seqlens_q=ints("cu_seqlens_q", cu_seqlens_q, (batch + 1,)),
        cu_seqlens_kv=ints("cu_seqlens_kv", cu_seqlens_kv, (batch + 1,)), seqused_q=ints("seqused_q", seqused_q, (batch,)),
        seqused_kv=ints("seqused_kv", seqused_kv, (batch,)),
        cmp_residual_kv=ints("cmp_residual_kv", cmp_residual_kv, (batch,)))
    _tensor("status", status, torch.int32, None, dev)
    with _Launch(dev, stream) as st:
        if out is None:
            out = torch.empty(tokens, max(max_seqlen_kv, 0), dtype=torch.float32, device=dev)
        else:
            _tensor("out", out, torch.float32, None, dev)
            _require(tuple(out.shape) == (tokens, max_seqlen_kv) and out.stride(1) == 1,
                     f"out: needs ({tokens}, {max_seqlen_kv}) with contiguous rows")
        if visible is None:
            visible = torch.empty(tokens, dtype=torch.int32, device=dev)
        seen = ints("visible", visible, (tokens,))
        stride = out.stride(0) if tokens > 1 else max(max_seqlen_kv, 1)
        _check("sfm_index_scores", lib().sfm_index_scores(C.byref(params), C.byref(tensors), out.data_ptr(), stride, seen,
                                                          _ptr(status), st))
    return out, visible


def select_topk(scores: torch.Tensor, k: int, *, lengths=None, block_size: int = 1, first_blocks: int = 0,
                last_blocks: int = 0, out=None, status=None, stream=None):
    """Indices (rows, k) int32, ascending and padded with -1, of the k largest
    scores of every row of ``scores`` (rows, n) fp32, or with ``block_size``
    of the k blocks with the largest score in them, the row's ``first_blocks``
    and ``last_blocks`` always among them (see sfm_topk_select).  They are what
    sparse_flash_mla takes as cmp_sparse_indices / ori_sparse_indices.
    lengths: int32 (rows), scores a row really has (None: n)."""
    _require(isinstance(scores, torch.Tensor) and scores.dim() == 2, "scores: needs (rows, n)")
    _tensor("scores", scores, torch.float32)
    rows, n = scores.shape
    _require(scores.stride(1) == 1 or n == 1, "scores: rows must be contiguous")
    args = _tensor("lengths", lengths, torch.int32, (rows,), scores.device)
    _tensor("status", status, torch.int32, None, scores.device)
    params = SfmTopkParams(rows=rows, n=n, k=k, block_size=block_size, first_blocks=first_blocks, last_blocks=last_blocks,
                           score_stride=scores.stride(0) if rows > 1 else n)
    with _Launch(scores.device, stream) as st:
        if out is None:
            out = torch.empty(rows, max(k, 0), dtype=torch.int32, device=scores.device)
        got = _tensor("out", out, torch.int32, (rows, k), scores.device)
        _check("sfm_topk_select", lib().sfm_topk_select(C.byref(params), scores.data_ptr(), args, got, _ptr(status), st))
    return out
