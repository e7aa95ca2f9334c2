"""CPU checks of the calls over many queries: struct layouts and refusals before anything is launched."""
import ctypes as C
import math
import subprocess

import pytest
import torch

import sparse_shared_kv_gb300 as sfm
from sparse_shared_kv_gb300 import buildlib

ADDR = 1 << 20      # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    sfm.build()
    return sfm.lib()


def _dense(**kw):
    base = dict(num_heads=64, head_dim=512, batch_size=2, max_seqlen_q=4, max_seqlen_kv=1000, mask_mode=3, win_left=-1,
                win_right=-1, layout_q=sfm.BSND, layout_kv=sfm.PAGED, dtype=sfm.BF16, block_size=64, softmax_scale=0.1)
    base.update(kw)
    return sfm.SfmDenseParams(**base)


def _tensors(**kw):
    base = dict(q=ADDR, kv=ADDR, kv_row_stride=1024, kv_rows=4096, block_table=ADDR, block_table_stride=16, seqused_kv=ADDR)
    base.update(kw)
    return sfm.SfmDenseTensors(**base)


PARAMS_BAD = [
    (dict(num_heads=0), 1), (dict(num_heads=129), 1), (dict(head_dim=576), 2), (dict(dtype=2), 1), (dict(dtype=-1), 1),
    (dict(layout_q=sfm.PAGED), 3), (dict(layout_kv=7), 3), (dict(layout_q=sfm.TND, layout_kv=sfm.BSND), 3), (dict(batch_size=0), 1),
    (dict(max_seqlen_q=-1), 1), (dict(layout_q=sfm.TND, total_q=-1), 1), (dict(max_seqlen_kv=0), 1), (dict(max_seqlen_kv=(1 << 30) + 1), 2),
    (dict(mask_mode=1), 1), (dict(mask_mode=4, win_left=-2), 1), (dict(mask_mode=4, win_right=-2), 1), (dict(block_size=8), 3),
    (dict(block_size=40), 3), (dict(block_size=2048), 3), (dict(tree_words=-1), 1), (dict(tree_words=17), 1), (dict(split_keys=-128), 1),
    (dict(split_keys=64), 1), (dict(softmax_scale=math.inf), 1), (dict(softmax_scale=math.nan), 1), (dict(softcap=-1.0), 1),
    (dict(softcap=math.inf), 1), (dict(softcap=math.nan), 1), (dict(softcap=1e-35), 1), (dict(batch_size=1 << 16, max_seqlen_q=1 << 10), 2),
]
TENSORS_BAD = [
    ({}, dict(kv_row_stride=1008), 3), ({}, dict(kv_row_stride=1032), 3), ({}, dict(kv_rows=0), 3), ({}, dict(kv_rows=1 << 31), 2),
    (dict(layout_kv=sfm.BSND), dict(block_table=None, kv_rows=1999), 3), (dict(layout_kv=sfm.BSND), {}, 1),
    (dict(layout_q=sfm.TND, total_q=3), {}, 1), (dict(layout_q=sfm.TND, layout_kv=sfm.TND, total_q=3), dict(cu_seqlens_q=ADDR, block_table=None), 1),
    ({}, dict(seqused_kv=None), 1), ({}, dict(block_table=None), 1), ({}, dict(block_table_stride=0), 1), ({}, dict(tree_mask=ADDR), 1),
    ({}, dict(positions=ADDR), 1), (dict(tree_words=1), {}, 1), (dict(tree_words=1), dict(tree_mask=ADDR), 1),
    (dict(tree_words=1), dict(tree_mask=ADDR, positions=ADDR, prefix_lens=ADDR), 1),
    (dict(tree_words=1), dict(tree_mask=ADDR, positions=ADDR, key_begin=ADDR), 1),
    (dict(tree_words=1), dict(tree_mask=ADDR, positions=ADDR, key_end=ADDR), 1),
    (dict(tree_words=1), dict(tree_mask=ADDR + 4, positions=ADDR), 3), ({}, dict(q=None), 1), ({}, dict(kv=None), 1),
    ({}, dict(q=ADDR + 8), 3), ({}, dict(kv=ADDR + 8), 3), ({}, dict(sinks=ADDR + 2), 3), ({}, dict(bias_slopes=ADDR + 1), 3),
]


@pytest.mark.parametrize("kw,code", PARAMS_BAD, ids=[str(b[0]) for b in PARAMS_BAD])
def test_params_are_refused(lib, kw, code):
    size = C.c_size_t(0)
    assert lib.sfm_dense_workspace_size(C.byref(_dense(**kw)), C.byref(size)) == code
    assert lib.sfm_dense_forward(C.byref(_dense(**kw)), C.byref(_tensors()), ADDR, ADDR, None, 0, None, None) == code


@pytest.mark.parametrize("kw,tkw,code", TENSORS_BAD, ids=[str(b[0]) + str(b[1]) for b in TENSORS_BAD])
def test_tensors_are_refused(lib, kw, tkw, code):
    assert lib.sfm_dense_forward(C.byref(_dense(**kw)), C.byref(_tensors(**tkw)), ADDR, ADDR, None, 0, None, None) == code


def test_pointers_are_refused(lib):
    p, t = C.byref(_dense()), C.byref(_tensors())
    assert lib.sfm_dense_forward(None, t, ADDR, ADDR, None, 0, None, None) == 1
    assert lib.sfm_dense_forward(p, None, ADDR, ADDR, None, 0, None, None) == 1
    assert lib.sfm_dense_forward(p, t, None, ADDR, None, 0, None, None) == 1
    assert lib.sfm_dense_forward(p, t, ADDR + 8, ADDR, None, 0, None, None) == 3
    assert lib.sfm_dense_forward(p, t, ADDR, ADDR + 2, None, 0, None, None) == 3
    assert lib.sfm_dense_workspace_size(p, None) == 1
    # nothing to do: nothing is read
    none = C.byref(_dense(max_seqlen_q=0))
    assert lib.sfm_dense_forward(none, t, None, None, None, 0, None, None) == 0


@pytest.mark.parametrize("name", ["block_table", "cu_seqlens_q", "cu_seqlens_kv", "seqused_q", "seqused_kv", "prefix_lens", "key_begin",
                                  "key_end", "positions", "status"])
def test_unaligned_integers_are_refused(lib, name):
    kw, tkw, status = {}, {}, None
    if name == "status":
        status = ADDR + 2
    else:
        tkw[name] = ADDR + 2
    if name == "positions":
        kw, tkw = dict(tree_words=1), dict(tkw, tree_mask=ADDR)
    if name.startswith("cu"):
        kw, tkw = dict(layout_q=sfm.TND, layout_kv=sfm.TND, total_q=4), {**dict(cu_seqlens_q=ADDR, cu_seqlens_kv=ADDR, block_table=None), **tkw}
    assert lib.sfm_dense_forward(C.byref(_dense(**kw)), C.byref(_tensors(**tkw)), ADDR, ADDR, None, 0, status, None) == 3


@pytest.mark.parametrize("rows", [1, 7, 63])
def test_a_cache_of_less_than_a_block_is_refused(lib, rows):
    assert lib.sfm_dense_forward(C.byref(_dense()), C.byref(_tensors(kv_rows=rows)), ADDR, ADDR, None, 0, None, None) == 3


@pytest.mark.parametrize("cap", [1.8e38, 3.4e38])
def test_caps_that_leave_fp32_in_steps_of_a_power_of_two_are_refused(lib, cap):
    size = C.c_size_t(0)
    assert lib.sfm_dense_workspace_size(C.byref(_dense(softcap=cap)), C.byref(size)) == 1
    assert lib.sfm_dense_forward(C.byref(_dense(softcap=cap)), C.byref(_tensors()), ADDR, ADDR, None, 0, None, None) == 1


@pytest.mark.parametrize("scale", [2.4e38, -3.4e38])
def test_scales_that_leave_fp32_in_steps_of_a_power_of_two_are_refused(lib, scale):
    size = C.c_size_t(0)
    assert lib.sfm_dense_workspace_size(C.byref(_dense(softmax_scale=scale)), C.byref(size)) == 1
    assert lib.sfm_dense_forward(C.byref(_dense(softmax_scale=scale)), C.byref(_tensors()), ADDR, ADDR, None, 0, None, None) == 1


@pytest.mark.parametrize("layout", [sfm.BSND, sfm.TND])
def test_contiguous_sources_may_have_no_row(lib, layout):
    size, kw = C.c_size_t(0), dict(layout_q=layout, layout_kv=layout, total_q=8, max_seqlen_kv=0)
    assert lib.sfm_dense_workspace_size(C.byref(_dense(**kw)), C.byref(size)) in (0, 5)          # 5: no GPU here
    assert lib.sfm_dense_workspace_size(C.byref(_dense(**{**kw, "max_seqlen_kv": -1})), C.byref(size)) == 1
    none = dict(block_table=None, kv_rows=0, cu_seqlens_q=ADDR, cu_seqlens_kv=ADDR)
    # refused for what else is missing, not for the rows
    assert lib.sfm_dense_forward(C.byref(_dense(**kw)), C.byref(_tensors(q=None, kv=None, **none)), ADDR, ADDR, None, 0, None, None) == 1
    assert lib.sfm_dense_forward(C.byref(_dense(**kw)), C.byref(_tensors(q=ADDR + 8, kv=None, **none)), ADDR, ADDR, None, 0, None, None) == 3
    assert lib.sfm_dense_forward(C.byref(_dense(**kw)), C.byref(_tensors(**{**none, "kv_rows": -1})), ADDR, ADDR, None, 0, None, None) == 3


@pytest.mark.parametrize("rest", [-1, 4, 1 << 20])
def test_rest_is_refused(lib, rest):
    size = C.c_size_t(0)
    assert lib.sfm_dense_workspace_size(C.byref(_dense(zero_rest=rest)), C.byref(size)) == 1


def test_lookups_of_drafted_keys_stay_with_their_sequence(tmp_path):
    """The keys of a word whose positions and bits the kernel looks up, on the host: the drafted ones, all of them, and no other."""
    source, program = tmp_path / "entry.cu", tmp_path / "entry"
    source.write_text("""#include "sfm_dense.cuh"
int main()
{
    const int sizes[] = {0, 1, 2, 5, 31, 32, 33, 63, 64, 65, 100, 128, 200, 1000, (1 << 30) - 7, 1 << 30};
    for (int len : sizes)
        for (int n : sizes) {
            const int first = len - n;
            for (int at : {0, first > 0 ? first : 0, len})
                for (int j0 = (at > 300 ? at - 300 : 0) & ~15; j0 < at + 300; j0 += 16) {
                    const uint32_t bits = sfm::drafted_keys(first, len, j0);
                    for (int c = 0; c < 32; ++c) {
                        const long long j = (long long)j0 + c, k = j - first;
                        const bool drafted = j >= 0 && j < len && k >= 0;
                        if (drafted != (bits >> c & 1) || (drafted && k >= n)) return 1;
                    }
                }
        }
    return 0;
}
""")
    subprocess.run([buildlib._nvcc(), *buildlib.ARCH, "-std=c++17", "-I", buildlib.INCLUDE, "-I", buildlib.CSRC, str(source), "-o", str(program)],
                   check=True)
    assert subprocess.run([str(program)]).returncode == 0


def _merge(**kw):
    return sfm.SfmMergeParams(**{**dict(tokens=3, heads=4, head_dim=512, parts=2, dtype=sfm.FP16), **kw})


@pytest.mark.parametrize("kw,code", [(dict(tokens=-1), 1), (dict(heads=0), 1), (dict(head_dim=0), 1), (dict(head_dim=12), 3), (dict(parts=0), 1),
                                     (dict(parts=9), 1), (dict(dtype=2), 1), (dict(reserved=1), 1), (dict(tokens=2 ** 31 - 1, heads=2 ** 31 - 1), 2)],
                         ids=str)
def test_merge_refusals(lib, kw, code):
    two = (C.c_void_p * 2)(ADDR, ADDR)
    assert lib.sfm_merge(C.byref(_merge(**kw)), two, two, None, ADDR, ADDR, None) == code


def test_merge_refuses_pointers(lib):
    p, two = C.byref(_merge()), (C.c_void_p * 2)(ADDR, ADDR)
    for outs, lses, sinks, out, lse, code in (
            (None, two, None, ADDR, ADDR, 1), (two, None, None, ADDR, ADDR, 1), (two, two, None, None, ADDR, 1),
            ((C.c_void_p * 2)(ADDR, None), two, None, ADDR, ADDR, 1), (two, (C.c_void_p * 2)(None, ADDR), None, ADDR, ADDR, 1),
            ((C.c_void_p * 2)(ADDR, ADDR + 8), two, None, ADDR, ADDR, 3), (two, (C.c_void_p * 2)(ADDR, ADDR + 2), None, ADDR, ADDR, 3),
            (two, two, ADDR + 1, ADDR, ADDR, 3), (two, two, None, ADDR + 8, ADDR, 3), (two, two, None, ADDR, ADDR + 2, 3)):
        assert lib.sfm_merge(p, outs, lses, sinks, out, lse, None) == code
    assert lib.sfm_merge(None, two, two, None, ADDR, ADDR, None) == 1
    assert lib.sfm_merge(C.byref(_merge(tokens=0)), two, two, None, None, None, None) == 0


def _move(**kw):
    return sfm.SfmMoveParams(**{**dict(batch_size=2, max_path=4, row_bytes=1024, block_size=64, max_seqlen_kv=0, block_table_stride=3,
                                       row_stride=1024, rows=640), **kw})


@pytest.mark.parametrize("kw,code", [(dict(batch_size=-1), 1), (dict(max_path=-1), 1), (dict(row_bytes=0), 1), (dict(row_bytes=24), 3),
                                     (dict(row_stride=1008), 3), (dict(row_stride=1032), 3), (dict(rows=0), 3), (dict(rows=1 << 31), 2),
                                     (dict(block_size=-1), 1), (dict(block_table_stride=0), 1), (dict(block_size=0, max_seqlen_kv=0), 1),
                                     (dict(block_size=0, max_seqlen_kv=50), 1), (dict(batch_size=65536), 2)], ids=str)
def test_move_refusals(lib, kw, code):
    assert lib.sfm_kv_move(C.byref(_move(**kw)), ADDR, ADDR, ADDR, ADDR, None, None) == code


def test_move_refuses_pointers(lib):
    p = C.byref(_move())
    for path, first, table, cache, status, code in (
            (None, ADDR, ADDR, ADDR, None, 1), (ADDR, None, ADDR, ADDR, None, 1), (ADDR, ADDR, None, ADDR, None, 1), (ADDR, ADDR, ADDR, None, None, 1),
            (ADDR + 2, ADDR, ADDR, ADDR, None, 3), (ADDR, ADDR + 1, ADDR, ADDR, None, 3), (ADDR, ADDR, ADDR + 2, ADDR, None, 3),
            (ADDR, ADDR, ADDR, ADDR + 8, None, 3), (ADDR, ADDR, ADDR, ADDR, ADDR + 2, 3)):
        assert lib.sfm_kv_move(p, path, first, table, cache, status, None) == code
    assert lib.sfm_kv_move(None, ADDR, ADDR, ADDR, ADDR, None, None) == 1
    for kw in (dict(batch_size=0), dict(max_path=0)):
        assert lib.sfm_kv_move(C.byref(_move(**kw)), None, None, ADDR, None, None, None) == 0


def test_packed_structs_match_the_ctypes_ones():
    for packer, kind in ((sfm._DENSE_PARAMS, sfm.SfmDenseParams), (sfm._DENSE_TENSORS, sfm.SfmDenseTensors),
                         (sfm._MERGE_PARAMS, sfm.SfmMergeParams), (sfm._MOVE_PARAMS, sfm.SfmMoveParams)):
        values = list(range(1, len(kind._fields_) + 1))
        made = kind(**{name: float(v) if t is C.c_float else v for v, (name, t) in zip(values, kind._fields_)})
        assert packer.size == C.sizeof(kind) and packer.pack(*values) == bytes(made), kind


def test_host_tensors_are_refused(lib):
    q, kv = torch.zeros(1, 2, 4, 512, dtype=torch.bfloat16), torch.zeros(1, 8, 512, dtype=torch.bfloat16)
    i = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sfm.masked_attention(q, kv)
    with pytest.raises(ValueError, match="CUDA"):
        sfm.tree_attention(q, kv, torch.zeros(1, 2, 1, dtype=torch.int64), i)
    with pytest.raises(ValueError, match="tree_mask"):
        sfm.tree_attention(q, kv, None, i)
    with pytest.raises(ValueError, match="CUDA"):
        sfm.merge_attention([q], [torch.zeros(1, 2, 4)])
    with pytest.raises(ValueError, match="not a tensor"):
        sfm.merge_attention([None], [None])
    with pytest.raises(ValueError, match="CUDA"):
        sfm.move_kv(kv, i, i[0])
