"""CPU checks of the operators around the attention: what the host refuses, the
rope frequencies, and the argument checks of the torch-level calls."""
import ctypes as C
import math

import pytest
import torch

import sparse_shared_kv_gb300 as sfm

ADDR = 1 << 20          # a 16-byte aligned address that is never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    sfm.build()
    return sfm.lib()


def _rope(**kw):
    base = dict(tokens=4, heads=2, head_dim=128, rope_dim=64, rope_offset=64, amplitude=1.0, x_token_stride=256,
                x_head_stride=128, y_token_stride=256, y_head_stride=128)
    base.update(kw)
    return sfm.SfmRopeParams(**base)


ROPE_BAD = [
    (dict(tokens=-1), 1), (dict(heads=0), 1), (dict(head_dim=0), 1), (dict(head_dim=4097, rope_offset=0), 1),
    (dict(rope_dim=0), 1), (dict(rope_dim=63), 1), (dict(rope_offset=-2), 1), (dict(rope_offset=65), 1),
    (dict(rope_dim=130, rope_offset=0), 1), (dict(rope_layout=2), 1), (dict(inverse=2), 1), (dict(dtype=2), 1),
    (dict(amplitude=math.inf), 1), (dict(amplitude=math.nan), 1), (dict(reserved=1), 1), (dict(x_token_stride=-1), 3),
    (dict(y_head_stride=-128), 3), (dict(y_head_stride=0), 3), (dict(y_token_stride=0), 3), (dict(y_head_stride=127), 3),
    (dict(y_token_stride=255), 3),
]


@pytest.mark.parametrize("kw,code", ROPE_BAD, ids=[str(b[0]) for b in ROPE_BAD])
def test_rope_refusals(lib, kw, code):
    assert lib.sfm_rope(C.byref(_rope(**kw)), ADDR, ADDR, ADDR, 2 * ADDR, None) == code


def test_rope_refuses_pointers(lib):
    p = C.byref(_rope())
    for args in ((None, ADDR, ADDR, ADDR), (ADDR, None, ADDR, ADDR), (ADDR, ADDR, None, ADDR), (ADDR, ADDR, ADDR, None)):
        assert lib.sfm_rope(p, *args, None) == 1
    for args in ((ADDR + 1, ADDR, ADDR, ADDR), (ADDR, ADDR + 2, ADDR, ADDR), (ADDR, ADDR, ADDR + 4, ADDR)):
        assert lib.sfm_rope(p, *args, None) == 3
    assert lib.sfm_rope(None, ADDR, ADDR, ADDR, ADDR, None) == 1
    # in place with other strides
    assert lib.sfm_rope(C.byref(_rope(y_token_stride=512)), ADDR, ADDR, ADDR, ADDR, None) == 3
    # nothing to do: no pointer is needed
    assert lib.sfm_rope(C.byref(_rope(tokens=0)), None, None, None, None, None) == 0
    # heads on top: (heads, tokens, dim) is a layout like any other
    assert lib.sfm_rope(C.byref(_rope(tokens=0, y_token_stride=128, y_head_stride=512)), None, None, None, None, None) == 0


def _store(**kw):
    base = dict(tokens=4, heads=1, head_dim=576, kv_format=sfm.KV_INT8_PACKED, norm=1, norm_eps=1e-6, rope_dim=64,
                rope_offset=512, amplitude=1.0, x_token_stride=576, x_head_stride=576, row_stride=656, rows=64)
    base.update(kw)
    return sfm.SfmStoreParams(**base)


STORE_BAD = [
    (dict(tokens=-1), 1), (dict(heads=0), 1), (dict(head_dim=640), 1), (dict(dtype=2), 1), (dict(kv_format=4), 1),
    (dict(kv_format=-1), 1), (dict(norm=2), 1), (dict(norm_eps=-1.0), 1), (dict(norm_eps=math.nan), 1),
    (dict(rope_dim=24), 1), (dict(rope_offset=516), 1), (dict(rope_offset=520), 1), (dict(rope_layout=2), 1),
    (dict(amplitude=math.inf), 1), (dict(reserved=1), 1), (dict(rows=-1), 2), (dict(rows=1 << 31), 2),
    (dict(tokens=1 << 20, heads=1 << 12), 2), (dict(row_stride=640), 3), (dict(row_stride=664), 3),
    (dict(x_token_stride=580), 3), (dict(x_head_stride=-8), 3),
    (dict(kv_format=sfm.KV_PLAIN, head_dim=576, row_stride=1152), 1), (dict(kv_format=sfm.KV_PLAIN, head_dim=24), 1),
]


@pytest.mark.parametrize("kw,code", STORE_BAD, ids=[str(b[0]) for b in STORE_BAD])
def test_store_refusals(lib, kw, code):
    assert lib.sfm_kv_store(C.byref(_store(**kw)), ADDR, ADDR, ADDR, ADDR, ADDR, ADDR, None, None, None) == code


def test_store_refuses_pointers(lib):
    p = C.byref(_store())
    good = [ADDR, ADDR, ADDR, ADDR, ADDR, ADDR, None, None, None]
    for i in (0, 2, 3, 5):
        assert lib.sfm_kv_store(p, *[None if j == i else g for j, g in enumerate(good)]) == 1
    for i in (0, 1, 5):
        assert lib.sfm_kv_store(p, *[ADDR + 8 if j == i else g for j, g in enumerate(good)]) == 3
    assert lib.sfm_kv_store(p, ADDR, ADDR, ADDR, ADDR, ADDR, ADDR, ADDR, None, None) == 1      # scales: not this format
    rows = C.byref(_store(kv_format=sfm.KV_FP8_ROWS, head_dim=128, rope_offset=0, row_stride=128))
    assert lib.sfm_kv_store(rows, ADDR, ADDR, ADDR, ADDR, ADDR, ADDR, None, None, None) == 1   # needs scales
    assert lib.sfm_kv_store(C.byref(_store(norm=0)), *good) == 1                               # a weight without a norm
    assert lib.sfm_kv_store(None, *good) == 1
    assert lib.sfm_kv_store(C.byref(_store(tokens=0)), *[None] * 9) == 0


def _index(**kw):
    base = dict(num_heads=64, index_dim=128, batch_size=2, max_seqlen_q=1, max_seqlen_kv=1000, cmp_ratio=4, mask_mode=3,
                layout_q=sfm.BSND, layout_kv=sfm.PAGED, dtype=sfm.BF16, block_size=64)
    base.update(kw)
    return sfm.SfmIndexParams(**base)


def _index_tensors(**kw):
    base = dict(q=ADDR, k=ADDR, k_row_stride=256, k_rows=4096, weights=ADDR, block_table=ADDR, block_table_stride=16,
                seqused_kv=ADDR, cmp_residual_kv=ADDR)
    base.update(kw)
    return sfm.SfmIndexTensors(**base)


INDEX_BAD = [
    (dict(num_heads=0), {}, 1), (dict(num_heads=129), {}, 1), (dict(index_dim=64), {}, 2), (dict(dtype=3), {}, 1),
    (dict(layout_q=sfm.PAGED), {}, 3), (dict(layout_q=sfm.TND, layout_kv=sfm.BSND), {}, 3), (dict(batch_size=0), {}, 1),
    (dict(max_seqlen_q=0), {}, 1), (dict(max_seqlen_kv=0), {}, 1), (dict(cmp_ratio=0), {}, 1), (dict(mask_mode=4), {}, 1),
    (dict(block_size=8), {}, 3), (dict(block_size=2048), {}, 3), (dict(block_size=40), {}, 3),
    (dict(batch_size=1 << 16, max_seqlen_q=1 << 10), {}, 2), (dict(layout_q=sfm.TND, total_q=-1), dict(cu_seqlens_q=ADDR), 1),
    ({}, dict(k_row_stride=240), 3), ({}, dict(k_row_stride=264), 3), ({}, dict(k_rows=0), 3),
    ({}, dict(k_rows=1 << 31), 2), ({}, dict(seqused_kv=None), 1), ({}, dict(block_table=None), 1),
    ({}, dict(block_table_stride=0), 1), ({}, dict(cmp_residual_kv=None), 1), (dict(layout_q=sfm.TND, total_q=5), {}, 1),
    (dict(layout_kv=sfm.BSND), {}, 1), ({}, dict(q=None), 1), ({}, dict(k=None), 1), ({}, dict(weights=None), 1),
    ({}, dict(q=ADDR + 8), 3), ({}, dict(k=ADDR + 8), 3), ({}, dict(weights=ADDR + 2), 3),
]


@pytest.mark.parametrize("kw,tkw,code", INDEX_BAD, ids=[str(b[0]) + str(b[1]) for b in INDEX_BAD])
def test_index_refusals(lib, kw, tkw, code):
    assert lib.sfm_index_scores(C.byref(_index(**kw)), C.byref(_index_tensors(**tkw)), ADDR, 1000, None, None, None) == code


def test_index_columns_are_counted_in_whole_tiles(lib):
    t = C.byref(_index_tensors())
    for n in (2 ** 31 - 1, 2 ** 31 - 128, 2 ** 31 - 256):
        assert lib.sfm_index_scores(C.byref(_index(max_seqlen_kv=n)), t, ADDR, n, None, None, None) == 2


def test_index_refuses_outputs(lib):
    p, t = C.byref(_index()), C.byref(_index_tensors())
    assert lib.sfm_index_scores(p, t, ADDR, 999, None, None, None) == 3
    assert lib.sfm_index_scores(p, t, None, 1000, None, None, None) == 1
    assert lib.sfm_index_scores(p, t, ADDR + 2, 1000, None, None, None) == 3
    assert lib.sfm_index_scores(None, t, ADDR, 1000, None, None, None) == 1
    assert lib.sfm_index_scores(p, None, ADDR, 1000, None, None, None) == 1
    empty = _index(layout_q=sfm.TND, total_q=0)
    assert lib.sfm_index_scores(C.byref(empty), C.byref(_index_tensors(cu_seqlens_q=ADDR, q=None)), None, 1000, None, None,
                                None) == 0


def _topk(**kw):
    base = dict(rows=3, n=100, k=8, block_size=1, score_stride=100)
    base.update(kw)
    return sfm.SfmTopkParams(**base)


TOPK_BAD = [
    (dict(rows=-1), 1), (dict(n=0), 1), (dict(k=0), 1), (dict(block_size=0), 1), (dict(block_size=3), 1),
    (dict(block_size=256), 1), (dict(first_blocks=-1), 1), (dict(last_blocks=-1), 1), (dict(first_blocks=5, last_blocks=4), 1),
    (dict(first_blocks=2 ** 31 - 1, last_blocks=2 ** 31 - 1), 1), (dict(score_stride=99), 3),
]


@pytest.mark.parametrize("kw,code", TOPK_BAD, ids=[str(b[0]) for b in TOPK_BAD])
def test_topk_refusals(lib, kw, code):
    assert lib.sfm_topk_select(C.byref(_topk(**kw)), ADDR, None, ADDR, None, None) == code


def test_topk_refuses_pointers(lib):
    p = C.byref(_topk())
    assert lib.sfm_topk_select(p, None, None, ADDR, None, None) == 1
    assert lib.sfm_topk_select(p, ADDR, None, None, None, None) == 1
    assert lib.sfm_topk_select(p, ADDR + 1, None, ADDR, None, None) == 3
    assert lib.sfm_topk_select(p, ADDR, ADDR + 2, ADDR, None, None) == 3
    assert lib.sfm_topk_select(None, ADDR, None, ADDR, None, None) == 1
    assert lib.sfm_topk_select(C.byref(_topk(rows=0)), None, None, None, None, None) == 0


def test_packed_structs_match_the_ctypes_ones():
    for packer, struct in ((sfm._ROPE_PARAMS, sfm.SfmRopeParams), (sfm._STORE_PARAMS, sfm.SfmStoreParams),
                           (sfm._INDEX_PARAMS, sfm.SfmIndexParams), (sfm._INDEX_TENSORS, sfm.SfmIndexTensors),
                           (sfm._TOPK_PARAMS, sfm.SfmTopkParams)):
        n = len(struct._fields_)
        values = list(range(1, n + 1))
        made = struct(**{name: float(v) if kind is C.c_float else v for v, (name, kind) in zip(values, struct._fields_)})
        assert packer.size == C.sizeof(struct) and packer.pack(*values) == bytes(made), struct


def test_row_dimensions_of_one_entry_may_have_any_stride():
    """Caches cut or unflattened to blocks of one row are rows like any other."""
    wide = torch.zeros(60, 144)
    for x, want in ((wide[:, :128].unflatten(0, (60, 1)), (60, 576)), (wide[:, :128].unflatten(0, (1, 60)), (60, 576)),
                    (wide[:, :128].unflatten(0, (10, 6)), (60, 576)), (wide[:1, :128].unflatten(0, (1, 1)), (1, 512)),
                    (torch.zeros(5, 4, 128)[:, :1], (5, 2048)), (torch.zeros(5, 4, 128)[:1], (4, 512)),
                    (torch.zeros(6, 4, 2, 144)[:, :1, :, :128], None), (torch.zeros(6, 4, 2, 144)[:, 1:2, :1, :128], (6, 4608)),
                    (torch.zeros(1, 7, 128).expand(5, 7, 128), None), (torch.zeros(5, 4, 128)[:, :2], None),
                    (torch.zeros(3, 0, 128), (0, 512)), (torch.zeros(0, 4, 128), (0, 512)), (torch.zeros(4, 128), (4, 512)),
                    (wide[:, :128], (60, 576)), (wide[:1, :128], (1, 512))):
        if want is None:
            with pytest.raises(ValueError, match="one stride"):
                sfm._rows(x, "cache")
        else:
            assert sfm._rows(x, "cache") == want, (x.shape, x.stride())


# ---------------------------------------------------------------------------
# frequencies
# ---------------------------------------------------------------------------
def test_frequencies_against_their_definitions(lib):
    f, a = sfm.rope_frequencies(64)
    want = torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64)
    assert a == 1.0 and f.dtype == torch.float64 and torch.allclose(f, want, rtol=1e-14, atol=0)
    lin, a = sfm.rope_frequencies(64, scaling="linear", factor=8.0)
    assert a == 1.0 and torch.allclose(lin, want / 8, rtol=1e-14, atol=0)
    ntk, a = sfm.rope_frequencies(64, scaling="ntk", factor=8.0)
    assert a == 1.0 and math.isclose(float(ntk[0]), 1.0) and math.isclose(float(ntk[-1] * 8), float(want[-1]), rel_tol=1e-12)
    yarn, a = sfm.rope_frequencies(64, scaling="yarn", factor=16.0, original_max_position=4096)
    assert math.isclose(a, 0.1 * math.log(16) + 1, rel_tol=1e-6)
    turns = 4096 * want / (2 * math.pi)
    assert torch.allclose(yarn[turns > 40], want[turns > 40], rtol=1e-14, atol=0)
    assert torch.allclose(yarn[turns < 0.7], want[turns < 0.7] / 16, rtol=1e-14, atol=0)
    assert bool((yarn <= want * (1 + 1e-14)).all()) and bool((yarn >= want / 16 * (1 - 1e-14)).all())
    assert torch.allclose(sfm.rope_frequencies(64, scaling="yarn", factor=1.0, original_max_position=4096)[0], want,
                          rtol=1e-14, atol=0)


@pytest.mark.parametrize("kw", [
    dict(rope_dim=0), dict(rope_dim=7), dict(base=1.0), dict(base=math.nan), dict(scaling="linear", factor=0.5),
    dict(scaling="ntk", rope_dim=2, factor=2.0), dict(scaling="yarn", factor=2.0),
    dict(scaling="yarn", factor=2.0, original_max_position=64, beta_fast=1.0, beta_slow=2.0)], ids=str)
def test_frequency_refusals(lib, kw):
    kw = dict(kw)
    with pytest.raises(sfm.SfmError):
        sfm.rope_frequencies(kw.pop("rope_dim", 64), **kw)


def test_unknown_scaling():
    with pytest.raises(ValueError):
        sfm.rope_frequencies(64, scaling="other")


# ---------------------------------------------------------------------------
# the torch-level calls refuse what the C entry points cannot see
# ---------------------------------------------------------------------------
def test_host_tensors_are_refused(lib):
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.float64)
    p = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sfm.apply_rope(x, p, f)
    with pytest.raises(ValueError, match="dtype"):
        sfm.apply_rope(x.float(), p, f)
    with pytest.raises(ValueError, match="CUDA"):
        sfm.store_kv(x, torch.zeros(8, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        sfm.index_scores(x.unsqueeze(0), torch.zeros(1, 8, 128, dtype=torch.bfloat16), torch.zeros(1, 4, 2), max_seqlen_kv=8)
    with pytest.raises(ValueError, match="CUDA"):
        sfm.select_topk(torch.zeros(2, 8), 4)
