"""The operators around the attention on the GPU, against their definitions in
64 bits (``_plain64``), and a run of them together with the attention.

Tolerances, from the arithmetic (u = 2^-24, one fp32 rounding; e = half a step of
the output type relative to the value):
* rotation: a coefficient (cos or sin times the amplitude) is off by the angle's
  error -- below 2^-31 pi of the truncated turn plus u pi of its rounding to fp32 --
  and by sincospif's two steps and the product with the amplitude, together below
  2^-21; the two products and the sum add 3 u of (|a| + |b|).  Bound: 2^-20 amplitude
  (|a| + |b|), then e of the value.
* RMS norm: the sum of squares of 512 values in runs of 24 and five shuffles is
  off by at most 32 u, its square root by half of that, the division and the two
  products by 5 u: below 2^-19 of the value.
* a stored code: half a step of the code times the scale, beside the value's own
  error (2^-19 of the tile's largest magnitude and, rotated, 2^-20 of the pair's);
  for E4M3 half a step is 2^-4 of the value, or 2^-10 scales below the normal range.
* scores: 128 products per head, exact, added in fp32 by the tensor cores, each
  step off by at most 2^-23 of the magnitudes so far, then at most 128 + 2 fp32
  steps over the heads: (128 2^-23 + 130 u) of the sum of all magnitudes.
* selected indices are whole numbers and equal.
"""
import math

import pytest
import torch

import oracle
import sfm_inputs as S
import sparse_shared_kv_gb300 as sfm
from tests import _plain64 as P, _sfm

pytestmark = pytest.mark.gpu

F64 = torch.float64
SCORE_TOL = 128 * 2.0 ** -23 + 130 * 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}


@pytest.fixture(scope="module", autouse=True)
def _built():
    sfm.build()
    torch.cuda.init()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g).to(dtype)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def floor_of(dtype):
    """Half the step of the smallest values of the type."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def assert_within(got, want, bound, what=""):
    off = (got.detach().cpu().to(F64) - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {float((off / bound.clamp(min=1e-300)).max()):.3g} bounds"


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def rope_check(got, x, pos, f, off, inter, inv, amp):
    want, mag = P.rope_parts(x.cpu(), pos.cpu().tolist(), f.cpu(), off, inter, inv, amp)
    turned = mag > 0
    bound = torch.where(turned, 2.0 ** -20 * abs(amp) * mag * (1 + half_step(x.dtype)) + half_step(x.dtype) * want.abs()
                        + floor_of(x.dtype), 0.0)
    assert_within(got, want, bound, "rope")


# tokens, heads, dim, rot, offset
ROPE_SHAPES = [(1, 1, 64, 64, 0), (3, 5, 128, 64, 0), (17, 2, 576, 64, 512), (2, 128, 512, 64, 448), (33, 3, 192, 128, 64),
               (700, 1, 64, 16, 48), (5, 3, 20, 10, 6), (4, 2, 66, 2, 64), (2, 1, 4096, 4096, 0), (3, 7, 130, 24, 8)]


@pytest.mark.parametrize("shape", ROPE_SHAPES, ids=str)
@pytest.mark.parametrize("inter", [True, False], ids=["pairs", "halves"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_rope(shape, inter, dt):
    T, H, D, rot, off = shape
    g = gen(T * 1000 + D)
    x = randn(g, T, H, D, dtype=DT[dt]).cuda()
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (T,), generator=g, dtype=torch.int64).to(torch.int32)
    pos[0] = 0 if T % 2 else (1 << 31) - 1
    f, _ = sfm.rope_frequencies(rot, device="cuda")
    for inv, amp in ((False, 1.0), (True, 1.25)):
        y = sfm.apply_rope(x, pos.cuda(), f, rope_offset=off, interleaved=inter, inverse=inv, amplitude=amp)
        rope_check(y, x, pos, f, off, inter, inv, amp)
        z = x.clone()
        assert sfm.apply_rope(z, pos.cuda(), f, rope_offset=off, interleaved=inter, inverse=inv, amplitude=amp, out=z) is z
        assert torch.equal(z, y)


@pytest.mark.parametrize("shape", [(100003, 8, 64, 16, 48), (40009, 17, 64, 64, 0), (1301, 64, 512, 64, 448), (3001, 200, 80, 48, 16)],
                         ids=str)
@pytest.mark.parametrize("inter", [True, False], ids=["pairs", "halves"])
def test_rope_many_rows_as_in_pieces(shape, inter):
    """Tokens that one block works on one after the other turn as they do alone."""
    T, H, D, rot, off = shape
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, H + 1, D, generator=g, device="cuda").to(torch.bfloat16)[:, :H]
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (T,), generator=g, device="cuda").to(torch.int32)
    f, _ = sfm.rope_frequencies(rot, device="cuda")
    kw = dict(rope_offset=off, interleaved=inter, inverse=True, amplitude=1.25)
    y = sfm.apply_rope(x, pos, f, **kw)
    for i in range(0, T, max(T // 64, 1)):
        e = min(i + max(T // 64, 1), T)
        assert torch.equal(y[i:e], sfm.apply_rope(x[i:e], pos[i:e], f, **kw))
    some = slice(T // 2, T // 2 + 40)
    rope_check(y[some], x[some], pos[some], f, off, inter, True, 1.25)


@pytest.mark.parametrize("inter", [True, False], ids=["pairs", "halves"])
def test_rope_strided_views(inter):
    g = gen(5)
    big = randn(g, 6, 4, 520, dtype=torch.bfloat16).cuda()
    pos = torch.tensor([0, 1, 7, 4095, 100000, 999999], dtype=torch.int32)
    f, amp = sfm.rope_frequencies(32, scaling="yarn", factor=16.0, original_max_position=4096, device="cuda")
    for x in (big[..., 456:], big[..., 3:67], big[:, 1:3, 8:136], big.transpose(0, 1).contiguous().transpose(0, 1)[..., 8:72]):
        before = big.clone()
        rope_check(sfm.apply_rope(x, pos.cuda(), f, interleaved=inter, amplitude=amp), x, pos, f, 0, inter, False, amp)
        out = torch.full((6, x.shape[1], x.shape[2] + 5), 7.0, dtype=x.dtype, device="cuda")
        got = sfm.apply_rope(x, pos.cuda(), f, interleaved=inter, amplitude=amp, out=out[..., :x.shape[2]])
        rope_check(got, x, pos, f, 0, inter, False, amp)
        assert bool((out[..., x.shape[2]:] == 7.0).all()) and torch.equal(big, before)
    # broadcast heads are fine to read, in place they are refused
    one = big[:, :1, :64].expand(6, 4, 64)
    rope_check(sfm.apply_rope(one, pos.cuda(), f, interleaved=inter), one, pos, f, 0, inter, False, 1.0)
    with pytest.raises(sfm.SfmError):
        sfm.apply_rope(one, pos.cuda(), f, out=one)


@pytest.mark.parametrize("inter", [True, False], ids=["pairs", "halves"])
def test_rope_angles_of_far_positions(inter):
    """The angle is reduced as exactly at 2^31 as at 1, for fast pairs too.  Pairs whose first result nearly cancels show
    it: its rounding to fp16 is 2^-11 of next to nothing, and what is left of the bound is that of the coefficients."""
    freq = torch.tensor([1000.3, -1000.7, 100.9, 33.3, 6.5, 1.0, -0.7, 0.01], dtype=F64)
    n = freq.numel()
    pos = torch.tensor([1, 3, -5, 1000, 2 ** 20 + 1, 2 ** 30 - 7, -(2 ** 31), 2 ** 31 - 1], dtype=torch.int64)
    T, g = pos.numel(), gen(21)
    unit = torch.zeros(T, 1, 2 * n, dtype=F64)
    first, second = (slice(0, None, 2), slice(1, None, 2)) if inter else (slice(0, n), slice(n, None))
    unit[..., first] = 1.0
    turned, _ = P.rope_parts(unit, pos.tolist(), freq, 0, inter)
    c, s = turned[..., first], turned[..., second]
    for _ in range(8):
        r = 0.5 + 0.5 * torch.rand(T, 1, n, generator=g, dtype=F64)
        x = torch.zeros(T, 1, 2 * n, dtype=torch.float16)
        x[..., first], x[..., second] = (r * s).to(torch.float16), (r * c).to(torch.float16)      # a cos = b sin, nearly
        y = sfm.apply_rope(x.cuda(), pos.to(torch.int32).cuda(), freq.cuda(), interleaved=inter)
        rope_check(y, x, pos, freq, 0, inter, False, 1.0)


def test_rope_gradient_is_the_inverse_call():
    g = gen(9)
    x, gy = randn(g, 3, 2, 64, dtype=torch.float16).cuda(), randn(g, 3, 2, 64, dtype=torch.float16).cuda()
    pos = torch.tensor([3, 70000, -5], dtype=torch.int32)
    f, _ = sfm.rope_frequencies(32, device="cuda")
    for inter in (True, False):
        gx = sfm.apply_rope(gy, pos.cuda(), f, rope_offset=16, interleaved=inter, inverse=True, amplitude=1.5)
        # differences of the formula's <y, gy>, which is linear in x: exact up to 64-bit rounding
        def loss(v):
            return float((P.rope_parts(v, pos.tolist(), f.cpu(), 16, inter, False, 1.5)[0] * gy.cpu().to(F64)).sum())
        base = torch.zeros(3, 2, 64, dtype=F64)
        for at in ((0, 0, 0), (0, 1, 16), (1, 0, 17), (1, 1, 40), (2, 0, 47), (2, 1, 63)):
            e = base.clone()
            e[at] = 1.0
            d = (loss(e) - loss(-e)) / 2
            lim = half_step(torch.float16) * abs(d) + 2.0 ** -20 * 1.5 * 8 + floor_of(torch.float16)
            assert abs(float(gx[at]) - d) <= lim, at
        # amplitude 1: there and back, two roundings of each member of a pair
        back = sfm.apply_rope(sfm.apply_rope(x, pos.cuda(), f, interleaved=inter), pos.cuda(), f, interleaved=inter, inverse=True)
        _, mag = P.rope_parts(x.cpu(), pos.tolist(), f.cpu(), 0, inter)
        lim = 2 * half_step(torch.float16) * mag * 1.01 + half_step(torch.float16) * x.cpu().to(F64).abs() + 2.0 ** -18 * mag
        assert_within(back, x.cpu().to(F64), torch.where(mag > 0, lim + 2 * floor_of(torch.float16), 0.0))


def test_rope_and_autograd():
    """No gradient is lost in silence: the call refuses to be recorded, works inside a Function of the caller's, and
    what it writes is noticed by graphs that saved it."""
    g = gen(15)
    x, gy = randn(g, 5, 3, 64, dtype=torch.float16).cuda(), randn(g, 5, 3, 64, dtype=torch.float16).cuda()
    pos, (f, _) = torch.arange(5, dtype=torch.int32).cuda(), sfm.rope_frequencies(32, device="cuda")
    want = sfm.apply_rope(x, pos, f, amplitude=1.5)
    leaf = x.clone().requires_grad_()
    for t in (leaf, leaf * 1):
        for kw in (dict(), dict(out=t), dict(out=torch.empty_like(x)), dict(stream=torch.cuda.Stream())):
            with pytest.raises(ValueError, match="gradient"):
                sfm.apply_rope(t, pos, f, **kw)
    with pytest.raises(ValueError, match="gradient"):
        sfm.apply_rope(x, pos, f, out=torch.empty_like(x).requires_grad_())
    with torch.no_grad():
        assert torch.equal(sfm.apply_rope(leaf, pos, f, amplitude=1.5), want)

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return sfm.apply_rope(x, pos, f, amplitude=1.5)

        @staticmethod
        def backward(ctx, gy):
            return sfm.apply_rope(gy, pos, f, amplitude=1.5, inverse=True)
    y = Rope.apply(leaf)
    y.backward(gy)
    assert torch.equal(y, want) and torch.equal(leaf.grad, sfm.apply_rope(gy, pos, f, amplitude=1.5, inverse=True))

    weight = torch.ones_like(x).requires_grad_()
    for place in (True, False):
        a = x.clone()
        loss = (a * weight).sum()
        sfm.apply_rope(a if place else x, pos, f, out=a)
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
    with torch.inference_mode():
        a = x.clone()
        assert torch.equal(sfm.apply_rope(a, pos, f, amplitude=1.5, out=a), want)
    with torch.inference_mode():
        a = x.clone()
    assert torch.equal(sfm.apply_rope(a, pos, f, amplitude=1.5, out=a), want)


def test_rope_without_tokens_and_on_another_stream():
    f, _ = sfm.rope_frequencies(64, device="cuda")
    assert sfm.apply_rope(torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"),
                          torch.empty(0, dtype=torch.int32, device="cuda"), f).shape == (0, 4, 64)
    g = gen(2)
    x, pos = randn(g, 64, 8, 128, dtype=torch.bfloat16).cuda(), torch.arange(64, dtype=torch.int32).cuda()
    want = sfm.apply_rope(x, pos, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for given in (s, s.cuda_stream):
        y = sfm.apply_rope(x, pos, f, stream=given)
        s.synchronize()
        assert torch.equal(y, want)


# ---------------------------------------------------------------------------
# cache rows
# ---------------------------------------------------------------------------
FORMATS = {"plain": sfm.KV_PLAIN, "int8": sfm.KV_INT8_PACKED, "fp8": sfm.KV_FP8_PACKED, "rows": sfm.KV_FP8_ROWS}


def make_cache(fmt, rows, dim, dtype, pad=0):
    """A cache of recognisable bytes; pad: extra bytes between rows (a multiple of 16)."""
    if fmt == "plain":
        kind, width = dtype, dim
    elif fmt == "rows":
        kind, width = torch.float8_e4m3fn, dim
    else:
        kind, width = torch.uint8, 512 + 2 * (dim - 512) + 16
    e = 2 if fmt == "plain" else 1
    raw = torch.full((rows, width * e + pad), 0x33, dtype=torch.uint8, device="cuda")
    return raw, raw[:, :width * e].view(kind) if kind != torch.uint8 else raw[:, :width]


def check_rows(fmt, cache, scales, rows, values, mag, dtype, amp=1.0):
    """Rows `rows` of the cache hold `values` (n, dim; 64 bits) within the format's rounding."""
    c = cache[rows.cuda()].cpu()
    n, D = values.shape
    u = values.abs() * 2.0 ** -19 + 2.0 ** -20 * abs(amp) * mag

    def plain_bound(v, err, dt):
        return half_step(dt) * (v.abs() + err) + err + floor_of(dt)
    if fmt == "plain":
        assert_within(c, values, plain_bound(values, u, dtype), "plain")
        return
    nd = D if fmt == "rows" else 512
    tile = nd if fmt == "rows" else 128
    most = 127.0 if fmt == "int8" else 448.0
    t, tu = values[:, :nd].reshape(n, -1, tile), u[:, :nd].reshape(n, -1, tile)
    if fmt == "rows":
        got_scale = scales[rows.cuda()].cpu().to(F64)[:, None]
    else:
        got_scale = c[:, -16:].contiguous().view(torch.float32).to(F64)
    want_scale = (t.abs().amax(-1) / most).clamp(min=P.TINY)
    err = tu.amax(-1)
    assert_within(got_scale, want_scale, err / most + 2.0 ** -22 * want_scale + 2.0 ** -149, "scale")
    codes = c[:, :nd].contiguous()
    codes = codes.view(torch.int8).to(F64) if fmt == "int8" else codes.view(torch.float8_e4m3fn).to(torch.float32).to(F64)
    if fmt == "int8":
        assert int(codes.abs().max()) <= 127
    back = codes.reshape(n, -1, tile) * got_scale[..., None]
    s = got_scale[..., None]
    # value / scale is rounded twice in fp32 (the reciprocal and the product) before the code's own rounding
    q = t.abs() * 2.0 ** -22 + tu
    bound = s / 2 + q if fmt == "int8" else 2.0 ** -4 * (t.abs() + q) + q + 2.0 ** -10 * s
    assert_within(back, t, bound, fmt)
    if D > nd:
        rope = c[:, 512:512 + 2 * (D - 512)].contiguous().view(dtype)
        assert_within(rope, values[:, 512:], plain_bound(values[:, 512:], u[:, 512:], dtype), "rope part")


STORE_CASES = [   # format, dim, rot, offset, interleaved, heads
    ("plain", 512, 64, 448, True, 1), ("plain", 512, 512, 0, False, 1), ("plain", 512, 0, 0, True, 1),
    ("plain", 128, 64, 0, False, 1), ("plain", 16, 16, 0, True, 3), ("plain", 272, 32, 8, False, 1),
    ("int8", 576, 64, 512, True, 1), ("int8", 576, 64, 512, False, 1), ("int8", 512, 0, 0, True, 1),
    ("int8", 512, 64, 448, False, 1), ("fp8", 576, 64, 512, True, 1), ("fp8", 576, 576, 0, False, 1),
    ("fp8", 512, 32, 480, True, 1), ("rows", 128, 64, 0, False, 1), ("rows", 128, 64, 64, True, 5),
    ("rows", 512, 64, 448, True, 1), ("rows", 48, 0, 0, True, 64),
]


@pytest.mark.parametrize("case", STORE_CASES, ids=str)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens", [1, 37])
def test_store(case, dt, tokens):
    fmt, D, rot, off, inter, H = case
    g = gen(D * 7 + tokens)
    dtype = DT[dt]
    x = randn(g, tokens, H, D, dtype=dtype) * (0.1 + torch.rand(tokens, 1, 1, generator=g).to(dtype))
    x = x.to(dtype)
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g).to(torch.int32)
    f = sfm.rope_frequencies(rot, device="cuda")[0] if rot else None
    slots = torch.randperm(tokens + 11, generator=g)[:tokens].to(torch.int32)
    if tokens > 1:
        slots[5] = -1
        slots[tokens - 1] = -7
    rows = (tokens + 11) * H
    for norm in (False, True):
        w = 1 + 0.2 * randn(g, min(D, 512)) if norm and tokens > 1 else None
        raw, cache = make_cache(fmt, rows, D, dtype, pad=32)
        scales = torch.full((rows,), 9.0, device="cuda") if fmt == "rows" else None
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        sfm.store_kv(x.cuda(), cache, slot_mapping=slots.cuda(), kv_format=FORMATS[fmt], norm_weight=w.cuda() if w is not None else None,
                     norm_eps=1e-5 if norm else None, positions=pos.cuda() if rot else None, inv_freq=f,
                     rope_offset=off if rot else None, interleaved=inter, scales=scales, status=status)
        v, mag = P.store_values(x, w, 1e-5 if norm else None, pos.tolist(), f.cpu() if rot else None, off, inter)
        if norm and rot:      # the pair's magnitudes after the norm
            _, mag = P.rope_parts(P.store_values(x, w, 1e-5, None, None, 0, True)[0], pos.tolist(), f.cpu(), off, inter)
        keep = slots >= 0
        at = (slots[keep].long()[:, None] * H + torch.arange(H)).reshape(-1)
        check_rows(fmt, cache, scales, at, v[keep].reshape(-1, D), mag[keep].reshape(-1, D), dtype)
        assert int(status) == 0
        left = torch.ones(rows, dtype=torch.bool)
        left[at] = False
        assert bool((raw[left.cuda()] == 0x33).all()), "rows that no slot names"
        assert bool((raw[:, -32:] == 0x33).all()), "bytes between rows"
        if scales is not None:
            assert bool((scales[left.cuda()] == 9.0).all())


MANY_ROWS = [      # format, dim, rot, offset, interleaved, heads, tokens
    ("rows", 128, 64, 0, False, 64, 701), ("rows", 128, 64, 64, True, 5, 9001), ("rows", 512, 64, 0, False, 3, 7001),
    ("plain", 48, 16, 8, False, 7, 9001), ("plain", 512, 64, 448, True, 1, 20011), ("plain", 272, 32, 240, False, 2, 9001),
    ("plain", 512, 512, 0, False, 2, 6001), ("int8", 576, 64, 512, False, 1, 12007), ("fp8", 512, 0, 0, True, 1, 12007),
    ("fp8", 576, 64, 512, True, 1, 12007),
]


@pytest.mark.parametrize("case", MANY_ROWS, ids=str)
def test_store_many_rows_as_in_pieces(case):
    """Rows that one group of lanes works on one after the other hold what they hold when each has its own."""
    fmt, D, rot, off, inter, H, tokens = case
    g = torch.Generator(device="cuda").manual_seed(D + H)
    dtype = torch.bfloat16
    wide = torch.randn(tokens, H + 1, D + 16, generator=g, device="cuda").to(dtype)
    x = wide[:, :H, 8:8 + D]
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g, device="cuda").to(torch.int32)
    f = sfm.rope_frequencies(rot, device="cuda")[0] if rot else None
    w = 1 + 0.2 * torch.randn(min(D, 512), generator=g, device="cuda")
    slots = torch.randperm(tokens, generator=g, device="cuda").to(torch.int32)
    slots[::13] = -1
    rows = (tokens - 5) * H + H // 2                 # a few slots lie outside, one with some of its heads
    got = []
    for piece in (tokens, 97):
        raw, cache = make_cache(fmt, rows, D, dtype, pad=16)
        scales = torch.full((rows,), 9.0, device="cuda") if fmt == "rows" else None
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        for i in range(0, tokens, piece):
            e = min(i + piece, tokens)
            sfm.store_kv(x[i:e], cache, slot_mapping=slots[i:e], kv_format=FORMATS[fmt], norm_weight=w, norm_eps=1e-5,
                         positions=pos[i:e] if rot else None, inv_freq=f, rope_offset=off if rot else None,
                         interleaved=inter, scales=scales, status=status)
        got.append((raw, scales, int(status)))
    (raw, scales, status), (raw1, scales1, status1) = got
    assert status == status1 == sfm.STATUS_BAD_BLOCK
    assert torch.equal(raw, raw1) and (scales is None or torch.equal(scales, scales1))


@pytest.mark.parametrize("fmt,D", [("plain", 512), ("int8", 576), ("fp8", 512), ("rows", 128)])
def test_store_slots_outside_the_cache(fmt, D):
    g = gen(3)
    x = randn(g, 6, 1, D, dtype=torch.bfloat16).cuda()
    raw, cache = make_cache(fmt, 4, D, torch.bfloat16)
    scales = torch.full((4,), 9.0, device="cuda") if fmt == "rows" else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([4, 2, (1 << 31) - 1, -(1 << 31), 0, -1], dtype=torch.int32).cuda()
    sfm.store_kv(x, cache, slot_mapping=slots, kv_format=FORMATS[fmt], scales=scales, status=status)
    assert int(status) == sfm.STATUS_BAD_BLOCK
    check_rows(fmt, cache, scales, torch.tensor([2, 0]), x.cpu()[[1, 4], 0].to(F64), torch.zeros(2, D, dtype=F64), torch.bfloat16)
    assert bool((raw[[1, 3]] == 0x33).all())


@pytest.mark.parametrize("fmt,D,H", [("plain", 128, 4), ("plain", 512, 3), ("int8", 512, 2), ("fp8", 576, 5), ("rows", 128, 64)])
def test_store_writes_all_heads_of_a_token_or_none(fmt, D, H):
    """A cache that ends inside a token's rows: that token is not written, with slots and without."""
    g = gen(13)
    x = randn(g, 3, H, D, dtype=torch.bfloat16)
    rows = 2 * H + H // 2
    for slots in (None, torch.tensor([2, 0, 1], dtype=torch.int32).cuda()):
        raw, cache = make_cache(fmt, rows, D, torch.bfloat16)
        scales = torch.full((rows,), 9.0, device="cuda") if fmt == "rows" else None
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        sfm.store_kv(x.cuda(), cache, slot_mapping=slots, kv_format=FORMATS[fmt], scales=scales, status=status)
        assert int(status) == sfm.STATUS_BAD_BLOCK
        kept = x[:2] if slots is None else x[1:]
        check_rows(fmt, cache, scales, torch.arange(2 * H), kept.reshape(-1, D).to(F64), torch.zeros(2 * H, D, dtype=F64), torch.bfloat16)
        assert bool((raw[2 * H:] == 0x33).all()) and (scales is None or bool((scales[2 * H:] == 9.0).all()))


@pytest.mark.parametrize("fmt", ["int8", "fp8", "rows"])
def test_store_extreme_tiles(fmt):
    """Zero tiles, tiny ones, large ones, and a NaN that spoils its own tile alone."""
    D = 128 if fmt == "rows" else 512
    x = torch.zeros(5, 1, D, dtype=torch.bfloat16)
    x[1, 0, :7] = 2.0 ** -130
    x[2, 0, ::3] = 3e38
    x[2, 0, 1] = -3e38
    x[3, 0] = 1.0
    x[3, 0, 5] = math.nan
    x[4, 0, 9] = math.inf
    raw, cache = make_cache(fmt, 5, D, torch.bfloat16)
    scales = torch.zeros(5, device="cuda") if fmt == "rows" else None
    sfm.store_kv(x.cuda(), cache, kv_format=FORMATS[fmt], scales=scales)
    check_rows(fmt, cache, scales, torch.tensor([0, 1, 2]), x[:3, 0].to(F64), torch.zeros(3, D, dtype=F64), torch.bfloat16)
    got = scales[:, None] if fmt == "rows" else cache[:, -16:].contiguous().view(torch.float32)
    assert bool(got[3, :1].isnan().all()) and bool(got[3, 1:].isfinite().all()) and bool(got[4, :1].isinf().all())
    assert bool((raw[0, :D] == 0).all())


@pytest.mark.parametrize("fmt", ["int8", "fp8", "rows"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_store_codes_are_the_rounded_quotients(fmt, dt):
    """Values that are neither normed nor rotated: scale = max |v| / M and code = v / scale, every operation one rounding
    to nearest with ties to even.  Quotients of 16-bit values meet ties of the codes; no code may be off."""
    D, n = (128, 6000) if fmt == "rows" else (512, 1500)
    tile, most = 128, torch.tensor(127.0 if fmt == "int8" else 448.0)
    dtype = DT[dt]
    x = randn(gen(77), n, D, dtype=dtype)
    lo = -24 if dt == "fp16" else -133
    for r, e in enumerate((1, 0, -3, -9, lo, lo + 3, lo + 7, lo + 12, lo + 20)):      # tiles of other sizes, the smallest among them
        x[r] = (randn(gen(r), D) * 2.0 ** e).to(dtype)
    x[9] = (randn(gen(9), D) * 0.2 * torch.finfo(dtype).max).clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max).to(dtype)
    x[10, 5] = math.inf
    raw, cache = make_cache(fmt, n, D, dtype)
    scales = torch.zeros(n, device="cuda") if fmt == "rows" else None
    sfm.store_kv(x.cuda(), cache, kv_format=FORMATS[fmt], scales=scales)
    v = x.float().view(n, -1, tile)
    scale = (v.abs().amax(-1) / most).clamp(min=P.TINY)
    quotient = v / scale[..., None]
    got = raw[:, :D].cpu()
    finite = quotient.isfinite().view(n, D)
    if fmt == "int8":
        want, got = quotient.nan_to_num().round().to(torch.int8).view(n, D), got.view(torch.int8)
    else:
        want, got = quotient.to(torch.float8_e4m3fn).float().view(n, D), got.view(torch.float8_e4m3fn).float()
    have = scales.cpu()[:, None] if fmt == "rows" else cache[:, -16:].contiguous().view(torch.float32).cpu()
    assert torch.equal(have, scale)
    wrong = (got != want) & finite
    assert not wrong.any(), f"{int(wrong.sum())} of {wrong.numel()} codes"


def test_store_without_tokens_and_noncontiguous_input():
    raw, cache = make_cache("plain", 3, 512, torch.bfloat16)
    sfm.store_kv(torch.empty(0, 512, dtype=torch.bfloat16, device="cuda"), cache)
    assert bool((raw == 0x33).all())
    g = gen(1)
    wide = randn(g, 3, 1024, dtype=torch.bfloat16).cuda()
    sfm.store_kv(wide[:, 512:], cache)
    assert torch.equal(cache, wide[:, 512:])
    with pytest.raises(sfm.SfmError):
        sfm.store_kv(wide[:, 4:516], cache)          # rows off their 16-byte boundaries
    with pytest.raises(ValueError):
        sfm.store_kv(wide[:, ::2], cache)
    with pytest.raises(ValueError):
        sfm.store_kv(wide[:, :512], cache, kv_format=sfm.KV_FP8_ROWS)


# ---------------------------------------------------------------------------
# index scores
# ---------------------------------------------------------------------------
def index_problem(seed, dt, heads, q_lens, lens, layout_q, layout_kv, block=64, ratio=1, pad=0, scales=None):
    """Keys of every sequence, and the same keys in a cache of the layout."""
    g = gen(seed)
    dtype = DT[dt]
    B = len(lens)

    def values(*shape):
        return (randn(g, *shape) * (50 if dt == "fp8" else 1)).clamp(-448, 448).to(dtype)
    keys = [values(n, 128) for n in lens]
    scales = dt == "fp8" if scales is None else scales
    ks = [0.01 + torch.rand(n, generator=g) for n in lens]
    maxk = max(max(lens), 1)
    if layout_kv == "PAGED":
        pages = [-(-n // block) for n in lens]
        total, cols = sum(pages) + 2, max(max(pages), 1)
        perm = torch.randperm(total, generator=g)
        table, pool, pool_s = torch.zeros(B, cols, dtype=torch.int32), torch.full((total * block, 128), math.nan), torch.full((total * block,), math.nan)
        at = 0
        for b, n in enumerate(lens):
            table[b, :pages[b]] = perm[at:at + pages[b]]
            at += pages[b]
            j = torch.arange(n)
            row = table[b].long()[j // block] * block + j % block
            pool[row], pool_s[row] = keys[b].float(), ks[b]
        shape = (total, block)
    elif layout_kv == "TND":
        pool, pool_s, table, shape = torch.cat(keys).float(), torch.cat(ks), None, (sum(lens),)
    else:
        pool, pool_s, table, shape = torch.full((B * maxk, 128), math.nan), torch.full((B * maxk,), math.nan), None, (B, maxk)
        for b, n in enumerate(lens):
            pool[b * maxk:b * maxk + n], pool_s[b * maxk:b * maxk + n] = keys[b].float(), ks[b]
    wide = torch.zeros(pool.shape[0], 128 + pad).to(dtype)
    wide.view(torch.uint8)[:, :128 * wide.element_size()] = pool.to(dtype).view(torch.uint8)
    cache = wide.cuda()[:, :128].unflatten(0, shape)
    S_ = max(q_lens)
    tokens = len(lens) * S_ if layout_q == "BSND" else sum(q_lens)
    q, w = values(tokens, heads, 128), randn(g, tokens, heads)
    first = [b * S_ for b in range(B)] if layout_q == "BSND" else [sum(q_lens[:b]) for b in range(B)]
    rest = [int(torch.randint(0, ratio, (1,), generator=g)) for _ in lens]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32).cuda()
    kw = dict(max_seqlen_kv=maxk, layout_q=layout_q, layout_kv=layout_kv, cmp_ratio=ratio, cmp_residual_kv=ints(rest),
              k_scales=pool_s.cuda().contiguous() if scales else None)
    if layout_kv == "PAGED":
        kw.update(block_table=table.cuda(), seqused_kv=ints(lens))
    elif layout_kv == "TND":
        kw.update(cu_seqlens_kv=ints([sum(lens[:b]) for b in range(B + 1)]))
    else:
        kw.update(seqused_kv=ints(lens))
    if layout_q == "TND":
        kw.update(cu_seqlens_q=ints([sum(q_lens[:b]) for b in range(B + 1)]), max_seqlen_q=S_)
    qd = q.cuda().view(B, S_, heads, 128) if layout_q == "BSND" else q.cuda()
    wd = w.cuda().view(B, S_, heads) if layout_q == "BSND" else w.cuda()
    return dict(q=q, w=w, keys=keys, ks=ks if scales else [None] * B, first=first, rest=rest, kw=kw, qd=qd, wd=wd,
                cache=cache, tokens=tokens, maxk=maxk, S=S_)


def check_scores(p, q_lens, lens, ratio, causal, got, seen, used_q=None):
    got, seen = got.cpu(), seen.cpu()
    for b, n in enumerate(lens):
        ql = used_q[b] if used_q else q_lens[b]
        vis = P.visible(ql, n, ratio, p["rest"][b], causal)
        t0 = p["first"][b]
        rows = p["S"] if p["kw"]["layout_q"] == "BSND" else q_lens[b]
        assert seen[t0:t0 + rows].tolist() == vis + [0] * (rows - ql), f"sequence {b}"
        want, mag = P.scores(p["q"][t0:t0 + ql], p["keys"][b], p["w"][t0:t0 + ql], p["ks"][b])
        block = got[t0:t0 + rows]
        shown = torch.arange(p["maxk"])[None] < torch.tensor(vis + [0] * (rows - ql))[:, None]
        assert bool(torch.isneginf(block[~shown]).all()), f"sequence {b}: hidden keys"
        if ql and n:
            s = shown[:ql, :n]
            assert_within(block[:ql, :n][s], want[s], SCORE_TOL * mag[s] + 1e-30, f"sequence {b}")


INDEX_CASES = [   # dtype, heads, q_lens, key counts, layouts, block, ratio
    ("bf16", 64, [1, 1, 1], [1, 127, 300], "BSND", "PAGED", 64, 1), ("fp8", 64, [1, 1], [1000, 129], "BSND", "PAGED", 128, 4),
    ("fp16", 64, [5, 5], [700, 64], "BSND", "PAGED", 16, 4), ("bf16", 1, [3], [200], "BSND", "PAGED", 48, 1),
    ("bf16", 5, [40], [260], "TND", "PAGED", 1024, 1), ("fp8", 16, [33, 1, 0, 7], [130, 50, 9, 0], "TND", "PAGED", 32, 1),
    ("bf16", 24, [9, 2], [300, 128], "TND", "TND", 0, 1), ("fp16", 32, [17, 17], [256, 77], "BSND", "BSND", 0, 2),
    ("bf16", 100, [3, 1], [400, 33], "TND", "PAGED", 64, 4), ("fp8", 128, [7], [513], "BSND", "PAGED", 64, 1),
    ("bf16", 128, [1, 1], [640, 250], "BSND", "PAGED", 128, 1), ("bf16", 128, [2, 2], [140, 250], "BSND", "PAGED", 128, 1),
    ("bf16", 64, [130], [1500], "TND", "TND", 0, 1), ("fp8", 33, [4], [90], "BSND", "BSND", 0, 1),
    ("bf16", 8, [16], [385], "BSND", "PAGED", 80, 1), ("fp16", 64, [2, 2], [5000, 129], "BSND", "PAGED", 64, 4),
    # enough work that a unit holds several tiles of keys
    ("fp8", 64, [96, 96, 96], [5000, 4100, 7000], "TND", "PAGED", 32, 1), ("bf16", 64, [200], [6001], "BSND", "PAGED", 128, 1),
    ("fp8", 16, [1] * 48, [6000 - 50 * b for b in range(48)], "BSND", "PAGED", 128, 4),
    ("bf16", 128, [1] * 30, [8000 - 99 * b for b in range(30)], "BSND", "PAGED", 16, 1),
    # sequences without keys among long ones, and more groups of queries than are shared out equally
    ("bf16", 16, [1] * 40, [0 if b % 3 else 3000 * (b % 2) + b for b in range(40)], "TND", "PAGED", 64, 1),
    ("fp8", 8, [1] * 1100, [5000 if b in (7, 1050) else b % 60 for b in range(1100)], "BSND", "PAGED", 64, 1),
]


@pytest.mark.parametrize("case", INDEX_CASES, ids=lambda c: f"{c[0]}-{c[1]}-{max(c[2])}x{len(c[2])}-{max(c[3])}-{c[4]}-{c[5]}-{c[6]}-{c[7]}")
@pytest.mark.parametrize("mask", [3, 0])
def test_index_scores(case, mask):
    dt, heads, q_lens, lens, lq, lkv, block, ratio = case
    p = index_problem(17 + heads, dt, heads, q_lens, lens, lq, lkv, block, ratio)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, seen = sfm.index_scores(p["qd"], p["cache"], p["wd"], mask_mode=mask, status=status, **p["kw"])
    torch.cuda.synchronize()
    assert int(status) == 0
    check_scores(p, q_lens, lens, ratio, mask == 3, got, seen)
    again, _ = sfm.index_scores(p["qd"], p["cache"], p["wd"], mask_mode=mask, **p["kw"])
    assert torch.equal(got, again)


def test_index_scores_of_quantised_queries():
    """Queries that store_kv wrote as E4M3 rows: their scales, multiplied into the weights, give the scores of the values."""
    p = index_problem(8, "fp8", 16, [3, 3], [300, 40], "BSND", "PAGED", 64)
    x = randn(gen(8), 6 * 16, 128, dtype=torch.bfloat16) * 3
    codes = torch.zeros(6 * 16, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    qs = torch.zeros(6 * 16, device="cuda")
    sfm.store_kv(x.cuda(), codes, kv_format=sfm.KV_FP8_ROWS, scales=qs)
    got, seen = sfm.index_scores(codes.view(2, 3, 16, 128), p["cache"], p["wd"] * qs.view(2, 3, 16), **p["kw"])
    p["q"] = (codes.float().cpu().to(F64) * qs.cpu().to(F64)[:, None]).view(6, 16, 128)
    check_scores(p, [3, 3], [300, 40], 1, True, got, seen)


def test_index_scores_padded_rows_strided_output_and_used_queries():
    for dt, scales in (("bf16", True), ("fp8", False)):
        p = index_problem(3, dt, 64, [6, 6], [300, 40], "BSND", "PAGED", 64, 1, pad=16, scales=scales)
        used = [4, 0]
        wide = torch.full((12, p["maxk"] + 7), 5.0, device="cuda")
        got, seen = sfm.index_scores(p["qd"], p["cache"], p["wd"], out=wide[:, :p["maxk"]],
                                     seqused_q=torch.tensor(used, dtype=torch.int32).cuda(), **p["kw"])
        check_scores(p, [6, 6], [300, 40], 1, True, got, seen, used)
        assert bool((wide[:, p["maxk"]:] == 5.0).all())


def test_index_scores_rows_behind_the_last_sequence_stay():
    p = index_problem(4, "bf16", 16, [5, 3], [70, 30], "TND", "PAGED", 16)
    q = torch.cat((p["qd"], p["qd"][:4]))
    w = torch.cat((p["wd"], p["wd"][:4]))
    out = torch.full((12, p["maxk"]), 5.0, device="cuda")
    vis = torch.full((12,), -9, dtype=torch.int32, device="cuda")
    sfm.index_scores(q, p["cache"], w, out=out, visible=vis, **p["kw"])
    check_scores(p, [5, 3], [70, 30], 1, True, out[:8], vis[:8])
    assert bool((out[8:] == 5.0).all()) and vis[8:].tolist() == [-9] * 4


def test_index_scores_padding_behind_the_last_sequence_selects_nothing():
    p = index_problem(4, "bf16", 16, [5, 3], [70, 30], "TND", "PAGED", 16)
    q = torch.cat((p["qd"], p["qd"][:4]))
    w = torch.cat((p["wd"], p["wd"][:4]))
    for junk in (-9, 1 << 20, 7):                    # what the allocator's last owner left
        rest = torch.full((12,), junk, dtype=torch.int32, device="cuda")
        del rest
        scores, seen = sfm.index_scores(q, p["cache"], w, **p["kw"])
        check_scores(p, [5, 3], [70, 30], 1, True, scores[:8], seen[:8])
        assert seen[8:].tolist() == [0] * 4
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        picked = sfm.select_topk(scores, 6, lengths=seen, status=status)
        assert int(status) == 0 and bool((picked[8:] == -1).all()) and bool((picked[:8, 0] >= 0).all())


@pytest.mark.parametrize("heads", [8, 64, 128])
def test_index_scores_take_any_bound_on_ragged_queries(heads):
    """max_seqlen_q of a ragged batch is an upper bound: loose ones, up to the largest there is, change nothing."""
    q_lens, lens = [5, 3, 0, 21], [70, 300, 9, 140]
    p = index_problem(4, "bf16", heads, q_lens, lens, "TND", "PAGED", 16)
    want, seen = sfm.index_scores(p["qd"], p["cache"], p["wd"], **p["kw"])
    check_scores(p, q_lens, lens, 1, True, want, seen)
    for bound in (29, 100, 1 << 20, (1 << 31) - 8, (1 << 31) - 1):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got, seen = sfm.index_scores(p["qd"], p["cache"], p["wd"], status=status, **{**p["kw"], "max_seqlen_q": bound})
        check_scores(p, q_lens, lens, 1, True, got, seen)
        assert torch.equal(got, want) and int(status) == 0


def test_index_scores_bad_blocks_and_lengths():
    p = index_problem(5, "bf16", 64, [1, 1], [300, 200], "BSND", "PAGED", 64)
    p["kw"]["block_table"][0, 2] = 1 << 20
    p["kw"]["block_table"][1, 0] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, seen = sfm.index_scores(p["qd"], p["cache"], p["wd"], status=status, **p["kw"])
    assert int(status) == sfm.STATUS_BAD_BLOCK and seen.tolist() == [300, 200]
    want, mag = P.scores(p["q"], p["keys"][0], p["w"])
    lost = (torch.arange(300) // 64) == 2
    assert bool(torch.isneginf(got[0, :300].cpu()[lost]).all())
    assert_within(got[0, :300].cpu()[~lost], want[0][~lost], SCORE_TOL * mag[0][~lost])
    assert bool(torch.isneginf(got[1, :64]).all()) and bool(torch.isfinite(got[1, 64:200]).all())
    p = index_problem(5, "bf16", 64, [1, 1], [300, 200], "BSND", "PAGED", 64)
    p["kw"]["seqused_kv"][1] = 5000
    status.zero_()
    _, seen = sfm.index_scores(p["qd"], p["cache"], p["wd"], status=status, **p["kw"])
    assert int(status) & sfm.STATUS_BAD_LENGTH and seen.tolist() == [300, 300]


def test_index_scores_keep_nan_and_infinities_where_they_are():
    p = index_problem(6, "bf16", 64, [2], [300], "BSND", "BSND")
    clean, _ = sfm.index_scores(p["qd"], p["cache"], p["wd"], **p["kw"])
    dirty = p["cache"].clone()
    dirty[0, 7, 3] = math.nan
    dirty[0, 200, 5] = math.inf
    got, _ = sfm.index_scores(p["qd"], dirty, p["wd"], **p["kw"])
    assert bool(got[:, 7].isnan().all()) and bool((~got[:, 200].isfinite()).all())
    keep = torch.ones(300, dtype=torch.bool)
    keep[[7, 200]] = False
    assert torch.equal(got[:, keep.cuda()], clean[:, keep.cuda()])


@pytest.mark.parametrize("heads", [1, 5, 16, 24, 33, 64, 100, 128])
def test_index_scores_of_infinite_keys(heads):
    """A key's infinity meets the heads that are there and nothing else."""
    p = index_problem(7, "bf16", heads, [2, 2], [300, 140], "BSND", "BSND")
    w = p["wd"].abs() + 0.25
    keys = p["cache"].clone()
    for j, d, v in ((3, 5, math.inf), (130, 127, -math.inf), (139, 0, math.inf)):
        keys[:, j, d] = v
    got, _ = sfm.index_scores(p["qd"], keys, w, mask_mode=0, **p["kw"])
    for b, n in enumerate([300, 140]):
        t0 = p["first"][b]
        want, _ = P.scores(p["q"][t0:t0 + 2], keys[b, :n].cpu(), w[b].cpu(), p["ks"][b])
        have = got[t0:t0 + 2, :n].cpu()
        assert torch.equal(have.isnan(), want.isnan()) and torch.equal(have.isinf(), want.isinf())


# ---------------------------------------------------------------------------
# selection
# ---------------------------------------------------------------------------
def topk_check(x, k, lengths=None, **kw):
    got = sfm.select_topk(x, k, lengths=lengths, **kw).cpu()
    host = x.cpu().tolist()
    ends = lengths.cpu().tolist() if lengths is not None else [x.shape[1]] * len(host)
    for r, row in enumerate(host):
        want = P.topk(row, k, ends[r], kw.get("block_size", 1), kw.get("first_blocks", 0), kw.get("last_blocks", 0))
        assert got[r].tolist() == want, f"row {r}"


@pytest.mark.parametrize("n", [1, 31, 32, 100, 1000, 4097, 20001])
@pytest.mark.parametrize("k", [1, 8, 512, 2048])
def test_topk(n, k):
    g = gen(n + k)
    x = torch.stack([randn(g, n), (randn(g, n) + 1).relu(), (randn(g, n) * 3).round(), torch.zeros(n),
                     torch.where(torch.rand(n, generator=g) < 0.9, -math.inf, randn(g, n))]).cuda()
    topk_check(x, k)
    topk_check(x, k, torch.tensor([n, n // 2, 0, 1, n - n // 3], dtype=torch.int32).cuda())


def test_topk_special_values():
    inf, nan, low = math.inf, math.nan, torch.finfo(torch.float32).min
    rows = [[nan, 1.0, -inf, 2.0, nan, inf], [-inf] * 6, [nan] * 6, [low, -inf, low, 0.0, -0.0, 1e-45], [-0.0, 0.0, -0.0, 0.0, -1e-45, nan],
            [inf, inf, -1.0, inf, inf, inf]]
    x = torch.tensor(rows).cuda()
    for k in (1, 2, 3, 4, 6, 9):
        topk_check(x, k)


@pytest.mark.parametrize("block", [2, 4, 16, 64, 128])
@pytest.mark.parametrize("n", [1, 130, 1000, 9001])
def test_topk_blocks(block, n):
    g = gen(n + block)
    x = torch.stack([randn(g, n), (randn(g, n) * 2).round(), torch.full((n,), -math.inf), randn(g, n)]).cuda()
    x[3, ::2] = math.nan
    lengths = torch.tensor([n, max(n - 5, 0), n, n // 2], dtype=torch.int32).cuda()
    for k, first, last in ((1, 0, 0), (8, 1, 2), (40, 0, 3), (3, 3, 0), (4, 2, 2)):
        topk_check(x, k, None, block_size=block, first_blocks=first, last_blocks=last)
        topk_check(x, k, lengths, block_size=block, first_blocks=first, last_blocks=last)


def test_topk_strided_rows_and_bad_lengths():
    g = gen(8)
    wide = randn(g, 5, 1003).cuda()
    topk_check(wide[:, 1:1000], 100)
    topk_check(wide[::2, :997], 100)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lengths = torch.tensor([-3, 2000, 5, 0, 1003], dtype=torch.int32).cuda()
    got = sfm.select_topk(wide, 4, lengths=lengths, status=status)
    assert int(status) == sfm.STATUS_BAD_LENGTH
    for r, n in enumerate([0, 1003, 5, 0, 1003]):
        assert got[r].tolist() == P.topk(wide[r].tolist(), 4, n)


@pytest.mark.parametrize("rows,n,k", [(1, 300001, 2048), (2, 900003, 1000), (400, 5000, 64), (1, 60000, 60001)])
def test_topk_long_and_many_rows(rows, n, k):
    g = torch.Generator(device="cuda").manual_seed(n)
    x = (torch.randn(rows, n, generator=g, device="cuda") * 50).round() / 8         # many equal values
    got = sfm.select_topk(x, k)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k].sort(1).values.to(torch.int32)
    assert torch.equal(got[:, :min(k, n)], order) and bool((got[:, n:] == -1).all())


@pytest.mark.parametrize("rows,n,k", [(5, 8192, 512), (300, 8191, 1000), (2, 70001, 64), (1, 200003, 2048), (3, 20000, 8)])
def test_topk_rows_that_mislead_a_sample(rows, n, k):
    """Orders and repetitions in which no part of a row is like the whole."""
    g = torch.Generator(device="cuda").manual_seed(n)
    r = torch.randn(rows, n, generator=g, device="cuda")
    j = torch.arange(n, device="cuda").expand(rows, n)
    cases = [r.sort(1).values, r.sort(1, descending=True).values, torch.where((j // 4) % 32 == 0, r, r - 10),
             torch.where((j // 4) % 32 == 0, r - 10, r), torch.where(j > n - 2 * k, r + 10, r),
             torch.where(j % 1000 == 0, math.inf, r), torch.where(j < n // 2, math.nan, r), torch.zeros_like(r),
             (r > 1).float(), torch.where(j < k + 1, r, -math.inf), torch.where(j < k - 1, r, -math.inf), -r.abs() * 1e38]
    lengths = torch.full((rows,), n, dtype=torch.int32, device="cuda")
    lengths[0] = n - n // 3
    for x in cases:
        for kw in (dict(), dict(lengths=lengths), dict(lengths=lengths, first_blocks=3, last_blocks=5)):
            got = sfm.select_topk(x, k, **kw)
            y = x.double().nan_to_num(nan=-math.inf, posinf=1e300, neginf=-math.inf)
            ends = lengths[:, None] if "lengths" in kw else n
            y = torch.where(j < ends, y, -math.inf)
            if "first_blocks" in kw:
                y = torch.where((j < ends) & ((j < 3) | (j >= ends - 5)), math.inf, y)
            best = torch.sort(y, dim=1, descending=True, stable=True)
            want = torch.where(best.values[:, :k] > -math.inf, best.indices[:, :k], n).sort(1).values
            assert torch.equal(got, torch.where(want < n, want, -1).to(torch.int32))


@pytest.mark.parametrize("n", [16385, 20003, 65536, 131075])
@pytest.mark.parametrize("k,first,last", [(1, 0, 0), (2048, 0, 0), (300, 2, 5), (60, 20, 40)])
def test_topk_many_long_rows(n, k, first, last):
    """Rows that are longer than a CTA's share and as many as there are SMs."""
    g = torch.Generator(device="cuda").manual_seed(n + k)
    rows = 160
    x = torch.randn(rows, n + 3, generator=g, device="cuda")[:, :n]
    x[1::4] = (x[1::4] * 2).round()
    x[2::8] = 0.25
    x[3::8, :n // 2] = -math.inf
    x[5::16, 7::3] = math.nan
    x[6::16] += 1e6
    lengths = torch.randint(0, n + 1, (rows,), generator=g, device="cuda").to(torch.int32)
    lengths[:8] = torch.tensor([0, 1, 2, 3, 511, 513, n - 1, n], dtype=torch.int32)
    j = torch.arange(n, device="cuda")
    for y in (x, x.contiguous()):
        for ends in (lengths, None):
            got = sfm.select_topk(y, k, lengths=ends, first_blocks=first, last_blocks=last)
            e = lengths[:, None] if ends is not None else torch.full((rows, 1), n, device="cuda")
            v = y.double().nan_to_num(nan=-math.inf, posinf=1e300, neginf=-math.inf)
            v = torch.where(j < e, v, -math.inf)
            v = torch.where((j < e) & ((j < first) | (j >= e - last)), math.inf, v)
            best = torch.sort(v, dim=1, descending=True, stable=True)
            want = torch.where(best.values[:, :k] > -math.inf, best.indices[:, :k], n).sort(1).values
            assert torch.equal(got, torch.where(want < n, want, -1).to(torch.int32))


# rows, scores, block: one to sixteen CTAs per row with 128 to 1024 threads each, and rows that no cluster holds
@pytest.mark.parametrize("rows,n,block", [
    (1, 131072, 64), (1, 300001, 4), (2, 600000, 16), (1, 600003, 64), (3, 524288, 128), (2, 100003, 2), (70, 60001, 2), (70, 70000, 4),
    (100, 100001, 2), (9, 200004, 16), (1, 1400001, 2), (2, 2700004, 4)])
def test_topk_blocks_of_long_rows(rows, n, block):
    g = torch.Generator(device="cuda").manual_seed(n)
    wide = torch.randn(rows, n + 3, generator=g, device="cuda")
    wide[0] = (wide[0] * 2).round()
    wide[-1, ::5] = math.nan
    wide[rows // 2, n // 3:n // 2] = -math.inf
    x = wide[:, :n]
    blocks, j = -(-n // block), torch.arange(n, device="cuda")
    each = torch.arange(blocks, device="cuda")
    ends = [n, 0, 1, block, n // 2 + 1, n // 16 // block * block + 3, n - 1, n - n // 5]     # some CTAs get a part, some nothing
    plans = [None] + [torch.tensor([ends[(r + i) % len(ends)] for r in range(rows)], dtype=torch.int32, device="cuda")
                      for i in range(len(ends) if rows < len(ends) else 1)]
    for y in (x.contiguous(), x):                    # rows on 16-byte boundaries (where n allows it) and off them
        for lengths in plans:
            e = lengths[:, None].long() if lengths is not None else torch.full((rows, 1), n, device="cuda")
            v = torch.where(j < e, y.double().nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf), -math.inf)
            v = torch.nn.functional.pad(v, (0, blocks * block - n), value=-math.inf).view(rows, blocks, block).amax(-1)
            have = -(-e // block)
            for k, first, last in ((31, 0, 0), (500, 1, 2), (1000, 300, 40)):
                got = sfm.select_topk(y, k, lengths=lengths, block_size=block, first_blocks=first, last_blocks=last)
                w = torch.where((each < have) & ((each < first) | (each >= have - last)), math.inf, v)
                best = torch.sort(w, dim=1, descending=True, stable=True)
                want = torch.where(best.values[:, :k] > -math.inf, best.indices[:, :k], blocks).sort(1).values
                assert torch.equal(got, torch.where(want < blocks, want, -1).to(torch.int32))


@pytest.mark.parametrize("n", [700, 9001, 70001])
@pytest.mark.parametrize("k,first,last", [(1, 0, 0), (8, 3, 5), (1, 0, 1), (700, 1, 2), (64, 40, 0), (600, 300, 300)])
def test_topk_short_lengths_in_long_rows(n, k, first, last):
    """Lengths that leave a part of a row's share-out with nothing, or with one to three scores."""
    ends = [e for e in (0, 1, 2, 3, 5, 127, 129, 700, 1923, 6273, 6274, 6275, 28801, 28802, 28803, 70001) if e <= n]
    g = gen(n + k)
    x = torch.stack([randn(g, n) for _ in ends]).cuda()
    x[1::2] = (x[1::2] * 2).round()
    lengths = torch.tensor(ends, dtype=torch.int32).cuda()
    topk_check(x, k, lengths, first_blocks=first, last_blocks=last)
    for r in range(len(ends)):
        topk_check(x[r:r + 1], k, lengths[r:r + 1], first_blocks=first, last_blocks=last)


def test_arguments_that_are_no_tensors_are_refused():
    """... by name, whatever they are instead."""
    x = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    pos, lens = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.full((1,), 8, dtype=torch.int32, device="cuda")
    f, cu = torch.zeros(8, dtype=F64, device="cuda"), torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    w, keys = torch.zeros(2, 4, device="cuda"), torch.zeros(2, 16, 128, dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros(8, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    cache = torch.zeros(8, 128, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")

    def rope(**kw):
        sfm.apply_rope(**{**dict(x=x, positions=pos, inv_freq=f), **kw})

    def store(**kw):
        sfm.store_kv(**{**dict(x=x, cache=cache, positions=pos, inv_freq=f), **kw})

    def rows(**kw):
        sfm.store_kv(**{**dict(x=x, cache=codes, kv_format=sfm.KV_FP8_ROWS), **kw})

    def scores(**kw):
        sfm.index_scores(**{**dict(q=x, index_k=keys, weights=w, max_seqlen_kv=16, max_seqlen_q=2, cu_seqlens_q=cu, seqused_kv=lens,
                                   block_table=table, layout_q="TND", layout_kv="PAGED"), **kw})

    def topk(**kw):
        sfm.select_topk(**{**dict(scores=w, k=2), **kw})
    rope(), store(), rows(scales=torch.zeros(8, device="cuda")), scores(), topk()
    for call, names in ((rope, ("x", "positions", "inv_freq", "out")), (store, ("x", "cache", "positions", "inv_freq", "slot_mapping", "status")),
                        (rows, ("scales",)), (topk, ("scores", "lengths", "out", "status")),
                        (scores, ("q", "index_k", "weights", "k_scales", "block_table", "cu_seqlens_q", "seqused_kv", "seqused_q",
                                  "cmp_residual_kv", "out", "visible", "status"))):
        for name in names:
            for other in ([0, 1], 3.5, "x"):
                with pytest.raises(ValueError, match=name):
                    call(**{name: other})


# ---------------------------------------------------------------------------
# calls behind each other: a kernel may be set up while the one before it runs
# ---------------------------------------------------------------------------
def test_calls_read_what_the_calls_before_them_wrote():
    """Every call's inputs are the outputs of the calls right before it; the same buffers hold other values each time."""
    g = torch.Generator(device="cuda").manual_seed(31)
    B, n, D, heads, block, k = 8, 700, 128, 64, 64, 96
    f, _ = sfm.rope_frequencies(64, device="cuda")
    x = torch.randn(B * n, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    q0 = torch.randn(B, heads, D, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.rand(B, heads, generator=g, device="cuda")
    pos = torch.arange(B * n, dtype=torch.int32, device="cuda")
    ones = torch.ones(B, dtype=torch.int32, device="cuda")
    pages = -(-n // block)
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
    slots = (torch.arange(B * n, device="cuda") // n * pages * block + torch.arange(B * n, device="cuda") % n).to(torch.int32)

    def run(between):
        rows, queries = x.clone(), q0.clone()
        cache = torch.zeros(B * pages, block, D, dtype=torch.bfloat16, device="cuda")
        out = torch.zeros(B, n, device="cuda")
        seen = torch.zeros(B, dtype=torch.int32, device="cuda")
        lens = torch.full((B,), n - 40, dtype=torch.int32, device="cuda")
        picked = torch.zeros(B, k, dtype=torch.int32, device="cuda")
        past = []
        torch.cuda.synchronize()
        for i in range(24):
            sfm.apply_rope(rows, pos, f, out=rows, interleaved=i % 2 == 0)
            between()
            sfm.store_kv(rows[:, 0], cache, slot_mapping=slots)
            between()
            sfm.apply_rope(queries, lens, f, out=queries, inverse=i % 3 == 0)
            between()
            sfm.index_scores(queries.view(B, 1, heads, D), cache, w.view(B, 1, heads), max_seqlen_kv=n, block_table=table,
                             seqused_kv=lens, layout_kv="PAGED", out=out, visible=seen)
            between()
            sfm.select_topk(out, k, lengths=seen, out=picked)
            between()
            sfm.index_scores(queries.view(B, 1, heads, D), cache, w.view(B, 1, heads), max_seqlen_kv=n, block_table=table,
                             seqused_kv=seen, layout_kv="PAGED", out=out, visible=lens)
            between()
            lens.add_(ones)
            between()
            past.append(picked.clone())
        torch.cuda.synchronize()
        return [rows, queries, cache, out, seen, lens, torch.stack(past)]
    apart = run(torch.cuda.synchronize)
    for _ in range(3):
        for a, b in zip(run(lambda: None), apart):
            assert torch.equal(a, b)


@pytest.mark.parametrize("batch", [6, 200], ids=["small planner", "large planner"])
def test_plans_read_the_lengths_the_call_before_them_wrote(batch):
    """`visible` of the index scores is a length tensor of the plan right behind them, eager and captured: the plan reads
    lengths before it waits for the kernel before it.  Each round's scores see one key less, or all again."""
    g = torch.Generator(device="cuda").manual_seed(batch)
    n, heads = 900, 16
    q = torch.randn(batch, 1, heads, 128, generator=g, device="cuda").to(torch.bfloat16)
    keys = torch.randn(batch, n, 128, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.rand(batch, 1, heads, generator=g, device="cuda")
    out, seen = torch.zeros(batch, n, device="cuda"), torch.zeros(batch, dtype=torch.int32, device="cuda")
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    first = torch.randint(1, n + 1, (batch,), generator=g, device="cuda").to(torch.int32)

    params = sfm.make_params(num_heads_q=64, batch_size=batch, max_seqlen_q=1, max_seqlen_ori_kv=n, ori_mask_mode=3)
    tensors = sfm.make_tensors(None, None, seqused_ori_kv=seen, ori_row_stride=0)
    words = sfm.sfm_metadata_size(params)

    def score():
        sfm.index_scores(q, keys, w, max_seqlen_kv=n, seqused_kv=lens, out=out, visible=seen)

    def run(between):
        lens.copy_(first)
        plans = [torch.zeros(words, dtype=torch.int32, device="cuda") for _ in range(12)]
        torch.cuda.synchronize()
        for p in plans:
            score()
            between()
            sfm.sfm_metadata(params, tensors, p)
            between()
            lens.sub_(1).clamp_(min=0)
        torch.cuda.synchronize()
        return torch.stack(plans)
    apart = run(torch.cuda.synchronize)
    assert not torch.equal(apart[0], apart[1])
    for _ in range(3):
        assert torch.equal(run(lambda: None), apart)
    planned = torch.zeros(words, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        score()
        sfm.sfm_metadata(params, tensors, planned)
    lens.copy_(first)
    for i in range(12):
        planned.zero_()
        graph.replay()
        assert torch.equal(planned, apart[i])
        lens.sub_(1).clamp_(min=0)


# ---------------------------------------------------------------------------
# offsets past 32 bits
# ---------------------------------------------------------------------------
def test_far_offsets():
    """Rows whose elements lie more than 2^32 bytes (and 2^31 elements) from the start of their tensors."""
    g = gen(11)
    far = torch.empty((1 << 31) + (1 << 20), dtype=torch.bfloat16, device="cuda")
    x = far.as_strided((2, 3, 128), ((1 << 31), 128, 1))
    x.copy_(randn(g, 2, 3, 128, dtype=torch.bfloat16))
    pos = torch.tensor([5, 70000], dtype=torch.int32)
    f, _ = sfm.rope_frequencies(64, device="cuda")
    for inter in (True, False):
        y = sfm.apply_rope(x, pos.cuda(), f, interleaved=inter)
        rope_check(y, x, pos, f, 0, inter, False, 1.0)
    rows = (1 << 32) // 1024 + 100
    cache = far[:rows * 512].view(rows, 512)
    values = randn(g, 2, 512, dtype=torch.bfloat16).cuda()
    slots = torch.tensor([rows - 1, 3], dtype=torch.int32).cuda()
    sfm.store_kv(values, cache, slot_mapping=slots)
    assert torch.equal(cache[rows - 1], values[0]) and torch.equal(cache[3], values[1])
    # index keys at the end of a pool of more than 2^32 bytes, scores in rows 2^31 elements apart
    blocks = (1 << 32) // (256 * 64) + 8
    pool = far[:blocks * 64 * 128].view(blocks, 64, 128)
    k, q, w = randn(g, 100, 128, dtype=torch.bfloat16), randn(g, 2, 16, 128, dtype=torch.bfloat16), randn(g, 2, 16)
    pool[blocks - 1] = k[:64].cuda()
    pool[blocks - 2, :36] = k[64:].cuda()
    wide = torch.empty((1 << 31) + 256, device="cuda")
    out = wide.as_strided((2, 100), (1 << 31, 1))
    sfm.index_scores(q.cuda().view(1, 2, 16, 128), pool, w.cuda().view(1, 2, 16), max_seqlen_kv=100, layout_kv="PAGED", mask_mode=0,
                     block_table=torch.tensor([[blocks - 1, blocks - 2]], dtype=torch.int32).cuda(),
                     seqused_kv=torch.tensor([100], dtype=torch.int32).cuda(), out=out)
    want, mag = P.scores(q, k, w)
    assert_within(out, want, SCORE_TOL * mag)
    host = out.cpu().tolist()
    got = sfm.select_topk(out, 10).tolist()
    assert got == [P.topk(host[r], 10, 100) for r in range(2)]


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def _slots(table, block, b, n):
    j = torch.arange(n, device="cuda")
    return (table[b].long()[j // block] * block + j % block).to(torch.int32)


def together(packed):
    """One decode step of a small batch through every operator into the
    attention; returns the problem as the attention saw it, and its output."""
    prob = S.build("together", seed=5, device="cuda", q_n=16, q_lens=[2, 2], kv_lens=[1003, 1500], layout_q="BSND",
                   layout_kv="PAGED", mode="ori_sparse" if packed else "csa", cmp_ratio=1 if packed else 4,
                   cmp_topk=0 if packed else 32, ori_topk=64 if packed else 0, win_left=63,
                   kv_format="fp8_packed" if packed else "plain", rope_head_dim=64 if packed else 0, sinks=not packed)
    t, g = prob.t, gen(1)
    which = "ori" if packed else "cmp"
    f, _ = sfm.rope_frequencies(64, device="cuda")
    lens = [1003, 1500] if packed else [1003 // 4, 1500 // 4]
    table, block = t[f"{which}_block_table"], 128
    dim = 576 if packed else 512
    for b, n in enumerate([1003, 1500]):
        x = randn(g, n, dim, dtype=torch.bfloat16).cuda()
        sfm.store_kv(x, t["ori_kv"].view(-1, t["ori_kv"].shape[-1]), slot_mapping=_slots(t["ori_block_table"], 128, b, n),
                     kv_format=sfm.KV_FP8_PACKED if packed else sfm.KV_PLAIN, norm_eps=1e-6,
                     positions=torch.arange(n, dtype=torch.int32, device="cuda"), inv_freq=f)
    if not packed:
        for b, n in enumerate(lens):
            sfm.store_kv(randn(g, n, 512, dtype=torch.bfloat16).cuda(), t["cmp_kv"].view(-1, 512),
                         slot_mapping=_slots(table, block, b, n), norm_eps=1e-6, inv_freq=f,
                         positions=torch.arange(0, 4 * n, 4, dtype=torch.int32, device="cuda"))
    rows = (int(table.max()) + 1) * block
    keys = torch.zeros(rows, 128, dtype=torch.float8_e4m3fn, device="cuda")
    ks = torch.zeros(rows, device="cuda")
    for b, n in enumerate(lens):
        sfm.store_kv(randn(g, n, 128, dtype=torch.bfloat16).cuda(), keys, slot_mapping=_slots(table, block, b, n),
                     kv_format=sfm.KV_FP8_ROWS, scales=ks)
    pos = torch.tensor([1001, 1002, 1498, 1499], dtype=torch.int32, device="cuda")
    t["q"].copy_(sfm.apply_rope(t["q"], pos, f, rope_offset=dim - 64))
    iq = torch.zeros(4 * 8, 128, dtype=torch.float8_e4m3fn, device="cuda")
    iqs = torch.zeros(4 * 8, device="cuda")
    sfm.store_kv(randn(g, 4, 8, 128, dtype=torch.bfloat16).cuda(), iq, kv_format=sfm.KV_FP8_ROWS, scales=iqs, positions=pos,
                 inv_freq=f, rope_offset=0, interleaved=False)
    w = torch.rand(4, 8, generator=g).cuda() * iqs.view(4, 8)
    state = dict(iq=iq.view(2, 2, 8, 128), w=w.view(2, 2, 8), keys=keys.view(-1, block, 128), ks=ks, table=table,
                 seqused_kv=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 rest=torch.tensor([1003 % 4, 1500 % 4] if not packed else [0, 0], dtype=torch.int32, device="cuda"),
                 k=64 if packed else 32, ratio=1 if packed else 4, name=f"{which}_sparse_indices", maxk=max(lens))
    return prob, state


def select(state, out=None):
    scores, seen = sfm.index_scores(state["iq"], state["keys"], state["w"], max_seqlen_kv=state["maxk"], k_scales=state["ks"],
                                    block_table=state["table"], seqused_kv=state["seqused_kv"],
                                    cmp_residual_kv=state["rest"], cmp_ratio=state["ratio"], layout_kv="PAGED")
    return scores, seen, sfm.select_topk(scores, state["k"], lengths=seen, out=out)


@pytest.mark.parametrize("packed", [False, True], ids=["csa", "packed"])
def test_operators_feed_the_attention(packed):
    prob, state = together(packed)
    scores, seen, picked = select(state)
    host = scores.cpu().tolist()
    for r in range(4):
        assert picked[r].tolist() == P.topk(host[r], state["k"], int(seen[r]))
    prob.t[state["name"]] = picked.view(2, 2, 1, state["k"])
    out, lse, status = _sfm.run(prob)
    assert status == 0
    O, L = oracle.forward(prob.to("cpu"))
    got = out.reshape(O.shape).float().cpu().numpy()
    assert (abs(got - O) <= 2e-2 + 2e-2 * abs(O)).all()
    assert abs(lse.reshape(L.shape).cpu().numpy() - L).max() <= 1e-3


def test_captured_step_replays_on_new_inputs():
    """The selection and attention of a step, captured once: new queries in the
    same buffers give what an eager step gives, bit for bit."""
    prob, state = together(False)
    idx = torch.empty(4, state["k"], dtype=torch.int32, device="cuda")
    prob.t[state["name"]] = idx.view(2, 2, 1, state["k"])
    f, _ = sfm.rope_frequencies(64, device="cuda")
    pos = torch.tensor([1001, 1002, 1498, 1499], dtype=torch.int32, device="cuda")
    q_in = prob.t["q"].clone()
    r = _sfm.Runner(prob)

    def step():
        sfm.apply_rope(q_in, pos, f, rope_offset=448, out=prob.t["q"])
        select(state, out=idx)
        r.plan()
        r.forward()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator(device="cuda").manual_seed(3)
    for _ in range(3):
        q_in.copy_(torch.randn(q_in.shape, generator=g, device="cuda").to(q_in.dtype))
        state["w"].copy_(torch.rand(state["w"].shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = r.out.clone(), r.lse.clone(), idx.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], r.out) and torch.equal(got[1], r.lse) and torch.equal(got[2], idx)


def test_calls_on_two_streams_at_once():
    a, b = together(False)[1], together(True)[1]
    want = [select(s)[2].clone() for s in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(10):
        for i, (s, st) in enumerate(zip(streams, (a, b))):
            with torch.cuda.stream(s):
                got[i].append(select(st)[2])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])
