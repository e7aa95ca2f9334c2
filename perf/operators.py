"""The operators around sparse shared-KV attention, as a serving program runs them.

Rotary positions of queries and outputs, the write side of the KV and index
caches (norm, rotation, quantisation, paged store), the index scores of new
queries against cached index keys, and the selection of the best positions or
blocks from those scores.  ``run`` computes each in plain torch operations, or,
with ``own`` set, through this repository's entry points.
"""
import math
import random

import torch

own = False

INDEX_DIM = 128
FP8_MAX = 448.0
TINY = 2.0 ** -126
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}
FORMATS = ("plain", "int8", "fp8", "fp8_rows")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the queries of one decode step: the last 64 of 512 dims carry positions, adjacent pairs
        dict(name="rope_decode", op="rope", tokens=32, heads=64, dim=512, rot=64, offset=448, interleaved=True,
             inverse=False, scaling="none", dtype="bf16"),
        # the attention output of a long prompt chunk, rotated back (the values carry positions too), long context
        dict(name="rope_output_back", op="rope", tokens=4093, heads=128, dim=512, rot=64, offset=448,
             interleaved=False, inverse=True, scaling="yarn", dtype="bf16"),
        # one new token per sequence into 656-byte packed rows
        dict(name="store_decode", op="store", tokens=64, heads=1, dim=576, rot=64, interleaved=True, norm=True,
             format="fp8", dtype="bf16"),
        # a prompt's rows into a plain paged cache
        dict(name="store_prefill", op="store", tokens=16381, heads=1, dim=512, rot=64, interleaved=True, norm=True,
             format="plain", dtype="bf16"),
        # index queries of a prompt chunk: rotated, then FP8 with one scale per head
        dict(name="store_index_queries", op="store", tokens=2048, heads=64, dim=128, rot=64, interleaved=False,
             norm=False, format="fp8_rows", dtype="bf16"),
        # few short sequences: latency
        dict(name="scores_short", op="scores", batch=4, q_len=1, heads=64, max_len=1000, ratio=4, block=64,
             dtype="bf16"),
        # a decode batch over compressed index keys
        dict(name="scores_decode", op="scores", batch=32, q_len=1, heads=64, max_len=32768, ratio=4, block=128,
             dtype="fp8"),
        # a prompt chunk over its cached prefix, one key per token
        dict(name="scores_prefill", op="scores", batch=1, q_len=2048, heads=64, max_len=8192, ratio=1, block=128,
             dtype="bf16"),
        # the selection of a decode batch
        dict(name="topk_decode", op="topk", rows=32, n=32768, k=512, block=1, first=0, last=0, causal=False),
        # one request with a very long context
        dict(name="topk_long", op="topk", rows=1, n=600001, k=2048, block=1, first=0, last=0, causal=False),
        # a prompt chunk, one key per token
        dict(name="topk_prefill", op="topk", rows=2048, n=8192, k=1024, block=1, first=0, last=0, causal=True),
        # the same over blocks of 64 tokens with the first block and the two newest always kept
        dict(name="topk_blocks", op="topk", rows=2048, n=16384, k=32, block=64, first=1, last=2, causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "store", "scores", "topk"))
    if op == "rope":
        dim = rng.choice((64, 128, 192, 512, 576))
        rot = rng.choice([r for r in (16, 32, 64, 128, 512) if r <= dim])
        heads = rng.choice((1, 7, 16, 64, 128))
        most = 4093 * 128 * 512 // (heads * dim)
        return dict(op=op, tokens=_log(rng, 1, min(most, 20000)), heads=heads, dim=dim, rot=rot,
                    offset=rng.choice((0, dim - rot)), interleaved=rng.random() < 0.5, inverse=rng.random() < 0.3,
                    scaling=rng.choice(("none", "linear", "ntk", "yarn")), dtype=rng.choice(("bf16", "fp16")))
    if op == "store":
        fmt = rng.choice(FORMATS)
        dim = rng.choice((512, 576)) if fmt in ("int8", "fp8") else 512 if fmt == "plain" else INDEX_DIM
        heads = rng.choice((1, 16, 64)) if fmt == "fp8_rows" else 1
        most = 4093 * 128 * 512 // (4 * heads * dim)
        return dict(op=op, tokens=_log(rng, 1, min(most, 30000)), heads=heads, dim=dim, rot=rng.choice((0, 32, 64)),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.7, format=fmt,
                    dtype=rng.choice(("bf16", "fp16")))
    if op == "scores":
        heads = rng.choice((8, 16, 24, 32, 64, 128))
        q_len = rng.choice((1, 1, 1, 2, 4, _log(rng, 5, 3000)))
        max_len = max(q_len, _log(rng, 1, 70000))
        pairs = 2048 * 64 * 8192 // heads
        max_len = max(q_len, min(max_len, pairs // q_len))
        batch = max(1, min(_log(rng, 1, 64), pairs // (q_len * max_len), 32 * 32768 // max_len))
        return dict(op=op, batch=batch, q_len=q_len, heads=heads, max_len=max_len, ratio=rng.choice((1, 4)),
                    block=rng.choice((16, 64, 128)), dtype=rng.choice(("bf16", "fp16", "fp8")))
    block = rng.choice((1, 1, 16, 64))
    n = _log(rng, 64, 600000)
    rows = max(1, min(_log(rng, 1, 3000), 2048 * 16384 // n))
    k = rng.choice((32, 512, 1000, 2048)) if block == 1 else rng.choice((8, 31, 64))
    return dict(op=op, rows=rows, n=n, k=k, block=block, first=rng.choice((0, 1)) if block > 1 else 0,
                last=rng.choice((0, 2)) if block > 1 else 0, causal=rows > 1 and rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _inv_freq(rot, scaling, device):
    """Angles per position (64 bits) and the amplitude of the rotated values."""
    base, factor, original = 10000.0, 16.0, 4096
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / max(rot - 2, 1))
    f = base ** (-2.0 * i / rot)
    amplitude = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        def at(turns):
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        f = f / factor * ramp + f * (1.0 - ramp)
        amplitude = 0.1 * math.log(factor) + 1.0
    return f.to(device), amplitude


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _prepare_rope(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    f, amplitude = _inv_freq(c["rot"], c["scaling"], "cuda")
    start = random.Random(seed).randrange(0, 120000)
    pos = (start + torch.arange(c["tokens"], device="cuda")) if c["tokens"] > 64 else torch.randint(
        0, 1 << 20, (c["tokens"],), generator=g, device="cuda")
    return dict(case=c, x=_randn(g, c["tokens"], c["heads"], c["dim"], dtype=dt), positions=pos.to(torch.int32),
                inv_freq=f, amplitude=amplitude)


def _row_shape(c):
    """(bytes or values of a cache row, its type)."""
    if c["format"] in ("int8", "fp8"):
        return 512 + 2 * (c["dim"] - 512) + 16, torch.uint8
    return c["dim"], DTYPES["fp8" if c["format"] == "fp8_rows" else c["dtype"]]


def _prepare_store(c, seed):
    g, dt, r = _gen(seed), DTYPES[c["dtype"]], random.Random(seed)
    T, H = c["tokens"], c["heads"]
    s = dict(case=c, x=_randn(g, T, H, c["dim"], dtype=dt) * (0.5 + r.random()))
    s["x"] = s["x"].to(dt)
    s["inv_freq"] = _inv_freq(c["rot"], "none", "cuda")[0] if c["rot"] else None
    s["positions"] = (r.randrange(0, 60000) + torch.arange(T, device="cuda")).to(torch.int32) if c["rot"] else None
    s["weight"] = (1.0 + 0.1 * _randn(g, min(c["dim"], 512))) if c["norm"] else None
    # pages in a shuffled pool a quarter larger than the tokens; every 97th token is padding (queries: none)
    groups = T if H > 1 else (T + T // 4 + 127) // 128 * 128
    if H > 1:
        s["slots"], s["rows"] = None, T * H
    else:
        page = torch.randperm(groups // 128, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        slots = page[t // 128] * 128 + t % 128
        s["slots"] = torch.where(t % 97 == 96, -1, slots).to(torch.int32)
        s["rows"] = groups
    width, kind = _row_shape(c)
    # one row behind the pool takes the padding's rows in the plain form; it is not part of the answer
    s["pool"] = torch.zeros(s["rows"] + 1, width, dtype=torch.uint8 if kind == DTYPES["fp8"] else kind, device="cuda")
    s["pool"] = s["pool"].view(kind)
    s["scales"] = torch.zeros(s["rows"] + 1, device="cuda") if c["format"] == "fp8_rows" else None
    return s


def _lens(c, seed):
    """Tokens so far and compressed keys of each sequence: between half and all of the longest."""
    r = random.Random(seed)
    most = c["max_len"] * c["ratio"]
    tokens = [r.randint(max(c["q_len"], most // 2), max(c["q_len"], most)) for _ in range(c["batch"])]
    tokens[r.randrange(c["batch"])] = max(c["q_len"], most)
    return [n // c["ratio"] for n in tokens], [n % c["ratio"] for n in tokens]


def _prepare_scores(c, seed):
    g, B, dt = _gen(seed), c["batch"], DTYPES[c["dtype"]]
    lens, rest = _lens(c, seed)
    cols = -(-c["max_len"] // c["block"])
    pages = [-(-n // c["block"]) for n in lens]
    total = max(1, sum(pages))
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist()
    table, at = torch.zeros(B, cols, dtype=torch.int32), 0
    for b, n in enumerate(pages):
        table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    s = dict(case=c, table=table.cuda(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             rest=torch.tensor(rest, dtype=torch.int32, device="cuda"))
    if c["dtype"] == "fp8":
        s["q"] = (_randn(g, B, c["q_len"], c["heads"], INDEX_DIM) * 100).clamp(-FP8_MAX, FP8_MAX).to(dt)
        s["k"] = (_randn(g, total, c["block"], INDEX_DIM) * 100).clamp(-FP8_MAX, FP8_MAX).to(dt)
        s["k_scales"] = 0.01 * (0.5 + torch.rand(total, c["block"], generator=g, device="cuda"))
    else:
        s["q"] = _randn(g, B, c["q_len"], c["heads"], INDEX_DIM, dtype=dt)
        s["k"] = _randn(g, total, c["block"], INDEX_DIM, dtype=dt)
        s["k_scales"] = None
    s["w"] = _randn(g, B, c["q_len"], c["heads"]) / (c["heads"] ** 0.5 * INDEX_DIM ** 0.5)
    return s


def _prepare_topk(c, seed):
    g = _gen(seed)
    # index scores: sums over clipped products, with the exact zeros that clipping leaves
    scores = (_randn(g, c["rows"], c["n"]) + 1.0).relu_()
    lengths = None
    if c["causal"]:
        r = torch.arange(c["rows"], device="cuda")
        lengths = (c["n"] - c["rows"] + 1 + r).clamp(min=1) if c["n"] >= c["rows"] else 1 + r % c["n"]
        lengths = lengths.to(torch.int32)
    return dict(case=c, scores=scores, lengths=lengths)


_PREPARE = dict(rope=_prepare_rope, store=_prepare_store, scores=_prepare_scores, topk=_prepare_topk)


def prepare(case, seed):
    return _PREPARE[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _rotate(x, positions, inv_freq, interleaved, inverse, amplitude):
    """x: (tokens, heads, rot) in 32 bits."""
    angle = positions.double()[:, None] * inv_freq
    cos, sin = angle.cos().float()[:, None] * amplitude, angle.sin().float()[:, None] * amplitude
    if inverse:
        sin = -sin
    half = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)


def _plain_rope(s):
    c, x = s["case"], s["x"]
    y, at = x.clone(), slice(c["offset"], c["offset"] + c["rot"])
    y[..., at] = _rotate(x[..., at].float(), s["positions"], s["inv_freq"], c["interleaved"], c["inverse"],
                         s["amplitude"]).to(x.dtype)
    return y


def _quantise(x, most):
    """x: (..., values of one scale) -> x / scale, scale."""
    scale = (x.abs().amax(-1, keepdim=True) / most).clamp(min=TINY)
    return x / scale, scale


def _plain_store(s):
    c, pool, x = s["case"], s["pool"], s["x"].float()
    T, H, D = x.shape
    nd = min(D, 512)
    if c["norm"]:
        n = x[..., :nd]
        n = n * torch.rsqrt(n.square().mean(-1, keepdim=True) + 1e-6) * s["weight"]
        x = torch.cat((n, x[..., nd:]), -1)
    if c["rot"]:
        r = _rotate(x[..., D - c["rot"]:], s["positions"], s["inv_freq"], c["interleaved"], False, 1.0)
        x = torch.cat((x[..., :D - c["rot"]], r), -1)
    x = x.reshape(T * H, D)
    rows = slice(0, T) if H > 1 else torch.where(s["slots"] < 0, s["rows"], s["slots"]).long()
    rows = slice(0, T * H) if H > 1 else rows
    if c["format"] == "plain":
        pool[rows] = x.to(pool.dtype)
    elif c["format"] == "fp8_rows":
        v, scale = _quantise(x, FP8_MAX)
        pool.view(torch.uint8)[rows] = v.to(DTYPES["fp8"]).view(torch.uint8)
        s["scales"][rows] = scale[:, 0]
    else:
        v, scale = _quantise(x[:, :512].reshape(-1, 4, 128), 127.0 if c["format"] == "int8" else FP8_MAX)
        v = v.round().to(torch.int8) if c["format"] == "int8" else v.to(DTYPES["fp8"])
        pool[rows] = torch.cat((v.view(torch.uint8).reshape(-1, 512),
                                x[:, 512:].to(s["x"].dtype).view(torch.uint8), scale.view(torch.uint8).reshape(-1, 16)), -1)


def _stored(s):
    """The pool's rows as the values they stand for: codes and scales, or int8 values times their scales."""
    c, pool = s["case"], s["pool"][:s["rows"]]
    if c["format"] == "plain":
        return pool
    if c["format"] == "fp8_rows":
        return dict(codes=pool, scales=s["scales"][:s["rows"]])
    rope = pool[:, 512:-16].view(s["x"].dtype)
    scales = pool[:, -16:].view(torch.float32)
    if c["format"] == "fp8":
        return dict(codes=pool[:, :512].view(DTYPES["fp8"]), rope=rope, scales=scales)
    values = pool[:, :512].view(torch.int8).view(-1, 4, 128).float() * scales[..., None]
    return dict(values=values.to(s["x"].dtype), rope=rope, scales=scales)


def _visible(s):
    """Keys each query may see: slot j is visible at position p when (j + 1) ratio <= p + 1."""
    c = s["case"]
    p = (s["lens"] * c["ratio"] + s["rest"] - c["q_len"])[:, None] + torch.arange(c["q_len"], device="cuda",
                                                                                  dtype=torch.int32)
    return torch.minimum(torch.div(p + 1, c["ratio"], rounding_mode="floor").clamp(min=0),
                         s["lens"][:, None]).to(torch.int32)


def _plain_scores(s):
    c = s["case"]
    B, S, H, L = c["batch"], c["q_len"], c["heads"], c["max_len"]
    bytes_of = s["k"].view(torch.uint8)
    k = bytes_of[s["table"].long()].view(s["k"].dtype).reshape(B, -1, INDEX_DIM)[:, :L]
    p = torch.matmul(s["q"].float().view(B, S * H, INDEX_DIM), k.float().transpose(1, 2)).relu_()
    scores = (p.view(B, S, H, L) * s["w"][..., None]).sum(2)
    if s["k_scales"] is not None:
        scores = scores * s["k_scales"][s["table"].long()].reshape(B, 1, -1)[..., :L]
    seen = _visible(s)
    j = torch.arange(L, device="cuda")
    return torch.where(j < seen[..., None], scores, -math.inf).view(B * S, L), seen.view(-1)


def _plain_topk(s):
    c, x = s["case"], s["scores"]
    rows, n = x.shape
    lengths = s["lengths"][:, None].long() if s["lengths"] is not None else torch.full((rows, 1), n, device="cuda")
    x = torch.where(torch.arange(n, device="cuda") < lengths, x, -math.inf)
    blocks = -(-n // c["block"])
    if c["block"] > 1:
        x = torch.nn.functional.pad(x, (0, blocks * c["block"] - n), value=-math.inf)
        x = x.view(rows, blocks, c["block"]).amax(-1)
    have = -(-lengths // c["block"])
    j = torch.arange(blocks, device="cuda")
    forced = ((j < c["first"]) | (j >= have - c["last"])) & (j < have)
    x = torch.where(forced, math.inf, x)
    order = torch.sort(x, dim=-1, descending=True, stable=True)
    k = min(c["k"], blocks)
    picked = torch.where(order.values[:, :k] > -math.inf, order.indices[:, :k], blocks).sort(-1).values
    picked = torch.where(picked < blocks, picked, -1)
    return torch.nn.functional.pad(picked, (0, c["k"] - k), value=-1).to(torch.int32)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own(s):
    import sparse_shared_kv_gb300 as sfm
    c = s["case"]
    if c["op"] == "rope":
        return sfm.apply_rope(s["x"], s["positions"], s["inv_freq"], amplitude=s["amplitude"],
                              rope_offset=c["offset"], interleaved=c["interleaved"], inverse=c["inverse"])
    if c["op"] == "store":
        kinds = dict(plain=sfm.KV_PLAIN, int8=sfm.KV_INT8_PACKED, fp8=sfm.KV_FP8_PACKED, fp8_rows=sfm.KV_FP8_ROWS)
        sfm.store_kv(s["x"], s["pool"][:s["rows"]], slot_mapping=s["slots"], kv_format=kinds[c["format"]],
                     norm_weight=s["weight"], norm_eps=1e-6 if c["norm"] else None, positions=s["positions"],
                     inv_freq=s["inv_freq"], interleaved=c["interleaved"],
                     scales=s["scales"][:s["rows"]] if s["scales"] is not None else None)
        return _stored(s)
    if c["op"] == "scores":
        return sfm.index_scores(s["q"], s["k"], s["w"], k_scales=s["k_scales"], block_table=s["table"],
                                seqused_kv=s["lens"], cmp_residual_kv=s["rest"], max_seqlen_kv=c["max_len"],
                                cmp_ratio=c["ratio"], layout_kv="PAGED")
    return sfm.select_topk(s["scores"], c["k"], lengths=s["lengths"], block_size=c["block"],
                           first_blocks=c["first"], last_blocks=c["last"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rope":
        return _plain_rope(state)
    if op == "store":
        _plain_store(state)
        return _stored(state)
    return _plain_scores(state) if op == "scores" else _plain_topk(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "rope":
        values = c["tokens"] * c["heads"] * c["dim"]
        return dict(bytes=4 * values + 4 * c["tokens"], flops=3 * c["tokens"] * c["heads"] * c["rot"])
    if c["op"] == "store":
        n, width = c["tokens"] * c["heads"], _row_shape(c)[0]
        size = width * (2 if c["format"] == "plain" else 1) + (4 if c["format"] == "fp8_rows" else 0)
        return dict(bytes=n * (2 * c["dim"] + size) + 8 * c["tokens"], flops=8 * n * c["dim"])
    if c["op"] == "scores":
        e = 1 if c["dtype"] == "fp8" else 2
        mean = 0.75 * c["max_len"] if c["batch"] > 1 else c["max_len"]      # lengths between half and all
        keys, queries = c["batch"] * mean, c["batch"] * c["q_len"]
        seen = max(1.0, mean - (c["q_len"] - 1) / (2 * c["ratio"]))
        return dict(bytes=keys * (INDEX_DIM * e + (4 if e == 1 else 0)) + queries * c["heads"] * (INDEX_DIM * e + 4)
                    + 4 * queries * c["max_len"], flops=queries * seen * c["heads"] * 2 * INDEX_DIM)
    read = c["rows"] * (c["n"] - (min(c["rows"], c["n"]) / 2 if c["causal"] else 0))
    return dict(bytes=4 * read + 4 * c["rows"] * c["k"], flops=read)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _turned(z, positions, inv_freq, interleaved, sign, amplitude):
    """Pairs of z (tokens, heads, rot; float64) as complex numbers times amplitude e^(i sign p f)."""
    T, H, rot = z.shape
    if interleaved:
        pairs = torch.view_as_complex(z.reshape(T, H, rot // 2, 2).contiguous())
    else:
        pairs = torch.complex(z[..., :rot // 2].contiguous(), z[..., rot // 2:].contiguous())
    angle = sign * positions.to(torch.float64).reshape(T, 1, 1) * inv_freq.reshape(1, 1, -1)
    pairs = pairs * torch.polar(torch.full_like(angle, amplitude), angle)
    if interleaved:
        return torch.view_as_real(pairs).reshape(T, H, rot)
    return torch.cat((pairs.real, pairs.imag), 2)


def _exact_rope(c, seed):
    s = prepare(c, seed)
    y = s["x"].double()
    a, b = c["offset"], c["offset"] + c["rot"]
    y[:, :, a:b] = _turned(y[:, :, a:b].clone(), s["positions"], s["inv_freq"], c["interleaved"],
                           -1.0 if c["inverse"] else 1.0, s["amplitude"])
    return y


def _exact_store(c, seed):
    s = prepare(c, seed)
    T, H, D = s["x"].shape
    y, m = s["x"].double(), min(D, 512)
    if c["norm"]:
        length = torch.linalg.vector_norm(y[:, :, :m], dim=2, keepdim=True)
        y[:, :, :m] = y[:, :, :m] / torch.sqrt(length * length / m + 1e-6) * s["weight"].double()
    if c["rot"]:
        y[:, :, D - c["rot"]:] = _turned(y[:, :, D - c["rot"]:].clone(), s["positions"], s["inv_freq"],
                                         c["interleaved"], 1.0, 1.0)
    y = y.reshape(T * H, D)
    if H == 1:                                # where each row of the pool comes from; the others keep their zeros
        kept = (s["slots"] >= 0).nonzero()[:, 0]
        all_rows = torch.zeros(s["rows"], D, dtype=torch.float64, device="cuda")
        all_rows[s["slots"][kept].long()] = y[kept]
        written = torch.zeros(s["rows"], 1, dtype=torch.float64, device="cuda")
        written[s["slots"][kept].long()] = 1.0
        y = all_rows
    else:
        written = torch.ones(T * H, 1, dtype=torch.float64, device="cuda")
    if c["format"] == "plain":
        return y
    tiles = y[:, :512].reshape(y.shape[0], -1, 128)
    most = 127.0 if c["format"] == "int8" else FP8_MAX
    scale = torch.clamp(torch.linalg.vector_norm(tiles, ord=math.inf, dim=2) / most, min=TINY) * written
    over = torch.where(scale > 0, scale, 1.0)
    if c["format"] == "fp8_rows":
        return dict(codes=(tiles / over[..., None]).reshape(-1, D), scales=scale[:, 0])
    if c["format"] == "fp8":
        return dict(codes=(tiles / over[..., None]).reshape(-1, 512), rope=y[:, 512:], scales=scale)
    return dict(values=tiles, rope=y[:, 512:], scales=scale)


def _exact_scores(c, seed):
    s = prepare(c, seed)
    B, S, H, L = c["batch"], c["q_len"], c["heads"], c["max_len"]
    out = torch.full((B, S, L), -math.inf, dtype=torch.float64, device="cuda")
    seen = torch.zeros(B, S, dtype=torch.int32)
    for b, (n, rest) in enumerate(zip(*_lens(c, seed))):
        at = torch.arange(n, device="cuda")
        page = s["table"][b].long()[at // c["block"]]
        keys = s["k"].float().reshape(-1, INDEX_DIM)[page * c["block"] + at % c["block"]].double()
        if s["k_scales"] is not None:
            keys = keys * s["k_scales"].reshape(-1)[page * c["block"] + at % c["block"]].double()[:, None]
        step = max(1, (1 << 28) // max(1, H * n))
        for i in range(0, S, step):
            q = s["q"][b, i:i + step].float().double()
            dots = torch.einsum("ihd,nd->ihn", q, keys).clamp_(min=0)
            out[b, i:i + step, :n] = torch.einsum("ihn,ih->in", dots, s["w"][b, i:i + step].double())
        for i in range(S):
            seen[b, i] = min(n, (n * c["ratio"] + rest - S + i + 1) // c["ratio"])
    hidden = torch.arange(L, device="cuda") >= seen.cuda()[..., None]
    return out.masked_fill_(hidden, -math.inf).reshape(B * S, L), seen.reshape(-1)


def _exact_topk(c, seed):
    s = prepare(c, seed)
    scores = s["scores"].double().cpu().numpy()
    ends = s["lengths"].tolist() if s["lengths"] is not None else [c["n"]] * c["rows"]
    out = torch.full((c["rows"], c["k"]), -1, dtype=torch.int32)
    import numpy as np
    for r, end in enumerate(ends):
        v = np.maximum.reduceat(scores[r, :end], np.arange(0, end, c["block"])) if c["block"] > 1 else scores[r, :end]
        v = v.copy()
        if c["first"]:
            v[:c["first"]] = np.inf
        if c["last"]:
            v[-c["last"]:] = np.inf
        best = np.argsort(-v, kind="stable")[:c["k"]]
        best = np.sort(best[v[best] > -np.inf])
        out[r, :len(best)] = torch.from_numpy(best.astype(np.int32))
    return out


def exact(case, seed):
    return dict(rope=_exact_rope, store=_exact_store, scores=_exact_scores, topk=_exact_topk)[case["op"]](case, seed)
