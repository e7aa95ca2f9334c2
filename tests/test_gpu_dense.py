"""Attention of many queries over the same rows, joined results and moved rows
on the GPU, against their definitions in 64 bits.

Tolerances, from the arithmetic (u = half a step of the output type relative to
the value, w_j the normalised weights, x the scores):
* a score: 512 exact products, added in fp32 in at most 32 runs of 16, each step
  off by at most 2^-23 of the magnitudes so far, counted twice for the alignment
  inside a run; scale, cap and bias add a few roundings of |x|, of the cap and
  of the bias: d = 64 2^-23 scale sum |q k| + 2^-20 (1 + cap + |bias|).
* LSE: the largest d of the row's visible keys, n 2^-24 of the sum of n weights and
  2^-20 of exp2, log2 and the change of base, relative to 1 + |LSE|.
* O: every weight is off by 2 d and rounded to the type once (u), the sum of n
  products by n 2^-23, the division by 2^-20; then u of the value:
  (u + 2 d + n 2^-23 + 2^-20) sum w |v| + u |O| + the type's smallest step.
"""
import math
import random

import pytest
import torch

import sparse_shared_kv_gb300 as sfm

pytestmark = pytest.mark.gpu

F64, INF = torch.float64, math.inf
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    sfm.build()
    torch.cuda.init()


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ---------------------------------------------------------------------------
# problems
# ---------------------------------------------------------------------------
def problem(seed=0, dt="bf16", heads=16, q_lens=(3,), lens=(50,), layout_q="TND", layout_kv="TND", block=64, mode=3, left=-1,
            right=-1, cap=0.0, bias=False, sinks=False, prefix=None, docs=False, tree=False, pad=0, q_scale=3.0, used_q=None,
            general_tree=False, rest=0):
    """A batch, its call's arguments, and per sequence its keys, positions and what each query sees."""
    g, r, dtype = gen(seed), random.Random(seed), DT[dt]
    B = len(q_lens)
    q_s = max(q_lens) if layout_q == "BSND" else 0
    caps = [q_s] * B if layout_q == "BSND" else list(q_lens)
    tokens = sum(caps) + rest
    q = (q_scale * randn(g, tokens, heads, 512)).to(dtype)
    keys = [randn(g, n, 512, dtype=dtype) for n in lens]
    args = dict(softmax_scale=512 ** -0.5, softcap=cap, mask_mode=mode, win_left=left, win_right=right, layout_q=layout_q,
                layout_kv=layout_kv)
    used = list(q_lens)
    if layout_q == "TND":
        args["cu_seqlens_q"] = ints([sum(q_lens[:b]) for b in range(B + 1)])
        if used_q is not None:
            used = list(used_q)
            args["seqused_q"] = ints(used)
    else:
        q = q.view(B, q_s, heads, 512)
        if len(set(q_lens)) > 1 or used_q is not None:
            used = list(used_q) if used_q is not None else used
            args["seqused_q"] = ints(used)
    if layout_kv == "PAGED":
        pages = [-(-n // block) for n in lens]
        cols, total = max(max(pages), 1) + 1, sum(pages) + 3
        ids = list(range(total))
        r.shuffle(ids)
        pool = torch.full((total, block, 512 + pad), math.nan, dtype=dtype, device="cuda")   # what nobody wrote
        table = [[-7] * cols for _ in lens]
        for b, n in enumerate(lens):
            for i in range(pages[b]):
                table[b][i] = ids.pop()
                part = keys[b][i * block:(i + 1) * block]
                pool[table[b][i], :len(part), :512] = part
        kv = pool[..., :512]
        args.update(block_table=ints(table), seqused_kv=ints(lens), max_seqlen_kv=max(max(lens), 1))
    elif layout_kv == "TND":
        kv = torch.full((sum(lens) + 5, 512 + pad), math.nan, dtype=dtype, device="cuda")[:, :512]
        kv[:sum(lens)] = torch.cat(keys)
        args.update(cu_seqlens_kv=ints([sum(lens[:b]) for b in range(B + 1)]), max_seqlen_kv=max(max(lens), 1))
    else:
        kv = torch.full((B, max(max(lens), 1), 512 + pad), math.nan, dtype=dtype, device="cuda")[..., :512]
        for b, n in enumerate(lens):
            kv[b, :n] = keys[b]
        args["seqused_kv"] = ints(lens)
    if sinks:
        args["sinks"] = 2.0 * randn(g, heads)
    if bias:
        args["bias_slopes"] = 2.0 ** (-8.0 * torch.arange(1, heads + 1, device="cuda") / heads)
    seqs, at = [], 0
    begin, end, masks, places = ([0] * tokens for _ in range(4))
    words = max(1, -(-max(max(caps), 1) // 64))
    for b, (n, ql) in enumerate(zip(lens, used)):
        j = torch.arange(n, device="cuda")
        p = (n - ql + torch.arange(ql, device="cuda"))[:, None]
        pos = j
        if tree:
            first, bits, depth = n - ql, [], []
            for i in range(ql):
                parent = r.randrange(max(-1, i - 6), i) if i else -1
                bits.append((bits[parent] if parent >= 0 else 0) | 1 << i)
                depth.append(depth[parent] + 1 if parent >= 0 else 0)
                if general_tree:
                    bits[i] = r.getrandbits(ql) if r.random() < 0.8 else 0
            place = [max(first, 0) + d for d in depth]
            for i in range(ql):
                masks[at + i], places[at + i] = bits[i], place[i]
            # keys before the drafted ones and their own (a negative first cuts the drafted ones off from the front)
            pos = torch.cat((torch.arange(max(first, 0), device="cuda"), ints(place, torch.int64)[max(-first, 0):]))
            p = ints(place, torch.int64)[:, None]
            seen = torch.zeros(ql, n, dtype=torch.bool)
            seen[:, :max(first, 0)] = True
            for i in range(ql):
                for k in range(max(-first, 0), ql):
                    seen[i, first + k] = bool(bits[i] >> k & 1)
            seen = seen.cuda()
            if mode == 4:
                seen &= (pos >= p - (left if left >= 0 else 1 << 30)) & (pos <= p + (right if right >= 0 else 1 << 30))
        else:
            seen = torch.ones(ql, n, dtype=torch.bool, device="cuda")
            if mode == 3:
                seen &= j <= p
            if mode == 4:
                seen &= (j >= p - (left if left >= 0 else 1 << 30)) & (j <= p + (right if right >= 0 else 1 << 30))
            if docs:
                cuts = [0] + sorted(r.randint(0, n) for _ in range(3)) + [n]
                for i in range(ql):
                    d = max(k for k in range(4) if cuts[k] <= max(n - ql + i, 0))
                    begin[at + i], end[at + i] = cuts[d], cuts[d + 1]
                    if r.random() < 0.1:
                        begin[at + i], end[at + i] = r.choice(((5, 5), (9, 2), (-3, n + 100), (n, n + 5), (-20, -10)))
                lo, hi = ints(begin[at:at + ql], torch.int64)[:, None], ints(end[at:at + ql], torch.int64)[:, None]
                seen &= (j >= lo) & (j < hi)
            if prefix is not None:
                seen |= j < prefix[b]
        seqs.append((at, ql, caps[b], keys[b], p - pos, seen))
        at += caps[b]
    lead = q.shape[:-2]
    if docs:
        args.update(key_begin=ints(begin).view(lead), key_end=ints(end).view(lead))
    if prefix is not None:
        args["prefix_lens"] = ints(list(prefix))
    call = sfm.masked_attention
    if tree:
        signed = [[(m >> 64 * w & (1 << 64) - 1) for w in range(words)] for m in masks]
        mask = ints([[v - (1 << 64) if v >> 63 else v for v in row] for row in signed], torch.int64).view(*lead, words)
        place = ints(places).view(lead)

        def call(q, kv, **kw):
            return sfm.tree_attention(q, kv, mask, place, **kw)
    return dict(q=q, kv=kv, args=args, seqs=seqs, call=call, heads=heads, dtype=dtype)


def run(p, **kw):
    status = ints([0])
    out, lse = p["call"](p["q"], p["kv"], status=status, **{**p["args"], **kw})
    return out.reshape(-1, p["heads"], 512), lse.reshape(-1, p["heads"]), int(status)


def check(p, out, lse, skip_nan=False):
    """Against the definition in 64 bits; returns it."""
    a, H, dtype = p["args"], p["heads"], p["dtype"]
    q = p["q"].reshape(-1, H, 512)
    u, tiny = half_step(dtype), torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    for at, ql, cap_q, keys, dist, seen in p["seqs"]:
        n = keys.shape[0]
        assert (out[at + ql:at + cap_q] == 0).all() and (lse[at + ql:at + cap_q] == -INF).all()
        step = max(1, (1 << 25) // max(1, H * n))
        for i in range(0, ql, step):
            e = min(ql, i + step)
            rows = slice(at + i, at + e)
            qq, kk = q[rows].double(), keys.double()
            x = torch.einsum("thd,nd->thn", qq, kk) * a["softmax_scale"]
            d = 64 * 2.0 ** -23 * torch.einsum("thd,nd->thn", qq.abs(), kk.abs()) * abs(a["softmax_scale"])
            cap = a["softcap"]
            if cap:
                x = cap * torch.tanh(x / cap)
            d = d + 2.0 ** -20 * (1 + cap)
            if a.get("bias_slopes") is not None:
                fall = a["bias_slopes"].double()[:, None] * dist[i:e].abs().double()[:, None]
                x = x - fall
                d = d + 2.0 ** -20 * fall
            vis = seen[i:e, None].expand_as(x)
            x = torch.where(vis, x, -INF)
            d = torch.where(vis, d, 0.0).amax(-1) if n else torch.zeros(e - i, H, dtype=F64, device="cuda")
            m = x.amax(-1, keepdim=True) if n else torch.full((e - i, H, 1), -INF, dtype=F64, device="cuda")
            m = torch.where(m == -INF, 0.0, m)
            w = torch.exp(x - m)
            total = w.sum(-1)
            L = m[..., 0] + torch.log(total)
            under = total + torch.exp(a["sinks"].double() - m[..., 0]) if a.get("sinks") is not None else total
            w = w / torch.where(under == 0, 1.0, under)[..., None]
            O, mag = torch.einsum("thn,nd->thd", w, kk), torch.einsum("thn,nd->thd", w, kk.abs())
            got_o, got_l = out[rows].double(), lse[rows].double()
            empty = L == -INF
            assert torch.equal(got_l == -INF, empty), "rows without keys"
            assert (got_o[empty] == 0).all()
            off = torch.where(empty, 0.0, (got_l - L).abs())
            bound = d + n * 2.0 ** -24 + 2.0 ** -20 * (1 + torch.where(empty, 0.0, L).abs())
            assert (off <= bound).all(), f"LSE off by {float((off / bound).max()):.3g} bounds"
            bound = (u + 2 * d[..., None] + n * 2.0 ** -23 + 2.0 ** -20) * mag + u * O.abs() + tiny
            off = (got_o - O).abs()
            assert (off <= bound).all(), f"O off by {float((off / bound).max()):.3g} bounds"


def go(**kw):
    p = problem(**kw)
    out, lse, status = run(p)
    assert status == 0
    check(p, out, lse)
    return p, out, lse


# ---------------------------------------------------------------------------
# shapes, layouts, types
# ---------------------------------------------------------------------------
SHAPES = [
    # heads, query lengths, key lengths
    (1, (1,), (1,)), (1, (131,), (200,)), (3, (5, 1, 40), (77, 1, 300)), (16, (1, 1, 1), (128, 129, 127)),
    (16, (9,), (1000,)), (48, (3, 7), (500, 64)), (64, (2, 3), (256, 1111)), (64, (1,), (5000,)), (100, (4,), (321,)),
    (127, (2,), (200,)), (128, (1, 2), (640, 13)), (128, (5,), (900,)), (20, (33, 0, 2), (700, 5, 0)), (64, (300,), (300,)),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["TND", "PAGED", "BSND"])
def test_causal(shape, dt, layout):
    heads, q_lens, lens = shape
    go(seed=1, heads=heads, q_lens=q_lens, lens=lens, dt=dt, layout_kv=layout, layout_q="TND" if layout == "TND" else "BSND")


@pytest.mark.parametrize("block", [16, 32, 48, 64, 80, 96, 128, 192, 1024])
@pytest.mark.parametrize("pad", [0, 8, 64])
def test_pages(block, pad):
    go(seed=2, heads=24, q_lens=(7, 3, 1), lens=(1030, 128, 1), layout_kv="PAGED", block=block, pad=pad)


@pytest.mark.parametrize("layout", ["TND", "BSND"])
def test_padded_rows(layout):
    go(seed=3, heads=8, q_lens=(20, 50), lens=(140, 50), layout_q=layout, layout_kv=layout, pad=24)


@pytest.mark.parametrize("mode,left,right", [(0, -1, -1), (3, -1, -1), (4, 0, 0), (4, 5, 0), (4, 127, 0), (4, 200, 3), (4, -1, 17),
                                             (4, 30, -1), (4, 2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("heads", [16, 128])
def test_masks(mode, left, right, heads):
    go(seed=4, heads=heads, q_lens=(60, 3, 9), lens=(60, 500, 4), mode=mode, left=left, right=right)


@pytest.mark.parametrize("cap", [0.0, 0.5, 30.0])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_scores(cap, bias, sinks, dt):
    go(seed=5, dt=dt, heads=48, q_lens=(40, 1), lens=(90, 700), cap=cap, bias=bias, sinks=sinks, mode=0)
    go(seed=6, dt=dt, heads=64, q_lens=(5, 2), lens=(600, 130), cap=cap, bias=bias, sinks=sinks, layout_kv="PAGED")


@pytest.mark.parametrize("scale", [0.0, -0.03, 0.3])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_scales(scale, cap):
    p = problem(seed=7, heads=16, q_lens=(9,), lens=(300,), cap=cap)
    p["args"]["softmax_scale"] = scale
    out, lse, _ = run(p)
    check(p, out, lse)


@pytest.mark.parametrize("mode", [0, 3, 4])
@pytest.mark.parametrize("prefix", [None, (0, 50, 3000, -5), (700, 128, 1, 40)])
def test_documents_and_prefixes(mode, prefix):
    go(seed=8, heads=16, q_lens=(80, 200, 31, 1), lens=(900, 210, 64, 41), mode=mode, left=40, right=5, docs=True, prefix=prefix)
    go(seed=9, heads=40, q_lens=(80, 20, 31, 1), lens=(900, 210, 64, 41), mode=mode, left=40, right=0, docs=prefix is None,
       prefix=prefix, layout_q="BSND", layout_kv="PAGED", block=48, bias=True)


def test_long_ranges_are_cut_and_joined():
    for split in (0, 128, 512, 4096):
        p = problem(seed=10, heads=16, q_lens=(1, 2), lens=(30000, 9000), sinks=True, bias=True, layout_kv="PAGED")
        out, lse, status = run(p, split_keys=split)
        assert status == 0
        check(p, out, lse)


@pytest.mark.parametrize("batch,heads,most_q,most_kv", [(33, 16, 3, 600), (40, 128, 1, 1500), (100, 128, 40, 300), (700, 8, 2, 90),
                                                        (1600, 3, 2, 40), (2000, 128, 1, 33), (70, 64, 60, 2000)])
@pytest.mark.parametrize("layout_q", ["TND", "BSND"])
def test_many_sequences(batch, heads, most_q, most_kv, layout_q):
    """More sequences than a warp reads at once, more tiles of queries than are shared evenly, and both."""
    r = random.Random(batch)
    q_lens = [r.randint(0 if layout_q == "TND" else 1, most_q) for _ in range(batch)]
    lens = [r.randint(0, most_kv) for _ in range(batch)]
    go(seed=batch, heads=heads, q_lens=q_lens, lens=lens, layout_q=layout_q, layout_kv="PAGED", sinks=batch < 50)


def test_one_long_sequence_among_short_ones():
    """Shares that begin and end inside of one tile's keys, and shares of many whole tiles."""
    lens = [60000] + [140] * 50 + [20000]
    for heads in (4, 64):
        go(seed=36, heads=heads, q_lens=[1] * 52, lens=lens, layout_kv="PAGED", block=128, bias=True)
    go(seed=37, heads=128, q_lens=[9, 0, 3, 1], lens=[40000, 0, 3, 0], tree=True)


def test_outputs_at_any_sixteen_bytes():
    p = problem(seed=38, heads=3, q_lens=(50, 7), lens=(300, 1500), rest=9)
    want = run(p)
    room = torch.zeros(want[0].numel() + 64, dtype=p["dtype"], device="cuda")
    for shift in (8, 16, 24):
        mine = room[shift:shift + want[0].numel()].view(want[0].shape)
        out, lse = sfm.masked_attention(p["q"], p["kv"], out=mine, **p["args"])
        assert torch.equal(mine[:57], want[0][:57])
    room = torch.zeros(p["q"].numel() + 64, dtype=p["dtype"], device="cuda")
    q = room[8:8 + p["q"].numel()].view(p["q"].shape)
    q.copy_(p["q"])
    assert torch.equal(sfm.masked_attention(q, p["kv"], **p["args"])[0], want[0])


def test_prefix_far_before_the_window_in_pieces():
    for split in (0, 128, 256):
        p = problem(seed=11, heads=8, q_lens=(20, 40), lens=(5000, 3000), mode=4, left=300, right=0, prefix=(1000, 2950))
        out, lse, _ = run(p, split_keys=split)
        check(p, out, lse)


@pytest.mark.parametrize("seed", range(40))
def test_random_problems(seed):
    r = random.Random(1000 + seed)
    B = r.randint(1, 6)
    heads = r.choice((1, 2, 5, 16, 17, 33, 48, 64, 96, 128))
    q_lens = [r.choice((0, 1, 1, 2, 5, r.randint(1, 6000 // heads))) for _ in range(B)]
    if not any(q_lens):
        q_lens[0] = 1
    lens = [r.choice((0, 1, q, q + r.randint(0, 200), q + r.randint(0, 2500))) for q in q_lens]
    layout_q = r.choice(("TND", "BSND"))
    layout_kv = r.choice((layout_q, "PAGED"))
    tree = r.random() < 0.4
    if tree:
        q_lens = [min(q, 1024) for q in q_lens]      # sixteen words of a mask
    go(seed=seed, dt=r.choice(("bf16", "fp16")), heads=heads, q_lens=q_lens, lens=lens, layout_q=layout_q, layout_kv=layout_kv,
       block=r.choice((16, 48, 64, 128)), mode=r.choice((0, 3, 4)), left=r.choice((-1, 0, 30, 200)), right=r.choice((-1, 0, 9)),
       cap=r.choice((0.0, 0.0, 10.0)), bias=r.random() < 0.4, sinks=r.random() < 0.4, tree=tree,
       prefix=None if tree or r.random() < 0.5 else [r.randint(0, 400) for _ in lens], docs=not tree and r.random() < 0.4,
       general_tree=r.random() < 0.4, pad=r.choice((0, 0, 16)))


# ---------------------------------------------------------------------------
# trees
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("drafts", [1, 2, 7, 63, 64, 65, 128, 200])
@pytest.mark.parametrize("heads", [1, 16, 64, 128])
def test_trees(drafts, heads):
    go(seed=12, heads=heads, q_lens=(drafts, drafts), lens=(drafts + 300, drafts), tree=True, layout_kv="PAGED")


@pytest.mark.parametrize("left,right", [(0, 0), (1, 0), (3, 0), (127, 0), (5, 2), (-1, 1)])
@pytest.mark.parametrize("general", [False, True])
def test_trees_in_a_window(left, right, general):
    go(seed=13, heads=20, q_lens=(40, 3, 70), lens=(140, 3, 1000), tree=True, mode=4, left=left, right=right, bias=True,
       general_tree=general, layout_q="BSND", layout_kv="PAGED", block=16)


def test_trees_of_any_mask():
    go(seed=14, heads=48, q_lens=(90, 130), lens=(130, 900), tree=True, general_tree=True, cap=20.0, sinks=True, dt="fp16")
    go(seed=15, heads=3, q_lens=(90, 130), lens=(50, 131), tree=True, general_tree=True, bias=True)


@pytest.mark.parametrize("mode", [3, 4])
def test_trees_whose_arrays_end_with_their_memory(mode):
    """Rows of a tile that do not count read no positions, masks or bounds: those of the last token are the last of 32 MB."""
    p = problem(seed=39, heads=3, q_lens=(5,), lens=(200,), tree=True, bias=True, mode=mode, left=60, right=0)
    want = run(p)
    mask, place = (x.cell_contents for x in p["call"].__closure__)
    ends = [torch.empty(4 << 20, dtype=x.dtype, device="cuda") for x in (mask, place)]
    for end, x in zip(ends, (mask, place)):
        end[-x.numel():] = x.flatten()
    got = sfm.tree_attention(p["q"], p["kv"], ends[0][-mask.numel():].view(mask.shape), ends[1][-place.numel():].view(place.shape), **p["args"])
    assert torch.equal(got[0].view(-1), want[0].view(-1)) and torch.equal(got[1].view(-1), want[1].view(-1))
    p = problem(seed=40, heads=3, q_lens=(5,), lens=(200,), docs=True, bias=True, mode=mode, left=60, right=0)
    want = run(p)
    args = dict(p["args"])
    for name in ("key_begin", "key_end"):
        end = torch.empty(8 << 20, dtype=torch.int32, device="cuda")
        end[-5:] = args[name]
        args[name] = end[-5:]
    got = sfm.masked_attention(p["q"], p["kv"], **args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_chain_is_causal_attention():
    p = problem(seed=16, heads=16, q_lens=(70,), lens=(400,))
    out, lse, _ = run(p)
    mask = [(1 << i + 1) - 1 for i in range(70)]
    words = [[m & (1 << 64) - 1, m >> 64] for m in mask]
    words = ints([[v - (1 << 64) if v >> 63 else v for v in w] for w in words], torch.int64)
    got, end = sfm.tree_attention(p["q"], p["kv"], words, ints(range(330, 400)), **p["args"])
    check(p, got, end)


# ---------------------------------------------------------------------------
# values that a row does not see
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("value", [math.nan, INF, -INF])
@pytest.mark.parametrize("heads", [1, 16, 64])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_hidden_values_have_no_part(value, heads, dt):
    """NaN and infinities in keys of other documents, of the future and of other branches change nothing, bit for bit."""
    p = problem(seed=17, dt=dt, heads=heads, q_lens=(150,), lens=(300,), docs=False)
    begin = ints([100 if i < 40 else 190 + i // 50 for i in range(150)])
    want = sfm.masked_attention(p["q"], p["kv"], key_begin=begin, **p["args"])
    hidden = [0, 7, 64, 99]
    p["kv"][hidden] = value
    p["kv"][50, 300:] = value
    got = sfm.masked_attention(p["q"], p["kv"], key_begin=begin, **p["args"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a key that only the last documents see
    p["kv"][hidden] = 1.0
    p["kv"][50] = 1.0
    p["kv"][191, 5] = value
    got = sfm.masked_attention(p["q"], p["kv"], key_begin=begin, **p["args"])
    sees = torch.tensor([b <= 191 <= 150 + i for i, b in enumerate(begin.tolist())], device="cuda")
    assert torch.equal(got[0][~sees], want[0][~sees]) and torch.equal(got[1][~sees], want[1][~sees])
    assert sees.any() and (~sees).any()
    if math.isnan(value):
        assert got[0][sees].isnan().all() and got[1][sees].isnan().all()
    tree = problem(seed=18, dt=dt, heads=heads, q_lens=(20,), lens=(60,), tree=True)
    seen = tree["seqs"][0][5][:, 45]
    want = run(tree)
    tree["kv"][45, 9] = value
    got = run(tree)
    assert torch.equal(got[0][~seen], want[0][~seen]) and (~seen).any()


def test_queries_that_are_nan_stay_alone():
    p, out, lse = go(seed=19, heads=16, q_lens=(40,), lens=(100,))
    q = p["q"].clone()
    q[5, 3] = math.nan
    q[17] = INF
    got, end = sfm.masked_attention(q, p["kv"], **p["args"])
    fine = torch.ones(40, 16, dtype=torch.bool, device="cuda")
    fine[5, 3] = fine[17] = False
    assert torch.equal(got[fine], out[fine]) and torch.equal(end[fine], lse[fine])
    assert got[5, 3].isnan().all() and got[17].isnan().all()


def test_large_scores():
    """Scores far outside of exp's range, both ways, and maxima that grow along the keys."""
    for q_scale in (100.0, 2000.0):
        p = problem(seed=20, heads=16, q_lens=(20,), lens=(700,), q_scale=q_scale)
        ramp = torch.linspace(0.1, 3.0, 700, device="cuda")[:, None]
        p["kv"][:700] = (p["kv"][:700].float() * ramp).to(p["dtype"])
        p["seqs"][0] = p["seqs"][0][:3] + (p["kv"][:700].clone(),) + p["seqs"][0][4:]
        out, lse, _ = run(p)
        check(p, out, lse)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_capped_scores_do_not_depend_on_what_rows_do_not_see(dt):
    """Large scores of the next sequence's rows, of rows behind a sequence's end and of hidden keys leave every bit as it was."""
    p = problem(seed=44, dt=dt, heads=5, q_lens=(3, 40), lens=(150, 90), layout_kv="PAGED", block=64, cap=20.0, q_scale=0.1, mode=4, left=100, right=0)
    kv, table = p["kv"].nan_to_num(0.0), p["args"]["block_table"]
    first = sfm.masked_attention(p["q"], kv, split_keys=128, **p["args"])
    check(p, first[0].view(-1, 5, 512), first[1].view(-1, 5))
    q = p["q"].clone()
    q[3:] *= 300.0
    # behind the first sequence's end, and a key that its window hides
    kv = kv.clone()
    kv[table[0, 2].long(), 150 - 128:] = 30.0
    kv[table[0, 0].long(), 40] = -30.0
    then = sfm.masked_attention(q, kv, split_keys=128, **p["args"])
    assert torch.equal(then[0][:3], first[0][:3]) and torch.equal(then[1][:3], first[1][:3])


def check_capped(p, out, lse):
    """As check(), but with capped scores x off by 2^-20 (1 + |x|) whatever the cap is (tanh z / z off by 2^-21 of itself and a few
    roundings up to |z| = 1; above, 1 - 2 / (e^2z + 1) by 2^-23 of the cap, which is at most 1.32 |x|), and up to a cap of 128,
    where the quotient comes for smaller z too, by 2^-21 of the cap."""
    a, H, dtype = p["args"], p["heads"], p["dtype"]
    q, cap, scale = p["q"].reshape(-1, H, 512).double(), a["softcap"], a["softmax_scale"]
    u, tiny = half_step(dtype), torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    for at, ql, _, keys, dist, seen in p["seqs"]:
        qq, kk, n = q[at:at + ql], keys.double(), keys.shape[0]
        x = cap * torch.tanh(torch.einsum("thd,nd->thn", qq, kk) * scale / cap)
        d = 64 * 2.0 ** -23 * torch.einsum("thd,nd->thn", qq.abs(), kk.abs()) * abs(scale) + 2.0 ** -20 * (1 + x.abs())
        if cap <= 128:
            d = d + 2.0 ** -21 * cap
        if a.get("bias_slopes") is not None:
            fall = a["bias_slopes"].double()[:, None] * dist.abs().double()[:, None]
            x, d = x - fall, d + 2.0 ** -20 * fall
        x = torch.where(seen[:, None], x, -INF)
        d = torch.where(seen[:, None], d, 0.0).amax(-1)
        L = x.logsumexp(-1)
        w = (x - L[..., None]).exp()
        O, mag = torch.einsum("thn,nd->thd", w, kk), torch.einsum("thn,nd->thd", w, kk.abs())
        off, bound = (lse[at:at + ql].double() - L).abs(), d + n * 2.0 ** -24 + 2.0 ** -20 * (1 + L.abs())
        assert (off <= bound).all(), f"LSE off by {float((off / bound).max()):.3g} bounds"
        off, bound = (out[at:at + ql].double() - O).abs(), (u + 2 * d[..., None] + n * 2.0 ** -23 + 2.0 ** -20) * mag + u * O.abs() + tiny
        assert (off <= bound).all(), f"O off by {float((off / bound).max()):.3g} bounds"


@pytest.mark.parametrize("cap", [20.0, 128.0, 129.0, 1e3, 1e4, 1e6, 1e9, 2.0 ** 60, 2.0 ** 127])
@pytest.mark.parametrize("q_scale", [0.05, 3.0])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_large_caps_leave_small_scores_as_they_are(cap, q_scale, dt):
    p = problem(seed=45, dt=dt, heads=20, q_lens=(7, 60), lens=(300, 1500), layout_kv="PAGED", cap=cap, q_scale=q_scale, mode=4, left=700, right=0,
                bias=dt == "fp16")
    out, lse, status = run(p)
    assert status == 0
    check_capped(p, out, lse)


@pytest.mark.parametrize("cap", [129.0, 1e3, 1e4])
def test_scores_about_as_large_as_a_large_cap(cap):
    """|z| on both sides of 1; what is above it elsewhere in a warp changes no bit of a row."""
    p = problem(seed=46, heads=20, q_lens=(40,), lens=(500,), cap=cap, q_scale=cap)
    out, lse, _ = run(p)
    check_capped(p, out, lse)
    small = problem(seed=46, heads=20, q_lens=(40,), lens=(500,), cap=cap, q_scale=0.1)
    mixed = small["q"].clone()
    mixed[::2] = p["q"][::2]
    one, both = sfm.masked_attention(small["q"], p["kv"], **p["args"]), sfm.masked_attention(mixed, p["kv"], **p["args"])
    for x, y, z in zip(one, (out, lse), both):
        assert torch.equal(z[1::2], x[1::2]) and torch.equal(z[::2], y.view(z.shape)[::2])


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_weights_far_below_the_largest_keep_their_bits(dt):
    """Key j has one value, in column j: every weight e^-distance shows, off by its rounding and the result's (2 u), and 2^-17 of the sums."""
    n, kind = 40, DT[dt]
    kv = torch.zeros(n, 512, dtype=kind, device="cuda")
    kv[range(n), range(n)] = 2.0 ** 14
    q = torch.zeros(1, 2, 512, dtype=kind, device="cuda")
    out, lse = sfm.masked_attention(q, kv, bias_slopes=torch.tensor([1.0, 0.5], device="cuda"), mask_mode=4, win_left=13, win_right=0,
                                    cu_seqlens_q=ints([0, 1]), cu_seqlens_kv=ints([0, n]), layout_q="TND", layout_kv="TND")
    far = (n - 1 - torch.arange(n, device="cuda", dtype=F64))
    for h, slope in enumerate((1.0, 0.5)):
        w = torch.where(far <= 13, torch.exp(-slope * far), 0.0)
        assert ((out[0, h, :n].double() * 2.0 ** -14 - w / w.sum()).abs() <= (2 * half_step(kind) + 2.0 ** -17) * w / w.sum()).all()
        assert abs(float(lse[0, h]) - float(torch.log(w.sum()))) < 2.0 ** -18


@pytest.mark.parametrize("far", [60.0, 87.0, 88.5, 91.0, 200.0])
def test_a_part_far_below_another_one_of_zeros(far):
    """What is left of it are values of the type, off by the roundings of the LSEs' difference, of the type and by a step at the end of the range."""
    outs = [torch.zeros(3, 2, 512, dtype=torch.bfloat16, device="cuda"), randn(gen(43), 3, 2, 512, dtype=torch.bfloat16)]
    ends = [torch.zeros(3, 2, device="cuda"), torch.full((3, 2), -far, device="cuda")]
    got, lse = sfm.merge_attention(outs, ends)
    want = outs[1].double() * math.exp(-far)
    assert ((got.double() - want).abs() <= (2.0 ** -8 + far * 2.0 ** -22) * want.abs() + 2.0 ** -133).all() and (lse == 0).all()


def test_sinks_far_above_all_scores_leave_what_the_type_holds():
    """Every visible key far away under a steep bias: the rows are e^-80 and less of the keys, which bf16 holds."""
    p = problem(seed=41, heads=8, q_lens=(3,), lens=(300,), bias=True, sinks=True, prefix=(100,), mode=4, left=-1, right=-1)
    p["args"].update(mask_mode=4, win_left=0, win_right=0, key_begin=ints([5] * 3), key_end=ints([5] * 3))
    at, ql, cap, keys, dist, seen = p["seqs"][0]
    p["seqs"][0] = (at, ql, cap, keys, dist, (torch.arange(300, device="cuda") < 100).expand(3, 300))
    _, alone, _ = run(p, sinks=None)
    for above in (60.0, 85.0, 88.5, 90.0, 95.0, 300.0):
        p["args"]["sinks"] = alone.amax(0) + above
        out, lse, _ = run(p)
        check(p, out, lse)
        part, end = sfm.masked_attention(p["q"], p["kv"], **{**p["args"], "sinks": None})
        joined, _ = sfm.merge_attention([part], [end], sinks=p["args"]["sinks"])
        # three roundings of 2^-8, of the LSE (below 2^8) a few of 2^-16, and at the end of the range a step of 2^-133 each
        off = (joined.double() - out.double()).abs()
        assert (off <= 2.0 ** -6 * out.double().abs() + 2.0 ** -132).all()


def test_sinks_above_all_scores():
    p = problem(seed=21, heads=16, q_lens=(4,), lens=(50,))
    p["args"]["sinks"] = torch.full((16,), 500.0, device="cuda")
    out, lse, _ = run(p)
    assert (out == 0).all() and lse.isfinite().all()


# ---------------------------------------------------------------------------
# rows and values outside of what counts
# ---------------------------------------------------------------------------
def test_rows_behind_the_last_sequence():
    p = problem(seed=22, heads=20, q_lens=(5, 8), lens=(30, 9), rest=40)
    out, lse, _ = run(p)
    check(p, out, lse)
    assert (out[13:] == 0).all() and (lse[13:] == -INF).all()
    mine, ends = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    got, end, _ = run(p, out=mine, lse=ends)
    assert torch.equal(got[:13], out[:13]) and torch.equal(end[:13], lse[:13])
    assert (mine[13:] == 7).all() and (ends[13:] == 7).all()


def test_rows_behind_the_last_sequence_with_one_given_output():
    p = problem(seed=42, heads=20, q_lens=(5, 8), lens=(30, 9), rest=40)
    out, lse, _ = run(p)
    torch.full_like(lse, 7.0)          # (memory that a new tensor may get)
    mine = torch.full_like(out, 7.0)
    got, end, _ = run(p, out=mine)
    assert (mine[13:] == 7).all() and (end[13:] == -INF).all() and torch.equal(mine[:13], out[:13]) and torch.equal(end, lse)
    ends = torch.full_like(lse, 7.0)
    got, end, _ = run(p, lse=ends)
    assert (got[13:] == 0).all() and (ends[13:] == 7).all() and torch.equal(got, out) and torch.equal(ends[:13], lse[:13])


@pytest.mark.parametrize("layout", ["TND", "BSND"])
def test_used_queries(layout):
    go(seed=23, heads=16, q_lens=(40, 40, 40), lens=(100, 30, 50), used_q=(0, 17, 40), layout_q=layout, layout_kv=layout)


def test_bad_blocks_and_lengths():
    p = problem(seed=24, heads=16, q_lens=(30, 2), lens=(500, 400), layout_q="BSND", layout_kv="PAGED", block=48, mode=0)
    out, lse, _ = run(p)
    table = p["args"]["block_table"]
    for bad in (-1, p["kv"].shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 2] = bad
        got, end, status = run(p, block_table=t)
        assert status == sfm.STATUS_BAD_BLOCK
        q = dict(p, seqs=list(p["seqs"]))
        at, ql, cap, keys, dist, seen = q["seqs"][0]
        seen = seen.clone()
        seen[:, 96:144] = False
        q["seqs"][0] = (at, ql, cap, keys, dist, seen)
        check(q, got, end)
    for lens in ([5000, 400], [500, -3], [500, 2 ** 31 - 1]):
        got, end, status = run(p, seqused_kv=ints(lens), max_seqlen_kv=500)
        assert status & sfm.STATUS_BAD_LENGTH
        if lens[1] == 400:
            assert torch.equal(got, out)
        if lens[1] < 0:
            assert (got[30:32] == 0).all() and (end[30:32] == -INF).all()
    p = problem(seed=25, heads=16, q_lens=(30, 2), lens=(500, 400))
    for cu in ([0, 300, 32], [0, -5, 32], [40, 30, 32], [0, 30, 2 ** 31 - 1], [-2 ** 31, 30, 32]):
        _, _, status = run(p, cu_seqlens_q=ints(cu))
        assert status & sfm.STATUS_BAD_LENGTH
    for cu in ([0, 300, 3 << 28], [0, -5, 32], [-9, 500, 900], [1 << 30, 1 << 30, 1 << 30], [900, 500, 0]):
        _, _, status = run(p, cu_seqlens_kv=ints(cu))
        assert status & sfm.STATUS_BAD_LENGTH


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("most,split", [(9000, 0), (1000, 0), (9000, 512)])
def test_offsets_that_fall_cut_lengths_and_nothing_else(seed, most, split):
    """Long keys (ranges cut evenly or into pieces) and short ones: such a batch ends, says so, and leaves its surroundings alone."""
    r = random.Random(seed)
    B, T, heads = r.randint(3, 120), r.randint(200, 900), r.choice((16, 64))
    pool = randn(gen(seed), 200, 64, 512, dtype=torch.bfloat16)
    cols = -(-most // 64)
    args = dict(softmax_scale=512 ** -0.5, layout_q="TND", layout_kv="PAGED", max_seqlen_kv=most, split_keys=split,
                seqused_kv=ints([r.choice((0, 100, 700, most)) for _ in range(B)]),
                block_table=ints([[r.randrange(200) for _ in range(cols)] for _ in range(B)]))
    q = randn(gen(100 + seed), T, heads, 512, dtype=torch.bfloat16)
    fine = [0] + sorted(r.randint(0, T) for _ in range(B - 1)) + [T]
    want = sfm.masked_attention(q, pool, cu_seqlens_q=ints(fine), **args)
    for n in range(4):
        cu = list(fine)
        if n < 3:
            for _ in range(n + 1):
                i = r.randint(1, B - 1)
                cu[i], cu[i - 1] = cu[i - 1], cu[i]
        else:
            r.shuffle(cu)
        if all(x <= y for x, y in zip(cu, cu[1:])):
            cu[0] = T
        room, ends = torch.full((T + 16, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((T + 16, heads), 7.0, device="cuda")
        status = ints([0])
        sfm.masked_attention(q, pool, cu_seqlens_q=ints(cu), out=room[8:-8], lse=ends[8:-8], status=status, **args)
        assert int(status) == sfm.STATUS_BAD_LENGTH
        for x in (room, ends):
            assert (x[:8] == 7).all() and (x[-8:] == 7).all()
    again = sfm.masked_attention(q, pool, cu_seqlens_q=ints(fine), **args)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])


def test_far_offsets():
    """A page more than 2^32 bytes behind the start of its cache."""
    blocks = (1 << 32) // (1024 * 64) + 3
    pool = torch.empty(blocks, 64, 512, dtype=torch.bfloat16, device="cuda")
    p = problem(seed=26, heads=16, q_lens=(5,), lens=(128,))
    pool[blocks - 1], pool[1] = p["kv"][:64], p["kv"][64:128]
    args = {k: v for k, v in p["args"].items() if k != "cu_seqlens_kv"}
    args.update(layout_kv="PAGED", block_table=ints([[blocks - 1, 1]]), seqused_kv=ints([128]))
    out, lse = sfm.masked_attention(p["q"], pool, **args)
    check(p, out, lse)
    del pool
    # the last rows of q and out lie more than 2^31 values behind their starts
    n = (1 << 31) // (128 * 512) + 3
    p = problem(seed=27, heads=128, q_lens=(3,), lens=(40,))
    q = torch.zeros(n, 128, 512, dtype=torch.bfloat16, device="cuda")
    q[-3:] = p["q"]
    out, lse = sfm.masked_attention(q, p["kv"], **{**p["args"], "cu_seqlens_q": ints([n - 3, n])})
    check(p, out[-3:], lse[-3:])
    assert (out[:4] == 0).all() and (lse[:4] == -INF).all()


def test_pieces_of_one_size_make_rows_independent_of_the_batch():
    lens = (3000, 900, 128, 5000, 40)
    p = problem(seed=28, heads=16, q_lens=(2, 1, 7, 3, 5), lens=lens, sinks=True, layout_kv="PAGED")
    out, lse, _ = run(p, split_keys=512)
    table, used = p["args"]["block_table"], p["args"]["seqused_kv"]
    for b, (at, ql, *_) in enumerate(p["seqs"]):
        got, end = sfm.masked_attention(p["q"][at:at + ql], p["kv"], split_keys=512, **{
            **p["args"], "block_table": table[b:b + 1].clone(), "seqused_kv": used[b:b + 1].clone(), "cu_seqlens_q": ints([0, ql])})
        assert torch.equal(got, out[at:at + ql]) and torch.equal(end, lse[at:at + ql])


@pytest.mark.parametrize("keys,same,apart", [(640, (384, 512), (128, 640)), (1024, (512, 640, 896), (384, 1024)), (1500, (512, 640), (384, 768))])
def test_pieces_are_as_even_as_tiles_allow(keys, same, apart):
    """5, 8 and 12 tiles: at most split_keys keys in a piece, and no more pieces than that takes."""
    p = problem(seed=51, heads=64, q_lens=(2,), lens=(keys,), mode=0)
    runs = [run(p, split_keys=n)[:2] for n in same]
    check(p, *runs[0])
    for o, l in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(l, runs[0][1])
    for n in apart:
        o, l, _ = run(p, split_keys=n)
        check(p, o, l)
        assert not torch.equal(l, runs[0][1])      # (sums of 128 rows in other groups)


def test_same_inputs_same_bits():
    p = problem(seed=29, heads=64, q_lens=(40, 1, 9), lens=(3000, 20000, 77), layout_kv="PAGED")
    first = run(p)
    for _ in range(5):
        again = run(p)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ---------------------------------------------------------------------------
# joined results
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("tokens,heads,dim", [(1, 1, 512), (7, 20, 512), (33, 128, 512), (5, 3, 8), (4, 2, 1000), (3000, 16, 128)])
@pytest.mark.parametrize("parts", [1, 2, 3, 8])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("sinks", [False, True])
def test_merge(tokens, heads, dim, parts, dt, sinks):
    g, dtype = gen(parts), DT[dt]
    outs = [randn(g, tokens, heads, dim, dtype=dtype) for _ in range(parts)]
    lses = [5 * randn(g, tokens, heads) for _ in range(parts)]
    for i in range(parts):
        none = torch.rand(tokens, heads, generator=g, device="cuda") < 0.3
        lses[i][none] = -INF
        outs[i][none] = math.nan            # what has no keys is not read
    s = 3 * randn(g, heads) if sinks else None
    out, lse = sfm.merge_attention(outs, lses, sinks=s)
    L = torch.stack([x.double() for x in lses]).logsumexp(0)
    under = torch.logaddexp(L, s.double().expand_as(L)) if sinks else L
    want, mag = (torch.zeros(tokens, heads, dim, dtype=F64, device="cuda") for _ in range(2))
    for o, l in zip(outs, lses):
        w = torch.where(l == -INF, 0.0, (l.double() - under).exp())[..., None]
        v = torch.where(l[..., None] == -INF, 0.0, o.double())
        want, mag = want + w * v, mag + w * v.abs()
    empty = L == -INF
    assert torch.equal(lse == -INF, empty) and (out[empty] == 0).all()
    # weights off by exp's two steps and the rounding of its argument (|l| + |L| <= 60), at most ten sums, a division
    rel = 2.0 ** -24 * (60 + 16)
    assert ((out.double() - want).abs() <= half_step(dtype) * want.abs() + rel * mag + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps).all()
    off = torch.where(empty, 0.0, (lse.double() - L).abs())
    assert (off <= rel + 2.0 ** -22 * torch.where(empty, 0.0, L).abs()).all()
    same, _ = sfm.merge_attention(outs, lses, sinks=s, out=outs[-1])        # in the place of a part
    assert same is outs[-1] and torch.equal(same, out)


def test_merge_of_pieces_is_attention_of_the_whole():
    p, _, _ = go(seed=30, heads=16, q_lens=(40,), lens=(500,), sinks=True)
    parts = []
    for lo, hi in ((0, 100), (100, 470), (470, 500)):
        bounds = dict(key_begin=ints([lo] * 40), key_end=ints([hi] * 40))
        parts.append(sfm.masked_attention(p["q"], p["kv"], **{**p["args"], "sinks": None}, **bounds))
    out, lse = sfm.merge_attention([o for o, _ in parts], [l for _, l in parts], sinks=p["args"]["sinks"])
    # three roundings of the parts more than the whole has
    a, kk = p["args"], p["seqs"][0][3].double()
    x = torch.einsum("thd,nd->thn", p["q"].double(), kk) * a["softmax_scale"]
    x = torch.where(p["seqs"][0][5][:, None], x, -INF)
    L = x.logsumexp(-1)
    w = (x - torch.logaddexp(L, a["sinks"].double().expand_as(L))[..., None]).exp()
    O, mag = torch.einsum("thn,nd->thd", w, kk), torch.einsum("thn,nd->thd", w, kk.abs())
    assert ((lse - L).abs() <= 2e-3).all()
    assert ((out.double() - O).abs() <= (3 * half_step(torch.bfloat16) + 5e-3) * mag).all()


def test_lses_come_in_the_order_of_the_rows():
    g = gen(49)
    outs = [randn(g, 2, 5, 8, 64, dtype=torch.bfloat16) for _ in range(2)]
    lses = [randn(g, 2, 5, 8) for _ in range(2)]
    want = sfm.merge_attention(outs, lses)
    for shape in ((80,), (10, 8), (2, 5, 8, 1), (1, 10, 8), (80, 1), (1, 1, 80)):
        got = sfm.merge_attention(outs, [lses[0], lses[1].view(shape)])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for shape in ((2, 8, 5), (8, 10), (8, 2, 5), (5, 2, 8), (2, 40), (10, 8, 1, 2), (16, 5), (40, 2)):
        with pytest.raises(ValueError, match="lses"):
            sfm.merge_attention(outs, [lses[0], lses[1].new_zeros(shape)])
    one = [o[:, :, :1].contiguous() for o in outs]          # one head: rows are tokens
    for shape in ((2, 5, 1), (1, 10), (10, 1), (10,), (2, 1, 5)):
        got = sfm.merge_attention(one, [x[..., 0].contiguous().view(shape) for x in lses])
        assert torch.equal(got[0], want[0][:, :, :1]) and torch.equal(got[1], want[1][..., :1])


@pytest.mark.parametrize("sinks", [False, True])
def test_merge_with_sparse_flash_mla(sinks):
    """A window by sparse_flash_mla, whose LSE is flat, joined with compressed rows by masked_attention."""
    g, H, n = gen(50), 16, 4
    q = 3 * randn(g, 2, n, H, 512)
    q, kv, cmp = q.bfloat16(), randn(g, 2, 300, 1, 512, dtype=torch.bfloat16), randn(g, 2, 75, 512, dtype=torch.bfloat16)
    s, scale = (randn(g, H) if sinks else None), 512 ** -0.5
    md = sfm.sparse_flash_mla_metadata(H, 1, 512, batch_size=2, max_seqlen_q=n, max_seqlen_ori_kv=300, ori_mask_mode=4, ori_win_left=63,
                                       ori_win_right=0, has_cmp_kv=False, return_softmax_lse=True)
    near = sfm.sparse_flash_mla(q, metadata=md, ori_kv=kv, softmax_scale=scale)
    visible = ints([[(297 + i) // 4 for i in range(n)]] * 2)
    far = sfm.masked_attention(q, cmp, softmax_scale=scale, mask_mode=0, key_end=visible)
    out, lse = sfm.merge_attention([near[0], far[0]], [near[1], far[1]], sinks=s)
    assert near[1].dim() == 1 and out.shape == q.shape and lse.shape == q.shape[:-1]
    for b in range(2):
        keys = torch.cat((kv[b, :, 0], cmp[b])).double()
        for i in range(n):
            p = 296 + i
            j = torch.arange(300, device="cuda")
            seen = torch.cat(((j > p - 64) & (j <= p), torch.arange(75, device="cuda") < (p + 1) // 4))
            x = torch.where(seen, torch.einsum("hd,nd->hn", q[b, i].double(), keys) * scale, -INF)
            L = x.logsumexp(-1)
            w = (x - (torch.logaddexp(L, s.double()) if sinks else L)[:, None]).exp()
            O, mag = w @ keys, w @ keys.abs()
            # the weights' rounding, the parts' and the result's
            assert ((out[b, i].double() - O).abs() <= (3 * 2.0 ** -8 + 5e-3) * mag).all()
            assert ((lse[b, i].double() - L).abs() <= 2e-3).all()


# ---------------------------------------------------------------------------
# moved rows
# ---------------------------------------------------------------------------
def moved(cache, paths, first, table, block):
    """The definition, row by row, on copies."""
    before, after = cache.clone(), cache.clone()
    for b, path in enumerate(paths):
        last = -1
        for i, k in enumerate(path):
            if k <= last:
                break
            last = k

            def at(j):
                if table is None:
                    return (b, j) if 0 <= j < cache.shape[1] else None
                if not 0 <= j < len(table[b]) * block or not 0 <= table[b][j // block] < cache.shape[0]:
                    return None
                return table[b][j // block], j % block
            src, dst = at(first[b] + k), at(first[b] + i)
            if src is None or dst is None:
                break
            after[dst] = before[src]
    return after


@pytest.mark.parametrize("width,dtype", [(512, torch.bfloat16), (128, torch.float16), (656, torch.uint8), (528, torch.uint8),
                                         (128, torch.float8_e4m3fn), (8, torch.bfloat16), (4096, torch.float32)])
@pytest.mark.parametrize("block", [0, 5, 16, 64])
def test_move(width, dtype, block):
    r = random.Random(width + block)
    B, n = 9, 40
    paths = [sorted(r.sample(range(n), r.choice((0, 1, 2, 8, 9, 17, n)))) for _ in range(B)]
    paths[0] = list(range(n))                       # nothing moves
    paths[1] = list(range(20)) + list(range(21, n))  # everything behind a gap moves by one
    first = [r.randint(0, 30) for _ in range(B)]
    first[3] = 0
    raw = torch.randint(0, 256, ((B * 20 if block else B) * (block or 80), width * dtype.itemsize + 32), generator=torch.Generator().manual_seed(1),
                        dtype=torch.uint8).cuda()
    cache = raw[:, :width * dtype.itemsize].view(-1, block or 80, width * dtype.itemsize)
    table = None
    if block:
        ids = list(range(cache.shape[0]))
        r.shuffle(ids)
        table = [[ids.pop() for _ in range(-(-80 // block) if block > 5 else 16)] for _ in range(B)]
    want = moved(cache, paths, first, table, block)
    got = sfm.move_kv(cache.view(dtype), ints([p + [-1] * (n - len(p)) for p in paths]), ints(first),
                      block_table=ints(table) if block else None)
    assert torch.equal(got.view(torch.uint8), want)


def test_move_refuses_bad_values():
    cache = torch.arange(6 * 16 * 8, device="cuda").view(6, 16, 8).to(torch.float16)
    table = [[0, 1], [4, 9], [2, -1], [3, 5]]
    paths = [[2, 1, 5], [3, 20, 21], [1, 3, 17], [0, 31, 32]]
    first = [0, 0, 0, 0]
    for b in range(4):
        status = ints([0])
        want = moved(cache, [paths[b]], [first[b]], [table[b]], 16)
        got = sfm.move_kv(cache.clone(), ints([paths[b]]), ints([first[b]]), block_table=ints([table[b]]), status=status)
        assert torch.equal(got, want)
        assert int(status) == (sfm.STATUS_BAD_INDEX if b == 0 else sfm.STATUS_BAD_BLOCK)
    for start in (-1, -2 ** 31, 2 ** 31 - 1, 32):
        status = ints([0])
        got = sfm.move_kv(cache.clone(), ints([[1, 2]]), ints([start]), block_table=ints([[0, 1]]), status=status)
        assert torch.equal(got, cache) and int(status) == sfm.STATUS_BAD_BLOCK


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def drafted_layer(seed=0):
    """One layer of a model with a window and compressed rows, for a drafted tree: the drafted rows go into the cache, the
    tree attends to its window and to every visible compressed row, the two are joined, the accepted rows move up."""
    g = gen(seed)
    H, n, ratio, window = 16, 12, 4, 64
    lens = [300, 77]                                     # tokens before the tree
    table, pages = ints([[0, 1, 2, 3, 4, 5], [6, 7, 8, 9, 10, 11]]), 12
    s = dict(H=H, n=n, lens=lens, table=table, window=window, g=g)
    s["cache"] = randn(g, pages, 64, 512, dtype=torch.bfloat16)
    s["cmp"] = randn(g, 2, 75, 512, dtype=torch.bfloat16)
    parents = [-1, 0, 0, 1, 1, 2, 3, 3, 6, 7, 8, 9]
    bits, depth = [], []
    for i, k in enumerate(parents):
        bits.append((bits[k] if k >= 0 else 0) | 1 << i)
        depth.append(depth[k] + 1 if k >= 0 else 0)
    s["bits"], s["depth"] = bits, depth
    s["tree"] = ints([bits, bits], torch.int64).view(2, n, 1)
    s["pos"] = ints([[L + d for d in depth] for L in lens])
    s["used"] = ints([L + n for L in lens])
    s["slots"] = ints([int(table[b, (L + i) // 64]) * 64 + (L + i) % 64 for b, L in enumerate(lens) for i in range(n)])
    s["seen"] = ints([[(L + d + 1) // ratio for d in depth] for L in lens])
    s["q"], s["new"] = 3 * randn(g, 2, n, H, 512), randn(g, 2 * n, 512)
    s["q"], s["new"] = s["q"].bfloat16(), s["new"].bfloat16()
    s["sinks"] = randn(g, H)
    path = [0, 1, 3, 7, 9, 11]
    s["path"], s["first"] = ints([path + [-1] * 6, path[:3] + [-1] * 9]), ints(lens)
    return s


def drafted_step(s):
    flat = s["cache"].view(-1, 512)
    sfm.store_kv(s["new"], flat, slot_mapping=s["slots"], norm_eps=1e-6)
    near = sfm.tree_attention(s["q"], s["cache"], s["tree"], s["pos"], softmax_scale=512 ** -0.5, mask_mode=4,
                              win_left=s["window"] - 1, win_right=0, layout_kv="PAGED", block_table=s["table"], seqused_kv=s["used"],
                              max_seqlen_kv=384)
    far = sfm.masked_attention(s["q"], s["cmp"], softmax_scale=512 ** -0.5, mask_mode=0, key_end=s["seen"])
    out, lse = sfm.merge_attention([near[0], far[0]], [near[1], far[1]], sinks=s["sinks"])
    sfm.move_kv(s["cache"], s["path"], s["first"], block_table=s["table"])
    return out, lse


def test_a_drafted_tree_through_a_layer():
    s = drafted_layer()
    before = s["cache"].clone()
    out, lse = drafted_step(s)
    x = s["new"].double()
    rows = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    for b, L in enumerate(s["lens"]):
        kept = torch.cat([before[int(s["table"][b, j])] for j in range(6)])[:L].double()
        new = rows[b * 12:(b + 1) * 12].bfloat16().double()
        keys = torch.cat((kept, new, s["cmp"][b].double()))
        pos = torch.tensor(list(range(L)) + [L + d for d in s["depth"]], device="cuda")
        for i in range(12):
            p = L + s["depth"][i]
            seen = torch.cat((pos > p - s["window"], torch.arange(75, device="cuda") < (p + 1) // 4))
            for k in range(12):
                seen[L + k] &= bool(s["bits"][i] >> k & 1)
            y = torch.einsum("hd,nd->hn", s["q"][b, i].double(), keys) * 512 ** -0.5
            y = torch.where(seen, y, -INF)
            LL = y.logsumexp(-1)
            w = (y - torch.logaddexp(LL, s["sinks"].double())[:, None]).exp()
            O, mag = w @ keys, w @ keys.abs()
            # the weights' rounding, the parts' and the result's, and stored rows that round the other way at a tie (2^-8 |v|)
            assert ((out[b, i].double() - O).abs() <= (4 * 2.0 ** -8 + 5e-3) * mag).all()
            assert ((lse[b, i].double() - LL).abs() <= 2e-2).all()
    for b, (L, n) in enumerate(zip(s["lens"], (6, 3))):
        got = torch.cat([s["cache"][int(s["table"][b, j])] for j in range(6)])[L:L + n].double()
        want = rows[b * 12:(b + 1) * 12][[0, 1, 3, 7, 9, 11][:n]]
        assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * want.abs()).all()


def test_captured_step_replays_on_new_inputs():
    s, eager = drafted_layer(1), drafted_layer(1)
    drafted_step(s)
    s["cache"].copy_(eager["cache"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = drafted_step(s)
    for k in range(3):
        g = gen(50 + k)
        q, new, cache = randn(g, *s["q"].shape).bfloat16(), randn(g, *s["new"].shape).bfloat16(), randn(g, *s["cache"].shape).bfloat16()
        for x in (s, eager):
            x["q"].copy_(q), x["new"].copy_(new), x["cache"].copy_(cache)
        graph.replay()
        want = drafted_step(eager)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(s["cache"], eager["cache"])


def test_calls_on_two_streams_at_once():
    ps = [problem(seed=31, heads=64, q_lens=(3, 1), lens=(9000, 20000), layout_kv="PAGED"),
          problem(seed=32, heads=16, q_lens=(200, 100), lens=(700, 3000), tree=True)]
    want = [run(p)[:2] for p in ps]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, (s, p) in enumerate(zip(streams, ps)):
            got[i].append(p["call"](p["q"], p["kv"], stream=s, **p["args"]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o.reshape(want[i][0].shape), want[i][0]) and torch.equal(l.reshape(want[i][1].shape), want[i][1])


def test_chained_calls_read_what_the_calls_before_them_wrote():
    """Each result is the next call's query, without anything between the launches."""
    p = problem(seed=33, heads=16, q_lens=(8, 1), lens=(64, 12000), layout_kv="PAGED")
    x, want = p["q"], p["q"]
    for _ in range(6):
        x, _ = sfm.masked_attention(x, p["kv"], **p["args"])
    torch.cuda.synchronize()
    for _ in range(6):
        want, _ = sfm.masked_attention(want, p["kv"], **p["args"])
        torch.cuda.synchronize()
    assert torch.equal(x, want)


def test_given_buffers_and_no_queries():
    p = problem(seed=34, heads=16, q_lens=(3, 1), lens=(5000, 12000), layout_kv="PAGED")
    out, lse, _ = run(p)
    mine, ends, room = torch.zeros_like(out), torch.zeros_like(lse), torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    version = mine._version
    got = sfm.masked_attention(p["q"], p["kv"], out=mine, lse=ends, workspace=room, **p["args"])
    assert got[0] is mine and got[1] is ends and torch.equal(mine, out) and torch.equal(ends, lse) and mine._version > version
    q = torch.empty(0, 16, 512, dtype=torch.bfloat16, device="cuda")
    none, end = sfm.masked_attention(q, p["kv"], **{**p["args"], "cu_seqlens_q": ints([0, 0, 0])})
    assert none.shape == q.shape and end.shape == (0, 16)
    sfm.merge_attention([q], [torch.empty(0, 16, device="cuda")])
    cache = torch.zeros(2, 4, 8, dtype=torch.float16, device="cuda")
    sfm.move_kv(cache, torch.empty(2, 0, dtype=torch.int32, device="cuda"), ints([0, 0]))


@pytest.mark.parametrize("layout", ["BSND", "TND"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_sources_without_a_row(layout, dt):
    """A compressed cache before its first row: no row sees a key, and the joined result is the other part."""
    g, kind = gen(48), DT[dt]
    q = randn(g, 2, 3, 16, 512, dtype=kind)
    near = randn(g, 2, 40, 512, dtype=kind)
    args = dict(softmax_scale=512 ** -0.5, layout_q=layout, layout_kv=layout)
    if layout == "BSND":
        none, some, kw, lens = near[:, :0], near, {}, {}
    else:
        q, none, some = q.view(6, 16, 512), near.new_empty(0, 512), near.view(80, 512)
        args["cu_seqlens_q"] = ints([0, 3, 6])
        kw, lens = dict(cu_seqlens_kv=ints([0, 0, 0])), dict(cu_seqlens_kv=ints([0, 40, 80]))
    sinks = randn(g, 16)
    mask, place = torch.full((*q.shape[:-2], 1), -1, dtype=torch.int64, device="cuda"), torch.zeros(q.shape[:-2], dtype=torch.int32, device="cuda")
    ends = torch.full(q.shape[:-2], 7, dtype=torch.int32, device="cuda")
    for more in ({}, dict(mask_mode=0, key_end=ends), dict(prefix_lens=ints([5, 0])), dict(split_keys=128), dict(softcap=20.0, max_seqlen_kv=5000)):
        status = ints([0])
        out, lse = sfm.masked_attention(q, none, sinks=sinks, status=status, **{**args, **kw, **more})
        assert (out == 0).all() and (lse == -INF).all() and out.shape == q.shape and int(status) == 0
    mine, end = torch.ones_like(q), torch.ones(q.shape[:-1], device="cuda")
    sfm.tree_attention(q, none, mask, place, out=mine, lse=end, **args, **kw)
    assert (mine == 0).all() and (end == -INF).all()
    part = sfm.masked_attention(q, some, **args, **lens)
    joined = sfm.merge_attention([part[0], out], [part[1], lse])
    assert torch.equal(joined[0], part[0])
    again = sfm.masked_attention(q, some, **args, **lens)
    assert torch.equal(again[0], part[0]) and torch.equal(again[1], part[1])
    if layout == "TND":
        status = ints([0])
        out, lse = sfm.masked_attention(q, none, status=status, **{**args, "cu_seqlens_kv": ints([0, 4, 9])})
        assert int(status) == sfm.STATUS_BAD_LENGTH and (out == 0).all() and (lse == -INF).all()


def test_batches_without_a_sequence():
    kv, none = torch.zeros(30, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    for layout, kw in (("BSND", dict(kv=kv[None, :0].expand(0, 0, 512))), ("BSND", dict(kv=kv.new_empty(0, 30, 512))),
                       ("PAGED", dict(kv=kv[:16][None], block_table=none.view(0, 1), seqused_kv=none))):
        q = torch.empty(0, 3, 16, 512, dtype=torch.bfloat16, device="cuda")
        out, lse = sfm.masked_attention(q, layout_kv=layout, sinks=torch.zeros(16, device="cuda"), **kw)
        assert out.shape == q.shape and lse.shape == (0, 3, 16) and out.dtype is q.dtype and lse.dtype is torch.float32
        out, lse = sfm.tree_attention(q, tree_mask=torch.empty(0, 3, 1, dtype=torch.int64, device="cuda"), positions=none.view(0, 3), layout_kv=layout, **kw)
        assert out.shape == q.shape and lse.shape == (0, 3, 16)
        joined = sfm.merge_attention([out, out], [lse, lse])
        assert joined[0].shape == q.shape and joined[1].shape == (0, 3, 16)
    # of a packed batch every row lies behind the last sequence
    q = torch.ones(5, 16, 512, dtype=torch.bfloat16, device="cuda")
    args = dict(cu_seqlens_q=ints([0]), cu_seqlens_kv=ints([0]), layout_q="TND", layout_kv="TND")
    out, lse = sfm.masked_attention(q, kv, **args)
    assert (out == 0).all() and (lse == -INF).all() and lse.shape == (5, 16)
    mine, end = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    got = sfm.masked_attention(q, kv, out=mine, lse=end, **args)
    assert got[0] is mine and got[1] is end and (mine == 7).all() and (end == 7).all()
    got = sfm.masked_attention(q, kv, out=mine, **args)
    assert (mine == 7).all() and (got[1] == -INF).all()
    with pytest.raises(ValueError, match="cu_seqlens_q"):
        sfm.masked_attention(q, kv, **{**args, "cu_seqlens_q": none})
    with pytest.raises(sfm.SfmError, match="invalid"):
        sfm.masked_attention(q, kv, softcap=-1.0, **args)


def test_refusals():
    p = problem(seed=35, heads=16, q_lens=(3, 1), lens=(50, 20))
    q, kv, a = p["q"], p["kv"], p["args"]
    mask, pos = torch.zeros(4, 1, dtype=torch.int64, device="cuda"), ints([0] * 4)

    def bad(match, fn, *args, **kw):
        with pytest.raises((ValueError, sfm.SfmError), match=match):
            fn(*args, **kw)
    for name, x, word in (("q", q.float(), "dtype"), ("q", q.cpu(), "CUDA"), ("q", None, "not a tensor"), ("q", q[0], "dimensions"),
                          ("q", q[:, ::2], "contiguous"), ("q", q.clone().requires_grad_(), "gradient")):
        bad(word, sfm.masked_attention, x, kv, **a)
    for x, word in ((kv.half(), "kv"), (kv.cpu(), "kv"), (None, "kv"), (kv[None], "kv"), (kv[:, :256], "kv"),
                    (kv.clone().requires_grad_(), "gradient")):
        bad(word, sfm.masked_attention, q, x, **a)
    for kw, word in ((dict(cu_seqlens_q=None), "cu_seqlens_q"), (dict(cu_seqlens_kv=None), "invalid"), (dict(mask_mode=1), "invalid"),
                     (dict(mask_mode=4, win_left=-2), "invalid"), (dict(softcap=-1.0), "invalid"), (dict(softcap=math.nan), "invalid"),
                     (dict(softmax_scale=INF), "invalid"), (dict(split_keys=100), "invalid"), (dict(sinks=torch.zeros(15, device="cuda")), "sinks"),
                     (dict(bias_slopes=torch.zeros(16, dtype=F64, device="cuda")), "bias_slopes"), (dict(prefix_lens=ints([1])), "prefix_lens"),
                     (dict(key_begin=ints([1])), "key_begin"), (dict(key_end=[1, 2]), "key_end"), (dict(layout_kv="BSND"), "kv"),
                     (dict(layout_q="PAGED"), "layout"), (dict(block_table=ints([[0], [0]])), "invalid"), (dict(out=q.half()), "out"),
                     (dict(lse=torch.zeros(4, 15, device="cuda")), "lse"), (dict(status=torch.zeros(1, device="cuda")), "status"),
                     (dict(max_seqlen_kv=-1), "invalid"), (dict(workspace=torch.zeros(8)), "workspace")):
        bad(word, sfm.masked_attention, q, kv, **{**a, **kw})
    for m, t, word in ((None, pos, "tree_mask"), (mask, None, "tree_mask"), (mask.int(), pos, "tree_mask"), (mask[:3], pos, "tree_mask"),
                       (mask, pos[:3], "positions"), (mask[:, :0], pos, "tree_mask"), (mask.expand(4, 17).contiguous(), pos, "invalid")):
        bad(word, sfm.tree_attention, q, kv, m, t, **a)
    o, l = torch.zeros(4, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 16, device="cuda")
    for outs, lses, kw, word in (([], [], {}, "outs"), ([o], [], {}, "outs"), ([o] * 9, [l] * 9, {}, "outs"), ([o, o[:2]], [l, l], {}, "outs"),
                                 ([o, o.half()], [l, l], {}, "outs"), ([o], [l[:1]], {}, "lses"), ([o], [l.double()], {}, "lses"),
                                 ([o], [l], dict(sinks=l), "sinks"), ([o], [l], dict(lse=l), "lse"), ([o[..., :4].contiguous()], [l], {}, "alignment"),
                                 ([o.clone().requires_grad_()], [l], {}, "gradient")):
        bad(word, sfm.merge_attention, outs, lses, **kw)
    c = torch.zeros(4, 16, 64, dtype=torch.float16, device="cuda")
    path, first = ints([[0, 1]]), ints([0])
    for args, kw, word in (((c, path, first), {}, "cache"), ((c.cpu(), path, first), {}, "CUDA"), ((None, path, first), {}, "not a tensor"),
                           ((c[..., :4], path, first), dict(block_table=ints([[0]])), "alignment"), ((c[..., ::2], path, first), dict(block_table=ints([[0]])), "contiguous"),
                           ((c, path[0], first), dict(block_table=ints([[0]])), "path"), ((c, path.long(), first), dict(block_table=ints([[0]])), "path"),
                           ((c, path, ints([0, 1])), dict(block_table=ints([[0]])), "first"), ((c, path, first), dict(block_table=ints([0])), "block_table"),
                           ((c[0], path, first), {}, "cache")):
        bad(word, sfm.move_kv, *args, **kw)


def test_gradients_of_parameters_and_tangents_are_not_lost():
    p = problem(seed=47, heads=16, q_lens=(3, 1), lens=(50, 20), sinks=True, bias=True)
    tree = problem(seed=47, heads=16, q_lens=(3, 1), lens=(50, 20), sinks=True, bias=True, tree=True)
    o, l = torch.zeros(4, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 16, device="cuda")
    s = torch.nn.Parameter(torch.ones(16, device="cuda"))
    for name in ("sinks", "bias_slopes"):
        for x in (p, tree):
            want = run(x, **{name: s.detach()})
            with pytest.raises(ValueError, match=name + ".*gradient"):
                run(x, **{name: s})
            with torch.no_grad():
                got = run(x, **{name: s})
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(ValueError, match="sinks.*gradient"):
        sfm.merge_attention([o], [l], sinks=s)
    with torch.no_grad():
        sfm.merge_attention([o], [l], sinks=s)
    c, path, first = torch.zeros(1, 16, 64, dtype=torch.float16, device="cuda"), ints([[0, 1]]), ints([0])
    with torch.autograd.forward_ad.dual_level():
        def dual(x):
            return torch.autograd.forward_ad.make_dual(x, torch.ones_like(x))
        for name, args, kw in (("q", (dual(p["q"]), p["kv"]), p["args"]), ("kv", (p["q"], dual(p["kv"])), p["args"]),
                               ("sinks", (p["q"], p["kv"]), {**p["args"], "sinks": dual(s.detach())}),
                               ("bias_slopes", (p["q"], p["kv"]), {**p["args"], "bias_slopes": dual(s.detach())})):
            with pytest.raises(ValueError, match=name + ".*tangent"):
                sfm.masked_attention(*args, **kw)
        for name, args, kw in (("outs", ([o, dual(o)], [l, l]), {}), ("lses", ([o, o], [l, dual(l)]), {}), ("sinks", ([o], [l]), dict(sinks=dual(s.detach())))):
            with pytest.raises(ValueError, match=name + ".*tangent"):
                sfm.merge_attention(*args, **kw)
        with pytest.raises(ValueError, match="cache.*tangent"):
            sfm.move_kv(dual(c), path, first)
        run(p), sfm.merge_attention([o], [l]), sfm.move_kv(c, path, first)       # others go on as they are


def test_moved_rows_through_tables_without_blocks_are_refused():
    c = torch.arange(4 * 16 * 64, device="cuda").view(4, 16, 64).half()
    was = c.clone()
    with pytest.raises(sfm.SfmError, match="invalid"):
        sfm.move_kv(c, ints([[1, 2]] * 4), ints([0] * 4), block_table=torch.empty(4, 0, dtype=torch.int32, device="cuda"))
    assert torch.equal(c, was)
