"""Attention over the shared KV rows with more kinds of masks and scores, and what drafted trees need around it.

Attention of prompts and single tokens whose scores may be capped by a tanh or
lowered with the distance, under document and prefix masks; attention of a tree
of drafted tokens over a cache; the joining of attention results over separate
sets of keys; and the moving of an accepted path's rows to the front of the
drafted ones.  ``run`` computes each in plain torch operations, or, with ``own``
set, through this repository's entry points.
"""
import math
import random

import torch

own = False

D = 512                                          # values of a shared KV row
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
MOST_PAIRS = 900_000_000                         # (query, head, key) triples of the largest case drawn


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _masked(name=None, **kw):
    c = dict(op="masked", batch=1, q_len=1, kv_len=1, ragged=False, heads=64, window=0, cap=0.0, bias=False, docs=0,
             prefix=0, sinks=False, block=0, dtype="bf16")
    c.update(kw)
    return dict(name=name, **c) if name else c


def _tree(name=None, **kw):
    c = dict(op="tree", batch=1, drafts=8, kv_len=1000, heads=64, window=0, cap=0.0, bias=False, sinks=False, block=64,
             dtype="bf16")
    c.update(kw)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one new token of two short sequences: latency
        _masked("capped_decode_short", batch=2, q_len=1, kv_len=300, heads=16, cap=30.0, block=16),
        # one new token per sequence over long caches, nearer keys count more
        _masked("distance_decode", batch=32, q_len=1, kv_len=32768, ragged=True, heads=64, bias=True, sinks=True, block=128),
        # a prompt packed of several documents
        _masked("document_prompt", batch=1, q_len=8191, kv_len=8191, heads=64, docs=5),
        # one prompt with capped scores
        _masked("capped_prompt", batch=1, q_len=4096, kv_len=4096, heads=64, cap=20.0, dtype="fp16"),
        # chunks of prompts behind cached tokens, the first of which every token sees; a window and falling scores behind them
        _masked("prefix_chunk", batch=4, q_len=2500, kv_len=6000, ragged=True, heads=48, bias=True, prefix=700, window=2048,
                block=64),
        # few drafted tokens of one sequence over a short cache with a window: latency
        _tree("tree_short", batch=1, drafts=7, kv_len=1000, heads=16, window=128, block=64),
        # a batch of drafted trees over medium caches
        _tree("tree_decode", batch=16, drafts=16, kv_len=16384, heads=128, sinks=True, block=128),
        # wide trees over long caches, capped scores that fall with the distance
        _tree("tree_wide", batch=4, drafts=61, kv_len=65000, heads=64, cap=30.0, bias=True, block=64, dtype="fp16"),
        # a decode batch: attention over the window joined with attention over selected rows, sinks counted once
        dict(name="merge_decode", op="merge", tokens=32, heads=64, parts=2, sinks=True, dtype="bf16"),
        # a prompt, three parts
        dict(name="merge_prompt", op="merge", tokens=4093, heads=64, parts=3, sinks=True, dtype="fp16"),
        # the accepted rows of a decode batch
        dict(name="move_decode", op="move", batch=32, drafts=16, kv_len=2000, most=5, width=512, block=64, dtype="bf16"),
        # a large batch of long drafts, rows of index keys
        dict(name="move_wide", op="move", batch=512, drafts=61, kv_len=900, most=24, width=128, block=16, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(("masked", "masked", "tree", "tree", "merge", "move"))
    dtype = rng.choice(("bf16", "fp16"))
    heads = rng.choice((1, 8, 16, 24, 48, 64, 100, 128))
    cap, bias, sinks = rng.choice((0.0, 0.0, 20.0, 50.0)), rng.random() < 0.4, rng.random() < 0.5
    if op == "masked":
        block = rng.choice((0, 16, 48, 64, 128))
        q_len = rng.choice((1, 1, 2, _log(rng, 3, 6000)))
        kv_len = q_len + _log(rng, 1, 40000)
        kv_len = max(q_len, min(kv_len, MOST_PAIRS // (q_len * heads)))
        batch = max(1, min(_log(rng, 1, 64), MOST_PAIRS // (q_len * kv_len * heads), 32 * 32768 // kv_len))
        return _masked(batch=batch, q_len=q_len, kv_len=kv_len, ragged=rng.random() < 0.6, heads=heads, cap=cap, bias=bias,
                       sinks=sinks, window=rng.choice((0, 0, 128, 1000)), docs=rng.choice((0, 0, 3, 9)) if q_len > 16 else 0,
                       prefix=rng.choice((0, 0, kv_len // 5)), block=block, dtype=dtype)
    if op == "tree":
        drafts, kv_len = _log(rng, 1, 128), _log(rng, 1, 65000)
        batch = max(1, min(_log(rng, 1, 64), MOST_PAIRS // (drafts * kv_len * heads), 32 * 32768 // kv_len))
        return _tree(batch=batch, drafts=drafts, kv_len=kv_len, heads=heads, cap=cap, bias=bias, sinks=sinks,
                     window=rng.choice((0, 0, 128)), block=rng.choice((16, 48, 64, 128)), dtype=dtype)
    if op == "merge":
        return dict(op=op, tokens=_log(rng, 1, 4093 * 64 // heads), heads=heads, parts=rng.randint(2, 4), sinks=sinks,
                    dtype=dtype)
    drafts = _log(rng, 2, 128)
    return dict(op=op, batch=_log(rng, 1, 512), drafts=drafts, kv_len=_log(rng, 1, 900), most=max(1, drafts // 3),
                width=rng.choice((64, 128, 512)), block=rng.choice((16, 48, 64)), dtype=dtype)


# ---------------------------------------------------------------------------
# what a case's sequences look like (the same for every seed)
# ---------------------------------------------------------------------------
def _rng(c):
    return random.Random("/".join(f"{k}={c[k]}" for k in sorted(c) if k != "name"))


def _sequences(c):
    """(new tokens, keys) of each sequence, the new ones among the keys."""
    r, out = _rng(c), []
    for b in range(c["batch"]):
        if c["op"] == "tree":
            out.append((c["drafts"], r.randint((c["kv_len"] + 1) // 2, c["kv_len"]) + c["drafts"]))
        elif c["ragged"]:
            q = r.randint((c["q_len"] + 1) // 2, c["q_len"])
            out.append((q, r.randint(max(q, (c["kv_len"] + 1) // 2), c["kv_len"])))
        else:
            out.append((c["q_len"], c["kv_len"]))
    return out


def _documents(c, q, n):
    """First key and one past the last key of the document of each of the last q of n tokens."""
    r = _rng(c)
    cuts = [0] + sorted(r.randint(1, n) for _ in range(c["docs"] - 1)) + [n]
    begin, end, d = [], [], 0
    for p in range(n - q, n):
        while p >= cuts[d + 1]:
            d += 1
        begin.append(cuts[d])
        end.append(cuts[d + 1])
    return begin, end


def _trees(c):
    """Per sequence the ancestors (bits, a token's own among them) and the depth of each drafted token."""
    r, out = _rng(c), []
    for b in range(c["batch"]):
        bits, depth = [1], [0]
        for i in range(1, c["drafts"]):
            parent = r.randrange(max(0, i - 8), i)
            bits.append(bits[parent] | 1 << i)
            depth.append(depth[parent] + 1)
        out.append((bits, depth))
    return out


def _paths(c):
    """Accepted tokens of each sequence, in order: the first one, then some behind the places that they move to."""
    r, out = _rng(c), []
    for b in range(c["batch"]):
        n = r.randint(1, min(c["most"], (c["drafts"] + 1) // 2))
        out.append([0] + sorted(r.sample(range(n, c["drafts"]), n - 1)))
    return out


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _pages(lens, block, seed):
    """A block table over a shuffled pool of pages, and the pages of the pool."""
    cols = max(-(-n // block) for n in lens)
    pages = [-(-n // block) for n in lens]
    perm = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table, at = torch.zeros(len(lens), cols, dtype=torch.int32), 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    return table.cuda(), sum(pages)


def _prepare_attention(c, seed):
    g, dt, H = _gen(seed), DTYPES[c["dtype"]], c["heads"]
    seqs = _sequences(c)
    q_lens, lens = [q for q, _ in seqs], [n for _, n in seqs]
    s = dict(case=c, seqs=seqs, scale=D ** -0.5)
    # scores of a few units, as trained heads have them
    s["q"] = (3.0 * _randn(g, sum(q_lens), H, D)).to(dt)
    s["cu_q"], s["cu_kv"] = _ints(_cu(q_lens)), _ints(_cu(lens))
    s["lens"] = _ints(lens)
    if c["block"]:
        s["table"], pool = _pages(lens, c["block"], seed)
        s["kv"] = _randn(g, pool, c["block"], D, dtype=dt)
    else:
        s["table"], s["kv"] = None, _randn(g, sum(lens), D, dtype=dt)
    s["sinks"] = _randn(g, H) if c["sinks"] else None
    s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, H + 1, device="cuda") / H) if c["bias"] else None
    s["begin"] = s["end"] = s["prefix"] = s["tree"] = s["positions"] = None
    if c["op"] == "tree":
        trees = _trees(c)
        words = -(-c["drafts"] // 64)
        flat = [[(m >> (64 * w)) & (1 << 64) - 1 for w in range(words)] for bits, _ in trees for m in bits]
        s["tree"] = _ints([[v - (1 << 64) if v >> 63 else v for v in row] for row in flat], torch.int64)
        s["positions"] = _ints([n - q + d for (q, n), (_, depth) in zip(seqs, trees) for d in depth])
        return s
    if c["docs"]:
        bounds = [_documents(c, q, n) for q, n in seqs]
        s["begin"], s["end"] = _ints([x for b, _ in bounds for x in b]), _ints([x for _, e in bounds for x in e])
    if c["prefix"]:
        s["prefix"] = _ints([min(c["prefix"], n) for n in lens])
    return s


def _prepare_merge(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    outs = [_randn(g, c["tokens"], c["heads"], D, dtype=dt) for _ in range(c["parts"])]
    lses = [3.0 + 2.0 * _randn(g, c["tokens"], c["heads"]) for _ in range(c["parts"])]
    # the last part has no keys at all for every seventh token (its result there is 0)
    none = torch.arange(c["tokens"], device="cuda") % 7 == 3
    lses[-1][none] = -math.inf
    outs[-1][none] = 0
    return dict(case=c, outs=outs, lses=lses, sinks=3.0 + _randn(g, c["heads"]) if c["sinks"] else None)


def _prepare_move(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    paths = _paths(c)
    first = [_rng(c).randint(0, c["kv_len"]) if b else c["kv_len"] for b in range(c["batch"])]
    table, pool = _pages([f + c["drafts"] for f in first], c["block"], seed)
    return dict(case=c, cache=_randn(g, pool, c["block"], c["width"], dtype=dt), table=table, first=_ints(first),
                path=_ints([p + [-1] * (c["drafts"] - len(p)) for p in paths]))


def prepare(case, seed):
    return dict(masked=_prepare_attention, tree=_prepare_attention, merge=_prepare_merge, move=_prepare_move)[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _keys(s, b):
    """The keys of sequence b in order."""
    q, n = s["seqs"][b]
    if s["table"] is None:
        at = sum(m for _, m in s["seqs"][:b])
        return s["kv"][at:at + n]
    block = s["case"]["block"]
    return s["kv"][s["table"][b, :-(-n // block)].long()].reshape(-1, D)[:n]


def _seen(s, b, at, i0, i1):
    """(visible, distance) of the keys of sequence b for its queries [i0, i1), which start at row `at`."""
    c, (q, n) = s["case"], s["seqs"][b]
    j = torch.arange(n, device="cuda")[None]
    rows = slice(at + i0, at + i1)
    if c["op"] == "tree":
        first = n - q
        p = s["positions"][rows].long()[:, None]
        place = torch.cat((torch.arange(first, device="cuda"), s["positions"][at:at + q].long()))[None]
        k = torch.arange(q, device="cuda")
        drafted = (s["tree"][rows][:, k // 64] >> (k % 64)) & 1 > 0
        seen = torch.cat((torch.ones(i1 - i0, first, dtype=torch.bool, device="cuda"), drafted), 1)
        if c["window"]:
            seen &= place > p - c["window"]
        return seen, p - place
    p = n - q + torch.arange(i0, i1, device="cuda")[:, None]
    seen = j <= p
    if c["window"]:
        seen = seen & (j > p - c["window"])
    if s["begin"] is not None:
        seen = seen & (j >= s["begin"][rows][:, None]) & (j < s["end"][rows][:, None])
    if s["prefix"] is not None:
        seen = seen | (j < s["prefix"][b])
    return seen, p - j


def _plain_attention(s):
    c, H = s["case"], s["case"]["heads"]
    out, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], device="cuda")
    at = 0
    for b, (q, n) in enumerate(s["seqs"]):
        k = _keys(s, b).float()
        step = max(1, (1 << 29) // (H * n))
        for i in range(0, q, step):
            e = min(q, i + step)
            x = torch.matmul(s["q"][at + i:at + e].float().view(-1, D), k.t()).view(e - i, H, n) * s["scale"]
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            seen, distance = _seen(s, b, at, i, e)
            if c["bias"]:
                x = x - s["slopes"][:, None] * distance.abs().float()[:, None]
            x = torch.where(seen[:, None], x, -math.inf)
            m = x.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, 0.0, m)
            p = torch.exp(x - m)
            total = p.sum(-1, keepdim=True)
            under = total + torch.exp(s["sinks"][:, None] - m) if c["sinks"] else total
            o = torch.matmul(p.view(-1, n), k).view(e - i, H, D) / torch.where(under == 0, 1.0, under)
            out[at + i:at + e] = o.to(out.dtype)
            lse[at + i:at + e] = (m + torch.log(total))[..., 0]
        at += q
    return out, lse


def _plain_merge(s):
    lses = torch.stack(s["lses"])
    m = lses.amax(0)
    m = torch.where(m == -math.inf, 0.0, m)
    w = torch.exp(lses - m)
    total = w.sum(0)
    under = total + torch.exp(s["sinks"] - m) if s["sinks"] is not None else total
    o = sum(w[i][..., None] * x.float() for i, x in enumerate(s["outs"])) / torch.where(under == 0, 1.0, under)[..., None]
    return o.to(s["outs"][0].dtype), m + torch.log(total)


def _plain_move(s):
    c = s["case"]
    rows = s["cache"].view(-1, c["width"])

    def at(i):
        j = s["first"].long()[:, None] + i
        return torch.gather(s["table"].long(), 1, j // c["block"]) * c["block"] + j % c["block"]

    path = s["path"].long()
    moved = path >= 0
    to, where = at(torch.arange(path.shape[1], device="cuda")[None].expand_as(path)), at(path.clamp(min=0))
    rows[to[moved]] = rows[where[moved]]
    return s["cache"]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own(s):
    import sparse_shared_kv_gb300 as sfm
    c = s["case"]
    if c["op"] == "merge":
        return sfm.merge_attention(s["outs"], s["lses"], sinks=s["sinks"])
    if c["op"] == "move":
        return sfm.move_kv(s["cache"], s["path"], s["first"], block_table=s["table"])
    lengths = dict(cu_seqlens_q=s["cu_q"], layout_q="TND", max_seqlen_q=max(q for q, _ in s["seqs"]),
                   max_seqlen_kv=max(n for _, n in s["seqs"]))
    if s["table"] is None:
        lengths.update(cu_seqlens_kv=s["cu_kv"], layout_kv="TND")
    else:
        lengths.update(block_table=s["table"], seqused_kv=s["lens"], layout_kv="PAGED")
    if c["window"]:
        lengths.update(mask_mode=4, win_left=c["window"] - 1, win_right=0)
    scores = dict(softmax_scale=s["scale"], softcap=c["cap"], bias_slopes=s["slopes"], sinks=s["sinks"])
    if c["op"] == "tree":
        return sfm.tree_attention(s["q"], s["kv"], s["tree"], s["positions"], **lengths, **scores)
    return sfm.masked_attention(s["q"], s["kv"], key_begin=s["begin"], key_end=s["end"], prefix_lens=s["prefix"], **lengths,
                                **scores)


def run(state):
    if own:
        return _own(state)
    return dict(masked=_plain_attention, tree=_plain_attention, merge=_plain_merge, move=_plain_move)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "merge":
        rows = c["tokens"] * c["heads"]
        return dict(bytes=rows * (c["parts"] + 1) * (2 * D + 4), flops=2 * rows * c["parts"] * D)
    if c["op"] == "move":
        rows = sum(len(p) - 1 for p in _paths(c))
        return dict(bytes=4 * c["width"] * rows + 4 * c["batch"] * (c["drafts"] + 1), flops=0)
    pairs = keys = queries = 0
    trees = _trees(c) if c["op"] == "tree" else None
    for b, (q, n) in enumerate(_sequences(c)):
        queries += q
        prefix = min(c.get("prefix", 0), n)
        bounds = _documents(c, q, n) if c.get("docs") else None
        low, high = n, 0
        for i in range(q):
            if trees:
                p = n - q + trees[b][1][i]
                own_keys = trees[b][1][i] + 1              # the path down to the token itself
                lo, hi = max(0, p - c["window"] + 1) if c["window"] else 0, n - q
                own_keys = min(own_keys, c["window"]) if c["window"] else own_keys
                pairs += max(0, hi - lo) + own_keys
                low, high = min(low, lo), n
                continue
            p = n - q + i
            lo, hi = max(0, p - c["window"] + 1) if c["window"] else 0, p + 1
            if bounds:
                lo, hi = max(lo, bounds[0][i]), min(hi, bounds[1][i])
            pairs += max(0, hi - max(lo, prefix)) + prefix
            low, high = min(low, max(lo, prefix)), max(high, hi)
        keys += prefix + max(0, high - low)
    rows = queries * c["heads"]
    return dict(bytes=rows * (4 * D + 4) + 2 * D * keys, flops=4 * D * pairs * c["heads"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_attention(c, seed):
    s = prepare(c, seed)
    H = c["heads"]
    slopes = s["slopes"].double() if c["bias"] else None
    outs, lses, at = [], [], 0
    trees = _trees(c) if c["op"] == "tree" else None
    for b, (q, n) in enumerate(s["seqs"]):
        rows = torch.arange(n, device="cuda")
        if s["table"] is None:
            rows = rows + sum(m for _, m in s["seqs"][:b])
        else:
            rows = s["table"][b].long()[rows // c["block"]] * c["block"] + rows % c["block"]
        keys = s["kv"].reshape(-1, D)[rows].double()
        place = list(range(n - q)) + [n - q + d for d in trees[b][1]] if trees else list(range(n))
        place = torch.tensor(place, device="cuda")
        bounds = _documents(c, q, n) if c.get("docs") else None
        step = max(1, (1 << 27) // (H * n))
        for i in range(0, q, step):
            e = min(q, i + step)
            allowed = torch.zeros(e - i, n, dtype=torch.bool)
            where = []
            for t in range(i, e):
                p = n - q + (trees[b][1][t] if trees else t)
                where.append(p)
                row = allowed[t - i]
                lo = max(0, p - c["window"] + 1) if c["window"] else 0
                if trees:
                    row[lo:n - q] = True
                    for k in range(t + 1):
                        if trees[b][0][t] >> k & 1 and n - q + trees[b][1][k] >= lo:
                            row[n - q + k] = True
                else:
                    hi = p + 1
                    if bounds:
                        lo, hi = max(lo, bounds[0][t]), min(hi, bounds[1][t])
                    row[lo:max(lo, hi)] = True
                    row[:min(c["prefix"], n)] = True
            allowed = allowed.cuda()
            last = int(allowed.any(0).nonzero().max()) + 1 if bool(allowed.any()) else 1
            y = torch.einsum("thd,nd->htn", s["q"][at + i:at + e].double(), keys[:last]) * s["scale"]
            if c["cap"]:
                y = torch.tanh(y / c["cap"]) * c["cap"]
            if c["bias"]:
                y -= slopes[:, None, None] * (torch.tensor(where, device="cuda")[:, None] - place[:last]).abs()
            y.masked_fill_(~allowed[:, :last], -math.inf)
            total = torch.logsumexp(y, -1)                               # heads, tokens
            under = torch.logaddexp(total, s["sinks"].double()[:, None].expand_as(total)) if c["sinks"] else total
            y.sub_(torch.where(under == -math.inf, 0.0, under)[..., None]).exp_()
            outs.append(torch.einsum("htn,nd->thd", y, keys[:last]))
            lses.append(total.t())
        at += q
    return torch.cat(outs), torch.cat(lses)


def _exact_merge(c, seed):
    s = prepare(c, seed)
    total = torch.full_like(s["lses"][0], -math.inf, dtype=torch.float64)
    for x in s["lses"]:
        total = torch.logaddexp(total, x.double())
    under = torch.logaddexp(total, s["sinks"].double().expand_as(total)) if c["sinks"] else total
    out = torch.zeros(s["outs"][0].shape, dtype=torch.float64, device="cuda")
    for x, y in zip(s["lses"], s["outs"]):
        out += (x.double() - under).exp()[..., None] * y.double()
    return out, total


def _exact_move(c, seed):
    s = prepare(c, seed)
    before = s["cache"].clone()
    table, first = s["table"].tolist(), s["first"].tolist()
    places = [[], []]
    for b, path in enumerate(_paths(c)):
        for i, k in enumerate(path):
            for j, out in ((first[b] + i, places[0]), (first[b] + k, places[1])):
                out.append(table[b][j // c["block"]] * c["block"] + j % c["block"])
    after = before.clone().view(-1, c["width"])
    after.index_copy_(0, _ints(places[0], torch.int64), before.view(-1, c["width"]).index_select(0, _ints(places[1], torch.int64)))
    return after.view_as(before)


def exact(case, seed):
    return dict(masked=_exact_attention, tree=_exact_attention, merge=_exact_merge, move=_exact_move)[case["op"]](case, seed)
