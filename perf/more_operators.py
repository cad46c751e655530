"""Cases of the operators on a cache whose slots are not simply one token after the other:
drafted trees, and caches that drop keys.

tree    : attention of a tree of drafted tokens over a cache (Model.op_attention_tree)
commit  : the accepted rows of a tree moved together in the cache (Model.op_cache_commit)
weights : decode attention that adds up the weight of every key (Model.op_attention_decode_weights)
evict   : the keys of least weight dropped, the others moved together (Model.op_cache_evict)

`run` computes an operator in its plain form (elementary torch operations in
fp32, rounded once at the end) or, with `own`, by the library's call on the
same state. `exact` is the definition in fp64.
"""
import math
import random

import numpy as np
import torch

own = False

SCALES = (0.011, 0.013)  # k_scale, v_scale of the E4M3 caches


# ---------------------------------------------------------------- cases
def _tree(name, **kw):
    # context: cached tokens of a sequence, at most; rows: drafted tokens of a sequence;
    # even: every sequence drafts `rows`, else 1 .. rows; chain: one path, no mask
    c = dict(op="tree", dtype="bf16", batch=1, rows=26, even=True, chain=False, context=1024, n_q=64, n_kv=8,
             d=128, page=16, cap=0.0, bias=False, spread=1)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _commit(name, **kw):
    c = dict(op="commit", dtype="bf16", layers=32, batch=1, rows=26, accepted=4, context=1024, n_kv=8, d=128,
             page=16, e4m3=False, spread=1)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _weights(name, **kw):
    c = dict(op="weights", dtype="bf16", batch=1, context=1024, n_q=32, n_kv=32, d=128, page=16, cap=0.0,
             bias=False, spread=1)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _evict(name, **kw):
    # context: filled slots of a sequence, at most; even: all have that many
    c = dict(op="evict", dtype="bf16", layers=1, batch=1, context=1088, even=True, keep=1024, first=4, recent=256,
             n_kv=8, d=128, page=16, e4m3=False, spread=1)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one user's verify step: a small tree over a chat's context, where latency counts
        _tree("tree one sequence"),
        # a batch that drafts short trees of different sizes, ragged contexts, no grouping
        _tree("tree batch ragged", batch=32, rows=9, even=False, context=4096, n_q=32, n_kv=32, spread=2),
        # wide trees with grouped heads: more arithmetic than bytes
        _tree("tree wide", batch=32, rows=64, context=8192, page=64, spread=3),
        # drafted chains of a model with a distance bias and capped scores, contiguous cache
        _tree("tree chain bias", batch=5, rows=13, chain=True, context=2000, n_q=40, n_kv=40, page=0, cap=50.0,
              bias=True, spread=4),
        # after the verify step of one user: every layer's accepted rows
        _commit("commit one sequence"),
        # after the verify step of a serving batch, E4M3 cache
        _commit("commit batch e4m3", batch=64, rows=64, accepted=9, n_kv=32, page=64, e4m3=True, spread=2),
        # one sequence decoding in a cache held to about a thousand keys
        _weights("weights one sequence"),
        # a batch with grouped heads
        _weights("weights batch", batch=32, context=4096, n_q=64, n_kv=8, page=64, spread=2),
        # the largest: long contexts in front of an eviction
        _weights("weights long", batch=64, context=16384, n_q=32, n_kv=8, page=64, spread=3),
        # the rolling eviction of one sequence and layer: 64 new keys since the last
        _evict("evict rolling"),
        # a prompt cut down for decoding, every layer at once
        _evict("evict prompt", layers=32, context=4096, keep=1500, n_kv=32, spread=2),
        # a batch of ragged contexts in an E4M3 cache, grouped heads
        _evict("evict batch e4m3", layers=8, batch=32, context=7001, even=False, keep=2048, first=16, recent=500,
               page=64, e4m3=True, spread=3),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((32, 32), (40, 40), (64, 8), (32, 8), (16, 4), (8, 8), (12, 4), (16, 1), (5, 5))


def draw(rng):
    op = rng.choice(("tree", "tree", "commit", "weights", "weights", "evict"))
    spread = rng.randrange(1 << 20)
    n_q, n_kv = rng.choice(HEADS)
    cap = rng.choice((0.0, 0.0, 0.0, 30.0, 50.0))
    bias = rng.random() < 0.3
    page = rng.choice((0, 16, 32, 64))
    if op == "tree":
        rows = _log_int(rng, 1, 90)
        if rng.random() < 0.15:
            return _tree(None, dtype="f32", batch=rng.randint(1, 6), rows=rows, even=False, context=_log_int(rng, 1, 600),
                         n_q=8, n_kv=rng.choice((2, 8)), d=rng.choice((64, 128, 40)), page=page, cap=cap, bias=bias,
                         spread=spread)
        batch = _log_int(rng, 1, 64)
        return _tree(None, batch=batch, rows=rows, even=rng.random() < 0.5, chain=rng.random() < 0.3,
                     context=_log_int(rng, 1, max(2, min(9000, 120000000 // (batch * rows * n_q)))), n_q=n_q, n_kv=n_kv,
                     page=page, cap=cap, bias=bias, spread=spread)
    if op == "commit":
        e4m3 = rng.random() < 0.3
        rows = _log_int(rng, 1, 64)
        return _commit(None, dtype="f32" if not e4m3 and rng.random() < 0.2 else "bf16", layers=_log_int(rng, 1, 32),
                       batch=_log_int(rng, 1, 32), rows=rows, accepted=rng.randint(1, rows), context=_log_int(rng, 1, 2000),
                       n_kv=n_kv, page=page, e4m3=e4m3, spread=spread)
    if op == "weights":
        if rng.random() < 0.15:
            return _weights(None, dtype="f32", batch=rng.randint(1, 8), context=_log_int(rng, 1, 900), n_q=8,
                            n_kv=rng.choice((2, 8)), d=rng.choice((64, 128, 40)), page=page, cap=cap, bias=bias,
                            spread=spread)
        batch = _log_int(rng, 1, 64)
        return _weights(None, batch=batch, context=_log_int(rng, 1, min(20000, 6000000 // (batch * n_kv))), n_q=n_q,
                        n_kv=n_kv, page=page, cap=cap, bias=bias, spread=spread)
    e4m3 = rng.random() < 0.3
    layers, batch = _log_int(rng, 1, 16), _log_int(rng, 1, 16)
    context = _log_int(rng, 2, max(2, min(9000, 4000000 // (layers * batch * n_kv))))
    keep = rng.randint(1, context)
    first = rng.randint(0, min(16, keep))
    return _evict(None, dtype="f32" if not e4m3 and rng.random() < 0.2 else "bf16", layers=layers, batch=batch,
                  context=context, even=rng.random() < 0.5, keep=keep, first=first, recent=rng.randint(0, keep - first),
                  n_kv=n_kv, page=page, e4m3=e4m3, spread=spread)


# ---------------------------------------------------------------- layout of a case
def _plan(c):
    """Cached tokens (tree, commit: without the drafted ones) and drafted rows of every sequence."""
    r = random.Random(c["spread"] + 11)
    rows = [0] * c["batch"]
    if c["op"] == "tree":
        rows = [c["rows"] if c["even"] else r.randint(1, c["rows"]) for _ in rows]
    elif c["op"] == "commit":
        rows = [c["rows"]] * c["batch"]
    if c["op"] == "evict":
        return [c["context"] if c["even"] else r.randint(1, c["context"]) for _ in rows], rows
    return [r.randint(max(1, c["context"] // 2 if c["batch"] == 1 else c["context"] // 16), c["context"]) for _ in rows], rows


def _trees(c):
    """Per sequence the parent of every drafted row: row 0 is the last token that is known, the
    others hang on earlier rows, mostly on late ones."""
    r = random.Random(c["spread"] + 29)
    got = []
    for n in _plan(c)[1]:
        got.append([-1] + [i - 1 if c.get("chain") else max(0, i - 1 - int(r.expovariate(0.3))) for i in range(1, n)])
    return got


def _ancestors(parents):
    """Bit j of row i: i attends j (its ancestors and itself), and the rows' depths."""
    bits, depth = [], []
    for i, p in enumerate(parents):
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return bits, depth


def _paths(c):
    """Accepted rows of every sequence, ascending: some of the drafted ones, row 0 among them."""
    r = random.Random(c["spread"] + 31)
    got = []
    for n in _plan(c)[1]:
        k = min(n, c["accepted"] if c["batch"] == 1 else r.randint(1, c["accepted"]))
        got.append([0] + sorted(r.sample(range(1, n), k - 1)))
    return got


def _size(c):
    return 1 if c.get("e4m3") else 2 if c["dtype"] == "bf16" else 4


def _type(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def work(c):
    lens, rows = _plan(c)
    d, es, nkv = c["d"], _size(c), c["n_kv"]
    if c["op"] == "tree":
        keys = sum(a + b for a, b in zip(lens, rows))
        seen = sum(n * len(t) + sum(bin(x).count("1") for x in _ancestors(t)[0]) for n, t in zip(lens, _trees(c)))
        words = 0 if c["chain"] else -(-max(rows) // 32)
        return {"bytes": 2 * keys * nkv * d * es + sum(rows) * (2 * c["n_q"] * d * es + 4 * words),
                "flops": 4 * d * c["n_q"] * seen}
    if c["op"] == "commit":  # rows that are where they belong do not move
        moved = sum(sum(i != x for i, x in enumerate(p)) for p in _paths(c))
        return {"bytes": c["layers"] * 2 * nkv * d * es * 2 * moved + 4 * sum(map(len, _paths(c))), "flops": 0}
    if c["op"] == "weights":
        keys = sum(lens)
        return {"bytes": keys * nkv * (2 * d * es + 8) + 2 * c["batch"] * c["n_q"] * d * es,
                "flops": 4 * d * c["n_q"] * keys}
    heads, b = c["layers"] * nkv, 0
    for n in lens:
        # weights in and out, the list, and the rows behind the first one that goes (of n - first -
        # recent candidates, the first that goes is 1 / share in)
        m = min(n, c["keep"])
        rest = n - c["first"] - c["recent"]
        stay = c["first"] + rest / max(1, n - c["keep"]) if n > c["keep"] else m
        b += heads * (4 * n + 4 * max(lens) + 4 * m + 4 * d * es * max(0.0, m - stay))
    return {"bytes": int(b), "flops": 0}


# ---------------------------------------------------------------- inputs
def _randn(g, shape, dtype, std=1.0):
    t = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return (t * std).to(dtype) if std != 1.0 else t.to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _deal(counts, seed, skip):
    """Pages of a shuffled pool: a table [B, width] whose row b has -1 for its first skip[b] pages
    (which nothing here reads) and its own pages behind them, and the pool's size."""
    order = list(range(sum(counts)))
    random.Random(seed).shuffle(order)
    width = max(s + n for s, n in zip(skip, counts))
    rows, at = [], 0
    for s, n in zip(skip, counts):
        rows.append([-1] * s + order[at:at + n] + [-1] * (width - s - n))
        at += n
    return rows, at


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nkv, d, dt, page = c["n_kv"], c["d"], _type(c["dtype"]), c["page"]
    nq, layers, B = c.get("n_q", nkv), c.get("layers", 1), c["batch"]
    lens, rows = _plan(c)
    s = {"case": c}
    slots = [a + b for a, b in zip(lens, rows)]
    if page:
        skip = [n // page if c["op"] == "commit" else 0 for n in lens]  # only what a commit touches
        table, pages = _deal([-(-n // page) - k for n, k in zip(slots, skip)], c["spread"], skip)
        s["pages"] = _ints(table)
        shape = (layers, pages, nkv, page, d)
    else:
        s["pages"] = None
        shape = (layers, B, nkv, max(slots), d)
    if c.get("e4m3"):
        k, v = (_randn(g, shape, torch.bfloat16, 40.0).to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2))
    else:
        k, v = _randn(g, shape, dt, 1.5), _randn(g, shape, dt)
    s["k"], s["v"] = k, v
    if c["op"] == "tree":
        n = sum(rows)
        s["q"] = _randn(g, (n, nq, d), dt, 1.5)
        cu = [0]
        for x in rows:
            cu.append(cu[-1] + x)
        words = -(-max(rows) // 32)
        bits, at = [], []
        for start, t in zip(lens, _trees(c)):
            b, depth = _ancestors(t)
            bits += [[(x >> 32 * w & 0xffffffff) - (x >> 32 * w + 31 & 1) * (1 << 32) for w in range(words)] for x in b]
            at += [start + x for x in depth]
        s["cu"], s["start"], s["at"] = _ints(cu), _ints(lens), _ints(at)
        s["bits"] = None if c["chain"] else _ints(bits)
        s["out"] = torch.empty(n, nq * d, dtype=dt, device="cuda")
    elif c["op"] == "commit":
        paths = _paths(c)
        width = max(map(len, paths))
        s["start"], s["count"] = _ints(lens), _ints([len(p) for p in paths])
        s["path"] = _ints([p + [-1] * (width - len(p)) for p in paths])
    elif c["op"] == "weights":
        top = max(lens)
        s["q"] = _randn(g, (B, nq, d), dt, 1.5)
        s["positions"] = _ints([n - 1 for n in lens])
        # what some six earlier steps have left: a few keys have much of the weight
        s["weights"] = torch.rand(B, nkv, top, generator=g, device="cuda").log_().neg_().pow_(3).mul_(nq / nkv / top)
        s["scratch"] = torch.empty(B, nq, top, device="cuda")
        s["out"] = torch.empty(B, nq * d, dtype=dt, device="cuda")
    else:
        top = max(lens)
        s["lens"] = _ints(lens)
        w = torch.rand(layers, B, nkv, top, generator=g, device="cuda").log_().neg_().pow_(3)
        w[torch.rand(w.shape, generator=g, device="cuda") < 0.05] = 0.0  # keys that nobody looked at
        s["weights"], s["weights_out"] = w, torch.empty_like(w)
        s["kept"] = torch.empty(layers, B, nkv, c["keep"], dtype=torch.int32, device="cuda")
    if "cap" in c:
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, nq + 1, device="cuda").float() / nq) if c["bias"] else None
    if own:
        _handle(s, c, nq, layers, max(slots))
    return s


def _handle(s, c, nq, layers, top):
    """The library context, cache and option objects that a user's program keeps."""
    from llama2_decoder_forward_gb300 import binding, synth
    nkv, d, dt = c["n_kv"], c["d"], _type(c["dtype"])
    shape = synth.Shape(layers, 256, nq, nkv, d, 256, 256, dtype=c["dtype"])
    sizes = dict(attn_norm=(256,), wqkv=((nq + 2 * nkv) * d, 256), wo=(256, nq * d), ffn_norm=(256,),
                 w_gate=(256, 256), w_up=(256, 256), w_down=(256, 256))
    layer = {n: torch.zeros(z, dtype=dt, device="cuda") for n, z in sizes.items()}
    s["model"] = binding.Model(shape, {"layers": [layer] * layers}, max_batch=c["batch"], max_tokens=0, max_seq=top,
                               has_embed_head=False)
    if "cap" in c:
        s["scores"] = binding.Scores(cap=c["cap"], slopes=s["slopes"])
    kind = dict(n_pages=s["k"].shape[1], page_size=c["page"], page_table=s["pages"]) if c["page"] else \
        dict(batch=s["k"].shape[1], capacity=s["k"].shape[3])
    if c.get("e4m3"):
        kind["e4m3"] = SCALES
    s["cache"] = binding.KVCache(shape, k=s["k"], v=s["v"], **kind)


# ---------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if c["op"] == "tree":
        if own:
            s["model"].op_attention_tree(s["q"], s["cu"], s["start"], 0, s["cache"], s["out"], mask=s["bits"],
                                         positions=s["at"], scores=s["scores"])
            return s["out"]
        return _plain_tree(s)
    if c["op"] == "weights":
        if own:
            s["model"].op_attention_decode_weights(s["q"], s["positions"], 0, s["cache"], s["out"], s["weights"],
                                                   s["scratch"], scores=s["scores"])
            out = s["out"]
        else:
            out = _plain_weights(s)
        return {"out": out, "weights": s["weights"]}
    if c["op"] == "commit":
        if own:
            s["model"].op_cache_commit(s["cache"], s["start"], s["path"], s["count"])
        else:
            _plain_commit(s)
        return _values(s)
    if own:
        s["model"].op_cache_evict(s["cache"], s["lens"], c["keep"], s["weights"], s["kept"], first=c["first"],
                                  recent=c["recent"], weights_out=s["weights_out"])
    else:
        _plain_evict(s)
    return {"kept": s["kept"], "weights": s["weights_out"], **_values(s)}


def _values(s):
    """The caches, as the values that they stand for."""
    if s["case"]["e4m3"]:
        return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn)}
    return {"k": s["k"], "v": s["v"]}


def _softmax(t, c, slopes, distance, hidden):
    """Scale, cap, bias and mask of scores t [B, n_kv, G, rows, keys] in place, exponentials and their sums."""
    t.mul_(1.0 / math.sqrt(c["d"]))
    if c["cap"]:
        t.div_(c["cap"]).tanh_().mul_(c["cap"])
    if slopes is not None:
        t.sub_(slopes.view(c["n_kv"], -1, 1, 1) * distance[:, None, None])
    t.masked_fill_(hidden[:, None, None], -math.inf)
    t.sub_(t.amax(-1, keepdim=True)).exp_()
    return t, t.sum(-1, keepdim=True)


def _gathered(s, cache, top):
    """Layer 0 of slots 0 .. top - 1 of each sequence in fp32, [B, n_kv, top, d]."""
    at = torch.arange(top, device="cuda")
    if s["pages"] is None:
        return cache[0, :, :, :top].float()
    page = s["case"]["page"]
    return cache[0][s["pages"].long()[:, at // page].clamp(min=0), :, at % page].transpose(1, 2).float()


def _plain_tree(s):
    c = s["case"]
    nq, nkv, d, B, R = c["n_q"], c["n_kv"], c["d"], c["batch"], c["rows"]
    G = nq // nkv
    n = s["q"].shape[0]
    cu, start = s["cu"].long(), s["start"].long()
    row = torch.arange(n, device="cuda")
    seq = torch.searchsorted(cu[1:], row, right=True)
    i = row - cu[seq]
    q = torch.zeros(B, R, nq, d, device="cuda")
    q[seq, i] = s["q"].float()
    j = torch.arange(R, device="cuda")
    sees = torch.zeros(B, R, R, dtype=torch.bool, device="cuda")
    sees[seq, i] = j <= i[:, None] if c["chain"] else (s["bits"][:, j // 32] >> (j % 32)) & 1 == 1
    top = s["k"].shape[3] if s["pages"] is None else s["pages"].shape[1] * c["page"]
    key = torch.arange(top, device="cuda")
    own_key = key - start[:, None]  # index in the tree, [B, top]
    inside = (own_key >= 0) & (own_key < (cu[1:] - cu[:-1])[:, None])
    pick = own_key.clamp(0, R - 1)
    hidden = ~(sees.gather(2, pick[:, None].expand(B, R, top)) & inside[:, None] | (own_key < 0)[:, None])
    far = None
    if c["bias"]:
        at = torch.zeros(B, R, dtype=torch.long, device="cuda")
        at[seq, i] = s["at"].long()
        where = torch.where(inside, at.gather(1, pick), key)
        far = (at[:, :, None] - where[:, None]).abs().float()
    k, v = _gathered(s, s["k"], top), _gathered(s, s["v"], top)
    t = torch.matmul(q.view(B, R, nkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, nkv, G * R, d), k.transpose(2, 3))
    hidden[:, :, 0] &= (hidden.all(-1) & (j >= (cu[1:] - cu[:-1])[:, None])) == 0  # padding rows: any one key
    t, total = _softmax(t.view(B, nkv, G, R, top), c, s["slopes"], far, hidden)
    o = torch.matmul(t.view(B, nkv, G * R, top), v).view(B, nkv, G, R, d) / total
    return o.permute(0, 3, 1, 2, 4)[seq, i].reshape(n, nq * d).to(_type(c["dtype"]))


def _plain_weights(s):
    c = s["case"]
    nq, nkv, d, B = c["n_q"], c["n_kv"], c["d"], c["batch"]
    top = s["weights"].shape[-1]
    pos = s["positions"].long()[:, None]
    key = torch.arange(top, device="cuda")
    k, v = _gathered(s, s["k"], top), _gathered(s, s["v"], top)
    t = torch.matmul(s["q"].float().view(B, nkv, nq // nkv, d), k.transpose(2, 3))
    t, total = _softmax(t[:, :, :, None], c, s["slopes"], (pos - key).float()[:, None] if c["bias"] else None,
                        (key > pos)[:, None])
    p = (t / total)[:, :, :, 0]
    s["weights"].add_(p.sum(2))
    return torch.matmul(p, v).reshape(B, nq * d).to(_type(c["dtype"]))


def _move(s, src, dst):
    """Rows of slots src [layers, B, n_kv, n] of the cache to slots dst; -1 in src: none."""
    c = s["case"]
    ok = src >= 0
    layer, b, g, _ = torch.where(ok)
    for cache in (s["k"], s["v"]):
        if s["pages"] is None:
            cache[layer, b, g, dst[ok]] = cache[layer, b, g, src[ok]]
        else:
            page, pages = c["page"], s["pages"].long()
            cache[layer, pages[b, dst[ok] // page], g, dst[ok] % page] = \
                cache[layer, pages[b, src[ok] // page], g, src[ok] % page]


def _plain_commit(s):
    c = s["case"]
    i = torch.arange(s["path"].shape[1], device="cuda")
    start = s["start"].long()[:, None]
    src = torch.where(i < s["count"][:, None], start + s["path"], -1)
    full = (c["layers"], c["batch"], c["n_kv"], len(i))
    _move(s, src[:, None].expand(full), (start + i)[:, None].expand(full))


def _plain_evict(s):
    c = s["case"]
    keep, top = c["keep"], s["weights"].shape[-1]
    n = s["lens"].long()[:, None, None]
    slot = torch.arange(top, device="cuda")
    w = s["weights"].masked_fill((slot < c["first"]) | (slot >= n - c["recent"]), math.inf).masked_fill(slot >= n, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True)[1][..., :keep]
    kept = torch.sort(order.masked_fill(order >= n, top), -1)[0]
    if keep > kept.shape[-1]:
        kept = torch.nn.functional.pad(kept, (0, keep - kept.shape[-1]), value=top)
    there = kept < top
    _move(s, torch.where(there, kept, -1), torch.arange(keep, device="cuda").expand(kept.shape))
    s["kept"].copy_(torch.where(there, kept, -1))
    m = min(keep, top)
    s["weights_out"].zero_()
    s["weights_out"][..., :m] = s["weights"].gather(-1, kept[..., :m].clamp(max=top - 1)).where(there[..., :m], 0.0)


# ---------------------------------------------------------------- the definition in fp64
def _rows_of(s, cache, layer, b, slots):
    """Rows [n, n_kv, d] of the given slots of a sequence."""
    page = s["case"]["page"]
    if not page:
        return cache[layer, b, :, slots].transpose(0, 1)
    return cache[layer][s["pages"][b].long()[slots // page], :, slots % page]


def _attend(q, K, V, c, slopes, far, hidden):
    """Query rows q [heads, m, d] of one K/V head over K, V [n, d]: (weights, outputs)."""
    x = (q @ K.T) / math.sqrt(c["d"])
    if c["cap"]:
        x = torch.tanh(x / c["cap"]) * c["cap"]
    if slopes is not None:
        x = x - slopes.double()[:, None, None] * far
    if hidden is not None:
        x = x.masked_fill(hidden, -math.inf)
    p = torch.softmax(x, -1)
    return p, p @ V


def exact(c, seed):
    s = prepare(c, seed)
    nkv, d = c["n_kv"], c["d"]
    lens, rows = _plan(c)
    if c["op"] == "tree":
        nq, G = c["n_q"], c["n_q"] // nkv
        out = torch.empty(sum(rows), nq, d, dtype=torch.float64, device="cuda")
        lo = 0
        for b, (n, m, t) in enumerate(zip(lens, rows, _trees(c))):
            bits, depth = _ancestors(t)
            hidden = torch.zeros(m, n + m, dtype=torch.bool)
            hidden[:, n:] = torch.tensor([[not x >> j & 1 for j in range(m)] for x in bits])
            at = torch.tensor([n + x for x in depth])
            far = (at[:, None] - torch.cat((torch.arange(n), at))[None]).abs().double().cuda()
            slots = torch.arange(n + m, device="cuda")
            K, V = (_rows_of(s, s[x], 0, b, slots).double() for x in ("k", "v"))
            for g in range(nkv):
                hs = slice(g * G, g * G + G)
                o = _attend(s["q"][lo:lo + m, hs].double().transpose(0, 1), K[:, g], V[:, g], c,
                            s["slopes"][hs] if c["bias"] else None, far, hidden.cuda())[1]
                out[lo:lo + m, hs] = o.transpose(0, 1)
            lo += m
        return out.view(sum(rows), nq * d)
    if c["op"] == "weights":
        nq, G = c["n_q"], c["n_q"] // nkv
        out = torch.empty(c["batch"], nq, d, dtype=torch.float64, device="cuda")
        total = s["weights"].double()
        for b, n in enumerate(lens):
            slots = torch.arange(n, device="cuda")
            K, V = (_rows_of(s, s[x], 0, b, slots).double() for x in ("k", "v"))
            for g in range(nkv):
                hs = slice(g * G, g * G + G)
                p, o = _attend(s["q"][b, hs].double()[:, None], K[:, g], V[:, g], c,
                               s["slopes"][hs] if c["bias"] else None, (n - 1 - slots).double(), None)
                out[b, hs] = o[:, 0]
                total[b, g, :n] += p.sum((0, 1))
        return {"out": out.view(c["batch"], nq * d), "weights": total}
    if c["op"] == "commit":  # nothing is computed: rows move
        return None
    # of an eviction only the weights are numbers that could be rounded
    want = s["weights"].double().cpu()
    new = torch.zeros_like(want)
    for layer in range(c["layers"]):
        for b, n in enumerate(lens):
            if n <= c["keep"]:
                new[layer, b, :, :n] = want[layer, b, :, :n]
                continue
            for g in range(nkv):
                w = want[layer, b, g, :n].numpy()
                middle = c["first"] + np.argsort(-w[c["first"]:n - c["recent"]], kind="stable")
                kept = sorted([*range(c["first"]), *middle[:c["keep"] - c["first"] - c["recent"]], *range(n - c["recent"], n)])
                new[layer, b, g, :c["keep"]] = torch.from_numpy(w[kept])
    return {"kept": None, "weights": new, "k": None, "v": None}
