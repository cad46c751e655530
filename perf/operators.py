"""Cases of the attention operators beside the plain Llama2 path.

append : head norms, rotation and cache append of new rows in one pass
         (Model.op_rope_norm_append)
docs   : prompt attention over packed documents, with capped scores, a
         distance bias or a bidirectional prefix (Model.op_attention_docs)
shared : decode attention of a batch whose first keys are the same for every
         sequence (Model.op_attention_decode_shared)

`run` computes an operator in its plain form (elementary torch operations in
fp32, rounded once at the end) or, with `own`, by the library's call on the
same state. `exact` is the definition in fp64.
"""
import math
import random

import torch

own = False

SCALES = (0.011, 0.013)  # k_scale, v_scale of the E4M3 caches


# ---------------------------------------------------------------- cases
def _append(name, **kw):
    c = dict(op="append", dtype="bf16", src="f32", rows=1, seqs=1, n_q=64, n_kv=8, d=128, rotary=128,
             half=True, norm=True, page=64, start=1000, e4m3=False, spread=1)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _docs(name, **kw):
    c = dict(op="docs", dtype="bf16", rows=1024, docs=1, n_q=32, n_kv=32, d=128, cap=0.0, bias=False,
             prefix=False, spread=1)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _shared(name, **kw):
    c = dict(op="shared", dtype="bf16", batch=32, n_q=32, n_kv=32, d=128, prefix=0, own_max=1024, page=16,
             cap=0.0, bias=False, spread=1)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a single user's next token: one row, where the launch is all the time
        _append("append one token", src="bf16", page=16),
        # a decode step of a batch on an E4M3 cache
        _append("append batch e4m3", rows=32, seqs=32, half=False, norm=False, e4m3=True, spread=2),
        # prompts of different lengths joining a serving batch, rotated in half of the head
        _append("append prompts", rows=8192, seqs=6, n_q=32, n_kv=32, rotary=64, start=3000, spread=3),
        # a chat turn: one short prompt of a model with capped scores
        _docs("docs short prompt", rows=100, cap=50.0),
        # training-style packing: many documents in one row of tokens, distance bias
        _docs("docs packed", rows=8192, docs=17, n_q=64, n_kv=8, bias=True, spread=2),
        # one long prompt, capped scores, grouped heads
        _docs("docs long prompt", rows=8192, n_q=64, n_kv=8, cap=30.0, spread=3),
        # prompts whose first part (an instruction, an image) attends both ways
        _docs("docs prefix", rows=2500, docs=3, prefix=True, spread=4),
        # the fp32 model of the parity tests, every score option at once
        _docs("docs fp32", dtype="f32", rows=700, docs=2, n_q=8, n_kv=2, d=64, cap=20.0, bias=True,
              prefix=True, spread=5),
        # one sequence decoding alone, capped scores: latency of the split-key path
        _shared("shared one sequence", batch=1, cap=50.0),
        # a batch over one system prompt, distance bias, no grouping
        _shared("shared batch bias", prefix=500, own_max=600, bias=True, spread=2),
        # a batch over a long shared document, grouped heads, capped scores
        _shared("shared long prefix", batch=64, n_q=64, n_kv=8, prefix=8192, own_max=512, page=64,
                cap=30.0, spread=3),
        # the largest serving batch: shared prefix and long own contexts
        _shared("shared large batch", batch=128, n_q=64, n_kv=8, prefix=16384, own_max=3500, page=64,
                spread=4),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((32, 32), (40, 40), (64, 8), (16, 4), (8, 8), (12, 4), (16, 1), (5, 5))


def draw(rng):
    op = rng.choice(("append", "docs", "shared"))
    spread = rng.randrange(1 << 20)
    n_q, n_kv = rng.choice(HEADS)
    cap = rng.choice((0.0, 0.0, 20.0, 30.0, 50.0))
    bias = rng.random() < 0.4
    if op == "append":
        seqs = _log_int(rng, 1, 64)
        rows = seqs if rng.random() < 0.4 else max(seqs, _log_int(rng, 1, 6000))
        page = rng.choice((0, 16, 32, 64, 128))
        e4m3 = rng.random() < 0.25 and n_q // n_kv <= 8
        return _append(None, src=rng.choice(("f32", "bf16")), rows=rows, seqs=seqs, n_q=n_q, n_kv=n_kv,
                       rotary=rng.choice((128, 128, 96, 64, 32, 24)), half=rng.random() < 0.6,
                       norm=rng.random() < 0.6, page=page, start=_log_int(rng, 1, 2000), e4m3=e4m3,
                       spread=spread)
    if op == "docs":
        if rng.random() < 0.2:
            return _docs(None, dtype="f32", rows=_log_int(rng, 1, 900), docs=rng.randint(1, 4), n_q=8,
                         n_kv=rng.choice((2, 8)), d=rng.choice((64, 128, 40)), cap=cap, bias=bias,
                         prefix=rng.random() < 0.4, spread=spread)
        return _docs(None, rows=_log_int(rng, 16, 4500), docs=_log_int(rng, 1, 16), n_q=n_q, n_kv=n_kv,
                     cap=cap, bias=bias, prefix=rng.random() < 0.3, spread=spread)
    if rng.random() < 0.15:
        return _shared(None, dtype="f32", batch=rng.randint(1, 8), n_q=8, n_kv=rng.choice((2, 8)), d=64,
                       prefix=rng.choice((0, 77, 300)), own_max=_log_int(rng, 1, 300),
                       page=rng.choice((0, 16)), cap=cap, bias=bias, spread=spread)
    batch = _log_int(rng, 1, 100)
    prefix = rng.choice((0, _log_int(rng, 16, 9000), _log_int(rng, 16, 9000)))
    page = rng.choice((0, 16, 32, 64)) if batch * n_kv * prefix < 3000000 else 64
    return _shared(None, batch=batch, n_q=n_q, n_kv=n_kv, prefix=prefix,
                   own_max=_log_int(rng, 1, min(1500, 3000000 // (batch * n_kv))), page=page, cap=cap, bias=bias,
                   spread=spread)


# ---------------------------------------------------------------- layout of a case
def _parts(total, n, seed):
    """total split into n positive lengths (n <= total)."""
    r = random.Random(seed)
    cuts = sorted(r.sample(range(1, total), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _plan(c):
    r = random.Random(c["spread"] + 7)
    if c["op"] == "append":
        lens = _parts(c["rows"], c["seqs"], c["spread"])
        return lens, [r.randint(0, c["start"]) for _ in lens]
    if c["op"] == "docs":
        n = min(c["docs"], c["rows"])
        lens = _parts(c["rows"], n, c["spread"])
        return lens, [r.randint(0, x) if c["prefix"] else 0 for x in lens]
    return [c["prefix"] + r.randint(1, c["own_max"]) for _ in range(c["batch"])], None


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def _type(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _pairs(lens, pre):
    """Kept (query, key) pairs of causal documents with a two-way prefix."""
    return sum(n * (n + 1) // 2 + p * (p - 1) // 2 for n, p in zip(lens, pre))


def work(c):
    nq, nkv, d, es = c["n_q"], c["n_kv"], c["d"], _size(c["dtype"])
    lens, more = _plan(c)
    if c["op"] == "append":
        rows, src = c["rows"], _size(c["src"])
        cache = 1 if c["e4m3"] else es
        side = 0 if c["rows"] == c["seqs"] else 2 * nkv * d * es
        positions = len({p for n, s in zip(lens, more) for p in range(s, s + n)})
        b = rows * ((nq + 2 * nkv) * d * src + nq * d * es + 2 * nkv * d * cache + side)
        b += positions * c["rotary"] * 4
        f = rows * (nq + nkv) * (3 * c["rotary"] + (4 * d if c["norm"] else 0))
        return {"bytes": b, "flops": f}
    if c["op"] == "docs":
        return {"bytes": c["rows"] * (2 * nq + 2 * nkv) * d * es, "flops": 4 * d * nq * _pairs(lens, more)}
    keys = c["prefix"] + sum(n - c["prefix"] for n in lens)
    return {"bytes": 2 * keys * nkv * d * es + 2 * c["batch"] * nq * d * es, "flops": 4 * d * nq * sum(lens)}


# ---------------------------------------------------------------- inputs
def _randn(g, shape, dtype, std=1.0):
    t = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return (t * std).to(dtype) if std != 1.0 else t.to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cumulative(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _page_table(counts, seed, width=None):
    """Pages of a shuffled pool dealt out in order: (table [B, width], pages)."""
    order = list(range(sum(counts)))
    random.Random(seed).shuffle(order)
    width = width or max(counts)
    rows, at = [], 0
    for n in counts:
        rows.append(order[at:at + n] + [-1] * (width - n))
        at += n
    return rows, at


def _rope_table(positions, rotary):
    """(cos, sin) [positions][rotary / 2][2] of a context stretched four times by linear scaling."""
    f = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] / 4.0 * f
    return torch.stack((a.cos(), a.sin()), -1).float().contiguous()


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nq, nkv, d, dt = c["n_q"], c["n_kv"], c["d"], _type(c["dtype"])
    lens, more = _plan(c)
    s = {"case": c}
    if c["op"] == "append":
        last = max(n + p for n, p in zip(lens, more))
        s["qkv"] = _randn(g, (c["rows"], (nq + 2 * nkv) * d), _type(c["src"]))
        s["q_gain"] = (1 + 0.1 * _randn(g, (d,), torch.float32)).to(dt) if c["norm"] else None
        s["k_gain"] = (1 + 0.1 * _randn(g, (d,), torch.float32)).to(dt) if c["norm"] else None
        s["table"] = _rope_table(last, c["rotary"])
        s["cu"], s["start"] = _ints(_cumulative(lens)), _ints(more)
        s["token"] = c["rows"] == c["seqs"]  # the single-token form
        page = c["page"]
        ct = torch.uint8 if c["e4m3"] else dt
        if page:
            # earlier pages of a sequence are its own too; only those that the rows reach are in the pool
            first = [p // page for p in more]
            count = [(n + p - 1) // page + 1 - f for n, p, f in zip(lens, more, first)]
            dealt, pages = _page_table(count, c["spread"])
            width = max(f + n for f, n in zip(first, count))
            table = [[-1] * f + row[:n] + [-1] * (width - f - n) for f, n, row in zip(first, count, dealt)]
            s["pages"] = _ints(table)
            shape = (1, pages, nkv, page, d)
        else:
            s["pages"] = None
            shape = (1, len(lens), nkv, last, d)
        s["k"], s["v"] = (torch.zeros(shape, dtype=ct, device="cuda") for _ in range(2))
        s["q_out"] = torch.empty(c["rows"], nq * d, dtype=dt, device="cuda")
        s["k_out"], s["v_out"] = (None if s["token"] else
                                  torch.empty(c["rows"], nkv * d, dtype=dt, device="cuda") for _ in range(2))
    elif c["op"] == "docs":
        s["q"] = _randn(g, (c["rows"], nq, d), dt, 1.5)
        s["k"] = _randn(g, (c["rows"], nkv, d), dt, 1.5)
        s["v"] = _randn(g, (c["rows"], nkv, d), dt)
        s["cu"] = _ints(_cumulative(lens))
        s["prefix"] = _ints(more) if c["prefix"] else None
        s["out"] = torch.empty(c["rows"], nq * d, dtype=dt, device="cuda")
    else:
        B, page, P = c["batch"], c["page"], c["prefix"]
        s["q"] = _randn(g, (B, nq, d), dt, 1.5)
        s["positions"] = _ints([n - 1 for n in lens])
        if page:
            # the prefix's whole pages are the same ones for every sequence; a page that it
            # fills in part is each sequence's own
            whole = P // page
            dealt, pages = _page_table([whole] + [-(-n // page) - whole for n in lens], c["spread"],
                                       -(-max(lens) // page))
            s["pages"] = _ints([dealt[0][:whole] + row[:len(row) - whole] for row in dealt[1:]])
            shape = (1, pages, nkv, page, d)
        else:
            s["pages"] = None
            shape = (1, B, nkv, max(lens), d)
        s["k"], s["v"] = _randn(g, shape, dt, 1.5), _randn(g, shape, dt)
        s["out"] = torch.empty(B, nq * d, dtype=dt, device="cuda")
    if c["op"] != "append":
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, nq + 1, device="cuda").float() / nq) if c["bias"] else None
    if own:
        _handle(s, c, lens)
    return s


def _handle(s, c, lens):
    """The library context, cache and option objects that a user's program keeps."""
    from llama2_decoder_forward_gb300 import binding, synth
    nq, nkv, d, dt = c["n_q"], c["n_kv"], c["d"], _type(c["dtype"])
    shape = synth.Shape(1, 256, nq, nkv, d, 256, 256, dtype=c["dtype"])
    sizes = dict(attn_norm=(256,), wqkv=((nq + 2 * nkv) * d, 256), wo=(256, nq * d), ffn_norm=(256,),
                 w_gate=(256, 256), w_up=(256, 256), w_down=(256, 256))
    layer = {n: torch.zeros(z, dtype=dt, device="cuda") for n, z in sizes.items()}
    top = s["table"].shape[0] if c["op"] == "append" else max(lens)
    s["model"] = binding.Model(shape, {"layers": [layer]}, max_batch=len(lens), max_tokens=0, max_seq=top,
                               has_embed_head=False)
    if c["op"] == "append":
        s["rope"] = binding.Rope(s["table"], binding.ROPE_HALF if c["half"] else binding.ROPE_ADJACENT)
    else:
        s["scores"] = binding.Scores(cap=c["cap"], slopes=s["slopes"])
    if c["op"] != "docs":
        kind = dict(n_pages=s["k"].shape[1], page_size=c["page"], page_table=s["pages"]) if c["page"] else \
            dict(batch=s["k"].shape[1], capacity=s["k"].shape[3])
        if c.get("e4m3"):
            kind["e4m3"] = SCALES
        s["cache"] = binding.KVCache(shape, k=s["k"], v=s["v"], **kind)


# ---------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if c["op"] == "append":
        if own:
            s["model"].op_rope_norm_append(s["qkv"], s["start"], 0, s["cache"], s["q_out"], rope=s["rope"],
                                           cu_rows=None if s["token"] else s["cu"], q_gain=s["q_gain"],
                                           k_gain=s["k_gain"], k_out=s["k_out"], v_out=s["v_out"])
            out = {"q": s["q_out"], "k_rows": s["k_out"], "v_rows": s["v_out"]}
        else:
            out = _plain_append(s)
        caches = (s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn)) if c["e4m3"] else \
            (s["k"], s["v"])
        out["k"], out["v"] = caches
        return out
    if c["op"] == "docs":
        if own:
            s["model"].op_attention_docs(s["q"], s["k"], s["v"], s["cu"], s["out"], prefix=s["prefix"],
                                         scores=s["scores"])
            return s["out"]
        return _plain_docs(s)
    if own:
        s["model"].op_attention_decode_shared(s["q"], s["positions"], 0, s["cache"], s["out"],
                                              shared_len=c["prefix"], scores=s["scores"])
        return s["out"]
    return _plain_shared(s)


def _plain_append(s):
    c = s["case"]
    nq, nkv, d, r, dt = c["n_q"], c["n_kv"], c["d"], c["rotary"], _type(c["dtype"])
    rows = torch.arange(c["rows"], device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), rows, right=True)
    pos = (s["start"].long() - s["cu"][:-1].long())[seq] + rows
    x = s["qkv"].float().view(c["rows"], nq + 2 * nkv, d)
    qk, v = x[:, :nq + nkv], x[:, nq + nkv:]
    if c["norm"]:
        gain = torch.cat((s["q_gain"].float().expand(nq, d), s["k_gain"].float().expand(nkv, d)))
        qk = qk / torch.sqrt((qk * qk).mean(-1, keepdim=True) + 1e-5) * gain
    cs = s["table"][pos][:, None]
    cos, sin = cs[..., 0], cs[..., 1]
    if c["half"]:
        a, b = qk[..., :r // 2], qk[..., r // 2:r]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    else:
        a, b = qk[..., 0:r:2], qk[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    qk = torch.cat((turned, qk[..., r:]), -1)
    k = qk[:, nq:]
    for cache, new, scale in ((s["k"], k, SCALES[0]), (s["v"], v, SCALES[1])):
        if c["e4m3"]:
            new = (new / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            new = new.to(dt)
        if c["page"]:
            page = s["pages"].long()[seq, pos // c["page"]]
            cache[0][page, :, pos % c["page"]] = new
        else:
            cache[0][seq, :, pos] = new
    side = s["k_out"] is not None
    return {"q": qk[:, :nq].to(dt).reshape(c["rows"], -1),
            "k_rows": k.to(dt).reshape(c["rows"], -1) if side else None,
            "v_rows": v.to(dt).reshape(c["rows"], -1) if side else None}


def _scores_plain(t, c, slopes, distance):
    """Cap and bias of scores t [n_kv, G, ...] in place; distance broadcasts over the last two axes."""
    t.mul_(1.0 / math.sqrt(c["d"]))
    if c["cap"]:
        t.div_(c["cap"]).tanh_().mul_(c["cap"])
    if slopes is not None:
        t.sub_(slopes.view(c["n_kv"], c["n_q"] // c["n_kv"], 1, 1) * distance)
    return t


def _plain_docs(s):
    c = s["case"]
    nq, nkv, d, n = c["n_q"], c["n_kv"], c["d"], c["rows"]
    G = nq // nkv
    rows = torch.arange(n, device="cuda")
    doc = torch.searchsorted(s["cu"][1:].long(), rows, right=True)
    at = rows - s["cu"].long()[doc]
    keep = doc[:, None] == doc
    if s["prefix"] is None:
        keep &= at[:, None] >= at
    else:
        keep &= (at[:, None] >= at) | (at < s["prefix"].long()[doc])
    q = s["q"].float().view(n, nkv, G, d).permute(1, 2, 0, 3).reshape(nkv, G * n, d)
    k = s["k"].float().permute(1, 2, 0)
    v = s["v"].float().transpose(0, 1)
    t = torch.matmul(q, k).view(nkv, G, n, n)
    _scores_plain(t, c, s["slopes"], (at[:, None] - at).abs().float() if c["bias"] else None)
    t.masked_fill_(~keep, -math.inf)
    t.sub_(t.amax(-1, keepdim=True)).exp_()
    total = t.sum(-1, keepdim=True)
    o = torch.matmul(t.view(nkv, G * n, n), v).view(nkv, G, n, d) / total
    return o.permute(2, 0, 1, 3).reshape(n, nq * d).to(_type(c["dtype"]))


def _gathered(s, cache):
    """Own keys of each sequence [B, own_max, n_kv, d] and the shared ones [P, n_kv, d] in fp32."""
    c = s["case"]
    P, page, top = c["prefix"], c["page"], s["case"]["prefix"] + c["own_max"]
    top = min(top, s["k"].shape[3] if not page else s["pages"].shape[1] * page)
    at = torch.arange(P, top, device="cuda")
    first = torch.arange(P, device="cuda")
    if page:
        pages = s["pages"].long()
        mine = cache[0][pages[:, at // page].clamp(min=0), :, at % page]
        both = cache[0][pages[0, first // page], :, first % page]
    else:
        mine, both = cache[0][:, :, P:top].transpose(1, 2), cache[0][0, :, :P].transpose(0, 1)
    return mine.float(), both.float(), at, first


def _plain_shared(s):
    c = s["case"]
    B, nq, nkv, d, P = c["batch"], c["n_q"], c["n_kv"], c["d"], c["prefix"]
    G = nq // nkv
    q = s["q"].float().view(B, nkv, G, d)
    k_own, k_both, at, first = _gathered(s, s["k"])
    v_own, v_both = _gathered(s, s["v"])[:2]
    pos = s["positions"].long()[:, None]
    t_own = torch.matmul(q, k_own.permute(0, 2, 3, 1)).permute(1, 2, 0, 3)  # [n_kv, G, B, own]
    t_both = torch.matmul(q.permute(1, 2, 0, 3).reshape(nkv, G * B, d), k_both.permute(1, 2, 0)).view(nkv, G, B, P)
    t = torch.cat((t_both, t_own), -1)
    keys = torch.cat((first, at))
    _scores_plain(t, c, s["slopes"], (pos - keys).float() if c["bias"] else None)
    t.masked_fill_(keys > pos, -math.inf)
    t.sub_(t.amax(-1, keepdim=True)).exp_()
    total = t.sum(-1, keepdim=True)
    v_own = v_own.masked_fill((at > pos)[:, :, None, None], 0.0)
    o = torch.matmul(t[..., P:].permute(2, 0, 1, 3), v_own.transpose(1, 2)).permute(1, 2, 0, 3)
    o = o + torch.matmul(t[..., :P].reshape(nkv, G * B, P), v_both.transpose(0, 1)).view(nkv, G, B, d)
    return (o / total).permute(2, 0, 1, 3).reshape(B, nq * d).to(_type(c["dtype"]))


# ---------------------------------------------------------------- the definition in fp64
def _attend(q, K, V, c, slopes, query_at, key_at, hidden):
    """One group of heads: q [G, m, d], K, V [n, d] -> [G, m, d]; hidden [m, n] marks masked keys."""
    w = (q @ K.T) / math.sqrt(c["d"])
    if c["cap"]:
        w = torch.tanh(w / c["cap"]) * c["cap"]
    if slopes is not None:
        w = w - slopes.double()[:, None, None] * (query_at[:, None] - key_at[None]).abs().double()
    if hidden is not None:
        w = w.masked_fill(hidden, -math.inf)
    return torch.softmax(w, -1) @ V


def exact(c, seed):
    s = prepare(c, seed)
    nq, nkv, d = c["n_q"], c["n_kv"], c["d"]
    G = nq // nkv
    lens, more = _plan(c)
    if c["op"] == "append":
        return _exact_append(s, c, lens, more)
    if c["op"] == "docs":
        out = torch.empty(c["rows"], nq, d, dtype=torch.float64, device="cuda")
        lo = 0
        for n, pre in zip(lens, more):
            at = torch.arange(n, device="cuda")
            hidden = (at[None] > at[:, None]) & (at[None] >= pre)
            for g in range(nkv):
                K, V = s["k"][lo:lo + n, g].double(), s["v"][lo:lo + n, g].double()
                for h in range(g * G, g * G + G):
                    sl = s["slopes"][h:h + 1] if c["bias"] else None
                    out[lo:lo + n, h] = _attend(s["q"][lo:lo + n, h].double()[None], K, V, c, sl, at, at, hidden)[0]
            lo += n
        return out.view(c["rows"], nq * d)
    out = torch.empty(c["batch"], nq, d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        at = torch.arange(n, device="cuda")
        # keys below the shared length are the same for everyone: sequence 0's
        if c["page"]:
            shared = s["pages"][0].long()[at[:c["prefix"]] // c["page"]]
            mine = s["pages"][b].long()[at[c["prefix"]:] // c["page"]]
            where = torch.cat((shared, mine))
            K, V = (s[x][0][where, :, at % c["page"]].double() for x in ("k", "v"))
        else:
            K, V = (torch.cat((s[x][0, 0, :, :c["prefix"]], s[x][0, b, :, c["prefix"]:n]), 1).double().transpose(0, 1)
                    for x in ("k", "v"))
        for g in range(nkv):
            hs = slice(g * G, g * G + G)
            out[b, hs] = _attend(s["q"][b, hs].double()[:, None], K[:, g], V[:, g], c,
                                 s["slopes"][hs] if c["bias"] else None, at[-1:], at, None)[:, 0]
    return out.view(c["batch"], nq * d)


def _exact_append(s, c, lens, more):
    nq, nkv, d, r = c["n_q"], c["n_kv"], c["d"], c["rotary"]
    x = s["qkv"].double().view(c["rows"], nq + 2 * nkv, d)
    heads = x[:, :nq + nkv].clone()
    if c["norm"]:
        heads *= torch.rsqrt(heads.pow(2).sum(-1, keepdim=True) / d + 1e-5)
        heads[:, :nq] *= s["q_gain"].double()
        heads[:, nq:] *= s["k_gain"].double()
    turn = torch.view_as_complex(s["table"].double().contiguous())  # [positions, r / 2]
    k_cache, v_cache = (torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in ("k", "v"))
    lo = 0
    for b, (n, p0) in enumerate(zip(lens, more)):
        part = heads[lo:lo + n]
        z = part[..., :r]
        z = torch.stack(z.chunk(2, -1), -1) if c["half"] else z.reshape(n, nq + nkv, r // 2, 2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn[p0:p0 + n, None])
        part[..., :r] = torch.cat((z[..., 0], z[..., 1]), -1) if c["half"] else z.flatten(-2)
        for cache, new, scale in ((k_cache, part[:, nq:], SCALES[0]), (v_cache, x[lo:lo + n, nq + nkv:], SCALES[1])):
            if c["e4m3"]:
                new = (new / scale).clamp(-448, 448)
            if c["page"]:
                at = torch.arange(p0, p0 + n, device="cuda")
                cache[0][s["pages"][b].long()[at // c["page"]], :, at % c["page"]] = new
            else:
                cache[0, b, :, p0:p0 + n] = new.transpose(0, 1)
        lo += n
    side = not s["token"]
    return {"q": heads[:, :nq].reshape(c["rows"], -1), "k": k_cache, "v": v_cache,
            "k_rows": heads[:, nq:].reshape(c["rows"], -1) if side else None,
            "v_rows": x[:, nq + nkv:].reshape(c["rows"], -1) if side else None}
