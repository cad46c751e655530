"""The operators beside the plain Llama2 path against plain fp64 forms: head
norms + rotation + append, attention over packed documents, decode attention
over a shared prefix; and the three together, as a server runs them.

Tolerances. A rounding is off by at most half a step, eps / 2 relative: 2^-8
for bf16, 2^-24 for fp32, 2^-4 for E4M3 (2^-10 absolute below its normals).

* Rows: bf16 outputs are one rounding of an fp32 value whose own error is
  some 2^-24 of the head's largest value: 2^-8 |ref| + 2^-18 max|head|.
* Attention, bf16: the output's rounding, 2^-8 |ref|; the weights are rounded
  once for the tensor cores, 2^-8 of sum p|v| (where the rounded weights are
  also the ones that are summed, the mean o moves by sum p e (v - o), |e| <= 2^-8,
  so sum p|v - o| stands there: the same for values of both signs); scores carry fp32 sums of 128
  products, below 2^-11 at these magnitudes, which moves every weight by that
  and the normalising sum by as much: 2^-10 of sum p|v|.
* Attention, fp32: a score is off by at most (d + 8) 2^-24 sum|q k| scale plus
  2^-22 of its bias, cap or size (a few fp32 roundings); twice that, and n/8 + 64
  roundings of the sums and exponentials, act on sum p|v|.
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from _common import f64, need_gpu, to_dev
from llama2_decoder_forward_gb300 import binding, synth
from oracle import attention_forms as A

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(shape, dtype, seed, std=1.0):
    return (torch.randn(*shape, generator=_gen(seed)) * std).to(dtype)


def _model(nq, nkv, d=128, dtype="bf16", max_batch=8, max_seq=4096, n_layers=1):
    need_gpu()
    shape = synth.Shape(n_layers, 256, nq, nkv, d, 256, 256, dtype=dtype)
    w = {"layers": [synth.layer_weights(shape, 3, l) for l in range(n_layers)]}
    return binding.Model(shape, to_dev(w), max_batch=max_batch, max_tokens=0, max_seq=max_seq,
                         has_embed_head=False), shape


def _within(got, ref, bound, what):
    got = f64(got)
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isfinite(err), err - bound, np.inf)), err.shape)
        raise AssertionError("%s: %d of %d out of tolerance; worst at %s: got %r ref %r bound %r"
                             % (what, bad.sum(), bad.size, i, got[i], ref[i], np.broadcast_to(bound, err.shape)[i]))


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# --------------------------------------------------------------------------- table
@pytest.mark.parametrize("kind,kw", [
    ("plain", {}), ("plain", dict(theta=1e6)), ("linear", dict(factor=4.0)),
    ("bands", dict(factor=8.0, low_turns=1.0, high_turns=4.0, original_len=8192)),
    ("bands", dict(factor=16.0, low_turns=1.0, high_turns=32.0, original_len=4096, magnitude=1.25)),
])
@pytest.mark.parametrize("n_pos,r", [(1, 8), (1000, 128), (70001, 24)])
def test_rope_table(kind, kw, n_pos, r):
    need_gpu()
    kinds = dict(plain=binding.ROPE_PLAIN, linear=binding.ROPE_LINEAR, bands=binding.ROPE_BANDS)
    t = binding.rope_table(n_pos, r, kind=kinds[kind], **kw)
    ref = A.rotation_table(n_pos, r, kind=kind, **kw)
    # one fp32 rounding of an fp64 value; the fp64 angle (up to 7e4 rad) of either side is off by 2^-36
    _within(t, ref, 2.0 ** -24 * np.abs(ref) + 2.0 ** -33, "table")


# --------------------------------------------------------------------------- rows
def _rows_case(nq, nkv, d, dtype, src, lens, starts, *, rotary=128, half=True, norm="qk", page=16,
               e4m3=None, side=True, token=False, lead=0, tail=0, ld_pad=0, layers=2, layer=1, seed=5,
               own_table=True, scaled=False):
    """Runs the operator and checks q, side rows, every written slot and that nothing else changed."""
    m, shape = _model(nq, nkv, d, dtype, max_batch=len(lens), n_layers=layers)
    dt = shape.torch_dtype
    n, width = lead + sum(lens) + tail, (nq + 2 * nkv) * d
    x = _randn((n, width + ld_pad), torch.float32 if src == "f32" else dt, seed, 1.5)
    gains = [(1 + 0.1 * torch.randn(d, generator=_gen(seed + i))).to(dt) for i in (1, 2)]
    qg, kg = (gains[0] if "q" in norm else None), (gains[1] if "k" in norm else None)
    top = max(s + l for s, l in zip(starts, lens)) or 1
    kw = dict(kind="linear", factor=4.0) if scaled else {}
    table = A.rotation_table(max(top, 1), rotary, **kw).astype(np.float32) if rotary else None
    rope = None
    if rotary and own_table:
        rope = binding.Rope(torch.from_numpy(table).cuda(), binding.ROPE_HALF if half else binding.ROPE_ADJACENT)
    elif rotary:
        rope = binding.Rope(None, binding.ROPE_HALF if half else binding.ROPE_ADJACENT, rotary)
    cu = [lead]
    for l in lens:
        cu.append(cu[-1] + l)
    if page:
        pages = [max(1, math.ceil((s + l) / page)) for s, l in zip(starts, lens)]
        pt, total = synth.page_table(pages, max(pages), seed)
        kv = binding.KVCache(shape, n_pages=total, page_size=page, page_table=pt.cuda(), e4m3=e4m3)
    else:
        kv = binding.KVCache(shape, batch=len(lens), capacity=top + 3, e4m3=e4m3)
    mark = 0x35 if e4m3 else 7.0
    kv.k.fill_(mark)
    kv.v.fill_(mark)
    q_out = torch.full((n, nq * d), 3.0, dtype=dt, device="cuda")
    ko = torch.full((n, nkv * d), 3.0, dtype=dt, device="cuda") if side else None
    vo = torch.full((n, nkv * d), 3.0, dtype=dt, device="cuda") if side else None
    xd = x.cuda()
    m.op_rope_norm_append(xd[:, :width], _i32(starts), layer, kv, q_out, rope=rope,
                          cu_rows=None if token else _i32(cu), q_gain=None if qg is None else qg.cuda(),
                          k_gain=None if kg is None else kg.cuda(), eps=1e-6, k_out=ko, v_out=vo)
    m.sync()
    xf = f64(x)[:, :width].reshape(n, nq + 2 * nkv, d)
    K, V = kv.k, kv.v
    if e4m3:
        K, V = (t.view(torch.float8_e4m3fn).float() for t in (K, V))
    K, V = f64(K)[layer].copy(), f64(V)[layer].copy()
    if e4m3:  # codes stand for value / scale
        mark = float(torch.tensor([0x35], dtype=torch.uint8).view(torch.float8_e4m3fn).float())

    def close(got, ref, what, scale=None):
        big = np.abs(ref).max(-1, keepdims=True)
        if scale is not None:
            ref = np.clip(ref / scale, -448, 448)
            _within(got, ref, 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 + 2.0 ** -18 * np.minimum(big / scale, 448), what)
        elif dtype == "bf16":
            _within(got, ref, 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * big, what)
        else:
            _within(got, ref, 2.0 ** -24 * np.abs(ref) + 32 * 2.0 ** -24 * big, what)

    for b, (l, p0) in enumerate(zip(lens, starts)):
        for i in range(l):
            r, p = cu[b] + i, p0 + i
            q, k, v = xf[r, :nq], xf[r, nq:nq + nkv], xf[r, nq + nkv:]
            q = q if qg is None else A.head_norm(q, f64(qg), 1e-6)
            k = k if kg is None else A.head_norm(k, f64(kg), 1e-6)
            if rotary:
                q, k = A.rotate(q, table[p].astype(np.float64), half), A.rotate(k, table[p].astype(np.float64), half)
            close(q_out[r].view(nq, d), q, "q row %d" % r)
            if side:
                close(ko[r].view(nkv, d), k, "k side row %d" % r)
                close(vo[r].view(nkv, d), v, "v side row %d" % r)
            at = (int(pt[b, p // page]), slice(None), p % page) if page else (b, slice(None), p)
            close(K[at], k, "cached k %d" % r, e4m3 and e4m3[0])
            close(V[at], v, "cached v %d" % r, e4m3 and e4m3[1])
            K[at], V[at] = mark, mark
    assert np.all(K == mark) and np.all(V == mark), "another slot of the layer was written"
    for t in (kv.k, kv.v):
        others = torch.cat((t[:layer].flatten(), t[layer + 1:].flatten()))
        assert torch.all(others == (0x35 if e4m3 else 7.0)), "another layer was written"
    outside = list(range(lead)) + list(range(cu[-1], n))
    if outside:
        assert torch.all(q_out[outside] == 3.0) and (not side or torch.all(ko[outside] == 3.0))


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("rotary", [0, 8, 24, 64, 128])
@pytest.mark.parametrize("norm", ["", "qk", "k"])
def test_rows_layouts(half, rotary, norm):
    _rows_case(8, 2, 128, "bf16", "f32", [5, 0, 17, 1], [0, 9, 30, 1500], half=half, rotary=rotary, norm=norm)


@pytest.mark.parametrize("src", ["f32", "bf16"])
@pytest.mark.parametrize("page", [0, 16, 48])
@pytest.mark.parametrize("e4m3", [None, (0.02, 0.004)])
def test_rows_caches(src, page, e4m3):
    _rows_case(16, 4, 128, "bf16", src, [1, 33, 2], [15, 40, 0], page=page, e4m3=e4m3, half=False)


@pytest.mark.parametrize("nq,nkv,d", [(4, 2, 64), (5, 5, 40), (3, 1, 256), (1, 1, 8)])
@pytest.mark.parametrize("half", [False, True])
def test_rows_fp32(nq, nkv, d, half):
    _rows_case(nq, nkv, d, "f32", "f32", [7, 1, 20], [0, 100, 3], rotary=d if d < 64 else d - 24, page=16,
               half=half)


def test_rows_single_tokens():
    _rows_case(64, 8, 128, "bf16", "bf16", [1] * 33, [3 * i for i in range(33)], token=True, side=False)


def test_rows_of_no_sequence_are_left():
    _rows_case(8, 8, 128, "bf16", "f32", [3, 1], [4, 0], lead=2, tail=5)


def test_rows_strided_source():
    _rows_case(12, 4, 128, "bf16", "f32", [9], [4], ld_pad=64)
    _rows_case(12, 4, 128, "bf16", "bf16", [9], [4], ld_pad=8)


def test_rows_many_sequences():
    g = _gen(9)
    lens = torch.randint(0, 3, (1500,), generator=g).tolist()
    _rows_case(1, 1, 128, "bf16", "f32", lens, [i % 5 for i in range(1500)], page=16, rotary=32)


def test_rows_context_table_matches_plain_append():
    # without a table the context's own angles; the same bits as the plain operator
    m, shape = _model(8, 2)
    x = _randn((6, shape.qkv_rows), torch.float32, 21).cuda()
    pos = _i32([0, 1, 77, 4095, 12, 3])
    outs = []
    for fused in (False, True):
        kv = binding.KVCache(shape, batch=6, capacity=4096)
        q = torch.empty(6, 8 * 128, dtype=torch.bfloat16, device="cuda")
        if fused:
            m.op_rope_norm_append(x, pos, 0, kv, q, rope=binding.Rope(None, binding.ROPE_ADJACENT, 128))
        else:
            m.op_rope_append(x, 1, pos, 0, kv, q)
        m.sync()
        outs.append((q, kv.k, kv.v))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_rows_out_of_range_are_flagged_and_skipped():
    m, shape = _model(4, 2, max_batch=4)
    d = 128
    x = _randn((4, shape.qkv_rows), torch.float32, 31).cuda()
    pt = _i32([[0, 1], [2, 9], [3, 4], [5, -1]])  # page 9 is not in the pool
    kv = binding.KVCache(shape, n_pages=6, page_size=16, page_table=pt)
    table = binding.rope_table(40, 128)
    q = torch.full((4, 4 * d), 3.0, dtype=torch.bfloat16, device="cuda")
    # in range; bad page; past the table; past the cache's pages (but in the table)
    m.op_rope_norm_append(x, _i32([5, 20, 40, 35]), 0, kv, q, rope=binding.Rope(table))
    rc, flags = m.sync_status()
    assert rc == 5 and flags == binding.FLAG_POS_RANGE | binding.FLAG_PAGE_RANGE
    assert torch.all(q[2] == 0) and torch.all(q[[0, 1, 3]].abs().sum(-1) > 0)
    assert int((kv.k != 0).any(-1).sum()) == 2  # one position's two K/V heads
    m.op_rope_norm_append(x, _i32([-1, 20, 0, 0]), 0, kv, q, rope=binding.Rope(table))
    rc, flags = m.sync_status()
    assert rc == 5 and flags & binding.FLAG_POS_RANGE and torch.all(q[0] == 0)


# --------------------------------------------------------------------------- attention
def _attn_bound(ref, mass, dtype, n, d, big, extra):
    if dtype == "bf16":
        return 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * mass
    score = (d + 8) * 2.0 ** -24 * big + 2.0 ** -22 * extra
    return 2.0 ** -24 * np.abs(ref) + (2 * score + (n / 8 + 64) * 2.0 ** -24) * mass


def _slopes(nq):
    return torch.exp2(-8.0 * torch.arange(1, nq + 1).float() / nq)


def _docs_case(nq, nkv, d, dtype, lens, *, prefix=None, cap=0.0, bias=False, scale=0.0, lead=0, tail=0,
               seed=7, std=1.5, rows=None, poison=False, slopes=None):
    m, shape = _model(nq, nkv, d, dtype)
    dt = shape.torch_dtype
    n = lead + sum(lens) + tail
    q, k, v = (_randn((n, h, d), dt, seed + i, s) for i, (h, s) in enumerate(((nq, std), (nkv, std), (nkv, 1.0))))
    cu = [lead]
    for l in lens:
        cu.append(cu[-1] + l)
    if poison:  # rows of no document may hold anything
        for t in (q, k, v):
            t[:lead] = float("nan")
            t[cu[-1]:] = float("inf")
    slopes = torch.tensor(slopes) if slopes is not None else _slopes(nq) if bias else None
    bias = slopes is not None
    out = torch.full((n, nq * d), 3.0, dtype=dt, device="cuda")
    m.op_attention_docs(q.cuda(), k.cuda(), v.cuda(), _i32(cu), out,
                        prefix=None if prefix is None else _i32(prefix),
                        scores=binding.Scores(scale, cap, None if slopes is None else slopes.cuda()))
    m.sync()
    sc = scale or 1 / math.sqrt(d)
    ref, mass = A.attend_documents(f64(q), f64(k), f64(v), cu, prefix, sc, cap,
                                   None if slopes is None else f64(slopes), rows)
    big = float(np.nanmax(np.abs(f64(q)[lead:cu[-1]]))) ** 2 * d * sc if dtype == "f32" else 0
    sel = sorted(rows) if rows is not None else list(range(lead, cu[-1]))
    _within(out.view(n, nq, d)[sel], ref[sel],
            _attn_bound(ref[sel], mass[sel], dtype, n, d, big, cap + (n if bias else 0)), "docs")
    outside = list(range(lead)) + list(range(cu[-1], n))
    if outside:
        assert torch.all(out[outside] == 3.0)
    return out


OPTIONS = [dict(), dict(cap=5.0), dict(bias=True), dict(cap=30.0, bias=True, scale=0.2)]


@pytest.mark.parametrize("nq,nkv", [(2, 2), (4, 1), (6, 2), (3, 1)])
@pytest.mark.parametrize("opt", range(4))
def test_docs_bf16(nq, nkv, opt):
    _docs_case(nq, nkv, 128, "bf16", [1, 0, 37, 130, 2], **OPTIONS[opt])


@pytest.mark.parametrize("n", [1, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
def test_docs_bf16_one_document(n):
    _docs_case(2, 1, 128, "bf16", [n], cap=20.0, bias=True)
    _docs_case(1, 1, 128, "bf16", [n])


@pytest.mark.parametrize("nq,nkv", [(2, 2), (4, 2), (1, 1)])
def test_docs_bf16_prefix(nq, nkv):
    # no prefix, all of it, past the document, one past a tile, negative
    _docs_case(nq, nkv, 128, "bf16", [20, 150, 90, 300, 5], prefix=[0, 150, 1000, 129, -3], bias=True)


def test_docs_bf16_long():
    rows = {0, 1, 127, 128, 700, 1023, 1024, 1999, 2300, 2301, 2399}
    _docs_case(4, 2, 128, "bf16", [2000, 400], cap=50.0, rows=rows)
    _docs_case(3, 3, 128, "bf16", [2000, 400], prefix=[900, 130], rows=rows)


def test_docs_rows_of_no_document():
    _docs_case(4, 2, 128, "bf16", [30, 140], lead=3, tail=40, poison=True)
    _docs_case(2, 2, 64, "f32", [30, 70], lead=3, tail=40, poison=True)


def test_docs_large_scores():
    # scores of some hundreds: the running maximum moves from tile to tile
    _docs_case(2, 1, 128, "bf16", [400], std=8.0)
    _docs_case(2, 1, 128, "bf16", [400], std=8.0, cap=400.0)
    _docs_case(2, 1, 64, "f32", [200], std=4.0)


def _nan_pattern(out, want):
    got = torch.isnan(out.float())
    assert torch.equal(got.all(-1), got.any(-1)) and torch.equal(got.all(-1).cpu(), want)
    assert torch.isfinite(out.float()[~got.any(-1)]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("opt", range(4))
def test_docs_nan_reaches_the_rows_that_see_it(dtype, opt):
    # a query, and the first 130 keys of the second document's K/V head 1: whole tiles of NaN scores
    nq, nkv, d, n = 4, 2, 128, 300
    m, shape = _model(nq, nkv, d, dtype)
    dt = shape.torch_dtype
    q, k, v = (_randn((n, h, d), dt, 120 + i) for i, h in enumerate((nq, nkv, nkv)))
    q[33, 2, 5] = float("nan")
    k[60:190, 1, 9] = float("nan")
    o = OPTIONS[opt]
    out = torch.empty(n, nq * d, dtype=dt, device="cuda")
    m.op_attention_docs(q.cuda(), k.cuda(), v.cuda(), _i32([0, 60, n]), out, scores=binding.Scores(
        o.get("scale", 0.0), o.get("cap", 0.0), _slopes(nq).cuda() if o.get("bias") else None))
    m.sync()
    want = torch.zeros(n, nq, dtype=torch.bool)
    want[33, 2] = True
    want[60:, 2:] = True
    _nan_pattern(out.view(n, nq, d), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("opt", range(4))
@pytest.mark.parametrize("nq,nkv", [(4, 2), (24, 2)])
@pytest.mark.parametrize("shared", [0, 150])
def test_shared_nan_reaches_the_rows_that_see_it(dtype, opt, nq, nkv, shared):
    # a query, the first 130 keys of every (or the shared) sequence, and one own key past a shorter position
    d, B, cap = 128, 3, 400
    m, shape = _model(nq, nkv, d, dtype, max_batch=B, max_seq=cap)
    dt = shape.torch_dtype
    q = _randn((B, nq, d), dt, 130)
    k, v = (_randn((1, B, nkv, cap, d), dt, 131 + i) for i in range(2))
    q[1, 1, 5] = float("nan")
    k[0, 0, 1, :130, 9] = float("nan")
    k[0, 2, 0, 320] = float("nan")
    o = OPTIONS[opt]
    half = nq // nkv
    kv = binding.KVCache(shape, batch=B, capacity=cap, k=k.cuda(), v=v.cuda())
    out = torch.empty(B, nq * d, dtype=dt, device="cuda")
    for pos in ([399, 399, 399], [200, 250, 319], [140, 100, 160]):
        m.op_attention_decode_shared(q.cuda(), _i32(pos), 0, kv, out, shared_len=shared, scores=binding.Scores(
            o.get("scale", 0.0), o.get("cap", 0.0), _slopes(nq).cuda() if o.get("bias") else None))
        m.sync()
        want = torch.zeros(B, nq, dtype=torch.bool)
        want[1, 1] = True
        want[slice(0, B) if shared else 0, half:] = True
        want[2, :half] = pos[2] >= 320
        _nan_pattern(out.view(B, nq, d), want)


SLOPES = [[5.0, -0.5, 0.0, 1.3], [1.3, 1.5, 0.1, 40.0], [-3.0, 0.0, -0.01, 2.0]]


@pytest.mark.parametrize("slopes", SLOPES)
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_docs_steep_and_negative_slopes(slopes, cap):
    # biases of some 100 between neighbouring tiles, rising and falling, per head
    _docs_case(4, 2, 128, "bf16", [330, 70], slopes=slopes, cap=cap)
    _docs_case(4, 4, 128, "bf16", [330, 70], slopes=slopes, cap=cap, prefix=[200, 70])


@pytest.mark.parametrize("slopes", SLOPES)
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_shared_steep_and_negative_slopes(slopes, cap):
    _shared_case(4, 1, 128, "bf16", [400, 260, 300], 256, slopes=slopes, cap=cap)
    _shared_case(4, 4, 128, "bf16", [400, 260, 300], 0, slopes=slopes, cap=cap)


@pytest.mark.parametrize("cap,scale", [(50.0, 0.0), (50.3, 0.0), (2.0, 0.5), (0.05, 1.0), (2000.0, 0.0), (300.0, 4.0)])
def test_docs_caps(cap, scale):
    # barely capped, far past the cap, and scale / cap outside the fitted range
    _docs_case(4, 2, 128, "bf16", [300, 40], cap=cap, scale=scale)
    _docs_case(3, 3, 128, "bf16", [300, 40], cap=cap, scale=scale, bias=True)


def test_docs_many_documents():
    lens = torch.randint(0, 4, (200,), generator=_gen(3)).tolist()
    _docs_case(2, 1, 128, "bf16", lens)


@pytest.mark.parametrize("nq,nkv", [(2, 1), (1, 1)])
def test_docs_many_ragged_documents(nq, nkv):
    # more documents than a warp's lanes, empty ones and prefixes of any length among them
    lens = [0] * 40 + [300, 1, 0, 129, 128, 257] + [0] * 30 + [64] * 5 + [0, 200]
    pre = torch.randint(0, 260, (len(lens),), generator=_gen(5)).tolist()
    _docs_case(nq, nkv, 128, "bf16", lens)
    _docs_case(nq, nkv, 128, "bf16", lens, prefix=pre, bias=True)


@pytest.mark.parametrize("nq,nkv,d", [(4, 2, 64), (2, 2, 40), (2, 1, 128), (1, 1, 256), (3, 1, 8)])
@pytest.mark.parametrize("opt", range(4))
def test_docs_fp32(nq, nkv, d, opt):
    _docs_case(nq, nkv, d, "f32", [1, 70, 0, 130], prefix=[0, 3, 0, 100] if opt & 1 else None, **OPTIONS[opt])


def test_docs_output_aligned_to_16_bytes_only():
    m, _ = _model(4, 2)
    n = 200
    q, k, v = (_randn((n, h, 128), torch.bfloat16, 210 + i).cuda() for i, h in enumerate((4, 2, 2)))
    want = torch.empty(n, 512, dtype=torch.bfloat16, device="cuda")
    buf = torch.full((n * 512 + 16,), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[8:8 + n * 512].view(n, 512)
    assert out.data_ptr() % 32 == 16
    for o in (want, out):
        m.op_attention_docs(q, k, v, _i32([0, 70, n]), o)
    m.sync()
    assert torch.equal(out, want) and torch.all(buf[:8] == 3.0) and torch.all(buf[8 + n * 512:] == 3.0)


def test_docs_matches_plain_prefill():
    m, shape = _model(4, 2)
    B, T = 2, 200
    q, k, v = (_randn((B * T, h, 128), torch.bfloat16, 40 + i).cuda() for i, h in enumerate((4, 2, 2)))
    a, b = (torch.empty(B * T, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.op_attention_prefill(q, k, v, B, T, a)
    m.op_attention_docs(q, k, v, _i32([0, T, 2 * T]), b)
    m.sync()
    ref, mass = A.attend_documents(f64(q), f64(k), f64(v), [0, T, 2 * T], None, 1 / math.sqrt(128))
    for t in (a, b):
        _within(t.view(B * T, 4, 128), ref, _attn_bound(ref, mass, "bf16", T, 128, 0, 0), "prefill")


def test_docs_bad_bounds_are_flagged():
    m, shape = _model(2, 2)
    q, k, v = (_randn((50, 2, 128), torch.bfloat16, 50 + i).cuda() for i in range(3))
    out = torch.full((50, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    m.op_attention_docs(q, k, v, _i32([0, 20, 70]), out)  # the second document ends past the rows
    rc, flags = m.sync_status()
    assert rc == 5 and flags == binding.FLAG_POS_RANGE
    ref, mass = A.attend_documents(f64(q), f64(k), f64(v), [0, 20, 50], None, 1 / math.sqrt(128))
    _within(out.view(50, 2, 128), ref, _attn_bound(ref, mass, "bf16", 50, 128, 0, 0), "cut document")


# --------------------------------------------------------------------------- decode
def _shared_case(nq, nkv, d, dtype, positions, shared, *, page=16, seq=0, cap=0.0, bias=False, scale=0.0,
                 seed=11, std=1.5, layers=1, layer=0, max_seq=None, poison=True, slopes=None):
    B = len(positions)
    top = max(max(positions) + 1, shared, 1)
    m, shape = _model(nq, nkv, d, dtype, max_batch=B, max_seq=max_seq or top, n_layers=layers)
    dt = shape.torch_dtype
    q = _randn((B, nq, d), dt, seed, std)
    extra = 1 if seq >= B else 0
    if page:
        whole = shared // page
        counts = [whole] + [max(math.ceil(max(p + 1, shared) / page) - whole, 0) for p in positions]
        t, total = synth.page_table(counts, max(math.ceil(top / page), 1), seed)
        pt = torch.full((B, t.shape[1]), -1, dtype=torch.int32)
        for b in range(B):
            pt[b, :whole] = t[0, :whole]
            pt[b, whole:whole + counts[b + 1]] = t[b + 1, :counts[b + 1]]
        size = (layers, max(total, 1), nkv, page, d)
    else:
        size = (layers, B + extra, nkv, top, d)
    k, v = _randn(size, dt, seed + 1, std), _randn(size, dt, seed + 2)

    def rows(t, b):  # (keys, values) as the definition reads them
        n = positions[b] + 1
        if page:
            at = lambda s, j: (layer, int(pt[s, j // page]), slice(None), j % page)
        else:
            at = lambda s, j: (layer, s, slice(None), j)
        return [at(seq if j < shared else b, j) for j in range(n)]
    if poison:  # slots that no key of any sequence is read from
        used = set()
        for b in range(B):
            used |= {(i[1], i[3]) for i in rows(None, b)}
        for i in range(size[1]):
            for j in range(size[3]):
                if (i, j) not in used:
                    k[layer, i, :, j] = float("nan")
                    v[layer, i, :, j] = float("nan") if (i + j) % 2 else float("inf")
    kv = binding.KVCache(shape, n_pages=size[1], page_size=page, page_table=pt.cuda(), k=k.cuda(), v=v.cuda()) \
        if page else binding.KVCache(shape, batch=size[1], capacity=top, k=k.cuda(), v=v.cuda())
    slopes = torch.tensor(slopes) if slopes is not None else _slopes(nq) if bias else None
    bias = slopes is not None
    out = torch.full((B, nq * d), 3.0, dtype=dt, device="cuda")
    m.op_attention_decode_shared(q.cuda(), _i32(positions), layer, kv, out, shared_len=shared, shared_seq=seq,
                                 scores=binding.Scores(scale, cap, None if slopes is None else slopes.cuda()))
    m.sync()
    sc = scale or 1 / math.sqrt(d)
    kf, vf, qf = f64(k), f64(v), f64(q)
    for b in range(B):
        where = rows(None, b)
        n = len(where)
        K = np.stack([kf[i] for i in where], 1)
        V = np.stack([vf[i] for i in where], 1)
        ref, mass = np.empty((nq, d)), np.empty((nq, d))
        for h in range(nq):
            g = h // (nq // nkv)
            ref[h], mass[h] = A.attend_row(qf[b, h], K[g], V[g], positions[b], np.ones(n, bool), sc, cap,
                                           0.0 if slopes is None else float(slopes[h]))
        big = float(np.abs(qf).max()) ** 2 * d * sc if dtype == "f32" else 0
        _within(out[b].view(nq, d), ref, _attn_bound(ref, mass, dtype, n, d, big, cap + (n if bias else 0)),
                "decode b=%d n=%d" % (b, n))


@pytest.mark.parametrize("nq,nkv", [(4, 4), (8, 1), (6, 2), (16, 1), (12, 1)])
@pytest.mark.parametrize("opt", range(4))
def test_shared_bf16(nq, nkv, opt):
    _shared_case(nq, nkv, 128, "bf16", [200, 150, 128, 333, 129], 128, **OPTIONS[opt])


@pytest.mark.parametrize("page", [0, 16, 64, 80])
@pytest.mark.parametrize("shared", [0, 1, 15, 64, 100, 257])
def test_shared_bf16_ends(page, shared):
    # the shared part ends inside a page or a tile; single own keys and long ones
    _shared_case(8, 2, 128, "bf16", [shared, shared + 1, shared + 63, shared + 64, shared + 300, shared + 7], shared,
                 page=page)


def test_shared_bf16_positions_inside_the_prefix():
    _shared_case(8, 2, 128, "bf16", [0, 10, 63, 64, 199, 200, 400], 200)
    _shared_case(2, 2, 128, "bf16", [0, 10, 63, 64, 199, 200, 400], 200, page=0, cap=10.0, bias=True)


@pytest.mark.parametrize("page,seq", [(0, 2), (0, 4), (16, 3)])
def test_shared_bf16_other_sequence(page, seq):
    _shared_case(4, 2, 128, "bf16", [300, 280, 260, 256], 256, page=page, seq=seq)


@pytest.mark.parametrize("B,nq,nkv", [(1, 32, 32), (1, 8, 1), (17, 16, 2), (40, 8, 1), (130, 2, 2), (9, 16, 1)])
def test_shared_bf16_batches(B, nq, nkv):
    # one row block, several, and the last one ragged
    _shared_case(nq, nkv, 128, "bf16", [140 + (7 * b) % 50 for b in range(B)], 130)


def test_shared_bf16_long_splits():
    _shared_case(8, 2, 128, "bf16", [4000, 2500], 2048, page=64, cap=30.0)
    _shared_case(4, 4, 128, "bf16", [5000], 0, page=0, bias=True)


@pytest.mark.parametrize("cap,scale", [(50.0, 0.0), (50.3, 0.0), (2.0, 0.5), (0.05, 1.0), (2000.0, 0.0), (300.0, 4.0),
                                       (3e4, 0.0), (1e6, 0.0), (1e8, 0.0)])
@pytest.mark.parametrize("nq,nkv", [(4, 2), (12, 1)])
@pytest.mark.parametrize("shared", [0, 128])
def test_shared_caps(cap, scale, nq, nkv, shared):
    # barely capped, far past the cap, and caps beside which the scores are small: own and shared keys
    # are capped alike, to an error relative to the score
    _shared_case(nq, nkv, 128, "bf16", [200, 150, 333], shared, cap=cap, scale=scale)
    _shared_case(nq, nkv, 128, "bf16", [200, 150, 333], shared, cap=cap, scale=scale, bias=True)


def test_shared_join_after_a_long_prefix():
    # the own keys' blocks leave partials: both row tiles with the same rows, and two blocks of rows;
    # own keys none, few and many, a position inside the prefix
    _shared_case(40, 40, 128, "bf16", [3299, 3163, 90], 3160, page=64, cap=20.0)
    _shared_case(40, 40, 128, "bf16", [3159, 3400], 3160, page=0, seq=2)
    _shared_case(640, 40, 128, "bf16", [1700 + 11 * b for b in range(8)] + [1500], 1700, page=64, bias=True)


def test_shared_longest_first():
    # more blocks than are resident: taken by length, with ties and the shortest of all
    g = _gen(9)
    pos = torch.randint(0, 200, (58,), generator=g).tolist()
    pos[3] = pos[40] = pos[41] = 479
    pos[7] = 0
    _shared_case(8, 8, 128, "bf16", pos, 0, page=16)
    _shared_case(16, 8, 128, "bf16", [p + 70 for p in pos], 70, page=0, cap=30.0, bias=True)


def test_shared_longest_first_beside_bad_positions():
    m, shape = _model(8, 8, max_batch=58, max_seq=480)
    q = _randn((58, 8, 128), torch.bfloat16, 190).cuda()
    k, v = (_randn((1, 58, 8, 480, 128), torch.bfloat16, 191 + i).cuda() for i in range(2))
    kv = binding.KVCache(shape, batch=58, capacity=480, k=k, v=v)
    out, want = (torch.full((58, 1024), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = [(37 * b) % 480 for b in range(58)]
    m.op_attention_decode_shared(q, _i32(pos), 0, kv, want)
    m.sync()
    bad = list(pos)
    bad[5], bad[6], bad[50] = -1, -2 ** 31, 2 ** 31 - 1
    m.op_attention_decode_shared(q, _i32(bad), 0, kv, out)
    rc, flags = m.sync_status()
    assert rc == 5 and flags == binding.FLAG_POS_RANGE
    assert torch.all(out[[5, 6]] == 0)
    keep = [b for b in range(58) if b not in (5, 6, 50)]
    assert torch.equal(out[keep], want[keep])


@pytest.mark.parametrize("dtype,nq,nkv,room,shared", [
    ("bf16", 4, 2, 400, 0), ("bf16", 4, 2, 400, 100), ("bf16", 40, 40, 3400, 3160), ("bf16", 16, 1, 3400, 0),
    ("f32", 4, 2, 400, 100)])
@pytest.mark.parametrize("bias", [False, True])
def test_shared_positions_past_the_cache(dtype, nq, nkv, room, shared, bias):
    # without a prefix, beside a short one, joined after a long one: the largest and the smallest
    # position are flagged, and the keys in range are attended as from the last one
    m, shape = _model(nq, nkv, 128, dtype, max_batch=4, max_seq=room)
    dt = shape.torch_dtype
    q = _randn((4, nq, 128), dt, 220).cuda()
    k, v = (_randn((1, 4, nkv, room, 128), dt, 221 + i).cuda() for i in range(2))
    kv = binding.KVCache(shape, batch=4, capacity=room, k=k, v=v)
    sc = binding.Scores(slopes=_slopes(nq).cuda()) if bias else None
    outs = []
    for pos in ([room - 1, room - 30, room - 1, -1], [2 ** 31 - 1, room - 30, room, -2 ** 31]):
        out = torch.full((4, nq * 128), 3.0, dtype=dt, device="cuda")
        m.op_attention_decode_shared(q, _i32(pos), 0, kv, out, shared_len=shared, scores=sc)
        rc, flags = m.sync_status()
        assert rc == 5 and flags == binding.FLAG_POS_RANGE
        outs.append(out)
    assert torch.all(outs[0][3] == 0) and torch.isfinite(outs[0]).all() and torch.all(outs[0][:3].abs().sum(-1) > 0)
    assert torch.equal(outs[0], outs[1])


def test_shared_second_layer():
    _shared_case(4, 2, 128, "bf16", [90, 70], 40, layers=3, layer=2)


def test_shared_large_scores():
    _shared_case(4, 2, 128, "bf16", [500, 300], 256, std=8.0)


@pytest.mark.parametrize("nq,nkv,d", [(4, 2, 64), (2, 2, 40), (20, 1, 128), (1, 1, 256)])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("opt", range(4))
def test_shared_fp32(nq, nkv, d, page, opt):
    _shared_case(nq, nkv, d, "f32", [0, 70, 99, 130], 50 if opt & 1 else 0, page=page, **OPTIONS[opt])


def test_shared_bad_positions_and_pages():
    m, shape = _model(4, 2, max_batch=4, max_seq=64)
    q = _randn((4, 4, 128), torch.bfloat16, 60).cuda()
    k, v = (_randn((1, 8, 2, 16, 128), torch.bfloat16, 61 + i) for i in range(2))
    pt = _i32([[0, 1, 2, 3], [0, 4, -1, -1], [0, 5, 6, 7], [0, 7, 90, -1]])
    kv = binding.KVCache(shape, n_pages=8, page_size=16, page_table=pt, k=k.cuda(), v=v.cuda())
    out = torch.full((4, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    # sequence 1 has no keys, 2 asks past max_seq (all 64 keys attended), 3 has a page outside the pool
    m.op_attention_decode_shared(q, _i32([40, -1, 64, 40]), 0, kv, out, shared_len=16)
    rc, flags = m.sync_status()
    assert rc == 5 and flags == binding.FLAG_POS_RANGE | binding.FLAG_PAGE_RANGE
    assert torch.all(out[1] == 0)
    for b, n in ((0, 41), (2, 64)):
        ids = pt[b].cpu().numpy()
        K = np.concatenate([f64(k)[0, ids[i]] for i in range(4)], 1)[:, :n]
        V = np.concatenate([f64(v)[0, ids[i]] for i in range(4)], 1)[:, :n]
        for h in range(4):
            ref, mass = A.attend_row(f64(q)[b, h], K[h // 2], V[h // 2], n - 1, np.ones(n, bool), 1 / math.sqrt(128))
            _within(out[b].view(4, 128)[h], ref, _attn_bound(ref, mass, "bf16", n, 128, 0, 0), "beside bad ones")
    m.op_attention_decode_shared(q, _i32([40, 20, 63, 30]), 0, kv, out, shared_len=16)
    m.sync()  # the context is usable again


# --------------------------------------------------------------------------- together
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_serving_run(dtype):
    """A system prompt and three user prompts are prefilled, then all sequences
    decode over the shared prompt: append -> documents -> append -> decode."""
    nq, nkv, d, page, P = 4, 2, 128, 16, 70
    m, shape = _model(nq, nkv, d, dtype, max_batch=4, max_seq=256)
    dt = shape.torch_dtype
    table = binding.rope_table(256, 96, kind=binding.ROPE_LINEAR, factor=2.0)
    rope = binding.Rope(table, binding.ROPE_HALF)
    qg, kg = ((1 + 0.1 * torch.randn(d, generator=_gen(i))).to(dt) for i in (1, 2))
    slopes = _slopes(nq)
    scores = binding.Scores(cap=20.0, slopes=slopes.cuda())
    own = [5, 40, 17]  # tokens after the shared prompt
    # table rows 0-2: users (own copy of the partly filled page); row 3: the prompt itself
    pt = torch.full((4, 16), -1, dtype=torch.int32)
    pt[3, :5] = torch.tensor([9, 2, 30, 7, 11])
    for b in range(3):
        pt[b, :4] = pt[3, :4]
        pt[b, 4:9] = torch.tensor([12, 13, 14, 15, 16]) + 5 * b
    kv = binding.KVCache(shape, n_pages=40, page_size=page, page_table=pt.cuda())
    tf = f64(table)

    def ref_rows(x, pos):
        x = f64(x).reshape(len(pos), nq + 2 * nkv, d)
        q, k = A.head_norm(x[:, :nq], f64(qg), 1e-5), A.head_norm(x[:, nq:nq + nkv], f64(kg), 1e-5)
        q = np.stack([A.rotate(q[i], tf[p], True) for i, p in enumerate(pos)])
        k = np.stack([A.rotate(k[i], tf[p], True) for i, p in enumerate(pos)])
        return q, k, x[:, nq + nkv:]

    # the prompt into sequence 3, attended as one document with a two-way part
    x = _randn((P, shape.qkv_rows), torch.float32, 70)
    q, o = (torch.empty(P, nq * d, dtype=dt, device="cuda") for _ in range(2))
    k, v = (torch.empty(P, nkv * d, dtype=dt, device="cuda") for _ in range(2))
    kw = dict(rope=rope, q_gain=qg.cuda(), k_gain=kg.cuda())
    m.op_rope_norm_append(x.cuda(), _i32([0, 0, 0, 0]), 0, kv, q, cu_rows=_i32([0, 0, 0, 0, P]), k_out=k, v_out=v, **kw)
    m.op_attention_docs(q, k, v, _i32([0, P]), o, prefix=_i32([20]), scores=scores)
    m.sync()
    ref, mass = A.attend_documents(f64(q).reshape(P, nq, d), f64(k).reshape(P, nkv, d), f64(v).reshape(P, nkv, d),
                                   [0, P], [20], 1 / math.sqrt(d), 20.0, f64(slopes))
    _within(o.view(P, nq, d), ref, _attn_bound(ref, mass, dtype, P, d, 400.0, 20 + P), "prompt")
    rq, rk, rv = ref_rows(x, range(P))
    tol = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -20
    for got, want in ((q, rq), (k, rk), (v, rv)):
        _within(got.view(P, -1, d), want, tol * np.abs(want) + 2.0 ** -16 * 6, "prompt rows")
    keys = [[k.view(P, nkv, d)[j] for j in range(P)] for _ in range(3)]
    vals = [[v.view(P, nkv, d)[j] for j in range(P)] for _ in range(3)]
    # the users' own tokens join one batch of packed rows, then two decode steps
    for step, lens in enumerate((own, [1] * 3, [1] * 3)):
        n = sum(lens)
        x = _randn((n, shape.qkv_rows), torch.float32, 80 + step)
        start = [len(keys[b]) for b in range(3)]
        cu = np.concatenate(([0], np.cumsum(lens))).tolist()
        q = torch.empty(n, nq * d, dtype=dt, device="cuda")
        k, v = (torch.empty(n, nkv * d, dtype=dt, device="cuda") for _ in range(2))
        m.op_rope_norm_append(x.cuda(), _i32(start), 0, kv, q, cu_rows=_i32(cu) if step == 0 else None, k_out=k,
                              v_out=v, **kw)
        m.sync()
        for b in range(3):
            for r in range(cu[b], cu[b + 1]):
                keys[b].append(k.view(n, nkv, d)[r])
                vals[b].append(v.view(n, nkv, d)[r])
        last = [c - 1 for c in cu[1:]]
        qd = torch.cat((q[last], q[:1] * 0)).contiguous()  # sequence 3 is only a prefix: no query
        pos = [len(keys[b]) - 1 for b in range(3)] + [-1]
        o = torch.full((4, nq * d), 3.0, dtype=dt, device="cuda")
        m.op_attention_decode_shared(qd, _i32(pos), 0, kv, o, shared_len=P, shared_seq=3, scores=scores)
        rc, flags = m.sync_status()
        assert rc == 5 and flags == binding.FLAG_POS_RANGE  # the row without keys
        assert torch.all(o[3] == 0)
        for b in range(3):
            K, V = f64(torch.stack(keys[b])), f64(torch.stack(vals[b]))
            for h in range(nq):
                ref, mass = A.attend_row(f64(qd)[b].reshape(nq, d)[h], K[:, h // 2], V[:, h // 2], pos[b],
                                         np.ones(len(K), bool), 1 / math.sqrt(d), 20.0, float(slopes[h]))
                _within(o[b].view(nq, d)[h], ref, _attn_bound(ref, mass, dtype, len(K), d, 400.0, 20 + len(K)),
                        "step %d user %d" % (step, b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [0, 64])
def test_cache_offsets_past_32_bits(dtype, page):
    # the last slots of a cache of more than 2^31 values: appended, then read as own and as shared keys
    nq, nkv, d, cap, B, n = 4, 2, 128, 1 << 17, 66, 150
    m, shape = _model(nq, nkv, d, dtype, max_batch=2, max_seq=256)
    dt = shape.torch_dtype
    if page:
        total = B * cap // page
        pt = torch.full((2, 4), -1, dtype=torch.int32)
        pt[0, :3] = torch.tensor([total - 3, total - 1, total - 2])
        pt[1] = torch.tensor([total - 3, total - 4, 0, 1])  # shares the first page only
        kv = binding.KVCache(shape, n_pages=total, page_size=page, page_table=pt.cuda())
        last = 0
    else:
        kv = binding.KVCache(shape, batch=B, capacity=cap)
        last = B - 1
    assert kv.k.numel() > 1 << 31
    x = _randn((n, shape.qkv_rows), torch.float32, 200)
    q = torch.empty(n, nq * d, dtype=dt, device="cuda")
    k, v = (torch.empty(n, nkv * d, dtype=dt, device="cuda") for _ in range(2))
    seqs = last + 1
    cu = _i32([0] * seqs + [n])
    m2 = m
    if not page:  # row counts by sequence need a context of that batch
        m2, _ = _model(nq, nkv, d, dtype, max_batch=B, max_seq=256)
    m2.op_rope_norm_append(x.cuda(), _i32([0] * seqs), 0, kv, q, cu_rows=cu, k_out=k, v_out=v)
    m2.sync()
    assert torch.equal(q, x[:, :nq * d].to(dt).cuda()) and torch.equal(v, x[:, -nkv * d:].to(dt).cuda())
    kf, vf = f64(k).reshape(n, nkv, d), f64(v).reshape(n, nkv, d)
    qd = q[:2].contiguous()
    # both sequences read the first 64 keys from the far slots
    pos = [63, 63]
    if page:
        pos[last] = n - 1
    o = torch.empty(2, nq * d, dtype=dt, device="cuda")
    m.op_attention_decode_shared(qd, _i32(pos), 0, kv, o, shared_len=64, shared_seq=last)
    m.sync()
    for b in range(2):
        for h in range(nq):
            ref, mass = A.attend_row(f64(qd)[b].reshape(nq, d)[h], kf[:pos[b] + 1, h // 2], vf[:pos[b] + 1, h // 2], pos[b],
                                     np.ones(pos[b] + 1, bool), 1 / math.sqrt(d))
            _within(o[b].view(nq, d)[h], ref, _attn_bound(ref, mass, dtype, n, d, 400.0, 0), "row %d" % b)
    if not page:  # as its own keys
        positions = _i32([-1] * last + [n - 1])
        qb = torch.zeros(B, nq * d, dtype=dt, device="cuda")
        qb[last] = q[0]
        ob = torch.empty_like(qb)
        m2.op_attention_decode_shared(qb, positions, 0, kv, ob)
        rc, flags = m2.sync_status()
        assert rc == 5 and flags == binding.FLAG_POS_RANGE
        for h in range(nq):
            ref, mass = A.attend_row(f64(q)[0].reshape(nq, d)[h], kf[:, h // 2], vf[:, h // 2], n - 1,
                                     np.ones(n, bool), 1 / math.sqrt(d))
            _within(ob[last].view(nq, d)[h], ref, _attn_bound(ref, mass, dtype, n, d, 400.0, 0), "own")


def test_captured_replays_follow_their_buffers():
    # append and decode captured on a stream, replayed with new inputs and positions
    m, shape = _model(8, 2, max_batch=3, max_seq=512)
    s = torch.cuda.Stream()
    pos = _i32([300, 310, 305])
    x = torch.empty(3, shape.qkv_rows, device="cuda")
    k, v = (_randn((1, 3, 2, 512, 128), torch.bfloat16, 90 + i).cuda() for i in range(2))
    kv = binding.KVCache(shape, batch=3, capacity=512, k=k, v=v)
    q, o = (torch.empty(3, 1024, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rope = binding.Rope(None, binding.ROPE_HALF, 128)
    sc = binding.Scores(cap=30.0)

    def step():
        m.op_rope_norm_append(x, pos, 0, kv, q, rope=rope)
        m.op_attention_decode_shared(q, pos, 0, kv, o, shared_len=200, scores=sc)
    torch.cuda.synchronize()
    m.set_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for i in range(3):
        x.copy_(_randn((3, shape.qkv_rows), torch.float32, 95 + i))
        before = (k.clone(), v.clone())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        captured = o.clone()
        k.copy_(before[0])
        v.copy_(before[1])
        o.fill_(3.0)
        torch.cuda.synchronize()
        step()
        m.sync()
        assert torch.equal(o, captured)
        pos += 1
    m.set_stream(torch.cuda.default_stream())


def test_two_contexts_on_two_streams_at_once():
    # each with its own workspace: the same results as alone, and the same bits every time
    runs = []
    for i, (nq, nkv, B) in enumerate(((8, 2, 6), (16, 16, 2))):
        m, shape = _model(nq, nkv, max_batch=B, max_seq=1024)
        s = torch.cuda.Stream()
        q = _randn((B, nq, 128), torch.bfloat16, 140 + i).cuda()
        k, v = (_randn((1, B, nkv, 1024, 128), torch.bfloat16, 150 + 2 * i + j).cuda() for j in range(2))
        kv = binding.KVCache(shape, batch=B, capacity=1024, k=k, v=v)
        pos = _i32([1023 - 7 * b for b in range(B)])
        dq = _randn((600, nq, 128), torch.bfloat16, 160 + i).cuda()
        dk, dv = (_randn((600, nkv, 128), torch.bfloat16, 170 + 2 * i + j).cuda() for j in range(2))
        cu = _i32([0, 350, 600])
        torch.cuda.synchronize()
        m.set_stream(s)
        runs.append((m, s, q, kv, pos, dq, dk, dv, cu))

    def once(r):
        m, s, q, kv, pos, dq, dk, dv, cu = r
        with torch.cuda.stream(s):
            o = torch.empty(q.shape[0], q.shape[1] * 128, dtype=q.dtype, device="cuda")
            do = torch.empty(600, q.shape[1] * 128, dtype=q.dtype, device="cuda")
        m.op_attention_decode_shared(q, pos, 0, kv, o, shared_len=700, scores=binding.Scores(cap=20.0))
        m.op_attention_docs(dq, dk, dv, cu, do)
        return o, do
    alone = []
    for r in runs:
        alone.append(once(r))
        r[0].sync()
    together = [[once(r) for r in runs] for _ in range(20)]
    for r in runs:
        r[0].sync()
    for pair in together:
        for got, want in zip(pair, alone):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for r in runs:
        r[0].set_stream(torch.cuda.default_stream())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_ranges(dtype):
    # caps and scales at the ends of their range; beyond it the constants that the kernels form
    # of them leave fp32
    lo, hi = 2.0 ** -100, 2.0 ** 100
    for cap, scale in ((hi, 0.0), (1e-29, 0.0), (lo, lo), (0.0, lo)):
        _docs_case(4, 2, 128, dtype, [150, 40], cap=cap, scale=scale)
        _docs_case(3, 3, 128, dtype, [150, 40], cap=cap, scale=scale, bias=True)
        _shared_case(4, 2, 128, dtype, [200, 140], 128, cap=cap, scale=scale, bias=True)
    m, shape = _model(4, 2, dtype=dtype, max_batch=2, max_seq=64)
    dt = shape.torch_dtype
    q, k = (torch.zeros(2, h * 128, dtype=dt, device="cuda") for h in (4, 2))
    kv = binding.KVCache(shape, batch=2, capacity=64)
    for cap, scale in ((3e38, 0.0), (2 * hi, 0.0), (lo / 2, 0.0), (1e-45, 0.0), (0.0, 2 * hi), (0.0, lo / 2),
                       (1e-20, 1e20), (1e20, 1e-20)):
        sc = binding.Scores(scale, cap)
        for call in (lambda: m.op_attention_docs(q, k, k, _i32([0, 2]), q.clone(), scores=sc),
                     lambda: m.op_attention_decode_shared(q, _i32([0, 1]), 0, kv, q.clone(), scores=sc)):
            with pytest.raises(binding.LlamaError) as e:
                call()
            assert e.value.rc == 1
    m.sync()


# --------------------------------------------------------------------------- several items per block
def _docs_reference(q, k, v, lens, prefix, scale, cap, slopes):
    """(out, mass) [n, n_q, d] in fp64 on the GPU, document by document."""
    q, k, v = (t.cuda().double() for t in (q, k, v))
    G = q.shape[1] // k.shape[1]
    out, mass, lo = torch.empty_like(q), torch.empty_like(q), 0
    for b, n in enumerate(lens):
        if n == 0:
            continue
        K, V = (t[lo:lo + n].repeat_interleave(G, 1) for t in (k, v))
        s = torch.einsum("ihd,jhd->hij", q[lo:lo + n], K) * scale
        if cap > 0:
            s = cap * torch.tanh(s / cap)
        at = torch.arange(n, device="cuda")
        if slopes is not None:
            s = s - slopes.cuda().double()[:, None, None] * (at[:, None] - at).abs()
        keep = at[:, None] >= at if prefix is None else (at[:, None] >= at) | (at < prefix[b])
        p = torch.softmax(s.masked_fill(~keep, -math.inf), -1)
        out[lo:lo + n] = torch.einsum("hij,jhd->ihd", p, V)
        mass[lo:lo + n] = torch.einsum("hij,jhd->ihd", p, V.abs())
        lo += n
    return f64(out), f64(mass)


def _one_key_per_dim(n, heads, dtype):
    """Values with a one in dim (key % 128): with weights near each other, a key too
    many or too few changes its dim by far more than a rounding. The values have one
    sign, so a weight's error moves the mean o by up to 2^-8 sum p|v - o| <= 2^-8
    (sum p|v| + |o|): 2^-8 |ref| more than values of both signs. And a dim may hold
    none but tiny weights: those below fp32's normals are lost, 2^-126 of a reference
    that lies up to 7 slopes of 2 octaves above the row's largest score, 2^-112 each
    for the 6 keys of a dim: below 2^-109."""
    v = torch.zeros(n, heads, 128)
    v[torch.arange(n), :, torch.arange(n) % 128] = 1.0
    return v.to(dtype)


ITEM_LENS = [1, 300, 128, 129, 0, 700, 64, 257, 5, 40, 1, 512, 90, 33, 0, 17, 256, 2, 127, 385] + [1, 3] * 10


@pytest.mark.parametrize("nq,nkv", [(32, 32), (40, 40), (64, 8)])
@pytest.mark.parametrize("cap,bias,two_way", [(0.0, False, False), (0.0, False, True), (0.0, True, False), (0.0, True, True),
                                              (20.0, False, False), (20.0, False, True), (60.0, True, True)])
def test_docs_many_items_per_block(nq, nkv, cap, bias, two_way):
    # each persistent block takes several work items, among them ones whose second row tile is
    # empty and ones beyond the first 32 documents
    pairs = nq // nkv % 2 == 0
    items = sum(-(-n // (128 if pairs else 256)) for n in ITEM_LENS) * (nq // 2 if pairs else nq)
    m, _ = _model(nq, nkv)
    assert items > 4 * torch.cuda.get_device_properties(0).multi_processor_count and len(ITEM_LENS) > 32
    n = sum(ITEM_LENS)
    cu = [0]
    for x in ITEM_LENS:
        cu.append(cu[-1] + x)
    pre = torch.randint(0, 280, (len(ITEM_LENS),), generator=_gen(8)).tolist() if two_way else None
    slopes = _slopes(nq) if bias else None
    sc = binding.Scores(cap=cap, slopes=None if slopes is None else slopes.cuda())
    q, k = (_randn((n, h, 128), torch.bfloat16, 230 + h) for h in (nq, nkv))
    for q, v, more in ((q, _randn((n, nkv, 128), torch.bfloat16, 232), 0.0),
                       ((q.float() * 0.3).bfloat16(), _one_key_per_dim(n, nkv, torch.bfloat16), 2.0 ** -8)):
        outs = []
        qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
        for _ in range(3):
            out = torch.full((n, nq * 128), 3.0, dtype=torch.bfloat16, device="cuda")
            m.op_attention_docs(qd, kd, vd, _i32(cu), out, prefix=None if pre is None else _i32(pre), scores=sc)
            outs.append(out)
        m.sync()
        ref, mass = _docs_reference(q, k, v, ITEM_LENS, pre, 128 ** -0.5, cap, slopes)
        _within(outs[0].view(n, nq, 128), ref, _attn_bound(ref, mass, "bf16", n, 128, 0, 0) +
                more * np.abs(ref) + 2.0 ** -109, "items")
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_docs_reference_is_the_definition():
    need_gpu()
    q, k, v = (_randn((45, h, 128), torch.bfloat16, 240 + h) for h in (4, 2, 2))
    lens, pre, sl = [30, 0, 15], [7, 3, 0], _slopes(4)
    cu = [0, 30, 30, 45]
    for cap in (0.0, 9.0):
        got = _docs_reference(q, k, v, lens, pre, 0.1, cap, sl)
        want = A.attend_documents(f64(q), f64(k), f64(v), cu, pre, 0.1, cap, f64(sl))
        for a, b in zip(got, want):
            np.testing.assert_allclose(a, b, atol=1e-12)


# --------------------------------------------------------------------------- many rows
@pytest.mark.parametrize("nq,nkv,d,dtype,src,rotary,half,norm,e4m3,page,side", [
    (32, 32, 128, "bf16", "f32", 128, True, "qk", None, 16, True),
    (32, 32, 128, "bf16", "bf16", 128, False, "", None, 0, False),
    (32, 32, 128, "bf16", "f32", 64, True, "k", (0.02, 0.004), 64, True),
    (32, 32, 128, "bf16", "bf16", 0, False, "q", None, 48, False),
    (40, 8, 128, "bf16", "f32", 96, False, "qk", (0.02, 0.004), 0, False),
    (40, 8, 128, "bf16", "bf16", 96, True, "qk", None, 16, True),
    (64, 8, 128, "bf16", "f32", 128, False, "qk", None, 64, True),
    (12, 4, 256, "f32", "f32", 256, True, "qk", None, 16, True),
    (12, 4, 256, "f32", "f32", 136, False, "", None, 0, True),
    (30, 5, 128, "f32", "f32", 128, False, "k", None, 0, False)])
def test_rows_one_block_walks_a_rows_heads(nq, nkv, d, dtype, src, rotary, half, norm, e4m3, page, side):
    # rows enough for one block per row, which walks several chunks of its heads (the last one
    # ragged in most of these) with the next one's values loaded ahead
    lens, starts, lead, tail = [1, 500, 0, 131, 2, 30, 64], [9, 0, 4, 1000, 300, 63, 16], 3, 5
    m, shape = _model(nq, nkv, d, dtype, max_batch=len(lens))
    dt, heads, n = shape.torch_dtype, nq + 2 * nkv, lead + sum(lens) + tail
    chunk = 256 // (1 << (d // 8 - 1).bit_length())  # heads that a block takes at a time
    chunks = -(-heads // chunk)
    assert chunks > 1 and chunks * n > 8 * torch.cuda.get_device_properties(0).multi_processor_count
    x = _randn((n, heads * d), torch.float32 if src == "f32" else dt, 250, 1.5)
    gains = [(1 + 0.1 * torch.randn(d, generator=_gen(251 + i))).to(dt) for i in range(2)]
    top = max(s + l for s, l in zip(starts, lens))
    table = A.rotation_table(top, rotary, kind="linear", factor=4.0).astype(np.float32) if rotary else None
    cu = [lead]
    for l in lens:
        cu.append(cu[-1] + l)
    if page:
        pages = [max(1, math.ceil((s + l) / page)) for s, l in zip(starts, lens)]
        pt, total = synth.page_table(pages, max(pages), 7)
        kv = binding.KVCache(shape, n_pages=total, page_size=page, page_table=pt.cuda(), e4m3=e4m3)
    else:
        kv = binding.KVCache(shape, batch=len(lens), capacity=top, e4m3=e4m3)
    mark = 0x35 if e4m3 else 7.0
    kv.k.fill_(mark)
    kv.v.fill_(mark)
    q_out = torch.full((n, nq * d), 3.0, dtype=dt, device="cuda")
    ko, vo = (torch.full((n, nkv * d), 3.0, dtype=dt, device="cuda") if side else None for _ in range(2))
    rope = binding.Rope(torch.from_numpy(table).cuda(), binding.ROPE_HALF if half else binding.ROPE_ADJACENT) \
        if rotary else None
    m.op_rope_norm_append(x.cuda(), _i32(starts), 0, kv, q_out, rope=rope, cu_rows=_i32(cu),
                          q_gain=gains[0].cuda() if "q" in norm else None,
                          k_gain=gains[1].cuda() if "k" in norm else None, eps=1e-6, k_out=ko, v_out=vo)
    m.sync()
    # all rows at once in fp64
    r = np.arange(cu[0], cu[-1])
    seq = np.searchsorted(np.array(cu[1:]), r, side="right")
    pos = np.array(starts)[seq] + r - np.array(cu)[seq]
    y = f64(x)[r].reshape(len(r), heads, d)
    q, k, v = y[:, :nq], y[:, nq:nq + nkv], y[:, nq + nkv:]
    q = A.head_norm(q, f64(gains[0]), 1e-6) if "q" in norm else q
    k = A.head_norm(k, f64(gains[1]), 1e-6) if "k" in norm else k
    if rotary:
        c, s = table.astype(np.float64)[pos][:, None, :, 0], table.astype(np.float64)[pos][:, None, :, 1]
        i0 = np.arange(rotary // 2) if half else 2 * np.arange(rotary // 2)
        i1 = i0 + rotary // 2 if half else i0 + 1
        q, k = q.copy(), k.copy()
        for t in (q, k):
            a, b = t[..., i0], t[..., i1]
            t[..., i0], t[..., i1] = a * c - b * s, a * s + b * c
    for got, ref, what in ((q_out, q, "q"),) + (((ko, k, "k rows"), (vo, v, "v rows")) if side else ()):
        big = np.abs(ref).max(-1, keepdims=True)
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * big if dtype == "bf16" else 2.0 ** -24 * np.abs(ref) + 32 * 2.0 ** -24 * big
        _within(got[cu[0]:cu[-1]].view(len(r), -1, d), ref, tol, what)
        assert torch.all(got[:lead] == 3.0) and torch.all(got[cu[-1]:] == 3.0)
    for cache, ref, scale in ((kv.k, k, e4m3 and e4m3[0]), (kv.v, v, e4m3 and e4m3[1])):
        big = np.abs(ref).max(-1, keepdims=True)
        c = cache.view(torch.float8_e4m3fn).float() if e4m3 else cache
        c = f64(c)[0]
        at = (pt.numpy()[seq, pos // page], slice(None), pos % page) if page else (seq, slice(None), pos)
        got = torch.from_numpy(c[at])
        if e4m3:
            ref = np.clip(ref / scale, -448, 448)
            tol = 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 + 2.0 ** -18 * np.minimum(big / scale, 448)
        elif dtype == "bf16":
            tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * big
        else:
            tol = 2.0 ** -24 * np.abs(ref) + 32 * 2.0 ** -24 * big
        _within(got, ref, tol, "cache")
        rest = np.ones(c.shape[:1] + c.shape[2:3], bool)
        rest[(at[0], at[2])] = False
        left = cache[0].permute(0, 2, 1, 3)[torch.from_numpy(rest).cuda()]
        assert left.numel() and torch.all(left == mark), "another slot was written"


# --------------------------------------------------------------------------- caches with room to grow
@pytest.mark.parametrize("room", [1024, 4096, 32768])
@pytest.mark.parametrize("dtype,nq,nkv,positions,shared", [
    ("bf16", 8, 8, [465], 0), ("bf16", 32, 32, [465], 0), ("bf16", 16, 1, [465, 0], 0),
    ("bf16", 8, 8, [499, 250, 3, 120], 0), ("bf16", 8, 2, [499, 250, 130, 640, 60], 130),
    ("bf16", 8, 8, [249 - b % 7 for b in range(64)], 0), ("bf16", 40, 8, [959, 900, 999], 900),
    ("f32", 8, 2, [465, 3, 64], 0), ("f32", 8, 8, [300, 200], 130)])
@pytest.mark.parametrize("page", [0, 16])
def test_shared_cache_with_room(room, dtype, nq, nkv, positions, shared, page):
    # the cache has room for many more keys than there are, which chooses other splits of them
    B, d, G = len(positions), 128, nq // nkv
    if page == 0 and B * nkv * room > 1 << 20:
        pytest.skip("the same plan as the paged cache's")
    m, shape = _model(nq, nkv, d, dtype, max_batch=B, max_seq=room)
    dt, top = shape.torch_dtype, max(positions) + 1
    q = _randn((B, nq, d), dt, 260, 0.4)
    k = _randn((B, nkv, top, d), dt, 261, 1.0)
    k[:, :, :shared] = k[:1, :, :shared]
    if page:
        width = -(-top // page)
        n_pages = B * width
        table = torch.full((B, room // page), -1, dtype=torch.int32)
        table[:, :width] = torch.randperm(n_pages, generator=_gen(262)).view(B, width).int()
        slots = (1, n_pages, nkv, page, d)
    else:
        slots = (1, B, nkv, room, d)
    one = _one_key_per_dim(top, B * nkv, dt).view(top, B, nkv, d).permute(1, 2, 0, 3).clone()
    for v, more in ((_randn((B, nkv, top, d), dt, 263), 0.0), (one, 2.0 ** -8)):
        v[:, :, :shared] = v[:1, :, :shared]
        caches = []
        for t in (k, v):
            c = torch.full(slots, float("nan"), dtype=dt, device="cuda")
            for b, p in enumerate(positions):
                n = max(p + 1, shared)
                if page:
                    at = torch.arange(n)
                    c[0][table[b].long()[at // page].cuda(), :, (at % page).cuda()] = t[b, :, :n].transpose(0, 1).cuda()
                else:
                    c[0, b, :, :n] = t[b, :, :n].cuda()
            caches.append(c)
        kw = dict(n_pages=n_pages, page_size=page, page_table=table.cuda()) if page else dict(batch=B, capacity=room)
        kv = binding.KVCache(shape, k=caches[0], v=caches[1], **kw)
        out = torch.full((B, nq * d), 3.0, dtype=dt, device="cuda")
        m.op_attention_decode_shared(q.cuda(), _i32(positions), 0, kv, out, shared_len=shared)
        m.sync()
        for b, p in enumerate(positions):
            K, V = (t[b, :, :p + 1].cuda().double().repeat_interleave(G, 0) for t in (k, v))
            w = torch.softmax(torch.einsum("hd,hjd->hj", q[b].cuda().double(), K) / math.sqrt(d), -1)
            ref, mass = f64(torch.einsum("hj,hjd->hd", w, V)), f64(torch.einsum("hj,hjd->hd", w, V.abs()))
            big = float(q.float().abs().max() * k.float().abs().max()) * math.sqrt(d) if dtype == "f32" else 0
            _within(out[b].view(nq, d), ref, _attn_bound(ref, mass, dtype, p + 1, d, big, 0) + more * np.abs(ref),
                    "b=%d" % b)


@pytest.mark.parametrize("cap,bias", [(0.0, False), (50.0, False), (50.0, True)])
def test_docs_values_scale(cap, bias):
    # the outputs of values times a power of two are the outputs times it, to the bit, with every
    # score at the cap or far below it
    m, _ = _model(4, 2)
    n = 400
    q, k, v = (_randn((n, h, 128), torch.bfloat16, 270 + h, s).cuda() for h, s in ((4, 8.0), (2, 8.0), (2, 1.0)))
    sc = binding.Scores(cap=cap, slopes=_slopes(4).cuda() if bias else None)
    outs = []
    for e in (0, 40, -30):
        out = torch.empty(n, 512, dtype=torch.bfloat16, device="cuda")
        m.op_attention_docs(q, k, v * 2.0 ** e, _i32([0, 250, n]), out, scores=sc)
        outs.append(out.float() * 2.0 ** -e)
    m.sync()
    assert torch.isfinite(outs[0]).all() and torch.equal(outs[0], outs[1])
    assert torch.equal(outs[0], outs[2])


def test_docs_all_empty_and_single_rows():
    for dtype in ("bf16", "f32"):
        m, shape = _model(4, 2, 128, dtype)
        q, k = (torch.ones(3, h, 128, dtype=shape.torch_dtype, device="cuda") for h in (4, 2))
        out = torch.full((3, 512), 3.0, dtype=shape.torch_dtype, device="cuda")
        m.op_attention_docs(q, k, k, _i32([3, 3, 3]), out, prefix=_i32([1, 2]))
        m.sync()
        assert torch.all(out == 3.0)
        _docs_case(4, 2, 128, dtype, [0] * 70 + [1] + [0] * 70, prefix=[5] * 141)
        _docs_case(1, 1, 128, dtype, [1])


@pytest.mark.parametrize("page", [1, 5, 12])
def test_fp32_pages_of_any_size(page):
    _shared_case(4, 2, 64, "f32", [0, 70, 99, 130], 52, page=page, cap=20.0)
    _rows_case(4, 2, 64, "f32", "f32", [7, 1, 20], [0, 100, 3], rotary=64, page=page)


@pytest.mark.parametrize("nq,nkv,shared,room", [(64, 8, 1100, 1600), (40, 40, 3200, 3400), (16, 16, 0, 700)])
def test_append_and_decode_without_a_wait_between(nq, nkv, shared, room):
    # the own keys' blocks start while the prefix kernel runs: they see what was appended just before it,
    # and what is enqueued behind them waits for both
    B, steps = 24, 12
    m, shape = _model(nq, nkv, max_batch=B, max_seq=room)
    k, v = (_randn((1, B, nkv, room, 128), torch.bfloat16, 280 + i).cuda() for i in range(2))
    first = [shared + (29 * b) % (room - shared - steps) for b in range(B)]
    xs = [_randn((B, shape.qkv_rows), torch.float32, 290 + i).cuda() for i in range(steps)]
    pos = [_i32([p + i for p in first]) for i in range(steps)]
    rope = binding.Rope(None, binding.ROPE_HALF, 128)
    runs = []
    for wait in (True, False):
        ck, cv = k.clone(), v.clone()
        cache = binding.KVCache(shape, batch=B, capacity=room, k=ck, v=cv)
        q = torch.empty(B, nq * 128, dtype=torch.bfloat16, device="cuda")
        outs = [torch.empty_like(q) for _ in range(steps)]
        torch.cuda.synchronize()
        for i in range(steps):
            m.op_rope_norm_append(xs[i], pos[i], 0, cache, q, rope=rope)
            if wait:
                torch.cuda.synchronize()
            m.op_attention_decode_shared(q, pos[i], 0, cache, outs[i], shared_len=shared, scores=binding.Scores(cap=30.0))
            if wait:
                torch.cuda.synchronize()
        m.sync()
        runs.append((outs, ck, cv))
    assert all(torch.equal(a, b) for a, b in zip(runs[0][0], runs[1][0]))
    assert torch.equal(runs[0][1], runs[1][1]) and torch.equal(runs[0][2], runs[1][2])


# --------------------------------------------------------------------------- refusals
def test_refusals():
    m, shape = _model(4, 2, max_batch=2, max_seq=64)
    m32, s32 = _model(2, 1, 64, "f32", max_batch=2, max_seq=64)
    d, dt = 128, torch.bfloat16
    x = torch.zeros(2, shape.qkv_rows, device="cuda")
    pos = _i32([0, 1])
    kv = binding.KVCache(shape, batch=2, capacity=64)
    q = torch.zeros(2, 4 * d, dtype=dt, device="cuda")
    k = torch.zeros(2, 2 * d, dtype=dt, device="cuda")
    table = binding.rope_table(64, 64)

    def refused(code, fn, *a, **kw):
        with pytest.raises(binding.LlamaError) as e:
            fn(*a, **kw)
        assert e.value.rc == code
    ap = m.op_rope_norm_append
    refused(1, ap, x, pos, 1, kv, q)                                          # layer
    refused(1, ap, x, pos, 0, kv, q, q_gain=q[0, :d].contiguous(), eps=0.0)   # eps
    refused(2, ap, x, pos, 0, kv, q, rope=binding.Rope(None, 0, 60))          # not a multiple of 8
    refused(1, ap, x, pos, 0, kv, q, rope=binding.Rope(None, 0, 64))          # the context turns whole heads
    refused(1, ap, x, pos, 0, kv, q, rope=binding.Rope(table, 2))             # layout
    refused(1, ap, x, pos, 0, kv, q, rope=binding.Rope(binding.rope_table(8, 136)))
    refused(1, ap, x[:1], pos, 0, kv, q[:1])                                  # one row per sequence
    with pytest.raises(ValueError):
        ap(x.half(), pos, 0, kv, q)
    with pytest.raises(ValueError):
        ap(x, pos.long(), 0, kv, q)
    with pytest.raises(ValueError):
        ap(x, pos, 0, kv, q[:1])
    bad = torch.zeros(2, shape.qkv_rows + 2, device="cuda")[:, :shape.qkv_rows]
    refused(1, ap, bad, pos, 0, kv, q)                                        # rows not 16-byte aligned
    docs = m.op_attention_docs
    cu = _i32([0, 2])
    for sc in (binding.Scores(cap=-1.0), binding.Scores(scale=float("nan")), binding.Scores(cap=float("inf"))):
        refused(1, docs, q, k, k, cu, q.clone(), scores=sc)
    with pytest.raises(ValueError):
        docs(q, q, k, cu, q.clone())
    with pytest.raises(ValueError):
        docs(q, k, k, cu, q.clone(), scores=binding.Scores(slopes=torch.ones(3, device="cuda")))
    with pytest.raises(ValueError):
        docs(q, k, k, cu, q.t().contiguous().t())
    dec = m.op_attention_decode_shared
    refused(3, dec, q, pos, 0, kv, q.clone(), shared_len=65)                  # past the cache
    refused(1, dec, q, pos, 0, kv, q.clone(), shared_len=8, shared_seq=2)
    refused(1, dec, q, pos, 0, kv, q.clone(), shared_len=-1)
    refused(2, dec, q, pos, 0, binding.KVCache(shape, batch=2, capacity=64, e4m3=(1.0, 1.0)), q.clone())
    three = torch.zeros(3, 4 * d, dtype=dt, device="cuda")
    refused(3, dec, three, _i32([0, 0, 0]), 0, binding.KVCache(shape, batch=3, capacity=64), three.clone())
    # tensors that are not on the context's device: each one by itself on the CPU, all of them elsewhere
    for bad in range(3):
        a = [t.cpu() if i == bad else t for i, t in enumerate((q, pos, q.clone()))]
        with pytest.raises(ValueError):
            dec(a[0], a[1], 0, kv, a[2])
        with pytest.raises(ValueError):
            docs(a[0], k, k, cu if bad != 1 else cu.cpu(), a[2])
    with pytest.raises(ValueError):
        ap(x, pos, 0, kv, q, rope=binding.Rope(table.cpu()))
    host = binding.KVCache(shape, batch=2, capacity=64, device="cpu")
    m._dev += 1
    try:
        for call in (lambda: ap(x, pos, 0, kv, q), lambda: docs(q, k, k, cu, q.clone()), lambda: dec(q, pos, 0, kv, q.clone())):
            with pytest.raises(ValueError):
                call()
    finally:
        m._dev -= 1
    with pytest.raises(ValueError):
        dec(q, pos, 0, host, q.clone())
    x32 = torch.zeros(2, s32.qkv_rows, device="cuda")
    with pytest.raises(ValueError):
        m32.op_rope_norm_append(x32.bfloat16(), pos, 0, binding.KVCache(s32, batch=2, capacity=64),
                                torch.zeros(2, 128, device="cuda"))
    m.sync()
    m32.sync()


# --------------------------------------------------------------------------- checked build
def test_suite_passes_on_the_bounds_check_build():
    # every kernel checks its shared-memory layout and index invariants there
    need_gpu()
    if os.environ.get("LLAMA_GB300_BOUNDS_CHECK") == "1":
        pytest.skip("this is that run")
    from llama2_decoder_forward_gb300 import build
    build.build_library(checked=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", os.path.abspath(__file__)],
                       cwd=root, env=dict(os.environ, LLAMA_GB300_BOUNDS_CHECK="1"), capture_output=True, text=True,
                       timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
