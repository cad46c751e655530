"""The operators on caches whose slots are not one token after the other against
plain fp64 forms: rows moved after a tree is accepted, eviction by accumulated
weight, rows appended with positions of their own.

Moves and selections are exact. Appended rows: as in the tests of
llama_op_rope_norm_append, one rounding (2^-8 relative in bf16, 2^-24 in fp32) of
an fp32 value whose own error is some 2^-24 of the head's largest value.
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
from oracle import cache_ops as C

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _model(nq, nkv, d=128, dtype="bf16", max_batch=8, max_seq=4096, n_layers=1):
    need_gpu()
    shape = synth.Shape(n_layers, 256, nq, nkv, d, 256, 256, dtype=dtype)
    w = {"layers": [synth.layer_weights(shape, 3, l) for l in range(n_layers)]}
    return binding.Model(shape, to_dev(w), max_batch=max_batch, max_tokens=0, max_seq=max_seq,
                         has_embed_head=False), shape


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _within(got, ref, bound, what):
    got = f64(got)
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isfinite(err), err - bound, np.inf)), err.shape)
        raise AssertionError("%s: %d of %d out of tolerance; worst at %s: got %r ref %r bound %r"
                             % (what, bad.sum(), bad.size, i, got[i], ref[i], np.broadcast_to(bound, err.shape)[i]))


def _cache(shape, B, slots, page, e4m3=False, seed=1, spare=3):
    """A cache for B sequences of `slots` slots, filled with numbers that tell the slots apart, and its page table."""
    kw = dict(e4m3=(0.5, 0.25)) if e4m3 else {}
    if page:
        n = -(-slots // page)
        order = torch.randperm(B * n + spare, generator=_gen(seed))[:B * n].view(B, n).to(torch.int32)
        kv = binding.KVCache(shape, n_pages=B * n + spare, page_size=page, page_table=order.cuda(), **kw)
    else:
        kv = binding.KVCache(shape, batch=B + 1, capacity=slots + 5, **kw)
    for i, t in enumerate((kv.k, kv.v)):
        x = torch.randint(0, 1 << 30, t.shape, generator=_gen(seed + 7 + i), dtype=torch.int32)
        # bit patterns: a move copies them, whatever they stand for
        if e4m3:
            t.copy_(x.to(torch.uint8))
        elif t.dtype == torch.bfloat16:
            t.view(torch.int16).copy_(x.to(torch.int16))
        else:
            t.view(torch.int32).copy_(x)
    return kv


def _bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu().numpy()


def _at(kv, b, slot):
    """Index of a slot's heads in one layer's bits."""
    if kv.page_size == 0:
        return (b, slice(None), slot)
    return (int(kv.page_table[b, slot // kv.page_size]), slice(None), slot % kv.page_size)


TYPES = [("bf16", False, 128), ("bf16", True, 128), ("f32", False, 64), ("f32", False, 40), ("f32", False, 256),
         ("f32", False, 8)]


# --------------------------------------------------------------------------- commit
def _commit_case(dtype, e4m3, d, page, starts, paths, nkv=3, layers=3, layer=None, width=None, pad=-7, seed=3):
    m, shape = _model(nkv, nkv, d, dtype, max_batch=len(starts), n_layers=layers)
    kv = _cache(shape, len(starts), 12 + max(s + max(p, default=0) for s, p in zip(starts, paths)), page, e4m3, seed)
    want = [_bits(t).copy() for t in (kv.k, kv.v)]
    for w in want:
        old = w.copy()
        for b, (s, p) in enumerate(zip(starts, paths)):
            for i, x in enumerate(p):
                for l in range(layers) if layer is None else [layer]:
                    w[l][_at(kv, b, s + i)] = old[l][_at(kv, b, s + x)]
    width = width or max(1, max(map(len, paths)))
    path = [p + [pad] * (width - len(p)) for p in paths]
    m.op_cache_commit(kv, _i32(starts), _i32(path), _i32([len(p) for p in paths]), layer=layer)
    m.sync()
    for t, w in zip((kv.k, kv.v), want):
        assert np.array_equal(_bits(t), w)


@pytest.mark.parametrize("dtype,e4m3,d", TYPES)
@pytest.mark.parametrize("page", [0, 16, 48])
def test_commit(dtype, e4m3, d, page):
    _commit_case(dtype, e4m3, d, page, [0, 30, 17, 5], [[0, 1, 2], [0, 3, 4, 11, 25], [], [7]])


@pytest.mark.parametrize("n", [1, 2, 31, 33, 64, 130, 700])
def test_commit_lengths(n):
    r = np.random.RandomState(n)
    _commit_case("bf16", False, 128, 16, [3, 40], [sorted(r.choice(2 * n, n, replace=False).tolist()), list(range(n))])


def test_commit_one_layer():
    _commit_case("bf16", False, 128, 16, [9, 0], [[0, 2], [1, 3, 4]], layer=1)


def test_commit_long_paths_of_wide_rows():
    r = np.random.RandomState(1)
    _commit_case("f32", False, 256, 16, [0], [sorted(r.choice(900, 500, replace=False).tolist())], nkv=1, layers=1)


def test_commit_bad_paths_are_flagged_and_skipped():
    m, shape = _model(2, 2, max_batch=6)
    kv = _cache(shape, 6, 64, 16, spare=0)
    kv.page_table[5, 1] = 99
    starts = [8, 60, -1, 0, 0, 14]
    paths = [[2, 1, 4], [1, 70, 71], [1, 2, 3], [0, 1, 2], [1, 2, 3], [1, 2, 3]]
    # 0: the 1 does not ascend, the 4 does again; 1 leaves the cache; 2 starts before it;
    # 3 and 4 have lengths out of range (4's is cut); 5 reaches a page that is not there
    want = [_bits(t).copy() for t in (kv.k, kv.v)]
    for w in want:
        old = w.copy()
        w[0][_at(kv, 0, 8)], w[0][_at(kv, 0, 10)] = old[0][_at(kv, 0, 10)], old[0][_at(kv, 0, 12)]
        w[0][_at(kv, 1, 60)] = old[0][_at(kv, 1, 61)]
        w[0][_at(kv, 4, 0)], w[0][_at(kv, 4, 1)], w[0][_at(kv, 4, 2)] = (old[0][_at(kv, 4, i)] for i in (1, 2, 3))
        w[0][_at(kv, 5, 14)] = old[0][_at(kv, 5, 15)]  # the others lie on page 99
    m.op_cache_commit(kv, _i32(starts), _i32(paths), _i32([3, 3, 3, -2, 9, 3]))
    rc, flags = m.sync_status()
    assert rc == 5 and flags == binding.FLAG_POS_RANGE | binding.FLAG_PAGE_RANGE
    for t, w in zip((kv.k, kv.v), want):
        assert np.array_equal(_bits(t), w)


# --------------------------------------------------------------------------- evict
def _evict_case(dtype, e4m3, d, page, lens, keep, first, recent, nkv=2, layers=2, layer=None, weights=None, ld=None,
                alias=False, seed=5):
    B, top = len(lens), max(max(lens), 1)
    m, shape = _model(nkv, nkv, d, dtype, max_batch=B, n_layers=layers)
    kv = _cache(shape, B, top, page, e4m3, seed)
    ld = ld or top
    n_l = layers if layer is None else 1
    if weights is None:
        weights = torch.rand(n_l, B, nkv, ld, generator=_gen(seed)).log().neg()
    w0 = weights.numpy().copy()
    want = [_bits(t).copy() for t in (kv.k, kv.v)]
    old = [w.copy() for w in want]
    kept = np.full((n_l, B, nkv, keep), -1, np.int32)
    wout = np.zeros_like(w0)
    for l in range(n_l):
        for b, n in enumerate(lens):
            for g in range(nkv):
                k = C.evict(w0[l, b, g, :n], keep, first, recent)
                kept[l, b, g, :len(k)] = k
                wout[l, b, g, :len(k)] = w0[l, b, g, k]
                for w, o in zip(want, old):
                    for i, x in enumerate(k):
                        li = l if layer is None else layer
                        to, fro = _at(kv, b, i), _at(kv, b, x)
                        w[li][to[0], g, to[2]] = o[li][fro[0], g, fro[2]]
    wd = weights.cuda()
    kd = torch.full(kept.shape, 77, dtype=torch.int32, device="cuda")
    od = wd if alias else torch.full_like(wd, 9.0)
    m.op_cache_evict(kv, _i32(lens), keep, wd, kd, layer=layer, first=first, recent=recent,
                     weights_out=None if alias else od)
    m.sync()
    assert np.array_equal(kd.cpu().numpy(), kept)
    assert np.array_equal(od.cpu().numpy(), wout, equal_nan=True)
    if not alias:
        assert np.array_equal(wd.cpu().numpy(), w0, equal_nan=True)
    for t, w in zip((kv.k, kv.v), want):
        assert np.array_equal(_bits(t), w)


@pytest.mark.parametrize("dtype,e4m3,d", TYPES)
@pytest.mark.parametrize("page", [0, 16, 48])
def test_evict(dtype, e4m3, d, page):
    _evict_case(dtype, e4m3, d, page, [90, 0, 41, 40, 1], 40, 3, 11)


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("lens,keep,first,recent", [
    ([1500, 700], 600, 4, 100), ([513, 512], 511, 0, 0), ([600], 1, 0, 0), ([600], 1, 1, 0), ([600], 1, 0, 1),
    ([700, 699], 20, 20, 0), ([700], 300, 0, 300), ([700], 300, 100, 200), ([2], 1, 0, 0), ([1025], 1024, 1000, 23),
    ([5000], 2100, 4, 64)])
def test_evict_sizes(lens, keep, first, recent, alias):
    _evict_case("bf16", False, 128, 16, lens, keep, first, recent, alias=alias, layers=1)


def test_evict_one_layer():
    _evict_case("bf16", False, 128, 16, [100, 50], 30, 2, 5, layers=3, layer=1)


def test_evict_room_behind():
    # weights with room for more slots than are filled: zeros there, nothing read
    w = torch.full((1, 2, 2, 400), float("nan"))
    w[..., :300] = torch.rand(1, 2, 2, 300, generator=_gen(8))
    _evict_case("bf16", False, 128, 0, [300, 200], 128, 4, 32, layers=1, weights=w, ld=400)


def test_evict_keep_above_everything():
    _evict_case("bf16", False, 128, 16, [30, 12], 64, 4, 32, layers=1)


@pytest.mark.parametrize("kind", ["zeros", "ties", "signs", "nan", "inf", "tiny", "steps"])
def test_evict_weights(kind):
    n = 900
    w = torch.rand(1, 2, 2, n, generator=_gen(11))
    if kind == "zeros":
        w.zero_()
    elif kind == "ties":
        w = (w * 5).floor()
    elif kind == "signs":
        w = (w - 0.5) * 3
        w[..., ::7] = -0.0
        w[..., 3::7] = 0.0
    elif kind == "nan":
        w[..., ::2] = float("nan")  # more than are dropped: some NaN stay
    elif kind == "inf":
        w[..., ::5] = float("inf")
        w[..., 1::5] = -float("inf")
    elif kind == "tiny":
        w = w * 1e-41  # below the normal numbers
    else:
        w = 1.0 + torch.randint(0, 40, w.shape, generator=_gen(12)) * 2.0 ** -23  # the last bits decide
    _evict_case("bf16", False, 128, 16, [n, n - 1], 600, 3, 50, layers=1, weights=w.float())


def test_evict_many_heads():
    # more (layer, sequence, head) items than the slices of one would fill
    _evict_case("bf16", False, 128, 16, [70, 64, 33, 71] * 5, 32, 1, 8, nkv=8, layers=4)


@pytest.mark.parametrize("layers,nkv,page,n,keep,dtype,d", [
    (8, 32, 16, 4000, 1500, "bf16", 128), (32, 32, 0, 2000, 1900, "bf16", 128), (1, 1, 16, 20000, 15000, "bf16", 128),
    (4, 8, 64, 3000, 2000, "f32", 256), (2, 3, 0, 6000, 5999, "f32", 40),
    (5, 32, 16, 3000, 1000, "bf16", 128), (40, 5, 0, 700, 300, "f32", 8), (9, 30, 64, 1500, 1490, "f32", 40)])
def test_evict_long_lists(layers, nkv, page, n, keep, dtype, d):
    # chunks follow one another in every CTA, and none may pass another one's rows by
    m, shape = _model(nkv, nkv, d, dtype, max_batch=1, max_seq=8, n_layers=layers)
    kv = _cache(shape, 1, n, page)
    for i in range(3):
        w = torch.rand(layers, 1, nkv, n, generator=_gen(i)).cuda()
        order = torch.sort(w, dim=-1, descending=True, stable=True)[1][..., :keep]
        kept = torch.sort(order, dim=-1)[0]
        got = torch.empty(layers, 1, nkv, keep, dtype=torch.int32, device="cuda")

        def rows(t, slot):  # [layers, nkv, slots, d]
            l, g = torch.arange(layers, device="cuda")[:, None, None], torch.arange(nkv, device="cuda")[None, :, None]
            if page:
                return t[l, kv.page_table[0].long()[slot // page], g, slot % page]
            return t[l, 0, g, slot]
        ints = {2: torch.int16, 4: torch.int32}[kv.k.element_size()]
        views = [t.view(ints) for t in (kv.k, kv.v)]
        want = [rows(t, kept[:, 0]) for t in views]
        m.op_cache_evict(kv, _i32([n]), keep, w, got, weights_out=torch.empty_like(w))
        m.sync()
        assert torch.equal(got.long(), kept)
        at = torch.arange(keep, device="cuda").expand(layers, nkv, keep)
        for t, x in zip(views, want):
            assert torch.equal(rows(t, at), x)


def test_evict_bad_lengths_and_pages_are_flagged():
    m, shape = _model(2, 2, max_batch=4)
    kv = _cache(shape, 4, 64, 16)
    kv.page_table[3, 2] = -5
    w = torch.rand(1, 4, 2, 64, generator=_gen(13)).cuda()
    old = [_bits(t).copy() for t in (kv.k, kv.v)]
    table = kv.page_table.cpu()
    kept = torch.zeros(1, 4, 2, 20, dtype=torch.int32, device="cuda")
    out = torch.empty_like(w)
    m.op_cache_evict(kv, _i32([-3, 70, 20, 64]), 20, w, kept, weights_out=out)
    rc, flags = m.sync_status()
    assert rc == 5 and flags == binding.FLAG_POS_RANGE | binding.FLAG_PAGE_RANGE
    assert torch.all(kept[0, 0] == -1) and torch.all(out[0, 0] == 0)
    wh = w.cpu().numpy()
    for b, n in ((1, 64), (2, 20), (3, 64)):  # 70 is cut to the cache's 64 slots
        for g in range(2):
            k = C.evict(wh[0, b, g, :n], 20, 0, 0)
            assert kept[0, b, g].tolist() == k
            for t, o in zip((kv.k, kv.v), old):
                got = _bits(t)[0]
                for i, x in enumerate(k):
                    a, f = (int(table[b, s // 16]) for s in (i, x))
                    from_bad = b == 3 and x // 16 == 2
                    src = o[0][f, g, x % 16] if not from_bad else o[0][a, g, i % 16]
                    assert np.array_equal(got[a, g, i % 16], src)


# --------------------------------------------------------------------------- rows with positions of their own
@pytest.mark.parametrize("dtype,d,rotary,half", [("bf16", 128, 128, True), ("bf16", 128, 64, False), ("f32", 64, 64, True)])
@pytest.mark.parametrize("token", [False, True])
def test_append_positions(dtype, d, rotary, half, token):
    nq, nkv, lens, starts = 4, 2, ([1, 1, 1] if token else [5, 0, 3]), [30, 4, 0]
    m, shape = _model(nq, nkv, d, dtype)
    n, dt = sum(lens), shape.torch_dtype
    pos = torch.randint(0, 90, (n,), generator=_gen(2)).tolist()
    x = torch.randn(n, shape.qkv_rows, generator=_gen(4))
    table = A.rotation_table(90, rotary).astype(np.float32)
    kv = binding.KVCache(shape, batch=3, capacity=40)
    q = torch.empty(n, nq * d, dtype=dt, device="cuda")
    cu = np.concatenate(([0], np.cumsum(lens))).tolist()
    rope = binding.Rope(torch.from_numpy(table).cuda(), binding.ROPE_HALF if half else binding.ROPE_ADJACENT)
    m.op_rope_norm_append(x.cuda(), _i32(starts), 0, kv, q, rope=rope, cu_rows=None if token else _i32(cu),
                          positions=_i32(pos))
    m.sync()
    xf, (K, V) = f64(x).reshape(n, nq + 2 * nkv, d), (f64(t)[0].copy() for t in (kv.k, kv.v))
    eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24

    def close(got, ref, what):
        _within(got, ref, eps * np.abs(ref) + (2.0 ** -18 if dtype == "bf16" else 2.0 ** -19) * np.abs(ref).max(), what)

    for b in range(3):
        for i in range(lens[b]):
            r, s = cu[b] + i, starts[b] + i
            cs = table[pos[r]].astype(np.float64)
            close(q[r].view(nq, d), A.rotate(xf[r, :nq], cs, half), "q")
            close(K[b, :, s], A.rotate(xf[r, nq:nq + nkv], cs, half), "k")
            close(V[b, :, s], xf[r, nq + nkv:], "v")
            K[b, :, s] = V[b, :, s] = 0
    assert not K.any() and not V.any()


def test_append_positions_out_of_range():
    m, shape = _model(4, 2)
    x = torch.randn(4, shape.qkv_rows, generator=_gen(6)).cuda()
    kv = binding.KVCache(shape, batch=4, capacity=16)
    q = torch.full((4, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    rope = binding.Rope(binding.rope_table(10, 128))
    # past the table; before it; a slot past the cache with a good position; all good
    m.op_rope_norm_append(x, _i32([1, 2, 16, 3]), 0, kv, q, rope=rope, positions=_i32([10, -1, 9, 0]))
    rc, flags = m.sync_status()
    assert rc == 5 and flags == binding.FLAG_POS_RANGE
    assert torch.all(q[:2] == 0) and torch.all(q[2:].abs().sum(-1) > 0)
    assert (kv.k != 0).any(-1).nonzero().tolist() == [[0, 3, 0, 3], [0, 3, 1, 3]]
    # without rotation positions do not count
    m.op_rope_norm_append(x, _i32([1, 2, 5, 3]), 0, kv, q, positions=_i32([-1, 1 << 30, 0, 0]))
    m.sync()
    assert torch.all(q.abs().sum(-1) > 0)


# --------------------------------------------------------------------------- key weights
def _slopes(nq):
    return torch.exp2(-8.0 * torch.arange(1, nq + 1).float() / nq)


def _randn(shape, dtype, seed, std=1.0):
    return (torch.randn(*shape, generator=_gen(seed)) * std).to(dtype)


def _filled(shape, B, slots, page, dtype, seed, std=1.5, read=None):
    """A random cache of layer 0 .. n_layers - 1; slots that `read` [B] does not cover hold NaN and infinities."""
    L, nkv, d = shape.n_layers, shape.n_kv_heads, shape.head_dim
    if page:
        n = -(-slots // page)
        pt = torch.randperm(B * n + 2, generator=_gen(seed))[:B * n].view(B, n).to(torch.int32)
        size = (L, B * n + 2, nkv, page, d)
    else:
        pt, size = None, (L, B, nkv, slots, d)
    k, v = _randn(size, dtype, seed + 1, std), _randn(size, dtype, seed + 2)
    if read is not None:
        used = torch.zeros(size[1], size[3], dtype=torch.bool)
        for b, n in enumerate(read):
            j = torch.arange(n)
            if page:
                used[pt[b].long()[j // page], j % page] = True
            else:
                used[b, :n] = True
        k.transpose(2, 3)[:, ~used] = float("nan")
        v.transpose(2, 3)[:, ~used] = torch.tensor(float("inf"))
    kw = dict(n_pages=size[1], page_size=page, page_table=pt.cuda()) if page else dict(batch=B, capacity=slots)
    kv = binding.KVCache(shape, k=k.cuda(), v=v.cuda(), **kw)
    return kv, k, v, pt


def _keys_of(t, pt, page, layer, b, n):
    """Rows 0 .. n - 1 of a sequence in fp64, [n_kv, n, d]."""
    j = torch.arange(n)
    if page:
        return f64(t[layer][pt[b].long()[j // page], :, j % page]).transpose(1, 0, 2)
    return f64(t[layer, b, :, :n])


def _score_error(q, K, scale, cap, bias_n):
    """What a score may be off by: fp32 sums of d products, each addition of which may cut
    (2^-23), and a few roundings of the scaled, capped and biased value."""
    d = q.shape[-1]
    S = float((np.abs(q) @ np.abs(K).T).max()) * scale
    return (d + 8) * 2.0 ** -23 * S + 16 * 2.0 ** -24 * (min(S, cap) if cap else S) + 16 * 2.0 ** -24 * (cap + bias_n)


def _out_bound(ref, mass, dtype, err, n):
    """An output's rounding, the weights' (bf16: one rounding to bf16 at most), the scores' on both
    a weight and the sum, and the sums' own."""
    eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    return eps * np.abs(ref) + mass * ((2.0 ** -8 if dtype == "bf16" else 0.0) + 2 * err + (n / 8 + 64) * 2.0 ** -24) + 1e-30


def _weights_case(nq, nkv, d, dtype, positions, *, page=16, cap=0.0, bias=False, scale=0.0, slots=None, ld=None, seed=31,
                  layers=1, layer=0, max_seq=None, calls=1, heads=None):
    B, top = len(positions), max(max(positions) + 1, 1)
    slots = slots or top
    ld = ld or top
    m, shape = _model(nq, nkv, d, dtype, max_batch=B, max_seq=max_seq or slots, n_layers=layers)
    dt = shape.torch_dtype
    kv, k, v, pt = _filled(shape, B, slots, page, dt, seed, read=[p + 1 for p in positions])
    q = _randn((B, nq, d), dt, seed + 5, 1.5)
    w0 = torch.rand(B, nkv, ld, generator=_gen(seed + 6))
    w, scratch = w0.cuda(), torch.full((B, nq, ld), float("nan"), device="cuda")
    out = torch.full((B, nq * d), 3.0, dtype=dt, device="cuda")
    sl = _slopes(nq) if bias else None
    sc = binding.Scores(scale, cap, None if sl is None else sl.cuda())
    for _ in range(calls):
        m.op_attention_decode_weights(q.cuda(), _i32(positions), layer, kv, out, w, scratch, scores=sc)
    m.sync()
    qf, got_w = f64(q), f64(w)
    sc = scale or 1 / math.sqrt(d)
    for b, p in enumerate(positions):
        n = p + 1
        K, V = _keys_of(k, pt, page, layer, b, n), _keys_of(v, pt, page, layer, b, n)
        where, all_keys = np.arange(n), np.ones(n, bool)
        for g in range(nkv):
            G = nq // nkv
            if heads is not None and g not in heads:
                continue
            add, tol = np.zeros(n), np.zeros(n)
            for h in range(g * G, g * G + G):
                e = _score_error(qf[b, h], K[g], sc, cap, n if bias else 0)
                pr = C.weigh(qf[b, h], K[g], p, where, all_keys, sc, cap, 0.0 if sl is None else float(sl[h]))
                add, tol = add + pr, tol + pr * (2 * e + (n / 8 + 64) * 2.0 ** -24)
                _within(out[b].view(nq, d)[h], pr @ V[g], _out_bound(pr @ V[g], pr @ np.abs(V[g]), dtype, e, n),
                        "out b=%d h=%d n=%d" % (b, h, n))
            want = f64(w0)[b, g].copy()
            want[:n] += calls * add
            bound = (G + calls) * 2.0 ** -24 * np.abs(want)
            bound[:n] += calls * tol + 1e-37
            bound[n:] = 0.0
            _within(got_w[b, g], want, bound, "weights b=%d g=%d n=%d" % (b, g, n))


OPTS = [dict(), dict(cap=30.0), dict(bias=True), dict(cap=20.0, bias=True, scale=0.11)]


@pytest.mark.parametrize("nq,nkv", [(4, 4), (8, 1), (6, 2), (16, 1), (12, 1), (5, 5)])
@pytest.mark.parametrize("opt", OPTS)
def test_weights_bf16(nq, nkv, opt):
    _weights_case(nq, nkv, 128, "bf16", [0, 14, 15, 16, 62, 63, 64, 300], **opt)


@pytest.mark.parametrize("page", [0, 16, 64, 80])
@pytest.mark.parametrize("slots,ld", [(700, 700), (5000, 5000), (700, 1000), (4000, 690)])
def test_weights_rooms(page, slots, ld):
    _weights_case(8, 2, 128, "bf16", [689, 3, 130], page=page, slots=slots, ld=ld)


@pytest.mark.parametrize("B,nq,nkv", [(1, 32, 32), (1, 8, 1), (40, 8, 1), (130, 2, 2)])
def test_weights_batches(B, nq, nkv):
    _weights_case(nq, nkv, 128, "bf16", [(37 * i + 5) % 290 for i in range(B)], heads=[0, nkv - 1])


def test_weights_long_splits():
    _weights_case(8, 1, 128, "bf16", [19999], page=64, cap=50.0)
    _weights_case(16, 1, 128, "bf16", [9000, 1], page=16, slots=30000)


def test_weights_more_splits_of_long_rows():
    # 320 pairs and 160: two to five splits each, of some rows one
    _weights_case(40, 40, 128, "bf16", [2999, 0, 511, 512, 1025, 2100, 64, -1 + 1024], slots=3000, heads=[0, 39])
    _weights_case(40, 40, 128, "bf16", [5999, 300, 4100, 65], page=64, cap=30.0, bias=True, heads=[0, 39])


def test_weights_add_up_over_calls_and_layers():
    _weights_case(4, 2, 128, "bf16", [70, 20], calls=3, layers=2, layer=1)


@pytest.mark.parametrize("nq,nkv,d", [(4, 2, 64), (2, 2, 40), (20, 1, 128), (40, 1, 64), (1, 1, 256), (3, 1, 8)])
@pytest.mark.parametrize("page", [0, 16, 5])
@pytest.mark.parametrize("opt", OPTS)
def test_weights_fp32(nq, nkv, d, page, opt):
    _weights_case(nq, nkv, d, "f32", [0, 15, 64, 300], page=page, **opt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_bad_positions_and_pages(dtype):
    m, shape = _model(4, 2, 128, dtype, max_batch=4, max_seq=64)
    kv, k, v, pt = _filled(shape, 4, 64, 16, shape.torch_dtype, 3)
    q = _randn((4, 4, 128), shape.torch_dtype, 4, 1.5).cuda()
    scratch = torch.empty(4, 4, 50, device="cuda")

    def call(positions):
        w, out = torch.ones(4, 2, 50, device="cuda"), torch.full((4, 512), 3.0, dtype=shape.torch_dtype, device="cuda")
        m.op_attention_decode_weights(q, _i32(positions), 0, kv, out, w, scratch)
        return m.sync_status(), w, out
    # no keys; past the weights' room; far past; in range
    (rc, flags), w, out = call([-1, 50, 2 ** 31 - 1, 49])
    assert rc == 5 and flags == binding.FLAG_POS_RANGE
    assert torch.all(out[0] == 0) and torch.all(w[0] == 1)
    (rc, _), w2, out2 = call([49, 49, 49, 49])
    assert rc == 0 and torch.equal(w[1:], w2[1:]) and torch.equal(out[1:], out2[1:])
    total = (w2 - 1).double().sum(-1)
    assert torch.all((total - 2).abs() < 1e-4)  # each of the two heads' weights add up to one
    kv.page_table[2, 1] = 77
    (rc, flags), w3, _ = call([49, 49, 49, 49])
    assert rc == 5 and flags == binding.FLAG_PAGE_RANGE and torch.isfinite(w3).all()
    kv.page_table = pt.cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("slots", [100, 4000])
def test_weights_nan_stays_in_its_heads(dtype, slots):
    m, shape = _model(4, 2, 128, dtype, max_batch=2, max_seq=slots)
    kv, k, v, pt = _filled(shape, 2, slots, 16, shape.torch_dtype, 5)
    kv.k[0, int(pt[0, 4]), 1, 3] = float("nan")  # key 67 of sequence 0, K/V head 1
    q = _randn((2, 4, 128), shape.torch_dtype, 6, 1.5).cuda()
    q[1, 0, 5] = float("nan")  # head 0 of sequence 1: K/V head 0
    w, out = torch.zeros(2, 2, slots, device="cuda"), torch.empty(2, 512, dtype=shape.torch_dtype, device="cuda")
    m.op_attention_decode_weights(q, _i32([90, 80]), 0, kv, out, w, torch.empty(2, 4, slots, device="cuda"))
    m.sync()
    bad = torch.isnan(w)
    assert bad[0, 1, :91].all() and not bad[0, 1, 91:].any() and not bad[0, 0].any()
    assert bad[1, 0, :81].all() and not bad[1, 0, 81:].any() and not bad[1, 1].any()
    bad = torch.isnan(out.view(2, 4, 128))
    assert bad[0, 2:].all() and not bad[0, :2].any() and bad[1, 0].all() and not bad[1, 1:].any()


def test_weights_give_the_plain_decode_output():
    m, shape = _model(8, 2, max_batch=3, max_seq=700)
    kv, *_ = _filled(shape, 3, 700, 16, torch.bfloat16, 7)
    q, pos = _randn((3, 8, 128), torch.bfloat16, 8, 1.5).cuda(), _i32([699, 5, 320])
    outs = [torch.empty(3, 1024, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    m.op_attention_decode_shared(q, pos, 0, kv, outs[0])
    m.op_attention_decode_weights(q, pos, 0, kv, outs[1], torch.zeros(3, 2, 700, device="cuda"),
                                  torch.empty(3, 8, 700, device="cuda"))
    m.sync()
    # the same sums merged in another order: a rounding apart
    assert torch.all((outs[0].float() - outs[1].float()).abs() <= 2.0 ** -7 * outs[0].float().abs() + 2.0 ** -18)


# --------------------------------------------------------------------------- trees
def _random_tree(n, seed):
    r = np.random.RandomState(seed)
    return [-1] + [int(r.randint(max(0, i - 6), i)) for i in range(1, n)]


def _tree_case(nq, nkv, d, dtype, starts, rows, *, page=16, cap=0.0, bias=False, scale=0.0, slopes=None, mask="tree",
               words=None, lead=0, tail=0, layers=1, layer=0, seed=51, std=1.5, heads=None, slots=None, positions=True,
               check=None, calls=1):
    """mask: "tree" (random parents), "chain" (none given), or "any" (random bits, some rows without any)."""
    B, n = len(starts), lead + sum(rows) + tail
    top = max(1, max(s + r for s, r in zip(starts, rows)))
    slots = slots or top
    m, shape = _model(nq, nkv, d, dtype, max_batch=B, max_seq=16, n_layers=layers)
    dt = shape.torch_dtype
    kv, k, v, pt = _filled(shape, B, slots, page, dt, seed, std, read=[s + r for s, r in zip(starts, rows)])
    q = _randn((n, nq, d), dt, seed + 5, std)
    cu = [lead]
    for r in rows:
        cu.append(cu[-1] + r)
    words = words or max(1, -(-max(rows) // 32))
    bits = np.full((n, words), -1, np.int32)  # rows of nobody: every bit
    sees, at = [], torch.randint(0, 9, (n,), generator=_gen(seed + 7)).tolist()
    r = np.random.RandomState(seed)
    for b, (s, c) in enumerate(zip(starts, rows)):
        if mask == "any":
            see = r.rand(c, c) < 0.4
            see[r.rand(c) < 0.3] = False
        else:
            parents = _random_tree(c, seed + b) if mask == "tree" else list(range(-1, c - 1))
            see = C.tree_visible(parents)
            for i in range(c):
                at[cu[b] + i] = at[cu[b] + parents[i]] + 1 if parents[i] >= 0 else s
        if c and mask != "chain":
            wide = np.concatenate((see, r.rand(c, max(0, 32 * words - c)) < 0.5), 1)  # bits past the rows: anything
            bits[cu[b]:cu[b] + c] = C.mask_words(wide, words)
            see[:, 32 * words:] = False
        sees.append(see)
    sl = torch.tensor(slopes) if slopes is not None else _slopes(nq) if bias else None
    out = torch.full((n, nq * d), 3.0, dtype=dt, device="cuda")
    args = (q.cuda(), _i32(cu), _i32(starts), layer, kv, out)
    kw = dict(mask=None if mask == "chain" else torch.from_numpy(bits).cuda(), positions=_i32(at) if positions else None,
              scores=binding.Scores(scale, cap, None if sl is None else sl.cuda()))
    for _ in range(calls):
        m.op_attention_tree(*args, **kw)
    m.sync()
    qf, got = f64(q), f64(out).reshape(n, nq, d)
    sc = scale or 1 / math.sqrt(d)
    for b, (s, c) in enumerate(zip(starts, rows)):
        K, V = _keys_of(k, pt, page, layer, b, s + c), _keys_of(v, pt, page, layer, b, s + c)
        lo = cu[b]
        pos = np.array(at[lo:lo + c]) if positions else s + np.arange(c)
        where = np.concatenate((np.arange(s), pos))
        for i in range(c) if check is None else [x for x in check if x < c]:
            keep = np.concatenate((np.ones(s, bool), sees[b][i]))
            for h in range(nq) if heads is None else heads:
                g, slope = h // (nq // nkv), 0.0 if sl is None else float(sl[h])
                far = float(np.abs(slope) * np.abs(pos[i] - where).max()) if sl is not None else 0.0
                e = _score_error(qf[lo + i, h], K[g], sc, cap, far)
                ref, mass = C.attend(qf[lo + i, h], K[g], V[g], pos[i], where, keep, sc, cap, slope)
                _within(got[lo + i, h], ref, _out_bound(ref, mass, dtype, e, s + c),
                        "tree b=%d row=%d head=%d start=%d rows=%d" % (b, i, h, s, c))
    outside = list(range(lead)) + list(range(cu[-1], n))
    assert np.all(got[outside] == 3.0)
    return got


@pytest.mark.parametrize("nq,nkv", [(4, 4), (8, 1), (6, 2), (5, 5), (16, 1), (12, 1)])
@pytest.mark.parametrize("opt", OPTS)
@pytest.mark.parametrize("mask", ["tree", "any"])
def test_tree_bf16(nq, nkv, opt, mask):
    _tree_case(nq, nkv, 128, "bf16", [130, 0, 0, 57, 255], [9, 5, 0, 1, 12], mask=mask, lead=2, tail=3, **opt)


@pytest.mark.parametrize("n", [1, 2, 15, 31, 32, 33, 63, 64, 65, 127, 128, 129, 130, 200, 300])
@pytest.mark.parametrize("start", [0, 1, 100, 128, 250])
def test_tree_rows_and_starts(n, start):
    _tree_case(2, 1, 128, "bf16", [start], [n], mask="any", check=[0, 1, 14, 31, 32, 62, 64, 100, 127, 128, 199, 257, 299])


@pytest.mark.parametrize("nq,nkv", [(2, 1), (8, 1)])
@pytest.mark.parametrize("mask", ["tree", "chain"])
def test_tree_mixed_batches(nq, nkv, mask):
    # some sequences fill several blocks of rows, some one row; both row-tile forms
    rows = [1, 130, 3, 0, 64, 17, 40]
    _tree_case(nq, nkv, 128, "bf16", [200, 5, 0, 90, 300, 128, 127], rows, mask=mask, check=[0, 2, 16, 39, 63, 64, 129])
    _tree_case(nq, nkv, 128, "bf16", [200, 5, 0, 90, 300, 128, 127], [1, 13, 3, 0, 6, 17, 4], mask=mask)


@pytest.mark.parametrize("page", [0, 16, 64, 80])
@pytest.mark.parametrize("slots", [None, 2000])
def test_tree_caches(page, slots):
    _tree_case(4, 2, 128, "bf16", [70, 500], [10, 7], page=page, slots=slots, layers=2, layer=1)


@pytest.mark.parametrize("nq,nkv,starts,rows", [
    (8, 1, [9000], [20]), (8, 8, [5000], [40]), (2, 2, [20000], [129]), (64, 8, [3000], [64]), (32, 32, [1000, 4000], [9, 5])])
def test_tree_shared_chunks(nq, nkv, starts, rows):
    # few items: their keys are cut over many CTAs and joined
    _tree_case(nq, nkv, 128, "bf16", starts, rows, page=64, check=[0, 4, 8, 19, 63, 128], heads=[0, nq // 2, nq - 1])


@pytest.mark.parametrize("B", [33, 90, 200])
def test_tree_many_sequences(B):
    r = np.random.RandomState(B)
    _tree_case(2, 1, 128, "bf16", r.randint(0, 400, B).tolist(), r.randint(0, 8, B).tolist(), check=[0, 5])


def test_tree_many_items_per_cta():
    # more items than SMs, of odd tile counts: chunks begin and end anywhere
    r = np.random.RandomState(3)
    _tree_case(16, 16, 128, "bf16", r.randint(0, 700, 30).tolist(), [6] * 30, check=[0, 5], heads=[0, 7, 15])
    _tree_case(16, 16, 128, "bf16", r.randint(0, 700, 20).tolist(), [150] * 20, check=[0, 149], heads=[0, 7, 15])


@pytest.mark.parametrize("rows", [9, 140])
def test_tree_long_items_per_cta(rows):
    # a CTA walks several items of many tiles, odd and even counts, and calls follow at once
    r = np.random.RandomState(rows)
    _tree_case(32, 32, 128, "bf16", r.randint(1, 4000, 12).tolist(), r.randint(1, rows + 1, 12).tolist(), check=[0, 5, 131],
               heads=[0, 13, 31], calls=6)


@pytest.mark.parametrize("nq,nkv", [(8, 1), (4, 4), (6, 2), (5, 1), (5, 5)])
@pytest.mark.parametrize("slots", [600, 3000, 20000])
@pytest.mark.parametrize("opt", OPTS)
def test_tree_few_rows(nq, nkv, slots, opt):
    # blocks of 8 (row, head) pairs, one, two and more per sequence; with room, and without keys
    _tree_case(nq, nkv, 128, "bf16", [300, 0, 17, 511, 130], [1, 2, 0, 3, 1], mask="any", slots=slots, lead=1, tail=1, **opt)


@pytest.mark.parametrize("B,rows", [(1, 1), (1, 8), (40, 2), (100, 8), (3, 13)])
@pytest.mark.parametrize("page", [0, 16, 64])
def test_tree_few_rows_batches(B, rows, page):
    r = np.random.RandomState(B + rows)
    _tree_case(2, 2, 128, "bf16", r.randint(0, 900, B).tolist(), r.randint(1, rows + 1, B).tolist(), page=page,
               check=[0, 1, 7, 12], calls=3)
    _tree_case(4, 1, 128, "bf16", r.randint(0, 900, B).tolist(), r.randint(0, rows + 1, B).tolist(), page=page, cap=20.0,
               bias=True, check=[0, 1, 7, 12])


@pytest.mark.parametrize("nq,nkv,starts,rows", [
    (64, 8, [700], [16]), (64, 8, [30, 0, 200, 61], [8, 3, 10, 9]), (16, 16, [800], [26]), (32, 8, [70, 150], [26, 31]),
    (16, 1, [700, 20, 0], [5, 9, 1]), (12, 1, [60, 0, 333], [1, 2, 1]), (18, 2, [100, 0, 33, 90], [2, 1, 3, 0]),
    (32, 2, [260, 1500], [1, 1]), (16, 1, [90] * 140, [1] * 140), (32, 32, [3, 0, 20, 7, 11, 2], [17, 20, 3, 24, 17, 17]), (8, 1, [500], [40]), (10, 5, [333, 2, 400], [30, 1, 12]), (64, 8, [5000, 3, 4100, 64, 900, 1, 0, 2500], [1] * 8)])
@pytest.mark.parametrize("opt", [OPTS[0], OPTS[3]])
def test_tree_several_blocks(nq, nkv, starts, rows, opt):
    # blocks of 8 (row, head) pairs enough to be resident at once, in clusters of up to 8 CTAs
    _tree_case(nq, nkv, 128, "bf16", starts, rows, mask="any", check=[0, 1, 7, 8, 15, 25, 39], heads=[0, nq // 2 - 1, nq - 1],
               lead=1, tail=1, **opt)


@pytest.mark.parametrize("opt", OPTS)
def test_tree_few_rows_cut_in_two(opt):
    # enough CTAs already, with keys for two each in some sequences
    _tree_case(40, 40, 128, "bf16", [1980, 0, 499, 505, 1020], [13, 13, 13, 8, 0], slots=2000, page=0, mask="any",
               check=[0, 7, 8, 12], heads=[0, 17, 39], calls=2, **opt)


@pytest.mark.parametrize("words", [1, 2, 7])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_mask_widths(words, dtype):
    # words that do not reach all rows hide them; words past the rows count for nothing
    _tree_case(2, 1, 128, dtype, [60, 3], [70, 20], mask="any", words=words)


@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("slopes", [[4.0, 0.01], [-0.5, 3.0], [0.0, 100.0]])
@pytest.mark.parametrize("positions", [True, False])
def test_tree_slopes(cap, slopes, positions):
    _tree_case(2, 1, 128, "bf16", [300, 40], [20, 9], cap=cap, slopes=slopes, positions=positions)


@pytest.mark.parametrize("cap,scale", [(50.0, 0.0), (50.3, 0.0), (2.0, 0.5), (0.05, 1.0), (2000.0, 0.0), (300.0, 4.0)])
def test_tree_caps(cap, scale):
    _tree_case(4, 2, 128, "bf16", [200], [30], cap=cap, scale=scale, check=[0, 13, 29])


def test_tree_large_scores():
    _tree_case(2, 1, 128, "bf16", [260], [30], std=12.0, check=[0, 11, 29])


@pytest.mark.parametrize("nq,nkv,d", [(4, 2, 64), (2, 2, 40), (20, 1, 128), (1, 1, 256), (3, 1, 8)])
@pytest.mark.parametrize("opt", OPTS)
@pytest.mark.parametrize("mask", ["tree", "any", "chain"])
def test_tree_fp32(nq, nkv, d, opt, mask):
    _tree_case(nq, nkv, d, "f32", [130, 0, 7, 64], [9, 40, 0, 1], mask=mask, page=5, lead=1, tail=2, **opt)


def test_tree_fp32_shared_keys():
    _tree_case(2, 1, 64, "f32", [3000], [40], page=0, check=[0, 39])


def test_tree_output_aligned_to_16_bytes_only():
    m, shape = _model(4, 2, max_batch=1)
    kv, *_ = _filled(shape, 1, 300, 16, torch.bfloat16, 9)
    for n in (2, 40):
        q = _randn((n, 4, 128), torch.bfloat16, 10).cuda()
        outs = [torch.empty(n * 512 + 8, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        for o, off in zip(outs, (0, 8)):
            m.op_attention_tree(q, _i32([0, n]), _i32([250]), 0, kv, o[off:off + n * 512])
        m.sync()
        assert torch.equal(outs[0][:n * 512], outs[1][8:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("opt", OPTS)
@pytest.mark.parametrize("slots", [1000, 200, 9000])
def test_tree_nan_reaches_the_rows_that_see_it(dtype, opt, slots):
    start = min(slots - 20, 980)
    m, shape = _model(4, 2, 128, dtype, max_batch=2)
    kv, k, v, pt = _filled(shape, 2, slots, 16, shape.torch_dtype, 12)
    parents = _random_tree(20, 4)
    see = C.tree_visible(parents)

    def poison(t, b, slot, g):
        t[0, int(pt[b, slot // 16]), g, slot % 16] = float("nan")
    poison(kv.k, 0, start + 7, 1)    # a tree row's K: the rows that see it, heads of K/V head 1
    poison(kv.k, 1, start // 2, 0)   # a cached key: every row of sequence 1, heads of K/V head 0
    q = _randn((40, 4, 128), shape.torch_dtype, 13).cuda()
    q[3, 0, 1] = float("nan")        # one query row and head
    out = torch.empty(40, 512, dtype=shape.torch_dtype, device="cuda")
    sl = _slopes(4).cuda() if opt.get("bias") else None
    bits = torch.from_numpy(np.concatenate((C.mask_words(see), C.mask_words(see)))).cuda()
    m.op_attention_tree(q, _i32([0, 20, 40]), _i32([start, start]), 0, kv, out, mask=bits,
                        scores=binding.Scores(opt.get("scale", 0.0), opt.get("cap", 0.0), sl))
    m.sync()
    bad = torch.isnan(out.view(40, 4, 128)).cpu().numpy()
    want = np.zeros((40, 4), bool)
    want[:20, 2:] = see[:, 7:8]
    want[20:, :2] = True
    want[3, 0] = True
    assert np.array_equal(bad.all(-1), want) and np.array_equal(bad.any(-1), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_bad_bounds_are_flagged(dtype):
    m, shape = _model(4, 2, 128, dtype, max_batch=4)
    dt = shape.torch_dtype
    kv, k, v, pt = _filled(shape, 4, 64, 16, dt, 21)
    q = _randn((12, 4, 128), dt, 22).cuda()

    def call(cu, starts):
        out = torch.full((12, 512), 3.0, dtype=dt, device="cuda")
        m.op_attention_tree(q, _i32(cu), _i32(starts), 0, kv, out)
        return m.sync_status(), out
    (rc, flags), base = call([0, 3, 6, 9, 12], [10, 20, 30, 40])
    assert rc == 0
    # a negative start: zeros; past the cache: what is in it is attended; far past
    (rc, flags), out = call([0, 3, 6, 9, 12], [-1, 62, 2 ** 31 - 2, 40])
    assert rc == 5 and flags == binding.FLAG_POS_RANGE
    assert torch.all(out[:3] == 0) and torch.equal(out[9:], base[9:])
    (_, _), all64 = call([0, 3, 6, 9, 12], [61, 61, 61, 61])
    assert torch.isfinite(out.float()).all()
    # sequence 2's rows, whose own slots are past the cache, attend all 64 cached slots: as row 8, the last, does there
    assert torch.allclose(out[8].float(), all64[8].float(), rtol=2.0 ** -6, atol=1e-3)
    # rows out of range, and decreasing
    (rc, flags), out = call([0, 3, 6, 9, 40], [10, 20, 30, 40])
    assert rc == 5 and flags == binding.FLAG_POS_RANGE and torch.equal(out, base)
    (rc, flags), out = call([0, 3, 2, 9, 12], [10, 20, 30, 40])  # (row 2 is sequence 0's and 2's)
    assert rc == 5 and flags == binding.FLAG_POS_RANGE and torch.equal(out[:2], base[:2]) and torch.equal(out[9:], base[9:])
    kv.page_table[1, 0] = 99
    (rc, flags), out = call([0, 3, 6, 9, 12], [10, 20, 30, 40])
    assert rc == 5 and flags == binding.FLAG_PAGE_RANGE
    assert torch.equal(out[:3], base[:3]) and torch.equal(out[6:], base[6:]) and torch.isfinite(out.float()).all()


# --------------------------------------------------------------------------- together, as they are used
def _place(kv, pt, layer, b, rows, values):
    """Puts values [n, n_kv, d] at slots `rows` of sequence b, for K and V."""
    for t, x in zip((kv.k, kv.v), values):
        if pt is None:
            t[layer, b, :, rows] = x.transpose(0, 1)
        else:
            t[layer, pt[b].long()[rows // kv.page_size].cuda(), :, (rows % kv.page_size).cuda()] = x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_verified_drafts_run(dtype):
    """Two sequences, two layers: prompts are cached, then three times a tree is drafted, appended
    at its depths' positions, attended, and its accepted path kept. The cache then is the one
    that plain appends of the accepted tokens give, to the bit, and each accepted row's output
    is its attention over that cache."""
    nq, nkv, d, layers, page = 4, 2, 128, 2, 16
    m, shape = _model(nq, nkv, d, dtype, max_batch=2, max_seq=256, n_layers=layers)
    dt = shape.torch_dtype
    pt = torch.randperm(20, generator=_gen(1)).view(2, 10).to(torch.int32)
    kv, plain = (binding.KVCache(shape, n_pages=20, page_size=page, page_table=pt.cuda()) for _ in range(2))
    rope = binding.Rope(None, binding.ROPE_HALF, d)
    kw = dict(rope=rope, k_gain=(1 + 0.1 * torch.randn(d, generator=_gen(2))).to(dt).cuda())
    slopes = _slopes(nq)
    scores = binding.Scores(cap=25.0, slopes=slopes.cuda())
    lens = [19, 33]
    cu = _i32([0, lens[0], sum(lens)])
    q = torch.empty(sum(lens), nq * d, dtype=dt, device="cuda")
    for l in range(layers):
        x = _randn((sum(lens), shape.qkv_rows), torch.float32, 300 + l).cuda()
        for c in (kv, plain):
            m.op_rope_norm_append(x, _i32([0, 0]), l, c, q, cu_rows=cu, **kw)
    for step in range(3):
        rows = [12, 7 + step]
        n = sum(rows)
        parents = [_random_tree(r, 60 + 2 * step + b) for b, r in enumerate(rows)]
        see = [C.tree_visible(p) for p in parents]
        pos, paths = [], []
        for b in range(2):
            pos += [lens[b] + int(see[b][i].sum()) - 1 for i in range(rows[b])]
            leaf = rows[b] - 1 - step * b
            paths.append([j for j in range(rows[b]) if see[b][leaf, j]])
        mask = torch.from_numpy(np.concatenate([C.mask_words(s) for s in see])).cuda()
        cu, start, at = _i32([0, rows[0], n]), _i32(lens), _i32(pos)
        outs, qs = [], []
        for l in range(layers):
            x = _randn((n, shape.qkv_rows), torch.float32, 320 + 2 * step + l).cuda()
            q, o = (torch.empty(n, nq * d, dtype=dt, device="cuda") for _ in range(2))
            m.op_rope_norm_append(x, start, l, kv, q, cu_rows=cu, positions=at, **kw)
            m.op_attention_tree(q, cu, start, l, kv, o, mask=mask, positions=at, scores=scores)
            outs.append(o)
            qs.append(q)
            keep = [p for p in paths[0]] + [rows[0] + p for p in paths[1]]
            q2 = torch.empty(len(keep), nq * d, dtype=dt, device="cuda")
            m.op_rope_norm_append(x[keep].contiguous(), start, l, plain, q2,
                                  cu_rows=_i32([0, len(paths[0]), len(keep)]), **kw)
            m.sync()
            assert torch.equal(q[keep], q2)
        width = max(map(len, paths))
        m.op_cache_commit(kv, start, _i32([p + [0] * (width - len(p)) for p in paths]), _i32([len(p) for p in paths]))
        m.sync()
        for b in range(2):
            lens[b] += len(paths[b])
            for l in range(layers):
                K, V = (_keys_of(t.cpu(), pt, page, l, b, lens[b]) for t in (plain.k, plain.v))
                for got, want in zip((kv.k, kv.v), (K, V)):
                    assert np.array_equal(_keys_of(got.cpu(), pt, page, l, b, lens[b]), want)
                for i, row in enumerate(paths[b]):
                    seen = lens[b] - len(paths[b]) + i + 1
                    r = row + (rows[0] if b else 0)
                    for h in range(nq):
                        g, qf = h // 2, f64(qs[l])[r].reshape(nq, d)[h]
                        ref, mass = C.attend(qf, K[g][:seen], V[g][:seen], seen - 1, np.arange(seen), np.ones(seen, bool),
                                             1 / math.sqrt(d), 25.0, float(slopes[h]))
                        e = _score_error(qf, K[g], 1 / math.sqrt(d), 25.0, seen)
                        _within(outs[l][r].view(nq, d)[h], ref, _out_bound(ref, mass, dtype, e, seen),
                                "step %d layer %d sequence %d row %d head %d" % (step, l, b, row, h))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bounded_cache_run(dtype):
    """Two sequences, two layers: tokens are appended behind the kept keys at their own positions,
    weigh the keys they attend, and whenever a cache is full its lightest keys are dropped.
    Every head's keys, their weights and the outputs are those of lists kept in fp64."""
    nq, nkv, d, layers, page, top, keep, first, recent = 4, 2, 128, 2, 16, 44, 24, 3, 6
    m, shape = _model(nq, nkv, d, dtype, max_batch=2, max_seq=256, n_layers=layers)
    dt = shape.torch_dtype
    pt = torch.randperm(6, generator=_gen(4)).view(2, 3).to(torch.int32)
    kv = binding.KVCache(shape, n_pages=6, page_size=page, page_table=pt.cuda())
    rope = binding.Rope(None, binding.ROPE_ADJACENT, d)
    w = torch.zeros(layers, 2, nkv, 48, device="cuda")
    scratch = torch.empty(2, nq, 48, device="cuda")
    kept = torch.empty(layers, 2, nkv, keep, dtype=torch.int32, device="cuda")
    # what is in the cache: [layer][sequence][head] of keys, values, weights and what those may be off by
    have = [[[dict(k=[], v=[], w=[], e=[]) for _ in range(nkv)] for _ in range(2)] for _ in range(layers)]
    token, lens, evictions = [0, 7], [0, 0], 0
    q, o = (torch.empty(2, nq * d, dtype=dt, device="cuda") for _ in range(2))
    k, v = (torch.empty(2, nkv * d, dtype=dt, device="cuda") for _ in range(2))
    for step in range(top + 2 * (top - keep) + 3):
        for l in range(layers):
            x = _randn((2, shape.qkv_rows), torch.float32, 400 + 2 * step + l, 1.3).cuda()
            m.op_rope_norm_append(x, _i32(lens), l, kv, q, rope=rope, positions=_i32(token), k_out=k, v_out=v)
            m.op_attention_decode_weights(q, _i32(lens), l, kv, o, w[l], scratch)
            m.sync()
            for b in range(2):
                for g in range(nkv):
                    H = have[l][b][g]
                    H["k"].append(f64(k)[b].reshape(nkv, d)[g])
                    H["v"].append(f64(v)[b].reshape(nkv, d)[g])
                    H["w"].append(0.0)
                    H["e"].append(0.0)
                    K, V, n = np.stack(H["k"]), np.stack(H["v"]), len(H["k"])
                    for h in (2 * g, 2 * g + 1):
                        qf = f64(q)[b].reshape(nq, d)[h]
                        p = C.weigh(qf, K, 0, np.arange(n), np.ones(n, bool), 1 / math.sqrt(d))
                        e = _score_error(qf, K, 1 / math.sqrt(d), 0.0, 0)
                        _within(o[b].view(nq, d)[h], p @ V, _out_bound(p @ V, p @ np.abs(V), dtype, e, n),
                                "step %d layer %d sequence %d head %d" % (step, l, b, h))
                        for j in range(n):
                            H["w"][j] += p[j]
                            # its error and, of the sum so far, a rounding
                            H["e"][j] += p[j] * (2 * e + (n / 8 + 64) * 2.0 ** -24) + 2 * 2.0 ** -24 * H["w"][j]
        lens = [n + 1 for n in lens]
        token = [t + 1 for t in token]
        got = f64(w)
        for l in range(layers):
            for b in range(2):
                for g in range(nkv):
                    H = have[l][b][g]
                    _within(got[l, b, g, :lens[b]], np.array(H["w"]), np.array(H["e"]) + 1e-37, "weights")
                    assert np.all(got[l, b, g, lens[b]:] == 0)
        if lens[0] == top:
            evictions += 1
            m.op_cache_evict(kv, _i32(lens), keep, w, kept, first=first, recent=recent)
            m.sync()
            for l in range(layers):
                for b in range(2):
                    for g in range(nkv):
                        stay = C.evict(got[l, b, g, :top], keep, first, recent)
                        assert kept[l, b, g].tolist() == stay
                        H = have[l][b][g]
                        for name in H:
                            H[name] = [H[name][i] for i in stay]
            lens = [keep] * 2
    assert evictions == 3


# --------------------------------------------------------------------------- streams, graphs, sizes
class _Step:
    """All five calls on buffers of their own; tree rows enough for the tensor-core kernel, and few."""

    def __init__(self, nq=8, nkv=2, seed=0, stream=None, B=2):
        self.m, shape = _model(nq, nkv, max_batch=B, max_seq=1024)
        self.kv, *_ = _filled(shape, B, 1024, 16, torch.bfloat16, 500 + seed)
        self.first = [self.kv.k.clone(), self.kv.v.clone()]
        self.rows = [40, 23]
        n = sum(self.rows)
        self.x = torch.empty(n, shape.qkv_rows, device="cuda")
        self.cu, self.start = _i32([0, 40, 63]), _i32([700, 300])
        self.one, self.few = _i32([0, 1, 3]), _randn((3, nq, 128), torch.bfloat16, 520 + seed).cuda()
        self.at = _i32([0] * n)
        self.mask = torch.empty(n, 2, dtype=torch.int32, device="cuda")
        self.path, self.path_len = _i32([[0] * 8] * 2), _i32([0, 0])
        self.lens = _i32([0, 0])
        self.w = torch.zeros(1, B, nkv, 1024, device="cuda")
        self.scratch = torch.empty(B, nq, 1024, device="cuda")
        self.rope = binding.Rope(None, binding.ROPE_HALF, 128)
        self.seed = seed
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.q, self.o, self.o2 = torch.empty(n, nq * 128, **bf), torch.empty(n, nq * 128, **bf), torch.empty(3, nq * 128, **bf)
        self.o3, self.kept = torch.empty(B, nq * 128, **bf), torch.empty(1, B, nkv, 200, dtype=torch.int32, device="cuda")
        if stream is not None:
            torch.cuda.synchronize()
            self.m.set_stream(stream)

    def inputs(self, i):
        r = np.random.RandomState(31 * i + self.seed)
        self.kv.k.copy_(self.first[0])
        self.kv.v.copy_(self.first[1])
        self.x.copy_(_randn(self.x.shape, torch.float32, 540 + i + self.seed))
        self.start.copy_(_i32(r.randint(250, 900, 2).tolist()))
        self.at.copy_(_i32(r.randint(0, 500, 63).tolist()))
        self.mask.copy_(torch.from_numpy(np.concatenate([C.mask_words(C.tree_visible(_random_tree(n, i)), 2) for n in self.rows])))
        paths = [sorted(r.choice(n, 8, replace=False).tolist()) for n in self.rows]
        self.path.copy_(_i32(paths))
        self.path_len.copy_(_i32([int(r.randint(0, 9)), 8]))
        self.lens.copy_(self.start + self.path_len)
        self.w.copy_(torch.rand(self.w.shape, generator=_gen(i)))

    def run(self):
        m, kv = self.m, self.kv
        m.op_rope_norm_append(self.x, self.start, 0, kv, self.q, cu_rows=self.cu, positions=self.at, rope=self.rope)
        m.op_attention_tree(self.q, self.cu, self.start, 0, kv, self.o, mask=self.mask, scores=binding.Scores(cap=30.0))
        m.op_attention_tree(self.few, self.one, self.start, 0, kv, self.o2)
        m.op_cache_commit(kv, self.start, self.path, self.path_len)
        m.op_attention_decode_weights(self.q[:2], self.start, 0, kv, self.o3, self.w, self.scratch)
        m.op_cache_evict(kv, self.lens, 200, self.w, self.kept, first=4, recent=20)

    def results(self):
        # (slots behind the kept ones hold anything: all of them are compared here, since the moves are the same)
        return [t.clone() for t in (self.q, self.o, self.o2, self.o3, self.w, self.kept, self.kv.k.view(torch.int16),
                                    self.kv.v.view(torch.int16))]


def test_captured_replays_follow_their_buffers():
    s = torch.cuda.Stream()
    steps = [_Step(stream=s), _Step(nq=16, nkv=16, seed=1, stream=s)]
    graphs = []
    for st in steps:
        st.inputs(9)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            st.run()
        graphs.append(g)
    # and a second graph of the first context: both use its one workspace, in turn
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        steps[0].run()
    for st, pair in ((steps[0], (graphs[0], g)), (steps[1], (graphs[1],))):
        for i in range(4):
            st.inputs(i)
            torch.cuda.synchronize()
            st.run()
            st.m.sync()
            want = st.results()
            for graph in pair:
                st.inputs(i)
                torch.cuda.synchronize()
                with torch.cuda.stream(s):
                    graph.replay()
                torch.cuda.synchronize()
                for a, b in zip(st.results(), want):
                    assert torch.equal(a.nan_to_num() if a.is_floating_point() else a,
                                       b.nan_to_num() if b.is_floating_point() else b)
        st.m.sync()


def test_two_contexts_on_two_streams_at_once():
    steps = [_Step(seed=i, nq=nq, nkv=nkv, stream=torch.cuda.Stream()) for i, (nq, nkv) in enumerate(((8, 2), (4, 4)))]
    alone = []
    for st in steps:
        st.inputs(3)
        torch.cuda.synchronize()
        st.run()
        st.m.sync()
        alone.append(st.results())
    for _ in range(10):
        for st in steps:
            st.inputs(3)
        torch.cuda.synchronize()
        for st in steps:
            st.run()
        for st in steps:
            st.m.sync()
        for st, want in zip(steps, alone):
            for a, b in zip(st.results(), want):
                assert torch.equal(a.nan_to_num() if a.is_floating_point() else a,
                                   b.nan_to_num() if b.is_floating_point() else b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [0, 64])
def test_cache_offsets_past_32_bits(dtype, page):
    # the last slots of a cache of more than 2^31 values
    nq, nkv, d, cap, n, rows = 4, 2, 128, 1 << 17, 150, 9
    B = 2 if page else 66
    m, shape = _model(nq, nkv, d, dtype, max_batch=B, max_seq=256)
    dt = shape.torch_dtype
    if page:
        total = 66 * cap // page
        pt = torch.full((2, 4), -1, dtype=torch.int32)
        pt[1, :3] = torch.tensor([total - 3, total - 1, total - 2])
        kv = binding.KVCache(shape, n_pages=total, page_size=page, page_table=pt.cuda())
    else:
        pt, kv = None, binding.KVCache(shape, batch=B, capacity=cap)
    assert kv.k.numel() > 1 << 31
    last = B - 1
    K, V = (_randn((n, nkv, d), dt, 600 + i, 1.5) for i in range(2))

    def fill():
        _place(kv, pt, 0, last, torch.arange(n), (K.cuda(), V.cuda()))

    def there():
        j = torch.arange(n)
        if page:
            return [t[0, pt[last].long()[j // page].cuda(), :, (j % page).cuda()].cpu() for t in (kv.k, kv.v)]
        return [t[0, last, :, :n].transpose(0, 1).cpu() for t in (kv.k, kv.v)]
    fill()
    kf, vf = f64(K).transpose(1, 0, 2), f64(V).transpose(1, 0, 2)
    # a chain of rows, few and more
    for r in (1, rows, 60):
        q = _randn((r, nq, d), dt, 610, 1.5)
        out = torch.empty(r, nq * d, dtype=dt, device="cuda")
        m.op_attention_tree(q.cuda(), _i32([0] * B + [r]), _i32([0] * last + [n - r]), 0, kv, out)
        m.sync()
        for i in range(r):
            for h in range(nq):
                qf, c = f64(q)[i, h], n - r + i + 1
                ref, mass = C.attend(qf, kf[h // 2, :c], vf[h // 2, :c], 0, np.arange(c), np.ones(c, bool), 1 / math.sqrt(d))
                e = _score_error(qf, kf[h // 2], 1 / math.sqrt(d), 0, 0)
                _within(out[i].view(nq, d)[h], ref, _out_bound(ref, mass, dtype, e, n), "tree")
    q = torch.zeros(B, nq, d, dtype=dt)
    q[last] = _randn((nq, d), dt, 611, 1.5)
    w, scratch = torch.zeros(B, nkv, 160, device="cuda"), torch.empty(B, nq, 160, device="cuda")
    out = torch.empty(B, nq * d, dtype=dt, device="cuda")
    m.op_attention_decode_weights(q.cuda(), _i32([-1] * last + [n - 1]), 0, kv, out, w, scratch)
    rc, flags = m.sync_status()
    assert rc == 5 and flags == binding.FLAG_POS_RANGE and torch.all(w[:last] == 0)
    for g in range(nkv):
        want, tol = np.zeros(n), np.zeros(n)
        for h in (2 * g, 2 * g + 1):
            p = C.weigh(f64(q)[last, h], kf[g], 0, np.arange(n), np.ones(n, bool), 1 / math.sqrt(d))
            e = _score_error(f64(q)[last, h], kf[g], 1 / math.sqrt(d), 0, 0)
            want, tol = want + p, tol + p * (2 * e + (n / 8 + 64) * 2.0 ** -24)
            _within(out[last].view(nq, d)[h], p @ vf[g], _out_bound(p @ vf[g], p @ np.abs(vf[g]), dtype, e, n), "weights")
        _within(w[last, g, :n], want, tol + 4 * 2.0 ** -24 * want + 1e-37, "weights")
    path = sorted(np.random.RandomState(5).choice(100, 30, replace=False).tolist())
    m.op_cache_commit(kv, _i32([0] * last + [40]), _i32([[0] * 30] * last + [path]), _i32([0] * last + [30]))
    m.sync()
    for got, was in zip(there(), (K, V)):
        want = was.clone()
        want[40:70] = was[[40 + p for p in path]]
        assert torch.equal(got, want)
    fill()
    kept = torch.empty(1, B, nkv, 50, dtype=torch.int32, device="cuda")
    was_w = f64(w)
    m.op_cache_evict(kv, _i32([0] * last + [n]), 50, w.view(1, B, nkv, 160), kept, first=2, recent=10)
    m.sync()
    for g in range(nkv):
        stay = C.evict(was_w[last, g, :n], 50, 2, 10)
        assert kept[0, last, g].tolist() == stay
        for got, was in zip(there(), (K, V)):
            assert torch.equal(got[:50, g], was[stay, g])
    # a row appended at a far slot, at a position of its own
    x = torch.zeros(B, shape.qkv_rows, device="cuda")
    x[last] = _randn((shape.qkv_rows,), torch.float32, 612).cuda()
    rope = binding.Rope(None, binding.ROPE_HALF, d)
    outs = [torch.empty(B, nq * d, dtype=dt, device="cuda") for _ in range(2)]
    got = []
    for o, slot, at in zip(outs, (n - 1, 30), (_i32([0] * last + [30]), None)):
        m.op_rope_norm_append(x, _i32([-1] * last + [slot]), 0, kv, o, rope=rope, positions=at)
        assert m.sync_status() == (5, binding.FLAG_POS_RANGE)
        got.append([t[slot] for t in there()])
    assert torch.equal(outs[0], outs[1]) and all(torch.equal(a, b) for a, b in zip(*got))


def test_weight_offsets_past_32_bits():
    # the last head's weights lie more than 2^31 values from the first's
    m, shape = _model(2, 2, max_batch=2, max_seq=256)
    kv, k, v, pt = _filled(shape, 2, 150, 16, torch.bfloat16, 620)
    ld = (1 << 31) // 3 + 8
    q = _randn((2, 2, 128), torch.bfloat16, 621, 1.5).cuda()
    w, scratch = (torch.empty(2, 2, ld, device="cuda") for _ in range(2))
    small, out, ref = torch.zeros(2, 2, 150, device="cuda"), *(torch.empty(2, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w[:, :, :200] = 0
    pos = _i32([149, 140])
    m.op_attention_decode_weights(q, pos, 0, kv, out, w, scratch)
    m.op_attention_decode_weights(q, pos, 0, kv, ref, small, torch.empty(2, 2, 150, device="cuda"))
    m.sync()
    assert torch.equal(out, ref) and torch.equal(w[:, :, :150], small) and torch.all(w[:, :, 150:200] == 0)
    kept = torch.empty(1, 2, 2, 50, dtype=torch.int32, device="cuda")
    m.op_cache_evict(kv, pos + 1, 50, w.unsqueeze(0), kept, recent=10)
    m.sync()
    for b in range(2):
        for g in range(2):
            stay = C.evict(f64(small)[b, g, :150 - 9 * b], 50, 0, 10)
            assert kept[0, b, g].tolist() == stay
            assert torch.equal(w[b, g, :50], small[b, g, stay]) and not w[b, g, 50:].any()


def test_tree_searched_blocks():
    # so many sequences that a CTA looks its own up, some without rows
    r = np.random.RandomState(7)
    for nq, nkv, B in ((2, 2, 129), (8, 1, 300), (4, 2, 1100)):
        rows = r.randint(0, 8 if nq == 2 else 3, B).tolist()
        rows[-1], rows[0] = 2, 0
        _tree_case(nq, nkv, 128, "bf16", r.randint(0, 60, B).tolist(), rows, check=[0, 6], heads=[0, nq - 1], lead=3, tail=2)
    _tree_case(2, 2, 128, "bf16", [5] * 200, [0] * 150 + [70] + [0] * 49, check=[0, 8, 69])


# --------------------------------------------------------------------------- refusals
def test_refusals():
    m, shape = _model(4, 2, max_batch=2, max_seq=64)
    m32, s32 = _model(2, 1, 40, "f32", max_batch=2, max_seq=64)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    kv = binding.KVCache(shape, batch=2, capacity=64)
    fp8 = binding.KVCache(shape, batch=2, capacity=64, e4m3=(1.0, 1.0))
    q, out, cu, start = torch.zeros(2, 512, **bf), torch.zeros(2, 512, **bf), _i32([0, 1, 2]), _i32([3, 4])
    w, scratch = torch.zeros(1, 2, 2, 64, device="cuda"), torch.zeros(2, 4, 64, device="cuda")
    path, n = _i32([[0, 1]] * 2), _i32([1, 1])
    kept = torch.zeros(1, 2, 2, 8, dtype=torch.int32, device="cuda")
    good = {
        "tree": (m.op_attention_tree, dict(q=q, cu_rows=cu, start_pos=start, layer=0, kv=kv, out=out)),
        "weights": (m.op_attention_decode_weights, dict(q=q, positions=start, layer=0, kv=kv, out=out, weights=w[0], scratch=scratch)),
        "commit": (m.op_cache_commit, dict(kv=kv, start_pos=start, path=path, path_len=n)),
        "evict": (m.op_cache_evict, dict(kv=kv, lens=start, keep=8, weights=w, kept=kept)),
    }

    def refused(rc, name, **kw):
        fn, base = good[name]
        if rc is None:
            with pytest.raises(ValueError):
                fn(**dict(base, **kw))
            return
        with pytest.raises(binding.LlamaError) as e:
            fn(**dict(base, **kw))
        assert e.value.rc == rc, (name, kw, e.value.rc)
    for fn, kw in good.values():
        fn(**kw)
    m.sync()
    three = _i32([0, 0, 0])
    kv3 = binding.KVCache(shape, batch=3, capacity=64)
    skew = torch.zeros(2 * 512 + 4, **bf)[4:].view(2, 512)  # 8 bytes past a 16-byte boundary
    for name in ("tree", "weights"):
        for layer in (-1, 1):
            refused(1, name, layer=layer)
        refused(2, name, kv=fp8)
        refused(1, name, q=skew)
        refused(1, name, out=skew)
        for sc in (binding.Scores(cap=-1.0), binding.Scores(scale=float("nan")), binding.Scores(cap=1e-35)):
            refused(1, name, scores=sc)
        refused(None, name, scores=binding.Scores(slopes=torch.ones(3, device="cuda")))
        for key in ("q", "out"):
            refused(None, name, **{key: torch.zeros(2, 512, device="cuda")})
            refused(None, name, **{key: torch.zeros(2, 511, **bf)})
            refused(None, name, **{key: torch.zeros(2, 512, dtype=torch.bfloat16)})
            refused(None, name, **{key: torch.zeros(512, 2, **bf).t()})
    for layer in (-2, 1):
        refused(1, "commit", layer=layer)
        refused(1, "evict", layer=layer)
    for name, key in (("tree", "cu_rows"), ("tree", "start_pos"), ("weights", "positions"), ("commit", "start_pos"),
                      ("commit", "path"), ("commit", "path_len"), ("evict", "lens"), ("evict", "kept")):
        t = good[name][1][key]
        refused(None, name, **{key: t.cpu()})
        refused(None, name, **{key: t.long()})
        if key != "kept":
            refused(None, name, **{key: torch.stack((t, t), -1)[..., 0]})  # with a stride
    # lengths that do not fit each other
    refused(None, "tree", cu_rows=_i32([0, 2]))
    refused(None, "tree", mask=torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    refused(None, "tree", mask=torch.zeros(2, dtype=torch.int32, device="cuda"))
    refused(None, "tree", mask=torch.zeros(2, 1, dtype=torch.int64, device="cuda"))
    refused(None, "tree", positions=_i32([0]))
    refused(None, "tree", mask=torch.zeros(2, 0, dtype=torch.int32, device="cuda"))
    refused(None, "weights", scratch=torch.zeros(2, 4, 63, device="cuda"))
    refused(None, "weights", weights=torch.zeros(2, 1, 64, device="cuda"))
    refused(None, "weights", weights=torch.zeros(2, 2, 64, **bf))
    refused(1, "weights", scratch=torch.zeros(2 * 4 * 64 + 1, device="cuda")[1:])
    refused(None, "commit", path_len=_i32([1]))
    refused(1, "commit", path=torch.zeros(2, 0, dtype=torch.int32, device="cuda"))
    for kw in (dict(keep=0, kept=kept[..., :0].contiguous()), dict(first=-1), dict(recent=-1), dict(first=5, recent=4), dict(first=2 ** 31 - 1, recent=2 ** 31 - 1)):
        refused(1, "evict", **kw)
    refused(None, "evict", keep=9)
    refused(None, "evict", weights=torch.zeros(1, 2, 1, 64, device="cuda"))
    refused(None, "evict", weights_out=torch.zeros(1, 2, 2, 32, device="cuda"))
    refused(None, "evict", weights_out=torch.zeros(1, 2, 2, 64))
    # more sequences than the context or the cache has
    many = {"tree": dict(cu_rows=_i32([0, 1, 2, 2]), start_pos=three),
            "weights": dict(q=torch.zeros(3, 512, **bf), out=torch.zeros(3, 512, **bf), positions=three,
                            weights=torch.zeros(3, 2, 64, device="cuda"), scratch=torch.zeros(3, 4, 64, device="cuda"))}
    refused(1, "tree", **many["tree"])
    refused(3, "weights", **many["weights"])
    refused(3, "weights", kv=kv3, **many["weights"])
    refused(1, "commit", start_pos=three, path=_i32([[0]] * 3), path_len=three)
    # fp32 contexts: caches of another type, or none that fits the heads
    with pytest.raises(ValueError):
        m32.op_cache_commit(kv, start, path, n)
    with pytest.raises(ValueError):
        m32.op_attention_tree(torch.zeros(2, 80, device="cuda"), cu, start, 0, kv, torch.zeros(2, 80, device="cuda"))
    # another device
    m._dev += 1
    try:
        for fn, kw in good.values():
            with pytest.raises(ValueError):
                fn(**kw)
    finally:
        m._dev -= 1
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
