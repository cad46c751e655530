"""Edges of the operators on caches whose slots are not one token after the other: starts far
past the cache, the largest lists in place, E4M3 rows at positions of their own. Tolerances
and helpers are those of the operators' other tests."""
import math

import numpy as np
import pytest
import torch

from llama2_decoder_forward_gb300 import binding
from oracle import cache_ops as C
from test_gpu_cache_ops import (_cache, _evict_case, _filled, _i32, _keys_of, _model, _out_bound, _randn, _score_error, _slopes,
                                _within)
from _common import f64

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------- trees that start past the cache
@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("start", [45, 70000, 2 ** 30 + 1, 2 ** 31 - 2])
def test_tree_starts_past_the_cache(dtype, d, rows, start):
    # Every cached key is attended and none of the rows, which is flagged. The bias goes by the rows'
    # slots: all keys are behind them, so that it differs between keys by slope x their distance.
    nq, nkv, limit = 4, 2, 40
    m, shape = _model(nq, nkv, d, dtype, max_batch=1)
    dt = shape.torch_dtype
    kv, k, v, pt = _filled(shape, 1, limit, 0, dt, 21)
    q = _randn((rows, nq, d), dt, 22, 1.5)
    sl = _slopes(nq)
    out = torch.full((rows, nq * d), 3.0, dtype=dt, device="cuda")
    m.op_attention_tree(q.cuda(), _i32([0, rows]), _i32([start]), 0, kv, out, scores=binding.Scores(slopes=sl.cuda()))
    rc, flags = m.sync_status()
    assert rc == 5 and flags == binding.FLAG_POS_RANGE
    K, V = _keys_of(k, pt, 0, 0, 0, limit), _keys_of(v, pt, 0, 0, 0, limit)
    qf, got, sc = f64(q), f64(out).reshape(rows, nq, d), 1 / math.sqrt(d)
    for i in range(rows):
        for h in range(nq):
            g = h // (nq // nkv)
            e = _score_error(qf[i, h], K[g], sc, 0.0, float(sl[h]) * (limit + rows))
            ref, mass = C.attend(qf[i, h], K[g], V[g], limit + i, np.arange(limit), np.ones(limit, bool), sc, 0.0, float(sl[h]))
            _within(got[i, h], ref, _out_bound(ref, mass, dtype, e, limit), "row=%d head=%d" % (i, h))


# --------------------------------------------------------------------------- the largest lists in place
@pytest.mark.parametrize("dtype,d,page,lens,keep,first,recent,ld", [
    ("bf16", 128, 16, [9000, 8192, 8193], 4000, 4, 300, None), ("bf16", 128, 0, [20000], 15000, 0, 0, 20011),
    ("f32", 8, 16, [17000, 30], 8500, 100, 8400, None), ("bf16", 128, 64, [16500], 1, 0, 0, None)])
def test_evict_long_lists_in_place(dtype, d, page, lens, keep, first, recent, ld):
    # more weights than a CTA holds, moved within their own buffer while later ones are still read
    _evict_case(dtype, False, d, page, lens, keep, first, recent, nkv=1, layers=1, ld=ld, alias=True)


@pytest.mark.parametrize("kind", ["ties", "nan", "steps"])
def test_evict_long_lists_of_equal_weights_in_place(kind):
    n = 18000
    g = torch.Generator().manual_seed(31)
    w = torch.rand(1, 1, 2, n, generator=g)
    if kind == "ties":
        w = (w * 5).floor()
    elif kind == "nan":
        w[..., ::2] = float("nan")
    else:
        w = 1.0 + torch.randint(0, 40, w.shape, generator=g) * 2.0 ** -23  # the last bits decide
    _evict_case("bf16", False, 128, 16, [n], 11000, 3, 50, layers=1, weights=w.float(), alias=True)


# --------------------------------------------------------------------------- E4M3 rows at positions of their own
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("gain", [False, True])
def test_append_positions_e4m3(page, half, gain):
    # The codes of a row at a position are those of the plain append to the slot of that number, bit by bit.
    nq, nkv, d, lens, starts = 8, 2, 128, [5, 0, 3, 1], [30, 4, 0, 62]
    m, shape = _model(nq, nkv, d)
    n = sum(lens)
    pos = torch.randint(0, 90, (n,), generator=torch.Generator().manual_seed(4)).tolist()
    x = _randn((n, shape.qkv_rows), torch.float32, 6).cuda()
    rope = binding.Rope(binding.rope_table(90, d), binding.ROPE_HALF if half else binding.ROPE_ADJACENT)
    gains = dict(q_gain=_randn((d,), torch.bfloat16, 7).cuda(), k_gain=_randn((d,), torch.bfloat16, 8).cuda()) if gain else {}
    kv = _cache(shape, len(lens), 64, page, e4m3=True)
    old = [t.clone() for t in (kv.k, kv.v)]
    plain = binding.KVCache(shape, batch=n, capacity=90, e4m3=(kv.k_scale, kv.v_scale))
    cu = np.concatenate(([0], np.cumsum(lens))).tolist()
    q, want = (torch.empty(n, nq * d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.op_rope_norm_append(x, _i32(starts), 0, kv, q, rope=rope, cu_rows=_i32(cu), positions=_i32(pos), **gains)
    m2, _ = _model(nq, nkv, d, max_batch=n)
    m2.op_rope_norm_append(x, _i32(pos), 0, plain, want, rope=rope, **gains)
    m.sync()
    m2.sync()
    assert torch.equal(q, want)
    for t, o, p in zip((kv.k, kv.v), old, (plain.k, plain.v)):
        for b in range(len(lens)):
            for i in range(lens[b]):
                s = starts[b] + i
                at = (0, int(kv.page_table[b, s // page]), slice(None), s % page) if page else (0, b, slice(None), s)
                assert torch.equal(t[at], p[0, cu[b] + i, :, pos[cu[b] + i]])
                o[at] = t[at]
        assert torch.equal(t, o)  # no other slot
