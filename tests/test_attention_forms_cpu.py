"""The plain fp64 forms of the attention operators against independent
restatements, and the refusals that need no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import __graft_entry__
from llama2_decoder_forward_gb300 import binding, synth
from oracle import attention_forms as A
from oracle import llama_oracle as O


def test_plain_rotation_is_the_oracles():
    x = np.random.RandomState(0).randn(5, 3, 16)
    pos = np.array([0, 1, 7, 300, 5])
    t = A.rotation_table(301, 16)
    got = np.stack([A.rotate(x[i], t[p], False) for i, p in enumerate(pos)])
    np.testing.assert_allclose(got, O.rope(x, pos, 1e4), atol=1e-12)


def test_half_layout_is_a_permutation_of_the_adjacent_one():
    x = np.random.RandomState(1).randn(2, 24)
    cs = A.rotation_table(9, 16)[8]
    perm = [i for j in range(8) for i in (j, j + 8)] + list(range(16, 24))
    np.testing.assert_allclose(A.rotate(x, cs, True)[:, perm], A.rotate(x[:, perm], cs, False), atol=1e-15)


def test_rotation_keeps_relative_positions():
    # q.k after rotation depends on the distance alone, whatever the scaling
    r = np.random.RandomState(2)
    q, k = r.randn(1, 32), r.randn(1, 32)
    for kw in (dict(kind="linear", factor=4.0), dict(kind="bands", factor=8.0, low_turns=1, high_turns=4, original_len=64)):
        t = A.rotation_table(200, 32, **kw)
        a = [float(np.sum(A.rotate(q, t[p + 11], True) * A.rotate(k, t[p], True))) for p in (0, 40, 188)]
        np.testing.assert_allclose(a, a[0], rtol=1e-9)


def test_bands_reach_both_limits():
    plain, wide = A.rotation_table(2, 64), A.rotation_table(2, 64, kind="bands", factor=10.0, low_turns=1.0, high_turns=8.0,
                                                             original_len=1000)
    ang = lambda t: np.arctan2(t[1, :, 1], t[1, :, 0])
    assert np.isclose(ang(wide)[0], ang(plain)[0]) and np.isclose(ang(wide)[-1], ang(plain)[-1] / 10)


def test_attend_row_plain_case_is_the_oracles():
    r = np.random.RandomState(3)
    q, K, V = r.randn(4, 16), r.randn(2, 9, 16), r.randn(2, 9, 16)
    ref = O.gqa_attention(q, K, V, 6)
    for h in range(4):
        o, _ = A.attend_row(q[h], K[h // 2], V[h // 2], 5, np.arange(9) <= 5, 1 / 4.0)
        np.testing.assert_allclose(o, ref[h], atol=1e-12)


def test_documents_against_a_masked_torch_softmax():
    g = torch.Generator().manual_seed(4)
    n, nq, nkv, d = 30, 4, 2, 8
    q, k, v = (torch.randn(n, h, d, generator=g, dtype=torch.float64) for h in (nq, nkv, nkv))
    cu, pre = [0, 11, 11, 30], [4, 0, 25]
    sl = torch.tensor([0.5, 0.25, 0.1, 0.0], dtype=torch.float64)
    doc = torch.tensor([0] * 11 + [2] * 19)
    at = torch.tensor(list(range(11)) + list(range(19)))
    keep = (doc[:, None] == doc) & ((at[:, None] >= at) | (at < torch.tensor(pre)[doc]))
    s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(2, 1)) * 0.3
    s = 5 * torch.tanh(s / 5) - sl[:, None, None] * (at[:, None] - at).abs()
    p = torch.softmax(s.masked_fill(~keep, -math.inf), -1)
    want = torch.einsum("hij,jhd->ihd", p, v.repeat_interleave(2, 1))
    got, _ = A.attend_documents(q.numpy(), k.numpy(), v.numpy(), cu, pre, 0.3, 5.0, sl.numpy())
    np.testing.assert_allclose(got, want.numpy(), atol=1e-12)


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return binding.lib()


def test_table_arguments(lib):
    buf = ctypes.create_string_buffer(4096 + 16)
    al = (ctypes.addressof(buf) + 15) // 16 * 16
    good = dict(kind=2, theta=1e4, factor=2.0, low_turns=1.0, high_turns=4.0, original_len=64, magnitude=1.0)

    def call(rotary=64, n_pos=4, table=al, **kw):
        a = dict(good, **kw)
        sc = binding.RopeScaling(*[a[n] for n, _ in binding.RopeScaling._fields_])
        return lib.llama_rope_table(ctypes.byref(sc), rotary, n_pos, table, None)
    assert lib.llama_rope_table(None, 64, 4, al, None) == 1
    for kw in (dict(table=None), dict(table=al + 8), dict(rotary=0), dict(rotary=12), dict(n_pos=0), dict(kind=3),
               dict(kind=-1), dict(theta=0.0), dict(theta=float("nan")), dict(factor=0.0), dict(factor=float("inf")),
               dict(low_turns=4.0), dict(low_turns=-1.0), dict(high_turns=float("inf")), dict(original_len=0),
               dict(magnitude=0.0), dict(magnitude=float("nan"))):
        assert call(**kw) == 1, kw
    assert call(rotary=1 << 20, n_pos=1 << 20) == 3  # more angles than a launch's grid


def test_null_context(lib):
    kv = binding.KV()
    assert lib.llama_op_rope_norm_append(None, None, 0, 0, 1, None, None, 1, None, None, None, 1e-5, 0,
                                         ctypes.byref(kv), None, None, None) == 1
    assert lib.llama_op_attention_docs(None, None, None, None, 1, None, 1, None, None, None) == 1
    assert lib.llama_op_attention_decode_shared(None, None, None, 1, 0, ctypes.byref(kv), 0, 0, None, None) == 1


def test_binding_refuses_wrong_tensors(lib):
    with pytest.raises(ValueError):
        binding.Rope()
    with pytest.raises(ValueError):
        binding.Rope(torch.zeros(4, 8, 2, dtype=torch.float64))
    with pytest.raises(ValueError):
        binding.Rope(torch.zeros(4, 8, 2), rotary_dim=24)
    with pytest.raises(ValueError):
        binding.Rope(torch.zeros(4, 2, 8).transpose(1, 2))
    with pytest.raises(ValueError):
        binding.Scores(slopes=torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError):
        binding.rope_table(4, 12)
    m = binding.Model.__new__(binding.Model)
    m.shape, m.ctx = synth.Shape(1, 256, 4, 2, 128, 256, 256), None
    m._bind(m.shape)
    q, k = torch.zeros(3, 512, dtype=torch.bfloat16), torch.zeros(3, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on the device
        m.op_attention_docs(q, k, k, torch.zeros(2, dtype=torch.int32), q)


# --------------------------------------------------------------------------- what reaches the C calls
class _Recorded:
    """A Model over CPU tensors whose three calls record the C structs they are given."""

    def __init__(self, nq=4, nkv=2, n_layers=1):
        self.shape = synth.Shape(n_layers, 256, nq, nkv, 128, 256, 256)
        self.m = m = binding.Model.__new__(binding.Model)
        m.shape, m.ctx = self.shape, None
        m._bind(m.shape)
        m._dev = -1  # what a CPU tensor's get_device() says
        m._append = lambda *a: self._take(rope=a[8], kv=a[13])
        m._docs = lambda *a: self._take(scores=a[8])
        m._shared = lambda *a: self._take(kv=a[5], scores=a[8])
        self.q = torch.zeros(2, nq * 128, dtype=torch.bfloat16)
        self.kv_rows = torch.zeros(2, nkv * 128, dtype=torch.bfloat16)
        self.qkv = torch.zeros(2, self.shape.qkv_rows)
        self.pos = torch.zeros(2, dtype=torch.int32)

    def _take(self, **structs):
        for name, ref in structs.items():
            s = None if ref is None else getattr(ref, "_obj", ref)
            setattr(self, name, None if s is None else {f: getattr(s, f) for f, _ in s._fields_})
        return 0

    def cache(self, **kw):
        kw = kw or dict(batch=2, capacity=64)
        return binding.KVCache(self.shape, device="cpu", **kw)

    def append(self, kv=None, rope=None):
        self.m.op_rope_norm_append(self.qkv, self.pos, 0, kv or self.cache(), self.q, rope=rope)

    def docs(self, scores):
        self.m.op_attention_docs(self.q, self.kv_rows, self.kv_rows, torch.tensor([0, 2], dtype=torch.int32),
                                 self.q.clone(), scores=scores)

    def decode(self, kv=None, scores=None):
        self.m.op_attention_decode_shared(self.q, self.pos, 0, kv or self.cache(), self.q.clone(), scores=scores)


def test_scores_follow_their_attributes(lib):
    r = _Recorded()
    sc = binding.Scores(cap=5.0, slopes=torch.zeros(4))
    for call in (r.docs, lambda s: r.decode(scores=s)):
        sc.slopes = torch.ones(4)
        call(sc)
        assert r.scores == dict(scale=0.0, cap=5.0, slopes=sc.slopes.data_ptr())
        sc.slopes = None
        call(sc)
        assert r.scores["slopes"] is None
        for bad in (torch.ones(3), torch.ones(4).double(), torch.ones(4, 2)[:, 0]):
            sc.slopes = bad
            with pytest.raises(ValueError):
                call(sc)


def test_rope_follows_its_table(lib):
    r = _Recorded()
    rope = binding.Rope(torch.zeros(9, 32, 2), binding.ROPE_HALF)
    r.append(rope=rope)
    assert r.rope == dict(layout=binding.ROPE_HALF, rotary_dim=64, table=rope.table.data_ptr(), n_pos=9)
    rope.table = torch.zeros(30, 32, 2)  # of more positions
    r.append(rope=rope)
    assert r.rope["table"] == rope.table.data_ptr() and r.rope["n_pos"] == 30
    for bad in (torch.zeros(9, 16, 2), torch.zeros(9, 32, 2).double(), torch.zeros(9, 2, 32).transpose(1, 2),
                torch.zeros(9, 64)):
        rope.table = bad
        with pytest.raises(ValueError):
            r.append(rope=rope)
    rope.table = torch.zeros(9, 32, 2)
    rope.table.get_device = lambda: 0  # (a device that the context is not on)
    with pytest.raises(ValueError):
        r.append(rope=rope)
    rope.table = None  # the context's own angles
    r.append(rope=rope)
    assert r.rope["table"] is None and r.rope["rotary_dim"] == 64


def _fields(kv):
    s = kv.struct()
    return {f: getattr(s, f) for f, _ in s._fields_}


def test_cache_layout_follows_its_attributes(lib):
    r = _Recorded()
    table = torch.zeros(2, 4, dtype=torch.int32)
    paged = r.cache(n_pages=8, page_size=16, page_table=table)
    flat = r.cache()
    for kv in (paged, flat):
        r.append(kv)
        assert r.kv == _fields(kv)
    # a server that widens its table, grows its pool, changes the page size
    paged.page_table, paged.max_pages = torch.zeros(2, 9, dtype=torch.int32), 9
    paged.k, paged.v = (torch.zeros(1, 24, 2, 16, 128, dtype=torch.bfloat16) for _ in range(2))
    paged.n_pages = 24
    flat.k, flat.v = (torch.zeros(1, 3, 2, 128, 128, dtype=torch.bfloat16) for _ in range(2))
    flat.batch, flat.capacity = 3, 128
    for call in (r.append, r.decode):
        for kv in (paged, flat):
            call(kv)
            assert r.kv == _fields(kv)
    paged.n_pages, paged.page_size = 48, 8
    r.decode(paged)
    assert r.kv == _fields(paged) and r.kv["page_size"] == 8


def test_page_table_is_checked(lib):
    # read past its end, as other integers or with another stride it would send writes anywhere
    r = _Recorded()
    good = torch.zeros(2, 4, dtype=torch.int32)
    kv = r.cache(n_pages=8, page_size=16, page_table=good)
    for bad in (torch.zeros(1, 4, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int64),
                torch.zeros(4, 2, dtype=torch.int32).t(), torch.zeros(2, 8, dtype=torch.int32)[:, :4],
                torch.zeros(2, 3, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), None):
        kv.page_table = bad
        for call in (r.append, r.decode):
            with pytest.raises(ValueError):
                call(kv)
    kv.page_table = torch.zeros(5, 4, dtype=torch.int32)  # more sequences than the batch
    r.append(kv)
    r.decode(kv)


def test_cache_tensors_cover_the_layout(lib):
    r = _Recorded(n_layers=2)
    for kw in (dict(batch=2, capacity=64), dict(n_pages=8, page_size=16, page_table=torch.zeros(2, 4, dtype=torch.int32))):
        kv = r.cache(**kw)
        k = kv.k
        for name in ("k", "v"):
            for bad in (k[:1], k.float(), k.transpose(3, 4), k[:, :-1].contiguous()):
                setattr(kv, name, bad)
                for call in (r.append, r.decode):
                    with pytest.raises(ValueError):
                        call(kv)
            setattr(kv, name, k)
        r.append(kv)
        kv.n_pages, kv.batch = kv.n_pages and 9, kv.batch and 3
        with pytest.raises(ValueError):
            r.append(kv)
        kv = r.cache(e4m3=(1.0, 1.0), **kw)
        r.append(kv)
        kv.k = k
        with pytest.raises(ValueError):
            r.append(kv)
    r.append(r.cache(**kw))  # of two layers
    one, kv = _Recorded(), _Recorded().cache(**kw)
    one.append(kv)
    with pytest.raises(ValueError):  # the same cache with a model of two
        r.append(kv)
