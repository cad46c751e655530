"""The plain fp64 forms of the operators on caches of drafted trees and dropped keys
against independent restatements, what reaches the C calls, and the refusals that
need no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import __graft_entry__
from llama2_decoder_forward_gb300 import binding, synth
from oracle import cache_ops as C
from oracle import llama_oracle as O


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return binding.lib()


# --------------------------------------------------------------------------- plain forms
def test_visible_rows_are_the_paths_to_the_root():
    # (I - P)^-1 of the parent matrix counts the paths from a row to its ancestors: one or none
    r = np.random.RandomState(0)
    for n in (1, 2, 9, 40):
        parents = [int(r.randint(-1, i)) for i in range(n)]
        P = np.zeros((n, n))
        for i, p in enumerate(parents):
            if p >= 0:
                P[i, p] = 1
        np.testing.assert_array_equal(C.tree_visible(parents), np.rint(np.linalg.inv(np.eye(n) - P)) > 0)


def test_mask_words_hold_the_bits():
    r = np.random.RandomState(1)
    for n, words in ((1, None), (32, None), (33, None), (70, 1), (5, 3)):
        see = r.rand(6, n) < 0.5
        got = C.mask_words(see, words)
        assert got.dtype == np.int32
        bits = np.unpackbits(got.view(np.uint8), axis=1, bitorder="little").astype(bool)
        m = min(n, bits.shape[1])
        np.testing.assert_array_equal(bits[:, :m], see[:, :m])
        assert not bits[:, m:].any()


def test_a_chain_is_plain_causal_attention():
    r = np.random.RandomState(2)
    q, K, V = r.randn(5, 16), r.randn(9, 16), r.randn(9, 16)
    see = C.tree_visible([-1, 0, 1, 2, 3])
    for i in range(5):
        keep = np.concatenate((np.ones(4, bool), see[i]))
        o, _ = C.attend(q[i], K, V, 4 + i, np.arange(9), keep, 0.25)
        ref = O.gqa_attention(q[i][None], K[None], V[None], 5 + i)
        np.testing.assert_allclose(o, ref[0], atol=1e-12)


def test_weigh_against_a_masked_torch_softmax():
    g = torch.Generator().manual_seed(3)
    q, K = torch.randn(8, generator=g, dtype=torch.float64), torch.randn(20, 8, generator=g, dtype=torch.float64)
    keep, where = torch.rand(20, generator=g) < 0.6, torch.randint(0, 50, (20,), generator=g)
    for cap, slope in ((0.0, 0.0), (2.0, 0.3)):
        s = K @ q * 0.4
        if cap:
            s = cap * torch.tanh(s / cap)
        s = (s - slope * (where - 17).abs().double()).masked_fill(~keep, -math.inf)
        got = C.weigh(q.numpy(), K.numpy(), 17, where.numpy(), keep.numpy(), 0.4, cap, slope)
        np.testing.assert_allclose(got, torch.softmax(s, 0).numpy(), atol=1e-14)
    assert not C.weigh(q.numpy(), K.numpy(), 0, where.numpy(), np.zeros(20, bool), 1.0).any()


def test_evict_against_a_stable_sort():
    r = np.random.RandomState(4)
    for n, keep, first, recent in ((30, 12, 3, 4), (30, 12, 0, 0), (30, 12, 12, 0), (30, 12, 5, 7), (12, 12, 1, 1), (3, 12, 1, 1),
                                   (40, 1, 0, 1), (40, 1, 0, 0)):
        w = r.randint(0, 6, n).astype(float)
        w[r.rand(n) < 0.1] = np.nan
        got = C.evict(w, keep, first, recent)
        if n <= keep:
            assert got == list(range(n))
            continue
        v = torch.tensor(w).nan_to_num(nan=-math.inf)
        v[:first], v[n - recent:] = math.inf, math.inf
        assert got == torch.sort(v, dim=0, descending=True, stable=True).indices[:keep].sort().values.tolist()


# --------------------------------------------------------------------------- without a GPU
def test_null_context(lib):
    kv = ctypes.byref(binding.KV())
    assert lib.llama_op_rope_norm_append_at(None, None, 0, 0, 1, None, None, 1, None, None, None, None, 1e-5, 0, kv,
                                            None, None, None) == 1
    assert lib.llama_op_attention_tree(None, None, 1, None, None, 1, None, 0, None, 0, kv, None, None) == 1
    assert lib.llama_op_attention_decode_weights(None, None, None, 1, 0, kv, None, None, 1, None, None) == 1
    assert lib.llama_op_cache_commit(None, kv, -1, None, 1, None, 1, None) == 1
    assert lib.llama_op_cache_evict(None, kv, -1, None, 1, 1, 0, 0, None, 1, None, None) == 1


class _Recorded:
    """A Model over CPU tensors whose calls record what they are given."""

    def __init__(self, monkeypatch, rc=0, n_layers=2):
        self.shape = synth.Shape(n_layers, 256, 4, 2, 128, 256, 256)
        self.m = m = binding.Model.__new__(binding.Model)
        m.shape, m.ctx = self.shape, None
        m._bind(m.shape)
        m._dev = -1  # what a CPU tensor's get_device() says
        self.calls = []

        def take(*a):
            self.calls.append(a)
            return rc
        m._append = m._append_at = m._tree = m._weights = take

        class Lib:
            llama_op_cache_commit = llama_op_cache_evict = staticmethod(take)
            llama_strerror = staticmethod(lambda code: b"")
        monkeypatch.setattr(binding, "lib", lambda: Lib)
        bf = dict(dtype=torch.bfloat16)
        self.kv = binding.KVCache(self.shape, device="cpu", batch=2, capacity=64)
        self.q, self.out = torch.zeros(3, 512, **bf), torch.zeros(3, 512, **bf)
        self.qkv = torch.zeros(3, self.shape.qkv_rows)
        self.cu, self.start = (torch.tensor(x, dtype=torch.int32) for x in ([0, 1, 3], [4, 5]))
        self.w, self.scratch = torch.zeros(2, 2, 2, 64), torch.zeros(2, 4, 64)
        self.kept = torch.zeros(2, 2, 2, 8, dtype=torch.int32)
        self.path = torch.zeros(2, 5, dtype=torch.int32)


def test_arguments_reach_the_calls(lib, monkeypatch):
    r = _Recorded(monkeypatch)
    m, kv = r.m, r.kv
    at, mask = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 4, dtype=torch.int32)
    m.op_attention_tree(r.q, r.cu, r.start, 1, kv, r.out)
    a = r.calls.pop()
    assert a[1:6] == (r.q.data_ptr(), 3, r.cu.data_ptr(), r.start.data_ptr(), 2)
    assert a[6:10] == (None, 0, None, 1) and a[11:] == (None, r.out.data_ptr())
    m.op_attention_tree(r.q, r.cu, r.start, 0, kv, r.out, mask=mask, positions=at, scores=binding.Scores(cap=3.0))
    a = r.calls.pop()
    assert a[6:10] == (mask.data_ptr(), 4, at.data_ptr(), 0) and a[11] is not None
    m.op_rope_norm_append(r.qkv, r.start, 0, kv, r.q, cu_rows=r.cu, positions=at)
    a = r.calls.pop()
    assert a[4:9] == (3, r.cu.data_ptr(), r.start.data_ptr(), 2, at.data_ptr()) and len(a) == 18
    m.op_rope_norm_append(r.qkv, r.start, 0, kv, r.q, cu_rows=r.cu)
    assert len(r.calls.pop()) == 17
    m.op_attention_decode_weights(r.q[:2], r.start, 1, kv, r.out[:2], r.w[1], r.scratch)
    a = r.calls.pop()
    assert a[1:5] == (r.q.data_ptr(), r.start.data_ptr(), 2, 1)
    assert a[7:] == (r.w[1].data_ptr(), 64, r.scratch.data_ptr(), r.out.data_ptr())
    m.op_cache_commit(kv, r.start, r.path, r.start)
    assert r.calls.pop()[2:] == (-1, r.start.data_ptr(), 2, r.path.data_ptr(), 5, r.start.data_ptr())
    m.op_cache_commit(kv, r.start, r.path, r.start, layer=1)
    assert r.calls.pop()[2] == 1
    m.op_cache_evict(kv, r.start, 8, r.w, r.kept, first=1, recent=2)
    assert r.calls.pop()[2:] == (-1, r.start.data_ptr(), 2, 8, 1, 2, r.w.data_ptr(), 64, r.w.data_ptr(), r.kept.data_ptr())
    other = torch.zeros(1, 2, 2, 64)
    m.op_cache_evict(kv, r.start, 8, r.w[0], r.kept[0], layer=0, weights_out=other)
    a = r.calls.pop()
    assert a[2] == 0 and a[8] == r.w.data_ptr() and a[10] == other.data_ptr()


def test_codes_become_errors(lib, monkeypatch):
    r = _Recorded(monkeypatch, rc=3)
    for call, name in ((lambda: r.m.op_attention_tree(r.q, r.cu, r.start, 0, r.kv, r.out), "llama_op_attention_tree"),
                       (lambda: r.m.op_attention_decode_weights(r.q[:2], r.start, 0, r.kv, r.out[:2], r.w[0], r.scratch),
                        "llama_op_attention_decode_weights"),
                       (lambda: r.m.op_cache_commit(r.kv, r.start, r.path, r.start), "llama_op_cache_commit"),
                       (lambda: r.m.op_cache_evict(r.kv, r.start, 8, r.w, r.kept), "llama_op_cache_evict")):
        with pytest.raises(binding.LlamaError, match=name) as e:
            call()
        assert e.value.rc == 3


def test_wrong_tensors_do_not_reach_the_calls(lib, monkeypatch):
    r = _Recorded(monkeypatch)
    good = {
        r.m.op_attention_tree: dict(q=r.q, cu_rows=r.cu, start_pos=r.start, layer=0, kv=r.kv, out=r.out),
        r.m.op_attention_decode_weights: dict(q=r.q[:2], positions=r.start, layer=0, kv=r.kv, out=r.out[:2], weights=r.w[0],
                                              scratch=r.scratch),
        r.m.op_cache_commit: dict(kv=r.kv, start_pos=r.start, path=r.path, path_len=r.start),
        r.m.op_cache_evict: dict(kv=r.kv, lens=r.start, keep=8, weights=r.w, kept=r.kept),
        r.m.op_rope_norm_append: dict(qkv=r.qkv, start_pos=r.start, layer=0, kv=r.kv, q_out=r.q, cu_rows=r.cu,
                                      positions=torch.zeros(3, dtype=torch.int32)),
    }
    for call, kw in good.items():
        for name, t in kw.items():
            if not isinstance(t, torch.Tensor):
                continue
            wrong = [t.double(), torch.stack((t, t), -1)[..., 0]]
            if name not in ("lens", "positions", "start_pos", "weights", "scratch", "path"):
                wrong.append(t[:-1].contiguous())  # too short for the others
            if name == "qkv":
                wrong = [t.double(), t[:, :-8]]
            for bad in wrong:
                with pytest.raises(ValueError):
                    call(**dict(kw, **{name: bad}))
    tree = good[r.m.op_attention_tree]
    for mask in (torch.zeros(3, dtype=torch.int32), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(3, 0, dtype=torch.int32),
                 torch.zeros(3, 1, dtype=torch.int64), torch.zeros(3, 2, dtype=torch.int32)[:, :1]):
        with pytest.raises(ValueError):
            r.m.op_attention_tree(**dict(tree, mask=mask))
    for kw in (dict(keep=9), dict(weights_out=r.w.double()), dict(weights_out=r.w[0]), dict(layer=0), dict(weights=r.w[:1])):
        with pytest.raises(ValueError):
            r.m.op_cache_evict(**dict(good[r.m.op_cache_evict], **kw))
    with pytest.raises(ValueError):
        r.m.op_attention_decode_weights(**dict(good[r.m.op_attention_decode_weights], scratch=r.scratch[:, :, :-1]))
    assert not r.calls
