"""Contexts with the least workspace: accepted, and every operation beside the plain path gives its results there,
trees with partial results for a few SMs or none included, without a byte written behind the buffer."""
import pytest
import torch

import test_gpu_cache_ops as ops
from _common import need_gpu, to_dev
from llama2_decoder_forward_gb300 import binding, synth
from test_gpu_cache_ops import OPTS

pytestmark = pytest.mark.gpu
GUARD = 1 << 16


@pytest.fixture
def least(monkeypatch):
    """_model of the operators' tests with the least workspace, in front of guard bytes that must stay."""
    guards, empty = [], torch.empty

    def guarded(*size, **kw):
        if kw.get("dtype") is not torch.uint8:
            return empty(*size, **kw)
        t = torch.full((size[0] + GUARD,), 0x5A, **kw)
        guards.append(t[size[0]:])
        return t[:size[0]]

    def model(nq, nkv, d=128, dtype="bf16", max_batch=8, max_seq=4096, n_layers=1):
        need_gpu()
        shape = synth.Shape(n_layers, 256, nq, nkv, d, 256, 256, dtype=dtype)
        w = to_dev({"layers": [synth.layer_weights(shape, 3, l) for l in range(n_layers)]})
        with monkeypatch.context() as mp:
            mp.setattr(torch, "empty", guarded)
            m = binding.Model(shape, w, max_batch=max_batch, max_tokens=0, max_seq=max_seq, has_embed_head=False, tree_room=False)
        assert m.workspace.numel() == binding.workspace_least_bytes(m.cfg)
        return m, shape
    monkeypatch.setattr(ops, "_model", model)
    yield model
    torch.cuda.synchronize()
    assert guards and all(bool((g == 0x5A).all()) for g in guards)


# nq, nkv, starts, rows: items of one row tile, of two, of several blocks; one CTA (no room for two), a few, many
@pytest.mark.parametrize("nq,nkv,starts,rows", [
    (1, 1, [3000, 9500], [100, 300]), (1, 1, [300], [129]), (8, 1, [9000], [20]), (8, 8, [5000], [40]), (64, 8, [3000, 10, 0], [64, 9, 30]),
    (16, 1, [2500] * 6, [70, 3, 0, 8, 9, 131])])
@pytest.mark.parametrize("opt", [OPTS[0], OPTS[3]])
@pytest.mark.parametrize("mask", ["tree", "any"])
def test_trees_in_the_least_workspace(least, nq, nkv, starts, rows, opt, mask):
    ops._tree_case(nq, nkv, 128, "bf16", starts, rows, page=64, mask=mask, check=[0, 4, 8, 63, 128], heads=[0, nq // 2, nq - 1], lead=1,
                   tail=1, calls=2, **opt)


@pytest.mark.parametrize("B", [33, 200])
def test_trees_of_many_sequences_in_the_least_workspace(least, B):
    r = ops.np.random.RandomState(B)
    ops._tree_case(2, 1, 128, "bf16", r.randint(0, 400, B).tolist(), r.randint(0, 8, B).tolist(), check=[0, 5])
    ops._tree_case(2, 2, 128, "bf16", r.randint(0, 400, B).tolist(), r.randint(60, 70, B).tolist(), check=[0, 59])


def test_trees_cut_in_two_in_the_least_workspace(least):
    ops._tree_case(40, 40, 128, "bf16", [1980, 0, 499, 505, 1020], [13, 13, 13, 8, 0], slots=2000, page=0, mask="any",
                   check=[0, 7, 8, 12], heads=[0, 17, 39], calls=2)


@pytest.mark.parametrize("nq,nkv,positions", [(8, 1, [19999]), (4, 4, [0, 14, 63, 64, 300]), (40, 40, [2999, 0, 511, 1025])])
def test_key_weights_in_the_least_workspace(least, nq, nkv, positions):
    ops._weights_case(nq, nkv, 128, "bf16", positions, page=64, heads=[0, nkv - 1])


@pytest.mark.parametrize("nq,nkv,d", [(40, 1, 64), (3, 1, 8), (4, 2, 40)])
def test_fp32_key_weights_in_the_least_workspace(least, nq, nkv, d):
    ops._weights_case(nq, nkv, d, "f32", [0, 15, 64, 300])


def test_less_than_the_least_is_refused(least):
    m, shape = least(4, 2, max_batch=1)
    ctx = binding.c_void_p()
    w = binding.Weights(None, None, None, binding.ctypes.cast(m._layers_arr, binding.ctypes.POINTER(binding.LayerWeights)))
    n = binding.workspace_least_bytes(m.cfg)
    assert binding.lib().llama_init(binding.ctypes.byref(m.cfg), binding.ctypes.byref(w), m.workspace.data_ptr(), n - 256, None,
                                    binding.ctypes.byref(ctx)) == 6
