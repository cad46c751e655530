"""The least workspace of a context: what it took before trees of drafted rows had room in it, so that
a buffer of that size still makes a context."""
import ctypes

import pytest

import __graft_entry__
from llama2_decoder_forward_gb300 import binding, synth


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return binding.lib()


F32 = synth.Shape(2, 256, 40, 40, 64, 256, 256, dtype="f32")
MQA = synth.Shape(2, 256, 16, 1, 128, 256, 256)


# bytes as llama_workspace_bytes gave them then, for 152 SMs
@pytest.mark.parametrize("shape,batch,tokens,seq,was", [
    (synth.LLAMA2_7B, 1, 0, 4096, 5709056), (synth.LLAMA2_7B, 32, 4096, 4096, 746300672), (synth.LLAMA2_7B, 64, 0, 16384, 57632000),
    (synth.LLAMA2_70B, 1, 512, 4096, 156971264), (synth.LLAMA2_70B, 16, 0, 32768, 55229696), (synth.TINY, 1, 16, 32, 298752),
    (synth.TINY, 8, 0, 512, 427008), (MQA, 200, 0, 1000, 35438336), (F32, 200, 0, 1000, 16633344)])
def test_least_workspace_is_that_without_trees(lib, shape, batch, tokens, seq, was):
    cfg = binding.make_config(shape, batch, tokens, seq)
    least, full = binding.workspace_least_bytes(cfg), binding.workspace_bytes(cfg)
    assert least == was
    assert least <= full <= least + 41_000_000 and full % 256 == 0
    if shape.dtype == "f32":
        assert full == least  # fp32 trees leave no partial results


def test_least_workspace_argument_checks(lib):
    n = ctypes.c_size_t()
    cfg = binding.make_config(synth.TINY, 1, 16, 32)
    assert lib.llama_workspace_least_bytes(ctypes.byref(cfg), ctypes.byref(n)) == 0 and n.value > 0
    assert lib.llama_workspace_least_bytes(ctypes.byref(cfg), None) == 1
    assert lib.llama_workspace_least_bytes(None, ctypes.byref(n)) == 1
    cfg.head_dim = 12
    assert lib.llama_workspace_least_bytes(ctypes.byref(cfg), ctypes.byref(n)) == 2
