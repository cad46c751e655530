"""Launches of the operators on caches of drafted trees and dropped keys: as many as their
descriptions say, and one or two by the path that the sizes choose (tests/test_attn_plans_cpu.py
has those paths)."""
import pytest
import torch

from llama2_decoder_forward_gb300 import binding
from test_gpu_cache_ops import _filled, _i32, _model, _randn

pytestmark = pytest.mark.gpu


def _count(m, call):
    n = m.launch_count()
    call()
    m.sync()
    return m.launch_count() - n


@pytest.mark.parametrize("want,nq,nkv,starts,rows,slots,page,dtype,d", [
    (1, 32, 32, [100, 20, 60, 3] * 4, [1] * 16, None, 16, "bf16", 128),  # a CTA per block
    (1, 64, 8, [700], [4], None, 16, "bf16", 128),  # a cluster of 8 per block
    (1, 32, 32, [700] * 4, [1] * 4, None, 16, "bf16", 128),  # and of 3
    (2, 40, 40, [1980, 0, 499, 505, 1020], [13, 13, 13, 8, 0], 2000, 0, "bf16", 128),  # cut in two and joined
    (2, 8, 1, [9000], [20], None, 64, "bf16", 128),  # the tensor cores and their join
    (2, 64, 8, [3000], [64], None, 64, "bf16", 128),
    (1, 4, 2, [130, 0], [9, 40], None, 5, "f32", 64)])
def test_tree_launches(want, nq, nkv, starts, rows, slots, page, dtype, d):
    m, shape = _model(nq, nkv, d, dtype, max_batch=len(starts))
    kv, *_ = _filled(shape, len(starts), slots or max(s + r for s, r in zip(starts, rows)), page, shape.torch_dtype, 3)
    n = sum(rows)
    q, out = _randn((n, nq, d), shape.torch_dtype, 4).cuda(), torch.empty(n, nq * d, dtype=shape.torch_dtype, device="cuda")
    cu = _i32([sum(rows[:i]) for i in range(len(rows) + 1)])
    assert _count(m, lambda: m.op_attention_tree(q, cu, _i32(starts), 0, kv, out)) == want
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("want,B,nq,nkv,keys,dtype,d", [
    (1, 64, 8, 8, 62, "bf16", 128), (1, 32, 32, 32, 200, "bf16", 128), (2, 1, 32, 32, 200, "bf16", 128), (2, 1, 8, 1, 20000, "bf16", 128),
    (2, 3, 4, 2, 300, "f32", 64)])
def test_key_weight_launches(want, B, nq, nkv, keys, dtype, d):
    m, shape = _model(nq, nkv, d, dtype, max_batch=B, max_seq=keys)
    kv, *_ = _filled(shape, B, keys, 0, shape.torch_dtype, 3)
    dt = shape.torch_dtype
    q, out = _randn((B, nq, d), dt, 4).cuda(), torch.empty(B, nq * d, dtype=dt, device="cuda")
    w, scratch = torch.zeros(B, nkv, keys, device="cuda"), torch.empty(B, nq, keys, device="cuda")
    pos = _i32([keys - 1] * B)
    assert _count(m, lambda: m.op_attention_decode_weights(q, pos, 0, kv, out, w, scratch)) == want
    # every head's weights are 1 in all, but for fp32 sums over the keys (the sum that divides them) and 2^x's own error
    assert abs(float(w.double().sum()) / (B * nq) - 1) < 2 * (keys / 8 + 64) * 2.0 ** -24 + 2.0 ** -20


@pytest.mark.parametrize("layer", [None, 1])
def test_move_launches(layer):
    m, shape = _model(4, 2, max_batch=2, n_layers=3)
    kv, *_ = _filled(shape, 2, 64, 16, torch.bfloat16, 3)
    path, n, at = _i32([[0, 2, 5]] * 2), _i32([3, 2]), _i32([10, 20])
    w = torch.rand(3 if layer is None else 1, 2, 2, 64, device="cuda")
    kept = torch.empty(len(w), 2, 2, 8, dtype=torch.int32, device="cuda")
    x, q = _randn((2, shape.qkv_rows), torch.float32, 5).cuda(), torch.empty(2, 4 * 128, dtype=torch.bfloat16, device="cuda")
    assert _count(m, lambda: m.op_cache_commit(kv, at, path, n, layer=layer)) == 1
    assert _count(m, lambda: m.op_cache_evict(kv, at, 8, w, kept, layer=layer)) == 1
    assert _count(m, lambda: m.op_rope_norm_append(x, at, layer or 0, kv, q, rope=binding.Rope(rotary_dim=128), positions=_i32([3, 4]))) == 1
