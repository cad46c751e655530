"""How decode attention over the cache is cut into CTAs (csrc/attn_plan.h), compiled for the
host: the workspace holds the partial results of every plan, no plan passes a launch's
limits, and the sizes of the GPU tests take the path that they are there for."""
import ctypes
import os
import random
import subprocess

import pytest

from llama2_decoder_forward_gb300 import build

SMS = 152
HARNESS = r"""
#include "attn_plan.h"
using namespace llgb;
extern "C" {
void shared(int B, int nq, int nkv, int keys, int len, int sms, int weights, long long* o) {
  const SharedPlan s = weights ? weights_plan(B, nq, nkv, keys, sms) : shared_plan(B, nq, nkv, keys, len, sms);
  o[0] = s.own_splits; o[1] = s.cluster; o[2] = s.join; o[3] = (long long)s.partials; o[4] = s.keep; o[5] = s.min_share; o[6] = s.keys;
}
void tree(int n, int B, int nq, int nkv, int keys, int scored, int sms, long long room, long long* o) {
  const TreePlan t = tree_plan(n, B, nq, nkv, keys, scored, sms, (size_t)room);
  o[0] = t.own; o[1] = t.splits; o[2] = t.cluster; o[3] = t.join; o[4] = t.shift; o[5] = t.slices; o[6] = t.per; o[7] = t.min_share;
}
long long shared_room(int B, int nq, int nkv, int seq, int sms) { return (long long)shared_partial_bytes(B, nq, nkv, seq, sms); }
long long weights_room(int B, int nq, int nkv, int seq, int sms) { return (long long)weights_partial_bytes(B, nq, nkv, seq, sms); }
}
"""
HEADS = [(nkv * G, nkv) for nkv in (1, 2, 3, 5, 8, 12, 32, 40, 100, 700) for G in (1, 2, 3, 5, 8, 9, 16)]
PARTIAL = 130 * 4


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plans")
    src, so = str(d / "plans.cpp"), str(d / "plans.so")
    with open(src, "w") as f:
        f.write(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", build.CSRC, src, "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.shared_room.restype = lib.weights_room.restype = ctypes.c_longlong
    lib.tree.argtypes = [ctypes.c_int] * 7 + [ctypes.c_longlong, ctypes.c_void_p]

    class Plans:
        @staticmethod
        def shared(B, nq, nkv, keys, length=0, weights=False):
            o = (ctypes.c_longlong * 7)()
            lib.shared(B, nq, nkv, keys, length, SMS, int(weights), o)
            return dict(zip(("splits", "cluster", "join", "partials", "keep", "min_share", "keys"), o))

        @staticmethod
        def tree(n, B, nq, nkv, keys, scored=False, room=1 << 26):
            o = (ctypes.c_longlong * 8)()
            lib.tree(n, B, nq, nkv, keys, int(scored), SMS, room, o)
            return dict(zip(("own", "splits", "cluster", "join", "shift", "slices", "per", "min_share"), o))
        rooms = staticmethod(lambda *a: (lib.shared_room(*a, SMS), lib.weights_room(*a, SMS)))
    return Plans


def _sizes(seed, n):
    r = random.Random(seed)
    for _ in range(n):
        nq, nkv = r.choice(HEADS)
        yield r, nq, nkv, r.choice((1, 2, 3, 8, 13, 40, 100, 129, 640, 4000)), int(2 ** r.uniform(0, 19))


def test_partial_results_fit_their_room(plans):
    for r, nq, nkv, most, seq in _sizes(1, 20000):
        shared, weights = plans.rooms(most, nq, nkv, seq)
        B, keys = r.randint(1, most), r.choice((seq, r.randint(1, seq)))
        at = (most, nq, nkv, seq, B, keys)
        assert plans.shared(B, nq, nkv, keys, r.randint(0, keys))["partials"] * PARTIAL + 16 <= shared, at
        assert plans.shared(B, nq, nkv, keys, 0)["partials"] * PARTIAL + 16 <= shared, at
        w = plans.shared(B, nq, nkv, keys, weights=True)
        assert w["partials"] * PARTIAL + 16 <= weights, at
        assert w["keep"] == 0 or w["keep"] >= keys and w["splits"] == 1 and not w["join"], at
        assert weights <= shared, at  # key weights cost a context nothing beyond the shared decode's room


def test_the_first_key_weights_plan_beyond_four_ctas_per_sm(plans):
    # 100 (sequence, K/V head) pairs in 8 splits of 1024 keys: 800 CTAs' partial results
    p = plans.shared(100, 1, 1, 8192, weights=True)
    assert p["splits"] == 8 and p["partials"] == 800 > 4 * SMS
    assert plans.rooms(100, 1, 1, 8192)[1] >= 800 * PARTIAL


def test_tree_plans_stay_within_a_launch(plans):
    for r, nq, nkv, B, keys in _sizes(2, 20000):
        G, n = nq // nkv, int(2 ** r.uniform(0, 16))
        room = int(2 ** r.uniform(10, 26))
        t = plans.tree(n, B, nq, nkv, keys, r.random() < 0.5, room)
        assert t["slices"] * t["per"] >= G > (t["slices"] - 1) * t["per"] and t["per"] << t["shift"] <= 8
        if not t["own"]:
            continue
        at = (n, B, nq, nkv, keys, room, t)
        assert (n >> t["shift"]) + B <= 65535 and nkv * t["slices"] <= 65535, at
        assert t["splits"] in (1, 2, 3, 4, 8) and not (t["cluster"] and t["join"]), at
        assert not t["join"] or n * nq * t["splits"] * PARTIAL <= room, at


def _tree(plans, nq, nkv, starts, rows, slots=None, page=16, lead=0, tail=0, scored=False):
    """The plan of a GPU test's call: rows in front and behind count among a call's, the cache's room in whole pages."""
    slots = slots or max(s + r for s, r in zip(starts, rows))
    return plans.tree(lead + sum(rows) + tail, len(starts), nq, nkv, -(-slots // page) * page if page else slots, scored)


@pytest.mark.parametrize("want,nq,nkv,starts,rows,kw", [
    # one CTA per block, clusters of 2, 3, 4 and 8
    (dict(own=1, splits=1), 32, 32, [100, 20, 60, 3] * 4, [1] * 16, {}),
    (dict(own=1, splits=8, cluster=1), 64, 8, [700], [4], {}),
    (dict(own=1, cluster=1, slices=2), 16, 1, [700, 20, 0], [5, 9, 1], dict(lead=1, tail=1)),
    (dict(own=1, splits=3, cluster=1), 32, 32, [700] * 4, [1] * 4, {}),
    # enough CTAs, long ones cut in two, a joining kernel
    (dict(own=1, splits=2, join=1, min_share=512), 40, 40, [1980, 0, 499, 505, 1020], [13, 13, 13, 8, 0], dict(slots=2000, page=0)),
    (dict(own=1, splits=8, join=1), 8, 8, [6600] * 8, [1] * 8, {}),
    # the tensor-core kernel: long keys of few rows, wide drafts, few items
    (dict(own=0), 8, 1, [9000], [20], dict(page=64)), (dict(own=0), 2, 2, [20000], [129], dict(page=64)),
    (dict(own=0), 64, 8, [3000], [64], dict(page=64)), (dict(own=0), 32, 32, [3000] * 12, [70] * 12, {})])
def test_paths_of_the_tree_tests(plans, want, nq, nkv, starts, rows, kw):
    t = _tree(plans, nq, nkv, starts, rows, **kw)
    assert {k: t[k] for k in want} == want, t


@pytest.mark.parametrize("want,B,nq,nkv,keys", [
    (dict(keep=62, splits=1, join=0), 64, 8, 8, 62), (dict(keep=200), 32, 32, 32, 200),  # weights added where they are scored
    (dict(keep=0, join=1, splits=2), 1, 32, 32, 200), (dict(keep=0, join=1), 1, 8, 1, 20000), (dict(keep=0, splits=2), 8, 40, 40, 3000)])
def test_paths_of_the_key_weight_tests(plans, want, B, nq, nkv, keys):
    p = plans.shared(B, nq, nkv, keys, weights=True)
    assert {k: p[k] for k in want} == want, p
