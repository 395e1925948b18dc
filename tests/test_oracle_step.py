"""Pins of the oracles of the step operators (block tables, norm and rotation,
windowed attention, sampling) against closed forms, brute force and one
another, and the refusals that the library makes on the host before anything
is launched (no GPU is needed for either)."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verification_19_gb300 as sv
from oracle import (oracle_block_tables, oracle_norm_rope, oracle_sample, oracle_verify_attn,
                    oracle_verify_attn_window)
from speculative_decoding_verification_19_gb300 import build as sv_build
from synth import kv_inputs_host, random_tree, workload


# --------------------------------------------------------------- block tables

def _pages(B, max_blocks, nb):
    return dict(block_table=np.full((B, max_blocks), -1, np.int32), span=np.zeros((B, 2), np.int32),
                pool=np.arange(nb, dtype=np.int32), pool_state=np.array([0, nb], np.int32))


def _step(st, ctx, row_start, rows, **kw):
    out = oracle_block_tables(np.asarray(ctx), row_start, kw.pop("parent", None), rows,
                              st["block_table"], st["span"], st["pool"], st["pool_state"],
                              np.full(rows, -9), np.full(rows, -9), kw.pop("M", 1), **kw)
    return out


def test_pages_are_conserved_and_cover_what_is_held():
    rng = np.random.default_rng(0)
    B, mb, nb = 7, 40, 90
    for window, sinks in ((0, 0), (50, 20), (16, 0)):
        st = _pages(B, mb, nb)
        ctx = np.full(B, -1)
        for _ in range(60):
            n = np.where(ctx < 0, 0, rng.integers(0, 40, B))
            start = np.concatenate([[0], np.cumsum(n)])
            out = _step(st, ctx, start, int(start[-1]) + 3, window=window, sinks=sinks)
            head, count = out["pool_state"]
            free = [int(out["pool"][(head + i) % nb]) for i in range(count)]
            used = out["block_table"][out["block_table"] >= 0].tolist()
            assert sorted(free + used) == list(range(nb))
            for b in range(B):
                if out["ok"][b]:
                    r = slice(start[b], start[b + 1])
                    assert np.array_equal(out["positions"][r], ctx[b] + np.arange(n[b]))
                    for t in range(ctx[b] + n[b]):
                        seen = t < sinks or t > ctx[b] - window or not window
                        if seen:
                            assert out["block_table"][b, t // 16] >= 0
            assert np.all(out["slots"][start[-1]:] == -9)
            st = out
            # commits keep a part of the new rows; requests end and begin
            ctx = np.where(out["ok"] > 0, ctx + rng.integers(0, n + 1), ctx)
            again = rng.random(B)
            ctx = np.where(again < 0.1, -1, np.where((ctx < 0) & (again > 0.5), 0, ctx))
            ctx = np.where(ctx > mb * 16 - 40, -1, ctx)


def test_pages_known_step():
    st = _pages(2, 4, 8)
    out = _step(st, [0, 30], np.array([0, 17, 19]), 20)
    # request 0: pages 0, 1 of 17 rows; request 1: pages 0, 1 of 32 positions
    assert out["block_table"].tolist() == [[0, 1, -1, -1], [2, 3, -1, -1]]
    assert out["slots"][15:20].tolist() == [15, 16, 3 * 16 + 14, 3 * 16 + 15, -9]
    assert out["pool_state"].tolist() == [4, 4] and out["status"] == 0
    # request 0 rolled back to 3 tokens, request 1 ended; one row each, none
    out = _step(out, [3, -1], np.array([0, 1, 1]), 1)
    assert out["block_table"].tolist() == [[0, -1, -1, -1], [-1, -1, -1, -1]]
    assert out["pool_state"].tolist() == [4, 7]
    assert [int(out["pool"][(4 + i) % 8]) for i in range(7)] == [4, 5, 6, 7, 1, 2, 3]
    assert out["ok"].tolist() == [1, 0]


# ----------------------------------------------------------- norm and rotation

def test_rotation_is_relative_and_keeps_lengths():
    rng = np.random.default_rng(1)
    f = 10000.0 ** (-np.arange(32) / 32)
    for inter in (False, True):
        x = rng.standard_normal((2, 1, 80))
        a = oracle_norm_rope(x, None, [5, 105], f, inter)
        b = oracle_norm_rope(x, None, [1005, 1105], f, inter)
        # the product of two rotated heads depends on the difference alone
        assert np.allclose(np.sum(a[0] * a[1]), np.sum(b[0] * b[1]))
        assert np.allclose(np.sum(a * a, -1), np.sum(x * x, -1))
        assert np.array_equal(a[..., 64:], x[..., 64:])
    y = oracle_norm_rope(x, np.ones(80), [0, -1], f, eps=0.0)
    assert np.allclose(np.mean(y[0] ** 2), 1.0) and np.all(y[1] == 0)


# ---------------------------------------------------------- windowed attention

@pytest.mark.parametrize("tree", [False, True])
def test_windowed_attention_against_a_mask(tree):
    wl = workload("tiny_chain").scaled(gamma=6)
    kv = kv_inputs_host(wl, seed=2, B=3, ctx=np.array([0, 5, 40]))
    parent = None
    if tree:
        parent = np.stack([random_tree(np.random.default_rng(s), 5, 2, 7) for s in range(3)])
    args = (kv["q"], kv["k_cache"], kv["v_cache"], kv["block_table"], kv["ctx_lens"], kv["k_new"],
            kv["v_new"])
    # a window of everything is the plain verify attention
    full = oracle_verify_attn(*args, parent=parent)
    wide = oracle_verify_attn_window(*args, window=1000, parent=parent)
    assert np.allclose(full[0], wide[0]) and np.allclose(full[1], wide[1])
    # by hand: keys outside the window moved out of reach
    for window, sinks in ((1, 0), (3, 0), (4, 2), (17, 20)):
        got = oracle_verify_attn_window(*args, window=window, sinks=sinks, parent=parent)
        b, i = 2, 6
        path = [i]
        while path[0] != 0:
            path.insert(0, path[0] - 1 if parent is None else int(parent[b, path[0]]))
        keys, vals = [], []
        for t in range(40 + len(path)):
            if t < sinks or t > 40 + len(path) - 1 - window:
                if t < 40:
                    blk = kv["block_table"][b, t // 16]
                    keys.append(kv["k_cache"][blk, 0, t % 16])
                    vals.append(kv["v_cache"][blk, 0, t % 16])
                else:
                    keys.append(kv["k_new"][b, path[t - 40], 0])
                    vals.append(kv["v_new"][b, path[t - 40], 0])
        s = np.array(keys, np.float64) @ kv["q"][b, i, 0] / 8.0
        p = np.exp(s) / np.exp(s).sum()
        assert np.allclose(got[0][b, i, 0], p @ np.array(vals, np.float64))
        assert np.allclose(got[1][b, i, 0], np.log(np.exp(s).sum()))


# -------------------------------------------------------------------- sampling

def test_sample_by_hand():
    z = np.log(np.array([[0.1, 0.4, 0.2, 0.3]]))
    one = lambda u, **kw: oracle_sample(z, [1.0], [u], **kw)  # noqa: E731
    assert [int(one(u)["tokens"][0]) for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.69, 0.71, 0.99)] == \
        [0, 0, 1, 1, 2, 2, 3, 3]
    # top-k 2 leaves tokens 1 and 3 with 4/7 and 3/7
    r = one(0.6, top_k=[2])
    assert r["tokens"][0] == 3 and np.isclose(r["prob"][0], 3 / 7)
    # top-p 0.65 needs 0.4 + 0.3; min-p 0.3 drops 0.1 (a quarter of 0.4)
    assert np.isclose(one(0.6, top_p=[0.65])["prob"][0], 3 / 7)
    assert np.isclose(one(0.0, min_p=[0.3])["prob"][0], 4 / 9)
    # ties go to the smaller index; greedy is the first largest
    t = oracle_sample(np.zeros((1, 4)), [1.0], [0.99], top_k=[3])
    assert t["tokens"][0] == 2
    assert oracle_sample(np.array([[1.0, 2.0, 2.0]]), [0.0], [0.9])["tokens"][0] == 1


def test_sample_follows_the_law():
    rng = np.random.default_rng(3)
    z = rng.standard_normal(6) * 1.5
    n = 4000
    u = (np.arange(n) + 0.5) / n  # a grid: every token as often as its probability
    r = oracle_sample(np.tile(z, (n, 1)), np.full(n, 0.7), u)
    p = np.exp(z / 0.7) / np.exp(z / 0.7).sum()
    assert np.all(np.abs(np.bincount(r["tokens"], minlength=6) / n - p) <= 1.01 / n)


# -------------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    sv_build.build()
    return sv.lib()


P = 1 << 20  # an address that nothing reads: these calls are refused on the host


def _dims(**kw):
    return sv.make_dims(**(dict(B=2, M=3, Hq=4, Hkv=2, D=128, max_blocks=4, num_blocks=9, V=64) | kw))


def test_sample_refusals(lib):
    good = dict(logits=P, stride=64, rows=2, V=64, dtype=0, T=P, u=P, out=P, ws=P, n=16)

    def call(**kw):
        a = good | kw
        return lib.spec_sample(a["logits"], a["stride"], a["rows"], a["V"], a["dtype"], a["T"], None,
                               None, None, a["u"], a["out"], None, a["ws"], a["n"], None)

    for kw in (dict(logits=None), dict(T=None), dict(u=None), dict(out=None), dict(ws=None),
               dict(n=15), dict(ws=P + 8), dict(V=0), dict(stride=63), dict(rows=-1), dict(dtype=2),
               dict(logits=P + 1)):
        assert call(**kw) == 1, kw
    assert call(V=(1 << 20) + 1, stride=1 << 21) == 3
    assert call(rows=0) == 0  # nothing to do, nothing launched


def test_window_refusals(lib):
    def call(d, window, sinks, q=P, n=1 << 30):
        return lib.spec_verify_attn_window(q, P, P, P, P, P, P, None, window, sinks, P, None,
                                           ctypes.byref(d), P, n, None)

    assert call(_dims(), 0, 0) == 1
    assert call(_dims(), -1, 0) == 1
    assert call(_dims(), 1, -1) == 1
    assert call(_dims(), 1, 0, q=None) == 1
    assert call(_dims(), 1, 0, q=P + 2) == 1
    assert call(_dims(), 1, 0, n=8) == 1
    assert call(_dims(D=96), 1, 0) == 3
    assert call(_dims(M=65), 1, 0) == 3  # 130 rows per KV head
    assert call(_dims(Hq=3), 1, 0) == 1
    assert call(_dims(max_blocks=1 << 27), 1, 0) == 3
    assert lib.spec_verify_attn_window(P, P, P, P, P, P, P, None, 1, 0, P, None, None, P, 9, None) == 1


def test_block_table_refusals(lib):
    good = dict(ctx=P, row_start=None, parent=None, rows=6, window=0, sinks=0, table=P, span=P,
                pool=P, state=P, slots=P, positions=P, ws=P, n=1 << 30)

    def call(d=None, **kw):
        a = good | kw
        d = d or _dims()
        return lib.spec_block_tables(a["ctx"], a["row_start"], a["parent"], a["rows"], a["window"],
                                     a["sinks"], a["table"], a["span"], a["pool"], a["state"],
                                     a["slots"], a["positions"], None, ctypes.byref(d), a["ws"],
                                     a["n"], None)

    for kw in (dict(ctx=None), dict(table=None), dict(span=None), dict(pool=None),
               dict(state=None), dict(slots=None), dict(positions=None), dict(ws=None), dict(n=4),
               dict(rows=5), dict(rows=-1, row_start=P), dict(window=-1), dict(sinks=-1),
               dict(row_start=P, parent=P)):
        assert call(**kw) == 1, kw
    assert call(_dims(max_blocks=0)) == 1 and call(_dims(num_blocks=0)) == 1
    assert call(_dims(max_blocks=1 << 27)) == 3
    # more rows or table entries than 32-bit counts hold
    assert call(rows=(1 << 30) + 1) == 3 and call(rows=(1 << 30) + 1, row_start=P) == 3
    assert call(_dims(B=17, max_blocks=1 << 26), rows=51) == 3


def test_norm_rope_refusals(lib):
    good = dict(q=P, k=P, v=P, qs=512, ks=256, vs=256, eps=1e-6, pos=P, f=P, rot=128, rows=5, qo=P,
                ko=P, slots=P, kc=P, vc=P, ws=P, n=1 << 30)

    def call(d=None, **kw):
        a = good | kw
        d = d or _dims()
        return lib.spec_qk_norm_rope(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], None, None,
                                     a["eps"], a["pos"], a["f"], a["rot"], 0, a["rows"], a["qo"],
                                     a["ko"], a["slots"], a["kc"], a["vc"], ctypes.byref(d), a["ws"],
                                     a["n"], None)

    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(pos=None), dict(f=None), dict(qo=None),
               dict(kc=None), dict(vc=None), dict(slots=None, ko=None), dict(qs=511), dict(qs=516),
               dict(ks=248), dict(vs=260), dict(q=P + 2), dict(ko=P + 8), dict(rot=130),
               dict(rot=-16), dict(eps=-1.0), dict(eps=float("nan")), dict(rows=-1), dict(n=4)):
        assert call(**kw) == 1, kw
    assert call(rot=24) == 3 and call(_dims(D=96)) == 3
    assert call(rows=0) == 0


def test_binding_checks_before_the_library():
    x = torch.zeros(2, 4)
    with pytest.raises(ValueError):
        sv.spec_sample(x, x[0], x[0], x[0], None, x[0])  # not on a GPU
    with pytest.raises(ValueError):
        sv.spec_verify_attn(x, x, x, x, x, x, x, None, x, None, _dims(), x, window=4)
