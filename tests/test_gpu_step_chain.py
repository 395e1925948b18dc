"""Calls of serving steps queued back to back, each reading what the one before
it writes, while its kernels already start: block tables, norm and rotation
with and without the cache written, attention, decisions, commit, and the
draft's draws read by the decisions.  The results of the same calls with a
synchronisation after each, which the oracles check.
"""
import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import speculative_decoding_verification_19_gb300 as sv  # noqa: E402
from harness import to_dev  # noqa: E402
from oracle import (oracle_block_tables, oracle_sample, oracle_verify_attn,  # noqa: E402
                    oracle_verify_attn_window)

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.mark.parametrize("impl", [sv.ATTN_TENSOR_CORES, sv.ATTN_CUDA_CORES])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 5)])
@pytest.mark.parametrize("cached", [False, True])
def test_steps_back_to_back(impl, window, sinks, cached):
    """Twenty steps whose tables change at every one: lengths jump, so pages
    come and go, and some requests end and begin."""
    steps, B, M, Hq, Hkv, D, mb, nb, V = 20, 3, 4, 4, 2, 128, 9, 29, 704
    rng = np.random.default_rng(window + 2 * cached)
    g = torch.Generator(device="cuda").manual_seed(31)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(BF)  # noqa: E731
    qkv, w = rand(steps, B * M, Hq + 2 * Hkv, D), rand(D)
    kc0, vc0 = rand(nb, Hkv, 16, D), rand(nb, Hkv, 16, D)
    inv = to_dev(10000.0 ** (-np.arange(D // 2) / (D // 2)), torch.float64)
    ctx = rng.integers(-1, mb * 16 - M + 1, (steps, B))
    if window:  # a window does not move back: lengths grow, and a request ends in between
        ctx = np.sort(ctx, axis=0)
        ctx[steps // 2] = -1
        ctx[steps // 2 + 1:] -= ctx[steps // 2 + 1:].min(0)
    ctxs = to_dev(ctx, I32)
    draft, target = rand(steps, B, M, V), rand(steps, B, M, V)
    T, u = torch.ones(B * M, device="cuda"), torch.rand(steps, B * M, device="cuda", generator=g)
    dims = sv.make_dims(B=B, M=M, Hq=Hq, Hkv=Hkv, D=D, max_blocks=mb, num_blocks=nb, V=V,
                        attn_impl=impl)
    kw = dict(window=window, sinks=sinks) if window else {}

    def state():
        e = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        return dict(table=torch.full((B, mb), -1, dtype=I32, device="cuda"), span=e(B, 2, dt=I32),
                    pool=torch.arange(nb, dtype=I32, device="cuda"), ring=to_dev([3, nb], I32),
                    kc=kc0.clone(), vc=vc0.clone(), slots=e(steps, B * M, dt=torch.int64),
                    pos=e(steps, B * M, dt=I32), q=e(steps, B, M, Hq, D), k=e(steps, B, M, Hkv, D),
                    v=qkv[:, :, Hq + Hkv:].contiguous().view(steps, B, M, Hkv, D),
                    out=e(steps, B, M, Hq, D), lse=e(steps, B, M, Hq, dt=F32),
                    drawn=e(steps, B, M, dt=I32), toks=e(steps, B, M, dt=I32),
                    path=e(steps, B, M, dt=I32), acc=e(steps, B, dt=I32), new=e(steps, B, dt=I32),
                    ws=sv.workspace(dims))

    def step(s, i, between=lambda *a: None):
        sv.spec_block_tables(ctxs[i], None, None, s["table"], s["span"], s["pool"], s["ring"],
                             s["slots"][i], s["pos"][i], None, dims, s["ws"], window=window,
                             sinks=sinks)
        between("tables")
        x = qkv[i]
        sv.spec_qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], w, w, s["pos"][i], inv,
                             s["q"][i].view(B * M, Hq, D), s["k"][i].view(B * M, Hkv, D), dims,
                             s["ws"], **(dict(slots=s["slots"][i], k_cache=s["kc"], v_cache=s["vc"])
                                         if cached else {}))
        between("rope")
        sv.spec_verify_attn(s["q"][i], s["k"][i], s["v"][i], s["kc"], s["vc"], s["table"], ctxs[i],
                            None, s["out"][i], s["lse"][i], dims, s["ws"], **kw)
        between("attention")
        sv.spec_sample(draft[i].view(B * M, V), T, u[i], s["drawn"][i].view(-1), None, s["ws"])
        between("sample")
        # the drawn tokens of the rows stand where the decisions read them
        sv.spec_reject_sample(target[i], draft[i], s["drawn"][i], None, T[:B], 5, i, s["toks"][i],
                              s["path"][i], s["acc"][i], None, dims, s["ws"])
        between("reject")
        sv.kv_commit(s["kc"], s["vc"], s["table"], ctxs[i], s["new"][i], s["path"][i], s["acc"][i],
                     dims, s["ws"])
        between("commit")

    alone = state()
    h = dict(block_table=np.full((B, mb), -1, np.int32), span=np.zeros((B, 2), np.int32),
             pool=np.arange(nb, dtype=np.int32), pool_state=np.array([3, nb], np.int32))
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    for i in range(steps):
        before = {}

        def check(after):
            torch.cuda.synchronize()
            if after == "tables":
                ref = oracle_block_tables(ctx[i], None, None, B * M, h["block_table"], h["span"],
                                          h["pool"], h["pool_state"], np.zeros(B * M),
                                          np.zeros(B * M), M, window=window, sinks=sinks)
                assert np.array_equal(alone["table"].cpu().numpy(), ref["block_table"])
                assert np.array_equal(alone["slots"][i].cpu().numpy(), ref["slots"])
                for k in h:
                    h[k] = ref[k].astype(np.int32)
                before["ok"] = np.nonzero(ref["ok"])[0]
            if after == "rope":
                before["kc"], before["vc"] = host(alone["kc"]), host(alone["vc"])
            if after == "attention" and len(before["ok"]):
                at = before["ok"]
                args = [host(alone["q"][i])[at], before["kc"], before["vc"], h["block_table"][at],
                        ctx[i][at], host(alone["k"][i])[at], host(alone["v"][i])[at]]
                o = (oracle_verify_attn_window(*args, window, sinks) if window
                     else oracle_verify_attn(*args))[0]
                got = host(alone["out"][i])[at]
                assert np.all(np.abs(got - o) <= 2e-2 + 1e-2 * np.abs(o))
            if after == "sample":
                ref = oracle_sample(host(draft[i]).reshape(B * M, V), np.ones(B * M),
                                    u[i].cpu().numpy())
                sure = ref["margin"] > 1e-8
                assert np.array_equal(alone["drawn"][i].cpu().numpy().reshape(-1)[sure],
                                      ref["tokens"][sure])

        step(alone, i, check)
    # places that do not run raise their bit
    assert sv.device_status(alone["ws"]) == ((1 << 2) if (ctx < 0).any() else 0)

    names = ("table", "span", "pool", "ring", "slots", "pos", "q", "k", "out", "lse", "kc", "vc",
             "drawn", "toks", "path", "acc", "new")
    for _ in range(10):  # queued
        s = state()
        torch.cuda.synchronize()
        for i in range(steps):
            step(s, i)
        for k in names:
            assert torch.equal(s[k], alone[k]), k
    s = state()  # and as one graph, whose kernels follow one another without a host between
    start = {k: s[k].clone() for k in names}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(steps):
            step(s, i)
    for _ in range(10):
        for k in names:
            s[k].copy_(start[k])
        graph.replay()
        for k in names:
            assert torch.equal(s[k], alone[k]), k


@pytest.mark.parametrize("tree", [False, True])
def test_logits_of_the_head_read_by_the_next_call(tree):
    """LM heads into one logits buffer, then the decisions and the draft's draws
    that read it, many times with other hidden states, queued back to back: the
    results of the calls one at a time."""
    from synth import random_tree

    steps, B, M, H, V = 8, 4, 8, 256, 8192
    g = torch.Generator(device="cuda").manual_seed(32)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(BF)  # noqa: E731
    hidden, w = rand(steps, 2, B * M, H), rand(2, V, H) * 0.1
    parent = None
    if tree:
        parent = to_dev(np.stack([random_tree(np.random.default_rng(b), 3, 3, M) for b in range(B)]),
                        I32)
    T, u = torch.ones(B * M, device="cuda"), torch.rand(B * M, device="cuda", generator=g)
    k = torch.full((B,), 40, dtype=I32, device="cuda")
    dims = sv.make_dims(B=B, M=M, V=V)

    def run(between):
        ws = sv.workspace(dims)
        target, draft = torch.zeros(2, B, M, V, dtype=BF, device="cuda")
        out = []
        for i in range(steps):
            e = lambda *s: torch.zeros(*s, dtype=I32, device="cuda")  # noqa: E731
            drawn, toks, path, acc = e(B, M), e(B, M), e(B, M), e(B)
            sv.spec_lm_head(hidden[i, 1], w[1], draft.view(B * M, V), ws)
            between()
            sv.spec_sample(draft.view(B * M, V), T, u, drawn.view(-1), None, ws)
            between()
            sv.spec_lm_head(hidden[i, 0], w[0], target.view(B * M, V), ws)
            between()
            kw = {} if i % 2 else dict(top_k=k)  # without a filter, and with one
            sv.spec_reject_sample(target, draft, drawn, parent, T[:B], 3, i, toks, path, acc, None,
                                  dims, ws, **kw)
            between()
            out += [drawn, toks, path, acc]
        torch.cuda.synchronize()
        assert sv.device_status(ws) == 0
        return out

    alone = run(torch.cuda.synchronize)
    for _ in range(20):
        for a, b in zip(run(lambda: None), alone):
            assert torch.equal(a, b)
