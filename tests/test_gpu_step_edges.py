"""Edges of the step operators on the GPU: large batches (the sampler's
second look, the attention plan past shared memory), nothing to do, values
that no row sees, side streams, captured calls that share a workspace, and
waits that run out.

Tolerances as in test_gpu_step.py.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import speculative_decoding_verification_19_gb300 as sv  # noqa: E402
from harness import to_dev  # noqa: E402
from oracle import oracle_verify_attn_window  # noqa: E402
from synth import kv_inputs_host, workload  # noqa: E402
from test_gpu_step import (BF, F32, I32, Pages, sample_check, sample_gpu,  # noqa: E402
                           window_case)


# -------------------------------------------------------------------- sampling

def sample_ref(x, T, u):
    """Token, probability and distance to the nearest step, in fp64 on the GPU
    (temperature alone)."""
    out = []
    for r in range(x.shape[0]):
        w = torch.exp((x[r].double() - x[r].double().max()) / float(T[r]))
        c = w.cumsum(0)
        t = float(u[r]) * float(c[-1])
        i = int((c <= t).sum())
        near = min(float(c[i]) - t, t - (float(c[i - 1]) if i else -math.inf)) / float(c[-1])
        out.append((i, float(w[i] / c[-1]), near))
    return [np.array(v) for v in zip(*out)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("scale", [0.05, 3.0])
def test_sample_many_rows_without_filters(dt, scale):
    """Rows enough for the streaming kernel to leave doubtful draws to the
    second one: nearly flat rows make most of them doubtful."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n, V = 700, 30011
    x = (torch.randn(n, V, device="cuda", generator=g) * scale).to(dt)
    rng = np.random.default_rng(4)
    T = rng.choice([0.3, 1.0, 4.0], n).astype(np.float32)
    u = (rng.integers(0, 1 << 24, n) / (1 << 24)).astype(np.float32)
    u[:3] = (0.0, 1 - 2.0 ** -24, 0.5)
    T[5:40], x[7, 100], x[8, :] = 0.0, float("nan"), -math.inf
    x[45, 30010], T[50], u[51] = math.inf, -1.0, 1.0
    x[60, 5:] = -math.inf               # five tokens left
    x[61] = float(torch.finfo(dt).min)  # flat at the lowest value
    bad = [7, 8, 45, 50, 51]
    tok, prob, status = sample_gpu(x, T, u)
    assert np.all(tok[bad] == -1) and np.all(prob[bad] == 0) and status == (1 << 5 | 1 << 1)
    greedy = [r for r in range(n) if T[r] == 0 and r not in bad]
    top = x[greedy].float().max(1, keepdim=True)[0]
    first = torch.where(x[greedy].float() == top, torch.arange(V, device="cuda"), V).amin(1)
    assert np.array_equal(tok[greedy], first.cpu().numpy()) and np.all(prob[greedy] == 1)
    rest = [r for r in range(n) if r not in bad and r not in greedy]
    i, p, near = sample_ref(x[rest], T[rest], u[rest])
    sure = near > 1e-9
    assert sure.mean() > 0.95
    assert np.array_equal(tok[rest][sure], i[sure])
    assert np.all(np.abs(prob[rest][sure] - p[sure]) <= 2.0 ** -21 * p[sure])
    # the same rows a few at a time, which draw exactly in one kernel
    few = rest[:20]
    again = sample_gpu(x[few], T[few], u[few])
    assert np.array_equal(again[0][sure[:20]], tok[few][sure[:20]])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("mask", ["lowest", "inf"])
def test_sample_masked_vocabulary(dt, mask):
    """Tokens masked by the type's lowest value or by -inf, to the row's end and
    in whole chunks between: the draws stay right, and no more rows than
    without a mask need the second look."""
    g = torch.Generator(device="cuda").manual_seed(18)
    n, V = 700, 30011
    x = (torch.randn(n, V, device="cuda", generator=g) * 2).to(dt)
    low = float(torch.finfo(dt).min) if mask == "lowest" else -math.inf
    x[:, 200:9000] = low
    x[:, 9300:] = low
    x[3, 1:] = low   # one token left
    x[4, :-1], x[4, -1] = low, 0.5  # the last one
    rng = np.random.default_rng(19)
    T = rng.choice([0.5, 1.0, 2.0], n).astype(np.float32)
    u = (rng.integers(0, 1 << 24, n) / (1 << 24)).astype(np.float32)
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    tok, prob = torch.empty(n, dtype=I32, device="cuda"), torch.empty(n, device="cuda")
    sv.spec_sample(x, to_dev(T, F32), to_dev(u, F32), tok, prob, ws)
    assert sv.device_status(ws) == 0
    assert int(ws.view(I32)[1]) < n // 10
    i, p, near = sample_ref(x, T, u)
    sure = near > 1e-9
    assert sure.mean() > 0.95
    assert np.array_equal(tok.cpu().numpy()[sure], i[sure])
    assert np.all(np.abs(prob.cpu().numpy()[sure] - p[sure]) <= 2.0 ** -21 * p[sure])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V,live", [(30011, 40), (30011, 700), (128256, 6000)])
def test_sample_masked_vocabulary_with_filters(dt, V, live):
    """A mask of the type's lowest value draws as one of -inf does: the masked
    tokens have no mass, and they are the last that top-k takes."""
    g = torch.Generator(device="cuda").manual_seed(20)
    n = 40
    x = torch.randn(n, V, device="cuda", generator=g).to(dt)
    masked = torch.rand(V, device="cuda", generator=g).argsort() >= live
    rng = np.random.default_rng(21)
    T = rng.choice([0.5, 1.0, 2.0], n).astype(np.float32)
    u = (rng.integers(0, 1 << 24, n) / (1 << 24)).astype(np.float32)
    k = rng.choice([0, 1, 30, 50, 1000, V - 1], n)
    p = rng.choice([1.0, 0.1, 0.9, 0.999], n).astype(np.float32)
    mp = rng.choice([0.0, 0.01, 0.3], n).astype(np.float32)
    for kw in (dict(k=k), dict(p=p), dict(mp=mp), dict(k=k, p=p), dict(k=k, p=p, mp=mp)):
        got = [sample_gpu(x.masked_fill(masked, low), T, u, **kw)
               for low in (float(torch.finfo(dt).min), -math.inf)]
        assert np.array_equal(got[0][0], got[1][0]) and got[0][2] == got[1][2] == 0
        assert np.all(np.abs(got[0][1] - got[1][1]) <= 2.0 ** -21 * got[1][1])
        assert not masked.cpu().numpy()[got[0][0]].any()


@pytest.mark.parametrize("V,dt", [(152064, F32), (1 << 20, BF)])
def test_sample_cut_inside_many_equal_tokens(V, dt):
    """Few distinct values, so that a filter's cut falls inside a value's
    tokens, and runs long enough to be shared out among a CTA's warps."""
    rng = np.random.default_rng(22)
    n = 10
    x = np.round(rng.normal(size=(n, V)) * 2) / 2
    u = rng.integers(0, 1 << 24, n) / (1 << 24)
    k = rng.choice([0, 5000, V // 3, V - 7], n)
    k[:2] = (5000, V // 3)
    p = rng.choice([1.0, 0.7, 0.98], n)
    mp = rng.choice([0.0, 0.02], n)
    sample_check(x, np.ones(n), u, k=k, dt=dt)
    sample_check(x, np.ones(n), u, p=p, dt=dt)
    sample_check(x, np.full(n, 0.8), u, k=k, p=p, mp=mp, dt=dt)


@pytest.mark.parametrize("shift,scale", [(0, 1.0), (-40, 2.0), (0, 1e-3), (3e4, 100.0), (0, 1e-5),
                                         (0, 1e30)])
def test_sample_deep_top_p_over_signs_and_scales(shift, scale):
    """Thresholds above, below and about zero, and past the values that the
    bf16 select holds."""
    rng = np.random.default_rng(23)
    n, V = 12, 40000
    x = rng.normal(size=(n, V)) * scale + shift
    T = rng.choice([1.0, 0.7], n) * max(1.0, scale / 2)
    u = rng.integers(0, 1 << 24, n) / (1 << 24)
    p = rng.choice([0.5, 0.9, 0.999], n)
    k = rng.choice([6000, 20000, 39000], n)
    for kw in (dict(p=p), dict(k=k, p=p), dict(k=k)):
        sample_check(x, T, u, dt=BF, **kw)
    x[:, ::2] = np.round(x[:, ::2] / scale * 2) / 2 * scale  # and many equal ones
    sample_check(x, T, u, k=k, p=p, dt=BF)


def test_sample_many_rows_of_the_largest_vocabulary():
    g = torch.Generator(device="cuda").manual_seed(5)
    n, V = 304, 1 << 20
    x = torch.randn(n, V, device="cuda", generator=g, dtype=BF)
    T = np.full(n, 1.0, np.float32)
    u = (np.random.default_rng(6).integers(0, 1 << 24, n) / (1 << 24)).astype(np.float32)
    tok, prob, status = sample_gpu(x, T, u)
    i, p, near = sample_ref(x, T, u)
    sure = near > 1e-9
    assert status == 0 and np.array_equal(tok[sure], i[sure])
    assert np.all(np.abs(prob[sure] - p[sure]) <= 2.0 ** -21 * p[sure])


def test_sample_filters_over_batch_sizes():
    """The number of CTAs a row takes goes by the batch; the law does not."""
    rng = np.random.default_rng(7)
    for n, V in ((40, 64000), (130, 64000), (300, 9000)):
        x = (rng.standard_normal((n, V)) * 3).astype(np.float32)
        k = rng.choice([0, 1, 60, 300, 900, 2500], n)
        p = rng.choice([1.0, 0.5, 0.9, 0.999], n)
        mp = rng.choice([0.0, 0.01], n)
        T, u = rng.choice([0.5, 1.0], n), (rng.integers(0, 1 << 20, n) + 0.5) / (1 << 20)
        for dt in (BF, F32):
            sample_check(x, T, u, k, p, mp, dt)
            sample_check(x, T, u, k=k, dt=dt)


def test_sample_two_captured_calls_share_a_workspace():
    """Two graphs on two streams over one workspace: large batches, so both
    count their doubtful rows in it."""
    g = torch.Generator(device="cuda").manual_seed(8)
    n, V = 640, 20000
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    runs = []
    for s in range(2):
        x = torch.randn(n, V, device="cuda", generator=g, dtype=F32) * 0.1
        T = torch.ones(n, device="cuda")
        u = torch.rand(n, device="cuda", generator=g)
        want = torch.empty(n, dtype=I32, device="cuda")
        sv.spec_sample(x, T, u, want, None, ws)
        tok = torch.empty(n, dtype=I32, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sv.spec_sample(x, T, u, tok, None, ws)
        runs.append((graph, tok, want, (x, T, u)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(5):
        for (graph, tok, _, _), st in zip(runs, streams):
            with torch.cuda.stream(st):
                tok.fill_(-7)
                graph.replay()
    torch.cuda.synchronize()
    for _, tok, want, _ in runs:
        assert torch.equal(tok, want)
    assert sv.device_status(ws) == 0


# ------------------------------------------------------------------- attention

@pytest.mark.parametrize("impl", [sv.ATTN_TENSOR_CORES, sv.ATTN_CUDA_CORES])
@pytest.mark.parametrize("window,sinks", [(40, 3), (50, 0), (7, 20)])
def test_window_values_that_no_row_sees(impl, window, sinks):
    """NaN at every cached position outside the window and the sinks, also in
    pages that are held."""
    wl = workload("chain_gqa_128k").scaled(gamma=4, Hq=4, Hkv=2)
    ctx = np.array([300, 45, 129])
    kv = kv_inputs_host(wl, seed=11, B=3, ctx=ctx)
    dims = sv.make_dims(B=3, M=5, Hq=4, Hkv=2, D=128, max_blocks=kv["max_blocks"],
                        num_blocks=kv["num_blocks"], attn_impl=impl)
    ws = sv.workspace(dims)
    kc, vc = to_dev(kv["k_cache"], BF), to_dev(kv["v_cache"], BF)
    for b in range(3):
        for t in range(ctx[b]):
            if t >= sinks and t <= ctx[b] - window:
                blk = kv["block_table"][b, t // 16]
                kc[blk, :, t % 16] = float("nan")
                vc[blk, :, t % 16] = float("inf")
    q = to_dev(kv["q"], BF)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    sv.spec_verify_attn(q, to_dev(kv["k_new"], BF), to_dev(kv["v_new"], BF), kc, vc,
                        to_dev(kv["block_table"], I32), to_dev(ctx, I32), None, out, lse, dims, ws,
                        window=window, sinks=sinks)
    o, l, _, _ = oracle_verify_attn_window(kv["q"], kv["k_cache"], kv["v_cache"], kv["block_table"],
                                           ctx, kv["k_new"], kv["v_new"], window, sinks)
    assert np.all(np.abs(out.double().cpu().numpy() - o) <= 2.0 ** -7 * 4.5)
    assert np.max(np.abs(lse.cpu().numpy() - l)) <= 1e-4


def test_window_of_many_requests():
    """More requests than the split plan keeps in shared memory."""
    wl = workload("chain_gqa_128k").scaled(gamma=1, Hq=2, Hkv=1)
    ctx = np.random.default_rng(12).integers(0, 90, 1100).tolist()
    window_case(wl, ctx, 30, 5, False, seed=12, impl=sv.ATTN_TENSOR_CORES)


def test_window_wait_gives_up_then_recovers():
    """A limit of a thousand clocks runs out in the copy pipeline or in the
    merge of a split pair; an ordinary call afterwards is right again."""
    wl = workload("chain_gqa_128k").scaled(gamma=3)
    kv = kv_inputs_host(wl, seed=13, B=1, ctx=np.array([40000]))
    buf = torch.empty(96 << 20, device="cuda")
    for limit in (1, 0):
        dims = sv.make_dims(B=1, M=4, Hq=wl.Hq, Hkv=wl.Hkv, D=128, max_blocks=kv["max_blocks"],
                            num_blocks=kv["num_blocks"], wait_limit_kcycles=limit)
        ws = sv.workspace(dims)
        args = [to_dev(kv[k], BF) for k in ("q", "k_new", "v_new", "k_cache", "v_cache")]
        out, lse = torch.empty_like(args[0]), torch.empty(1, 4, wl.Hq, device="cuda")
        buf.fill_(1.0)  # the cache out of L2
        sv.spec_verify_attn(*args, to_dev(kv["block_table"], I32), to_dev(kv["ctx_lens"], I32), None,
                            out, lse, dims, ws, window=20000, sinks=4)
        status = sv.device_status(ws)
        assert (status & (1 << 7)) if limit else status == 0
    o, l, _, _ = oracle_verify_attn_window(kv["q"], kv["k_cache"], kv["v_cache"], kv["block_table"],
                                           kv["ctx_lens"], kv["k_new"], kv["v_new"], 20000, 4)
    assert np.all(np.abs(out.double().cpu().numpy() - o) <= 2e-2 + 1e-2 * np.abs(o))


def test_new_values_that_a_row_does_not_see():
    """Without a window, CUDA cores: the last new rows stand in a key range of
    their own (the ranges are 256 keys here); what they hold does not reach the
    rows that see none of them."""
    M, ctx = 8, 254
    g = torch.Generator(device="cuda").manual_seed(15)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    dims = sv.make_dims(B=1, M=M, Hq=4, Hkv=2, D=64, max_blocks=20, num_blocks=20, kv_dtype=F32)
    ws = sv.workspace(dims)
    q, kn, vn = r(1, M, 4, 64), r(1, M, 2, 64), r(1, M, 2, 64)
    kc, vc = r(20, 2, 16, 64), r(20, 2, 16, 64)
    bt = torch.arange(20, dtype=I32, device="cuda")[None]
    outs = []
    for value in (0.5, float("nan"), float("inf")):
        vn[0, 5] = value
        out, lse = torch.empty_like(q), torch.empty(1, M, 4, device="cuda")
        sv.spec_verify_attn(q, kn, vn, kc.clone(), vc.clone(), bt,
                            torch.tensor([ctx], dtype=I32, device="cuda"), None, out, lse, dims, ws)
        outs.append(out[0, :2])
    assert torch.isfinite(outs[0]).all()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# --------------------------------------------- offsets that pass 32 bits

@pytest.mark.parametrize("dt,D,impl", [(BF, 128, sv.ATTN_TENSOR_CORES), (BF, 128, sv.ATTN_CUDA_CORES),
                                       (F32, 64, sv.ATTN_CUDA_CORES)])
def test_a_cache_of_more_than_2_31_values(dt, D, impl):
    """Norm and rotation with the cache written, and windowed attention, on the
    last blocks of a cache of 2.3e9 values, against the same blocks in a cache
    of their own: the same bits."""
    B, M, Hq, Hkv, mb, need = 2, 3, 4, 2, 7, 14
    nb = int(2.3e9) // (Hkv * 16 * D)
    g = torch.Generator(device="cuda").manual_seed(16)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(dt)  # noqa: E731
    q, k, v = rand(B * M, Hq, D), rand(B * M, Hkv, D), rand(B * M, Hkv, D)
    kc0, vc0 = rand(need, Hkv, 16, D), rand(need, Hkv, 16, D)
    inv = to_dev(10000.0 ** (-np.arange(D // 2) / (D // 2)), torch.float64)
    ctx = np.array([100, 47])
    table = torch.arange(need, device="cuda", dtype=I32).flip(0).view(B, mb).contiguous()
    runs = []
    for blocks, first in ((need, 0), (nb, nb - need)):
        kc = torch.zeros(blocks, Hkv, 16, D, dtype=dt, device="cuda")
        vc = torch.zeros(blocks, Hkv, 16, D, dtype=dt, device="cuda")
        kc[first:], vc[first:] = kc0, vc0
        dims = sv.make_dims(B=B, M=M, Hq=Hq, Hkv=Hkv, D=D, max_blocks=mb, num_blocks=blocks,
                            kv_dtype=dt, attn_impl=impl)
        ws = sv.workspace(dims)
        t = np.concatenate([np.arange(c, c + M) for c in ctx])
        page = (table.cpu().numpy()[np.arange(B * M) // M, t // 16] + first).astype(np.int64)
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        sv.spec_qk_norm_rope(q, k, v, None, None, to_dev(t, I32), inv, qo, ko, dims, ws,
                             slots=to_dev(page * 16 + t % 16, torch.int64), k_cache=kc, v_cache=vc)
        written = kc[first:].clone(), vc[first:].clone()
        out, lse = torch.empty_like(qo).view(B, M, Hq, D), torch.empty(B, M, Hq, device="cuda")
        sv.spec_verify_attn(qo.view(B, M, Hq, D), ko.view(B, M, Hkv, D), v.view(B, M, Hkv, D), kc, vc,
                            table + first, to_dev(ctx, I32), None, out, lse, dims, ws, window=60,
                            sinks=2)
        assert sv.device_status(ws) == 0
        assert not kc[:first].any() and not vc[:first].any()
        runs.append((qo, ko, *written, out, lse, kc[first:].clone(), vc[first:].clone()))
        del kc, vc
    for x, y in zip(*runs):
        assert torch.equal(x, y)
    assert torch.isfinite(runs[0][4]).all() and not torch.equal(runs[0][2], kc0)
    torch.cuda.empty_cache()


def test_rows_of_more_than_2_31_values():
    """Many rows of queries (in place), and logits whose rows stand far apart."""
    rows, Hq = 265000, 64
    q = torch.zeros(rows, Hq, 128, dtype=BF, device="cuda")
    k = torch.zeros(rows, 1, 128, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(17)
    some = torch.randn(6, Hq, 128, device="cuda", generator=g).to(BF)
    q[-6:], k[-6:] = some, some[:, :1]
    w = torch.full((128,), 1.5, dtype=BF, device="cuda")
    inv = to_dev(10000.0 ** (-np.arange(64) / 64), torch.float64)
    pos = torch.arange(rows, device="cuda", dtype=I32)
    dims = sv.make_dims(B=1, M=1, Hq=Hq, Hkv=1, D=128)
    ws = sv.workspace(dims)
    few_q, few_k = torch.empty_like(some), torch.empty_like(k[-6:])
    sv.spec_qk_norm_rope(some, k[-6:].clone(), None, w, w, pos[-6:], inv, few_q, few_k, dims, ws)
    sv.spec_qk_norm_rope(q, k, None, w, w, pos, inv, q, k, dims, ws)
    assert torch.equal(q[-6:], few_q) and torch.equal(k[-6:], few_k)
    assert not q[:-6].any() and not k[:-6].any()
    del q, k

    V, stride = 50021, 1 << 30
    far = torch.empty(2 * stride + V, dtype=BF, device="cuda")
    x = far.as_strided((3, V), (stride, 1))
    x.copy_(torch.randn(3, V, device="cuda", generator=g).to(BF))
    one, u = torch.ones(3, device="cuda"), torch.full((3,), 0.625, device="cuda")
    for kw in ({}, dict(top_k=torch.full((3,), 50, dtype=I32, device="cuda")),
               dict(top_p=one * 0.99), dict(min_p=one * 0.01)):
        got = []
        for logits in (x, x.contiguous()):
            tok = torch.empty(3, dtype=I32, device="cuda")
            sv.spec_sample(logits, one, u, tok, None, ws, **kw)
            got.append(tok)
        assert torch.equal(*got) and (got[0] >= 0).all()
    assert sv.device_status(ws) == 0
    del far, x
    torch.cuda.empty_cache()


# ----------------------------------------------------------- lengths and streams

def test_nothing_to_do():
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    e = lambda *s, dt=F32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    sv.spec_sample(e(0, 50), e(0), e(0), e(0, dt=I32), e(0), ws)
    dims = sv.make_dims(B=1, M=1, Hq=2, Hkv=1, D=64, kv_dtype=F32)
    w = sv.workspace(dims)
    f = torch.ones(32, dtype=torch.float64, device="cuda")
    sv.spec_qk_norm_rope(e(0, 2, 64), e(0, 1, 64), None, None, None, e(0, dt=I32), f, e(0, 2, 64),
                         e(0, 1, 64), dims, w)
    # requests without new rows: lengths change, pages come and go
    st = Pages(3, 5, 9)
    st.call(np.array([40, 0, -1]), np.zeros(4, np.int64), 0)
    st.call(np.array([12, 17, -1]), np.zeros(4, np.int64), 0)
    st.call(np.array([-1, -1, -1]), np.zeros(4, np.int64), 0)
    assert st.h["pool_state"][1] == 9


def test_step_operators_on_a_side_stream_and_in_a_graph():
    """Tables, norm and rotation with the cache written, attention, captured
    as one graph on a stream of its own, against the same calls one by one."""
    B, M, Hq, Hkv, mb, nb = 2, 3, 4, 2, 8, 24
    dims = sv.make_dims(B=B, M=M, Hq=Hq, Hkv=Hkv, D=128, max_blocks=mb, num_blocks=nb)
    g = torch.Generator(device="cuda").manual_seed(14)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(BF)  # noqa: E731
    qkv, w = rand(B * M, Hq + 2 * Hkv, 128), rand(128)
    inv = to_dev(10000.0 ** (-np.arange(64) / 64), torch.float64)
    kc0, vc0 = rand(nb, Hkv, 16, 128), rand(nb, Hkv, 16, 128)
    ctx = to_dev(np.array([50, 7]), I32)

    def state():
        return dict(table=torch.full((B, mb), -1, dtype=I32, device="cuda"),
                    span=torch.zeros(B, 2, dtype=I32, device="cuda"),
                    pool=torch.arange(nb, dtype=I32, device="cuda"),
                    ring=to_dev(np.array([5, nb]), I32), kc=kc0.clone(), vc=vc0.clone(),
                    slots=torch.empty(B * M, dtype=torch.int64, device="cuda"),
                    pos=torch.empty(B * M, dtype=I32, device="cuda"),
                    q=torch.empty(B * M, Hq, 128, dtype=BF, device="cuda"),
                    k=torch.empty(B * M, Hkv, 128, dtype=BF, device="cuda"),
                    out=torch.empty(B, M, Hq, 128, dtype=BF, device="cuda"),
                    lse=torch.empty(B, M, Hq, device="cuda"), ws=sv.workspace(dims))

    def step(s, stream=None):
        sv.spec_block_tables(ctx, None, None, s["table"], s["span"], s["pool"], s["ring"], s["slots"],
                             s["pos"], None, dims, s["ws"], window=20, sinks=2, stream=stream)
        sv.spec_qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], w, w, s["pos"], inv,
                             s["q"], s["k"], dims, s["ws"], slots=s["slots"], k_cache=s["kc"],
                             v_cache=s["vc"], stream=stream)
        v = qkv[:, Hq + Hkv:].contiguous().view(B, M, Hkv, 128) if stream is None else s["v"]
        sv.spec_verify_attn(s["q"].view(B, M, Hq, 128), s["k"].view(B, M, Hkv, 128), v, s["kc"],
                            s["vc"], s["table"], ctx, None, s["out"], s["lse"], dims, s["ws"],
                            window=20, sinks=2, stream=stream)

    a, b, c = state(), state(), state()
    step(a)
    b["v"] = qkv[:, Hq + Hkv:].contiguous().view(B, M, Hkv, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(b, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    c["v"] = b["v"]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, stream=torch.cuda.current_stream())
    graph.replay()
    torch.cuda.synchronize()
    for o in (b, c):
        for k in ("table", "span", "pool", "ring", "slots", "pos", "q", "k", "out", "lse", "kc", "vc"):
            assert torch.equal(a[k], o[k]), k
        assert sv.device_status(o["ws"]) == 0
    assert torch.isfinite(a["out"]).all()


def test_calls_on_two_streams_at_once():
    """Sampling calls that share a workspace, and windowed attention with a
    workspace each, queued on two streams: the results of the calls alone."""
    g = torch.Generator(device="cuda").manual_seed(24)
    x = torch.randn(400, 40007, device="cuda", generator=g).to(BF)
    one, u = torch.ones(400, device="cuda"), torch.rand(400, device="cuda", generator=g)
    k = torch.randint(0, 9000, (400,), dtype=I32, device="cuda", generator=g)
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    kinds = [({}, 400), (dict(top_k=k, top_p=one * 0.95), 400), (dict(min_p=one[:90] * 0.01), 90),
             ({}, 30)]

    def sample(i, tok, prob, stream=None):
        kw, n = kinds[i]
        sv.spec_sample(x[:n], one[:n], u[:n], tok[:n], prob[:n], ws, stream=stream, **kw)

    B, M, Hq, Hkv, mb = 6, 5, 16, 4, 130
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(BF)  # noqa: E731
    q, kn, vn = rand(B, M, Hq, 128), rand(B, M, Hkv, 128), rand(B, M, Hkv, 128)
    table = torch.randperm(B * mb, device="cuda", generator=g).to(I32).view(B, mb)
    ctx = to_dev(np.array([0, 100, 600, 1000, 1500, 2000]), I32)
    dims = sv.make_dims(B=B, M=M, Hq=Hq, Hkv=Hkv, D=128, max_blocks=mb, num_blocks=B * mb)
    states = [dict(kc=rand(B * mb, Hkv, 16, 128), vc=rand(B * mb, Hkv, 16, 128),
                   out=torch.empty_like(q), lse=torch.empty(B, M, Hq, device="cuda"),
                   ws=sv.workspace(dims), tok=torch.zeros(400, dtype=I32, device="cuda"),
                   prob=torch.zeros(400, device="cuda")) for _ in range(2)]

    def attn(s, stream=None):
        sv.spec_verify_attn(q, kn, vn, s["kc"], s["vc"], table, ctx, None, s["out"], s["lse"], dims,
                            s["ws"], stream=stream, window=700, sinks=5)

    alone = []
    for i, s in enumerate(states):
        for j in range(4):
            sample(j, s["tok"], s["prob"])
            alone.append((s["tok"].clone(), s["prob"].clone()))
        attn(s)
        alone.append((s["out"].clone(), s["lse"].clone()))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [[], []]
        for j in range(4):
            for i, (s, st) in enumerate(zip(states, streams)):
                with torch.cuda.stream(st):
                    sample(j, s["tok"], s["prob"])
                    got[i].append((s["tok"].clone(), s["prob"].clone()))
                    attn(s)
        torch.cuda.synchronize()
        for i, s in enumerate(states):
            for j in range(4):
                for a, b in zip(got[i][j], alone[5 * i + j]):
                    assert torch.equal(a, b), (i, j)
            assert torch.equal(s["out"], alone[5 * i + 4][0])
            assert torch.equal(s["lse"], alone[5 * i + 4][1])
            assert sv.device_status(s["ws"]) == 0
    assert sv.device_status(ws) == 0


def test_binding_refusals():
    x = torch.zeros(2, 64, device="cuda")
    one = torch.ones(2, device="cuda")
    tok = torch.zeros(2, dtype=I32, device="cuda")
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    for bad in (dict(temperature=one[:1]), dict(uniform=one.double()), dict(out_tokens=tok.long()),
                dict(uniform=one.cpu()), dict(logits=x.t()), dict(logits=x.half()),
                dict(uniform=torch.ones(4, device="cuda")[::2])):
        kw = dict(logits=x, temperature=one, uniform=one, out_tokens=tok, out_prob=None, ws=ws) | bad
        with pytest.raises(ValueError):
            sv.spec_sample(**kw)
    with pytest.raises(sv.SpecError):
        sv.spec_sample(x[:, :40].expand(2, 40).as_strided((2, 40), (8, 1)), one, one, tok, None, ws)
    sv.spec_sample(x, one, one * 0.5, tok, None, ws)
    assert sv.device_status(ws) == 0
