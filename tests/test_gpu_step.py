"""GPU parity of the step operators against the CPU oracles: block tables,
norm and rotation, windowed attention, sampling, and a serving loop that runs
them together with the verify step's own calls.

Tolerances.  Roundings to bf16 are off by at most half a step, 2^-8 of the
value.  Norm and rotation: fp32 throughout; the sum of squares of 128 terms,
the reciprocal root, five products and sums, sine and cosine come to less than
2^-20 of the pair's length, the angle to position * 2^-50 of a radian; one
rounding at the end.  Attention, bf16: the probabilities are rounded to bf16
before their product with V, so an output is off by at most 2^-8 of
sum p |v|, then rounded; fp32: scores of 128 terms are off by at most
128 * 2^-24 * max|q||k| * scale < 2e-5 for standard normal data, outputs by
about twice that times max|v| < 5.  Sampling: tokens are compared exactly
where u is more than 1e-9 from a step and a cut more than 1e-9 from its
target (the sums carry about 2^-32 of their value), probabilities to 2^-22.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import speculative_decoding_verification_19_gb300 as sv  # noqa: E402
from harness import to_dev  # noqa: E402
from oracle import (oracle_block_tables, oracle_kv_commit, oracle_norm_rope,  # noqa: E402
                    oracle_reject_sample, oracle_sample, oracle_verify_attn_window)
from synth import kv_inputs_host, random_tree, workload  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


# --------------------------------------------------------------- block tables

class Pages:
    """A page state on the GPU beside the oracle's."""

    def __init__(self, B, mb, nb, M=1, head=0):
        self.B, self.mb, self.nb, self.M = B, mb, nb, M
        pool = np.roll(np.random.default_rng(nb).permutation(nb), head).astype(np.int32)
        self.h = dict(block_table=np.full((B, mb), -1, np.int32), span=np.zeros((B, 2), np.int32),
                      pool=pool, pool_state=np.array([head, nb], np.int32))
        self.d = {k: to_dev(v, I32) for k, v in self.h.items()}
        self.dims = sv.make_dims(B=B, M=M, max_blocks=mb, num_blocks=nb)
        self.ws = sv.workspace(self.dims)

    def call(self, ctx, start, rows, parent=None, window=0, sinks=0, check=True):
        slots = torch.full((rows,), -9, dtype=torch.int64, device="cuda")
        pos = torch.full((rows,), -9, dtype=I32, device="cuda")
        ok = torch.full((self.B,), -9, dtype=I32, device="cuda")
        dev = lambda x: None if x is None else to_dev(x, I32)  # noqa: E731
        d = self.d
        sv.spec_block_tables(dev(ctx), dev(start), dev(parent), d["block_table"], d["span"],
                             d["pool"], d["pool_state"], slots, pos, ok, self.dims, self.ws,
                             window=window, sinks=sinks)
        got = {k: v.cpu().numpy() for k, v in d.items()}
        got.update(slots=slots.cpu().numpy(), positions=pos.cpu().numpy(), ok=ok.cpu().numpy(),
                   status=sv.device_status(self.ws))
        h = self.h
        ref = oracle_block_tables(ctx, start, parent, rows, h["block_table"], h["span"], h["pool"],
                                  h["pool_state"], np.full(rows, -9), np.full(rows, -9), self.M,
                                  window=window, sinks=sinks)
        for k in ("ok", "status", "pool_state", "span", "block_table", "positions", "slots", "pool"):
            assert np.array_equal(got[k], ref[k]), k
        for k in h:
            self.h[k] = ref[k].astype(np.int32)
        return ref


@pytest.mark.parametrize("B,nb,window,sinks", [(1, 9, 0, 0), (5, 60, 0, 0), (5, 60, 40, 17),
                                               (33, 300, 16, 0), (33, 300, 1, 1), (600, 5000, 0, 0),
                                               (600, 5000, 100, 40), (1100, 2500, 64, 300)])
def test_pages_over_a_life(B, nb, window, sinks):
    rng = np.random.default_rng(B + window)
    st = Pages(B, 24, nb, head=nb // 2)
    ctx = np.full(B, -1)
    short = 0
    for _ in range(12):
        n = np.where(ctx < 0, rng.integers(0, 2, B), rng.integers(0, 50, B))
        start = np.concatenate([[0], np.cumsum(n)])
        out = st.call(ctx, start, int(start[-1]) + 2, window=window, sinks=sinks)
        short += out["status"] != 0
        ctx = np.where(out["ok"] > 0, ctx + rng.integers(0, n + 1), ctx)
        r = rng.random(B)
        ctx = np.where(r < 0.1, -1, np.where((ctx < 0) & (r > 0.4), 0, ctx))
        ctx = np.where(ctx > 24 * 16 - 50, -1, ctx)
    assert short or nb != 2500  # the tightest ring runs out of pages


@pytest.mark.parametrize("M", [1, 5, 64, 128])
def test_pages_of_trees(M):
    rng = np.random.default_rng(M)
    st = Pages(4, 30, 130, M=M)
    for ctx in ([0, 3, 16, 200], [1, 4, 100, 201], [-1, 4, 100, 202]):
        parent = np.stack([random_tree(rng, max(1, M - 1), 3, M) for _ in range(4)])
        st.call(np.array(ctx), None, 4 * M + 1, parent=parent)
    st.call(np.array([2, 5, 101, 210]), None, 4 * M)


def test_pages_large_build_over_several_ctas():
    st = Pages(40, 700, 20000)
    n = np.full(40, 9000)
    n[3], n[7] = 0, 1
    start = np.concatenate([[0], np.cumsum(n)])
    st.call(np.zeros(40, np.int64), start, int(start[-1]) + 100)
    st.call(np.where(np.arange(40) % 2, -1, 8999), np.zeros(41, np.int64), 3)


def test_pages_refused_requests_stay_as_they_are():
    st = Pages(4, 4, 12, M=2)
    st.call(np.array([10, 20, 30, 40]), None, 8)
    # past the table; bad length; window pages needed again; rows out of range
    out = st.call(np.array([63, -2, 30, 40]), None, 8)
    assert out["ok"].tolist() == [0, 0, 1, 1] and out["status"] == (1 << 2 | 1 << 1)
    # one row out of order or out of range leaves no request's rows certain
    for start in ([0, 2, 1, 3, 4], [0, 2, 4, 6, 99], [-1, 2, 4, 6, 8], [0, 500, 4, 6, 8]):
        out = st.call(np.array([10, 20, 30, 40]), np.array(start), 8)
        assert out["ok"].sum() == 0 and out["status"] == 1 << 1
        assert np.all(out["slots"] == -1) and np.all(out["positions"] == -1)
    st.call(np.array([60, 20, 30, 40]), None, 8, window=17)
    out = st.call(np.array([3, 20, 30, 40]), None, 8, window=17)
    assert out["ok"].tolist()[0] == 0
    bad = np.array([[-1, 0], [0, 0], [-1, 1], [-1, 0]])
    out = st.call(np.array([60, 20, 30, 41]), None, 8, parent=bad, window=17)
    assert out["ok"].tolist() == [1, 0, 0, 1]
    # a span or a ring state that cannot be
    st.h["span"][2] = (3, 2)
    st.d["span"][2] = torch.tensor([3, 2])
    out = st.call(np.array([60, 20, 30, 42]), None, 8, window=17)
    assert out["ok"].tolist() == [1, 1, 0, 1]
    st.h["pool_state"][1] = 13
    st.d["pool_state"][1] = 13
    out = st.call(np.array([60, 20, 30, 43]), None, 8, window=17)
    assert out["ok"].sum() == 0 and out["status"] == 1 << 6


def test_pages_state_in_one_buffer():
    """Tables, spans, ring and ring state as views of one buffer, at odd
    offsets."""
    st = Pages(3, 5, 13)
    buf, at = torch.empty(3 * 5 + 6 + 13 + 2, dtype=I32, device="cuda"), 0
    for k in ("block_table", "span", "pool", "pool_state"):
        view = buf[at:at + st.d[k].numel()].view(st.d[k].shape)
        view.copy_(st.d[k])
        st.d[k], at = view, at + view.numel()
    for ctx in ([0, 10, 31], [3, 20, 33], [40, -1, 35]):
        assert st.call(np.array(ctx), np.array([0, 3, 8, 10]), 11)["ok"].sum() >= 2


def test_pages_rows_out_of_order_among_many_requests():
    st = Pages(1200, 4, 3000)
    start = np.arange(1201)
    st.call(np.full(1200, 5), start, 1203)
    for at, value in ((1100, 3), (600, 1300), (0, -1)):
        bad = start.copy()
        bad[at] = value
        out = st.call(np.full(1200, 20), bad, 1203)
        assert out["ok"].sum() == 0 and np.all(out["slots"] == -1)
    assert st.call(np.full(1200, 20), start, 1203)["ok"].all()


def test_pages_captured_and_replayed():
    st = Pages(3, 8, 20)
    ctx, start = torch.zeros(3, dtype=I32, device="cuda"), to_dev(np.array([0, 5, 5, 22]), I32)
    slots = torch.full((24,), -9, dtype=torch.int64, device="cuda")
    pos, ok = torch.full((24,), -9, dtype=I32, device="cuda"), torch.zeros(3, dtype=I32, device="cuda")
    d = st.d
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_block_tables(ctx, start, None, d["block_table"], d["span"], d["pool"],
                             d["pool_state"], slots, pos, ok, st.dims, st.ws)
    h = st.h
    for c in ([0, 0, 0], [5, 0, 17], [-1, 40, 30], [7, 41, 31]):
        ctx.copy_(torch.tensor(c))
        g.replay()
        ref = oracle_block_tables(np.array(c), start.cpu().numpy(), None, 24, h["block_table"],
                                  h["span"], h["pool"], h["pool_state"], np.full(24, -9),
                                  np.full(24, -9), 1)
        for k in ("block_table", "span", "pool", "pool_state"):
            assert np.array_equal(d[k].cpu().numpy(), ref[k]), k
            h[k] = ref[k].astype(np.int32)
        assert np.array_equal(slots.cpu().numpy(), ref["slots"])


# ----------------------------------------------------------- norm and rotation

def rope_check(got, x, w, pos, f, inter, dt, eps=1e-6):
    ref = oracle_norm_rope(x, w, pos, f, inter, eps)
    half = len(f)
    size = np.abs(ref)
    if half:  # an element's error scales with its pair's length
        a, b = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if inter
                else (slice(0, half), slice(half, 2 * half)))
        size[..., a] = size[..., b] = np.hypot(ref[..., a], ref[..., b])
    tol = size * (2.0 ** -20 + np.maximum(pos, 0)[:, None, None] * 2.0 ** -50) + 1e-30
    if dt == BF:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= tol), float((err / tol).max())


ROPE = [  # dtype, rows, Hq, Hkv, D, rot, interleaved, norm, strided
    (BF, 1, 32, 8, 128, 128, False, True, True), (BF, 7, 5, 1, 128, 128, True, True, False),
    (BF, 33, 7, 7, 64, 64, False, True, True), (BF, 19, 3, 1, 128, 64, False, True, True),
    (BF, 19, 3, 1, 64, 16, True, False, True), (BF, 5, 64, 8, 128, 0, False, True, False),
    (BF, 5000, 9, 3, 128, 128, False, True, True), (F32, 1, 1, 1, 64, 64, False, True, False),
    (F32, 17, 6, 2, 128, 128, False, True, True), (F32, 23, 4, 4, 64, 32, True, True, True),
    (F32, 40, 16, 2, 128, 48, False, False, False), (F32, 3000, 5, 1, 64, 64, True, True, True)]


@pytest.mark.parametrize("dt,rows,Hq,Hkv,D,rot,inter,norm,strided", ROPE)
@pytest.mark.parametrize("cached", [False, True])
def test_norm_rope(dt, rows, Hq, Hkv, D, rot, inter, norm, strided, cached):
    rng = np.random.default_rng(rows + D)
    g = torch.Generator(device="cuda").manual_seed(rows)
    H = Hq + 2 * Hkv
    qkv = (torch.randn(rows, H, D, device="cuda", generator=g) * 2).to(dt)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    wq = (torch.rand(D, device="cuda", generator=g) + 0.5).to(dt) if norm else None
    wk = (torch.rand(D, device="cuda", generator=g) - 1.5).to(dt) if norm else None
    f = 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
    pos = rng.integers(0, 200000, rows)
    pos[0] = 2 ** 31 - 1
    if rows > 4:
        pos[2:4] = (-1, 0)
    nb = -(-rows // 16) + 2
    dims = sv.make_dims(B=1, M=1, Hq=Hq, Hkv=Hkv, D=D, num_blocks=nb, kv_dtype=dt)
    ws = sv.workspace(dims)
    qo = torch.full((rows, Hq, D), 77.0, device="cuda", dtype=dt)
    ko = torch.full((rows, Hkv, D), 77.0, device="cuda", dtype=dt)
    kw = {}
    if cached:
        slots = rng.permutation(nb * 16)[:rows]
        if rows > 8:
            slots[5], slots[6] = -1, nb * 16  # no slot; past the cache
        kc = torch.full((nb, Hkv, 16, D), 55.0, device="cuda", dtype=dt)
        vc = torch.full((nb, Hkv, 16, D), 56.0, device="cuda", dtype=dt)
        kw = dict(slots=to_dev(slots, torch.int64), k_cache=kc, v_cache=vc)
    inv = to_dev(f, torch.float64) if rot else None
    sv.spec_qk_norm_rope(q, k, v, wq, wk, to_dev(pos, I32), inv, qo, ko, dims, ws,
                         interleaved=inter, **kw)
    np64 = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    rope_check(qo, np64(q), np64(wq), pos, f, inter, dt)
    rope_check(ko, np64(k), np64(wk), pos, f, inter, dt)
    assert sv.device_status(ws) == ((1 << 6) if cached and rows > 8 else 0)
    if cached:
        live = (pos >= 0) & (slots >= 0) & (slots < nb * 16)
        want_k, want_v = torch.full_like(kc, 55.0), torch.full_like(vc, 56.0)
        at = torch.from_numpy(slots[live]).cuda()
        rows_ = torch.from_numpy(np.nonzero(live)[0]).cuda()
        want_k[at // 16, :, at % 16] = ko[rows_]
        want_v[at // 16, :, at % 16] = v[rows_]
        assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
        # without k_out, and in place: the same caches and queries
        kc2, vc2, q2 = torch.full_like(kc, 55.0), torch.full_like(vc, 56.0), q.contiguous().clone()
        kw.update(k_cache=kc2, v_cache=vc2)
        sv.spec_qk_norm_rope(q2, k, v, wq, wk, to_dev(pos, I32), inv, q2, None, dims, ws,
                             interleaved=inter, **kw)
        assert torch.equal(q2, qo) and torch.equal(kc2, kc) and torch.equal(vc2, vc)


def test_norm_rope_special_values():
    """Zeros stay zeros; a NaN or infinity stays in its head."""
    dims = sv.make_dims(B=1, M=1, Hq=3, Hkv=1, D=128, kv_dtype=BF)
    ws = sv.workspace(dims)
    x = torch.randn(2, 4, 128, device="cuda").to(BF)
    x[0, 0], x[0, 1, 5], x[1, 2, 9] = 0, float("nan"), float("inf")
    w = torch.ones(128, device="cuda", dtype=BF)
    f = to_dev(10000.0 ** (-np.arange(64) / 64), torch.float64)
    pos = torch.tensor([3, 9], dtype=I32, device="cuda")
    qo, ko = torch.empty(2, 3, 128, device="cuda", dtype=BF), torch.empty(2, 1, 128, device="cuda", dtype=BF)
    sv.spec_qk_norm_rope(x[:, :3], x[:, 3:], None, w, w, pos, f, qo, ko, dims, ws)
    assert torch.all(qo[0, 0] == 0) and torch.isnan(qo[0, 1]).all()
    assert torch.isnan(qo[1, 2]).any() and torch.isfinite(qo[0, 2]).all()
    assert torch.isfinite(qo[1, :2]).all() and torch.isfinite(ko).all()


# ---------------------------------------------------------- windowed attention

def window_case(wl, ctx, window, sinks, tree, seed, impl, D=128):
    B, M = len(ctx), wl.M
    kv = kv_inputs_host(wl, seed=seed, B=B, ctx=np.array(ctx))
    rng = np.random.default_rng(seed)
    parent = None
    if tree:
        parent = np.stack([random_tree(rng, max(1, M - 1), 2, M) for _ in range(B)])
    # entries of pages that no row sees hold anything
    page = np.arange(kv["max_blocks"])
    for b in range(B):
        lo = max(0, ctx[b] - window + 1) // 16
        gone = (page >= -(-sinks // 16)) & (page < lo)
        kv["block_table"][b, gone] = rng.choice([-1, 1 << 30], gone.sum())
    dt = BF if wl.dtype == "bf16" else F32
    # what the rows do not see must not reach them: NaN in free blocks
    used = np.unique(kv["block_table"][(kv["block_table"] >= 0) &
                                       (kv["block_table"] < kv["num_blocks"])])
    free = np.setdiff1d(np.arange(kv["num_blocks"]), used)
    dims = sv.make_dims(B=B, M=M, Hq=wl.Hq, Hkv=wl.Hkv, D=wl.D, max_blocks=kv["max_blocks"],
                        num_blocks=kv["num_blocks"], kv_dtype=dt, attn_impl=impl)
    ws = sv.workspace(dims)
    kc, vc = to_dev(kv["k_cache"], dt), to_dev(kv["v_cache"], dt)
    if len(free):
        kc[torch.from_numpy(free).cuda()] = float("nan")
        vc[torch.from_numpy(free).cuda()] = float("nan")
    q = to_dev(kv["q"], dt)
    out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:3], float("nan"), device="cuda")
    sv.spec_verify_attn(q, to_dev(kv["k_new"], dt), to_dev(kv["v_new"], dt), kc, vc,
                        to_dev(kv["block_table"], I32), to_dev(kv["ctx_lens"], I32),
                        None if parent is None else to_dev(parent, I32), out, lse, dims, ws,
                        window=window, sinks=sinks)
    assert sv.device_status(ws) == 0
    args = (kv["q"], kv["k_cache"], kv["v_cache"], kv["block_table"], kv["ctx_lens"], kv["k_new"])
    o, l, ko, vo = oracle_verify_attn_window(*args, kv["v_new"], window, sinks, parent=parent)
    a = oracle_verify_attn_window(*args[:2], np.abs(kv["v_cache"]), *args[3:],
                                  np.abs(kv["v_new"]), window, sinks, parent=parent)[0]
    err = np.abs(out.double().cpu().numpy() - o)
    tol = 2.0 ** -8 * 1.02 * (a + np.abs(o)) + 2.0 ** -16 if dt == BF else 1e-4
    assert np.all(err <= tol), float((err / tol).max())
    assert np.max(np.abs(lse.cpu().numpy() - l)) <= 1e-4
    kc[torch.from_numpy(free).cuda()] = 0
    vc[torch.from_numpy(free).cuda()] = 0
    ko[free] = vo[free] = 0
    assert np.array_equal(kc.float().cpu().numpy(), ko.astype(np.float32))
    assert np.array_equal(vc.float().cpu().numpy(), vo.astype(np.float32))


CTX = [0, 1, 15, 16, 63, 64, 65, 200, 333, 1000]
WINDOWS = [(1, 0), (1, 1), (5, 0), (16, 4), (17, 16), (63, 70), (64, 0), (65, 20), (130, 200),
           (400, 1), (5000, 3)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("impl", [sv.ATTN_TENSOR_CORES, sv.ATTN_CUDA_CORES])
def test_window_bf16(window, sinks, tree, impl):
    wl = workload("chain_gqa_128k").scaled(gamma=8, Hq=6, Hkv=2)
    window_case(wl, CTX, window, sinks, tree, seed=window + sinks, impl=impl)


@pytest.mark.parametrize("gamma,Hq,Hkv", [(0, 8, 1), (0, 1, 1), (127, 2, 2), (63, 4, 2), (30, 4, 1),
                                          (69, 1, 1)])
@pytest.mark.parametrize("window,sinks", [(20, 3), (100, 80)])
def test_window_shapes(gamma, Hq, Hkv, window, sinks):
    wl = workload("chain_gqa_128k").scaled(gamma=gamma, Hq=Hq, Hkv=Hkv)
    for tree in (False, True):
        window_case(wl, [3, 70, 500, 129], window, sinks, tree, seed=gamma, impl=sv.ATTN_TENSOR_CORES)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (33, 31), (32, 64), (500, 5), (100, 0)])
def test_window_fp32(D, window, sinks):
    wl = workload("tiny_chain").scaled(gamma=9, Hq=6, Hkv=3, D=D)
    for tree in (False, True):
        window_case(wl, CTX, window, sinks, tree, seed=D, impl=0)


def test_window_long_contexts_split_over_ctas():
    wl = workload("chain_gqa_128k").scaled(gamma=3, Hq=8, Hkv=2)
    window_case(wl, [9000, 20, 12345, 4097], 4096, 100, False, seed=3, impl=sv.ATTN_TENSOR_CORES)
    window_case(wl, [9000, 20, 12345, 4097], 4096, 100, True, seed=4, impl=sv.ATTN_CUDA_CORES)


@pytest.mark.parametrize("impl", [sv.ATTN_TENSOR_CORES, sv.ATTN_CUDA_CORES])
def test_window_of_everything_equals_verify_attn(impl):
    """The same terms, over other ranges of keys: each probability is rounded
    to bf16 relative to another running maximum (2^-8 of sum p |v| on either
    side), and the outputs are rounded once each (2^-8 of the value)."""
    wl = workload("chain_gqa_128k").scaled(gamma=6)
    kv = kv_inputs_host(wl, seed=5, B=3, ctx=np.array([0, 700, 3333]))
    parent = np.stack([random_tree(np.random.default_rng(s), 4, 3, 7) for s in range(3)])
    dims = sv.make_dims(B=3, M=7, Hq=wl.Hq, Hkv=wl.Hkv, D=128, max_blocks=kv["max_blocks"],
                        num_blocks=kv["num_blocks"], attn_impl=impl)
    ws = sv.workspace(dims)
    res = []
    size = []
    for kw in (None, {}, dict(window=3340), dict(window=2 ** 31 - 1, sinks=2 ** 31 - 1)):
        vn, vc = (kv[k] if kw is not None else np.abs(kv[k]) for k in ("v_new", "v_cache"))
        for par in (None, to_dev(parent, I32)):
            q = to_dev(kv["q"], BF)
            out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
            sv.spec_verify_attn(q, to_dev(kv["k_new"], BF), to_dev(vn, BF),
                                to_dev(kv["k_cache"], BF), to_dev(vc, BF),
                                to_dev(kv["block_table"], I32), to_dev(kv["ctx_lens"], I32), par,
                                out, lse, dims, ws, **(kw or {}))
            (size if kw is None else res).append((out, lse))
    for i in (2, 4):
        for j in (0, 1):
            o, r, a = res[i + j][0].float(), res[j][0].float(), size[j][0].float() * (1 + 2.0 ** -6)
            assert torch.all((o - r).abs() <= 2 * 2.0 ** -8 * (a + r.abs()) * 1.01)
            assert torch.all((res[i + j][1] - res[j][1]).abs() <= 1e-5)


def test_window_failed_requests():
    wl = workload("chain_gqa_128k").scaled(gamma=2, Hq=4, Hkv=2)
    kv = kv_inputs_host(wl, seed=6, B=3, ctx=np.array([100, 200, 150]))
    kv["block_table"][1, 10] = -1  # inside the window
    for impl in (sv.ATTN_TENSOR_CORES, sv.ATTN_CUDA_CORES):
        dims = sv.make_dims(B=3, M=3, Hq=4, Hkv=2, D=128, max_blocks=kv["max_blocks"],
                            num_blocks=kv["num_blocks"], attn_impl=impl)
        ws = sv.workspace(dims)
        ctx = np.array([100, 200, kv["max_blocks"] * 16 - 2])
        kc, vc = to_dev(kv["k_cache"], BF), to_dev(kv["v_cache"], BF)
        q = to_dev(kv["q"], BF)
        out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:3], 9.0, device="cuda")
        sv.spec_verify_attn(q, to_dev(kv["k_new"], BF), to_dev(kv["v_new"], BF), kc, vc,
                            to_dev(kv["block_table"], I32), to_dev(ctx, I32), None, out, lse, dims,
                            ws, window=64, sinks=2)
        assert sv.device_status(ws) == (1 << 6 | 1 << 2)
        assert torch.all(out[1:] == 0) and torch.all(lse[1:] == -math.inf)
        assert torch.isfinite(lse[0]).all()


# -------------------------------------------------------------------- sampling

def sample_gpu(x, T, u, k=None, p=None, mp=None, dt=F32, ws=None):
    n = x.shape[0]
    x = x if torch.is_tensor(x) else to_dev(x, dt)
    tok = torch.full((n,), -9, dtype=I32, device="cuda")
    prob = torch.full((n,), -9.0, device="cuda")
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda") if ws is None else ws
    f = lambda a: None if a is None else to_dev(np.asarray(a), F32)  # noqa: E731
    sv.spec_sample(x, f(T), f(u), tok, prob, ws, top_k=None if k is None else to_dev(k, I32),
                   top_p=f(p), min_p=f(mp))
    return tok.cpu().numpy(), prob.cpu().numpy(), sv.device_status(ws)


def sample_check(x, T, u, k=None, p=None, mp=None, dt=F32, clear=1e-9):
    f32 = lambda a: None if a is None else np.asarray(a, np.float32)  # noqa: E731
    T, u, p, mp = f32(T), f32(u), f32(p), f32(mp)
    xd = to_dev(x, dt)
    tok, prob, status = sample_gpu(xd, T, u, k, p, mp)
    ref = oracle_sample(xd.double().cpu().numpy(), T, u, k, p, mp)
    sure = ref["margin"] > clear
    assert np.array_equal(tok[sure], ref["tokens"][sure])
    assert np.all(np.abs(prob[sure] - ref["prob"][sure]) <= 2.0 ** -22 * ref["prob"][sure] + 1e-37)
    assert status == np.bitwise_or.reduce(np.where(ref["status"] > 0, 1 << ref["status"], 0))
    return ref, sure


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [1, 2, 7, 100, 1023, 4096, 32001, 128256, 152064])
def test_sample_filters(V, dt):
    rng = np.random.default_rng(V)
    n = 48 if V < 100000 else 24
    x = rng.standard_normal((n, V)).astype(np.float32) * rng.choice([0.3, 1, 3, 8], (n, 1))
    on = rng.random((3, n)) < 0.5
    k = np.where(on[0], rng.choice([1, 2, 50, 600, 5000, 10 ** 9], n), 0)
    p = np.where(on[1], rng.choice([1e-6, 0.3, 0.9, 0.99, 0.9999], n), 1.0)
    mp = np.where(on[2], rng.choice([1e-8, 0.01, 0.5, 1.0], n), 0.0)
    T = rng.choice([0.0, 0.3, 1.0, 5.0], n)
    u = rng.integers(0, 1 << 24, n) / (1 << 24)
    u[:2] = (0.0, 1 - 2.0 ** -24)
    _, sure = sample_check(x, T, u, k, p, mp, dt)
    assert sure.mean() > 0.7
    sample_check(x, T, u, dt=dt)                 # temperature alone
    sample_check(x, T, u, p=p, dt=dt)
    sample_check(x, T, u, k=k, dt=dt)
    sample_check(x, T, u, mp=mp, dt=dt)


def test_sample_largest_vocabulary():
    rng = np.random.default_rng(5)
    V = 1 << 20
    x = rng.standard_normal((3, V)).astype(np.float32) * 2
    for dt in (BF, F32):
        sample_check(x, [1.0, 0.5, 0.0], [0.25, 0.75, 0.5], [0, 3000, 0], [0.8, 0.9, 1.0], None, dt)


@pytest.mark.parametrize("dt", [BF, F32])
def test_sample_ties_and_masks(dt):
    """Rows of few values: the cut falls among equal logits.  Masked tokens
    (-inf, the lowest finite value) are not drawn."""
    rng = np.random.default_rng(6)
    n, V = 40, 5000
    x = rng.integers(-3, 4, (n, V)).astype(np.float32) / 2
    x[0:4] = 1.25                        # one value
    x[4:8, rng.permutation(V)[:4000]] = -np.inf
    low = float(torch.finfo(dt).min)
    x[8:12, rng.permutation(V)[:4990]] = low
    x[12] = -np.inf
    x[12, 77] = -5.0                     # a single token
    x[13] = low                          # the lowest value everywhere: uniform
    x[14] = np.where(rng.random(V) < 0.5, 0.0, -0.0)  # zeros of both signs are ties
    k = rng.choice([0, 1, 3, 500, 4999, 5000], n)
    p = rng.choice([1.0, 0.5, 0.999], n)
    mp = rng.choice([0.0, 0.05, 1.0], n)
    T = rng.choice([0.0, 0.7, 1.0], n)
    u = (rng.integers(0, 1 << 20, n) + 0.5) / (1 << 20)
    ref, sure = sample_check(x, T, u, k, p, mp, dt)
    assert sure.mean() > 0.8 and np.all(ref["tokens"] >= 0)
    sample_check(x, T, u, k=k, dt=dt)
    sample_check(x, T, u, p=p, dt=dt)


def test_sample_failed_rows():
    V = 3000
    x = np.random.default_rng(7).standard_normal((12, V)).astype(np.float32)
    x[0, 2999], x[1, 5], x[2] = np.nan, np.inf, -np.inf
    T, u = np.ones(12), np.full(12, 0.5)
    k, p, mp = np.zeros(12, int), np.ones(12), np.zeros(12)
    T[3], T[4], T[5] = -1.0, np.nan, np.inf
    u[6], u[7] = 1.0, np.nan
    k[8], p[9], mp[10] = -1, 0.0, 1.5
    for dt in (BF, F32):
        ref, _ = sample_check(x, T, u, k, p, mp, dt)
        assert np.array_equal(ref["tokens"] == -1, np.arange(12) < 11)


@pytest.mark.parametrize("dt", [BF, F32])
def test_sample_views_and_repeats(dt):
    """Rows at any element of memory and any stride; two runs are equal bit
    for bit, also captured, and rows do not depend on their batch."""
    rng = np.random.default_rng(8)
    n, V = 9, 20011
    base = to_dev(rng.standard_normal((n, V + 13)) * 3, dt)
    T, u = rng.uniform(0.5, 1.5, n), rng.random(n).astype(np.float32)
    k, p = rng.choice([0, 40], n), rng.choice([0.9, 1.0], n)
    for off in (0, 1, 5, 8):
        x = base[:, off:off + V]
        a = sample_gpu(x, T, u, k, p)
        b = sample_gpu(x.contiguous(), T, u, k, p)
        assert np.array_equal(a[0], b[0]) and np.allclose(a[1], b[1], rtol=1e-6)
        again = sample_gpu(x, T, u, k, p)
        assert np.array_equal(a[0], again[0]) and np.array_equal(a[1], again[1])
        one = sample_gpu(x[4:5], T[4:5], u[4:5], k[4:5], p[4:5])
        assert one[0][0] == a[0][4] and one[1][0] == a[1][4]
    x = base[:, :V]
    tok, prob = torch.zeros(n, dtype=I32, device="cuda"), torch.zeros(n, device="cuda")
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    Td, ud, kd, pd = to_dev(T, F32), to_dev(u, F32), to_dev(k, I32), to_dev(p, F32)
    sv.spec_sample(x, Td, ud, tok, prob, ws, top_k=kd, top_p=pd)
    first = tok.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_sample(x, Td, ud, tok, prob, ws, top_k=kd, top_p=pd)
    tok.zero_()
    g.replay()
    assert torch.equal(tok, first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    tok.zero_()
    torch.cuda.synchronize()
    sv.spec_sample(x, Td, ud, tok, prob, ws, top_k=kd, top_p=pd, stream=s)
    s.synchronize()
    assert torch.equal(tok, first)


# ------------------------------------------------------------- the step's loop

def test_serving_loop_with_a_window():
    """Prefill, then verify steps: tables -> norm and rotation -> windowed
    attention -> decisions -> commit, tokens and caches checked against the
    oracles at every step; a request ends and another takes its place."""
    rng = np.random.default_rng(9)
    B, M, Hq, Hkv, D, V, W, S = 3, 4, 4, 2, 128, 500, 40, 5
    mb, nb = 16, 14
    f = 10000.0 ** (-np.arange(64) / 64)
    inv = to_dev(f, torch.float64)
    wq, wk = (to_dev(rng.uniform(0.5, 1.5, D), BF) for _ in range(2))
    dims = sv.make_dims(B=B, M=M, Hq=Hq, Hkv=Hkv, D=D, max_blocks=mb, num_blocks=nb, V=V)
    ws = sv.workspace(dims)
    d = dict(table=torch.full((B, mb), -1, dtype=I32, device="cuda"),
             span=torch.zeros(B, 2, dtype=I32, device="cuda"),
             pool=torch.arange(nb, dtype=I32, device="cuda"),
             state=torch.tensor([0, nb], dtype=I32, device="cuda"))
    h = dict(block_table=d["table"].cpu().numpy(), span=d["span"].cpu().numpy(),
             pool=d["pool"].cpu().numpy(), pool_state=d["state"].cpu().numpy())
    kc = torch.zeros(nb, Hkv, 16, D, device="cuda", dtype=BF)
    vc = torch.zeros_like(kc)
    ctx = torch.tensor([0, 0, -1], dtype=I32, device="cuda")

    def tables(n, rows):
        start = None if n is None else np.concatenate([[0], np.cumsum(n)])
        slots = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
        pos = torch.full((rows,), -1, dtype=I32, device="cuda")
        ok = torch.zeros(B, dtype=I32, device="cuda")
        sv.spec_block_tables(ctx, None if n is None else to_dev(start, I32), None, d["table"],
                             d["span"], d["pool"], d["state"], slots, pos, ok, dims, ws, window=W,
                             sinks=S)
        ref = oracle_block_tables(ctx.cpu().numpy(), start, None, rows, h["block_table"], h["span"],
                                  h["pool"], h["pool_state"], np.full(rows, -1), np.full(rows, -1),
                                  M, window=W, sinks=S)
        for k, t in (("block_table", "table"), ("span", "span"), ("pool", "pool"),
                     ("pool_state", "state")):
            assert np.array_equal(d[t].cpu().numpy(), ref[k])
            h[k] = ref[k].astype(np.int32)
        assert np.array_equal(slots.cpu().numpy(), ref["slots"])
        assert np.array_equal(ok.cpu().numpy(), ref["ok"])
        return slots, pos, ref["ok"]

    def qkv(rows):
        x = to_dev(rng.standard_normal((rows, Hq + 2 * Hkv, D)), BF)
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]

    def prefill(n):
        nonlocal ctx
        rows = int(sum(n)) + 3
        slots, pos, ok = tables(n, rows)
        q, k, v = qkv(rows)
        qo = torch.empty(rows, Hq, D, device="cuda", dtype=BF)
        ko = torch.empty(rows, Hkv, D, device="cuda", dtype=BF)
        sv.spec_qk_norm_rope(q, k, v, wq, wk, pos, inv, qo, ko, dims, ws, slots=slots, k_cache=kc,
                             v_cache=vc)
        rope_check(ko, k.double().cpu().numpy(), wk.double().cpu().numpy(), pos.cpu().numpy(), f,
                   False, BF)
        ctx = ctx + to_dev(np.where(ok > 0, n, 0), I32)

    prefill([37, 90, 0])
    for step in range(8):
        if step == 3:
            ctx[0] = -1                   # a request ends,
        if step == 5:
            ctx[0], ctx[2] = 0, 0         # two begin
            n = [21, 0, 50]
            prefill(n)
        slots, pos, ok = tables(None, B * M)
        q, k, v = qkv(B * M)
        qo = torch.empty(B * M, Hq, D, device="cuda", dtype=BF)
        ko = torch.empty(B * M, Hkv, D, device="cuda", dtype=BF)
        sv.spec_qk_norm_rope(q, k, v, wq, wk, pos, inv, qo, ko, dims, ws)
        out = torch.empty(B, M, Hq, D, device="cuda", dtype=BF)
        lse = torch.empty(B, M, Hq, device="cuda")
        before = kc.double().cpu().numpy(), vc.double().cpu().numpy()
        vn = v.contiguous().view(B, M, Hkv, D)
        run = torch.where(to_dev(ok, I32) > 0, ctx, -1)  # places without a request do not run
        sv.spec_verify_attn(qo.view(B, M, Hq, D), ko.view(B, M, Hkv, D), vn, kc, vc, d["table"], run,
                            None, out, lse, dims, ws, window=W, sinks=S)
        live = np.nonzero(ok)[0]
        np64 = lambda t: t.double().cpu().numpy()[live]  # noqa: E731
        o, _, _, _ = oracle_verify_attn_window(
            np64(qo.view(B, M, Hq, D)), *before, h["block_table"][live], ctx.cpu().numpy()[live],
            np64(ko.view(B, M, Hkv, D)), np64(vn), W, S)
        assert np.all(np.abs(np64(out) - o) <= 2e-2 + 1e-2 * np.abs(o))
        # decisions on the verify rows, a bonus token each, then the commit
        tl = rng.standard_normal((B, M, V)).astype(np.float32) * 2
        dl = (tl + rng.standard_normal((B, M, V)) * 0.3).astype(np.float32)
        # the draft's tokens come from the sampling call
        T, u = np.full(B * M, 0.9, np.float32), rng.random(B * M).astype(np.float32)
        dl_d = to_dev(dl, BF)
        drafted = sample_gpu(dl_d.view(B * M, V), T, u)[0].reshape(B, M)
        tokens = np.zeros((B, M), np.int64)
        tokens[:, 1:] = drafted[:, :-1]   # node n's token comes from row n - 1
        path = torch.empty(B, M, dtype=I32, device="cuda")
        toks = torch.empty(B, M, dtype=I32, device="cuda")
        acc = torch.empty(B, dtype=I32, device="cuda")
        sv.spec_reject_sample(to_dev(tl, BF), dl_d, to_dev(tokens, I32), None,
                              to_dev(np.full(B, 0.9), F32), 11, step, toks, path, acc, None, dims, ws)
        ref = oracle_reject_sample(to_dev(tl, BF).float().cpu().numpy(), dl_d.float().cpu().numpy(),
                                   tokens, None, np.full(B, 0.9, np.float32), 11, step)
        clear = ref["acc_margin"] >= 1e-6
        assert np.array_equal(acc.cpu().numpy()[clear], ref["accepted_len"][clear])
        acc = torch.where(to_dev(ok, I32) > 0, acc, -1)  # no commit where nothing ran
        old = ctx.cpu().numpy()
        sv.kv_commit(kc, vc, d["table"], ctx, ctx, path, acc, dims, ws)
        _, _, new = oracle_kv_commit(kc.float().cpu().numpy(), vc.float().cpu().numpy(),
                                     h["block_table"], old, path.cpu().numpy(), acc.cpu().numpy())
        assert np.array_equal(ctx.cpu().numpy(), new)
        sv.device_status(ws)  # places that do not run raise their bits
    assert int(ctx[1]) > 95 and h["pool_state"][1] > 0
