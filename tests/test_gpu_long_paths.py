"""The forms of the attention on views, by the path that each size takes: a shared prefix
in a pass of its own or read by the requests, few pairs merged by a kernel of their own.
Every case says how many launches its path has (spec_verify_attn returns the count), so a
rule that sends it another way is noticed.

A plain attention in fp64 on the GPU is the reference (it agrees with the CPU oracle, see
the first test).  Tolerances as in test_gpu_long.py."""
import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import speculative_decoding_verification_19_gb300 as sv  # noqa: E402
from harness import to_dev  # noqa: E402
from oracle import oracle_kv_append, oracle_verify_attn, oracle_verify_attn_pages  # noqa: E402
from test_gpu_long import AUTO, BF, CORES, F32, I32, TC, Step, choose  # noqa: E402

PASS, REQUESTS, GATHERED, CORES_SPLIT = 4, 2, 3, 3  # launches


def tree(rng, B, M, width):
    """Trees whose nodes hang from one of the `width` nodes before them."""
    n = np.arange(M)
    parent = np.maximum(0, n - 1 - rng.integers(0, width, (B, M)))
    parent[:, 0] = -1
    return parent


def attention64(st, pages=None, counts=None):
    """((out, lse, caches), the outputs' sums of p |v|), all numpy fp64."""
    f = lambda x: to_dev(x, torch.float64)  # noqa: E731
    q, kn, vn, k, v = (f(x) for x in (st.q, st.kn, st.vn, st.k, st.v))
    M, Hkv, D, group = st.M, st.Hkv, st.D, st.Hq // st.Hkv
    anc = np.tril(np.ones((st.B, M, M), bool))
    if st.parent is not None:
        anc = np.zeros((st.B, M, M), bool)
        for b in range(st.B):
            for i in range(M):
                if st.parent[b, i] >= 0:
                    anc[b, i] = anc[b, st.parent[b, i]]
                anc[b, i, i] = True
    out, lse, size = (torch.empty(*s, dtype=torch.float64, device="cuda")
                      for s in (q.shape, q.shape[:3], q.shape))
    for b in range(st.B):
        c = int(st.ctx[b])
        for h in range(Hkv):
            t = np.arange(c)
            if pages is not None:
                t = np.concatenate([(pages[b, h, :counts[b], None] * 16 + np.arange(16)).ravel(),
                                    np.arange(c // 16 * 16, c)]).astype(np.int64)
            blk, at = to_dev(st.table[b, t // 16], torch.int64), to_dev(t % 16, torch.int64)
            K = torch.cat([k[blk, h, at], kn[b, :, h]])
            V = torch.cat([v[blk, h, at], vn[b, :, h]])
            rows = q[b, :, h * group:(h + 1) * group]
            s = rows.reshape(-1, D) @ K.T / D ** 0.5
            hide = np.concatenate([np.zeros((M, len(t)), bool), ~anc[b]], 1).repeat(group, 0)
            s[to_dev(hide, torch.bool)] = -float("inf")
            p = torch.softmax(s, 1)
            where = (b, slice(None), slice(h * group, (h + 1) * group))
            out[where] = (p @ V).reshape(M, group, D)
            size[where] = (p @ V.abs()).reshape(M, group, D)
            lse[where] = torch.logsumexp(s, 1).reshape(M, group)
    kc, vc = oracle_kv_append(st.k, st.v, st.table, st.ctx, st.kn, st.vn)
    return (out.cpu().numpy(), lse.cpu().numpy(), kc, vc), size.cpu().numpy()


def run(st, launches, ref, size, **kw):
    q = to_dev(st.q, st.dt)
    st.out = torch.full_like(q, float("nan"))
    st.lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    n = sv.spec_verify_attn(q, to_dev(st.kn, st.dt), to_dev(st.vn, st.dt), st.kc, st.vc,
                            to_dev(st.table, I32), to_dev(st.ctx, I32),
                            None if st.parent is None else to_dev(st.parent, I32), st.out, st.lse,
                            st.dims, st.ws, **kw)
    assert sv.device_status(st.ws) == 0
    st.check(ref, size)
    st.check_cache(ref)
    assert n == launches


def test_the_reference_agrees_with_the_oracle():
    st = Step([70, 33], 5, 6, 2, 64, F32, 1)
    st.parent = tree(st.rng, 2, 5, 3)
    args = (st.q, st.k, st.v, st.table, st.ctx, st.kn, st.vn)
    lists, cnt = choose(st.rng, st.ctx, 2, 3)
    for got, want in ((attention64(st), oracle_verify_attn(*args, parent=st.parent)),
                      (attention64(st, lists, cnt),
                       oracle_verify_attn_pages(*args, lists, cnt, parent=st.parent))):
        for x, y in zip(got[0], want):
            assert np.allclose(x, y, rtol=1e-12, atol=1e-12)


PREFIX = [  # B, P, own positions to, M, Hq, Hkv, D, dt, tree's width, impl, launches
    # a pass on tensor cores, the own keys of up to 128 rows per KV head there too
    (52, 8000, 90, 128, 2, 2, 128, BF, 3, TC, PASS),    # 128 rows, masks of two words
    (52, 8000, 90, 64, 4, 2, 128, BF, 1, TC, PASS),     # 128 rows, masks of one
    (40, 8000, 200, 33, 6, 2, 128, BF, 4, TC, PASS),    # 99 rows
    (34, 6000, 40, 65, 3, 3, 128, BF, 9, TC, PASS),     # 65 rows, masks of two words
    (47, 6000, 40, 100, 4, 4, 128, BF, 0, TC, PASS),    # chains of 100
    (48, 9600, 70, 25, 10, 2, 128, BF, 2, TC, PASS),    # 125 rows, groups of five
    (24, 6000, 1500, 5, 21, 3, 128, BF, 2, TC, PASS),   # groups of seven, long own parts
    (60, 3200, 60, 9, 8, 8, 128, BF, 3, TC, PASS),      # one row of queries a head
    (13, 12816, 33, 1, 8, 8, 128, BF, 0, TC, PASS),     # single tokens
    # heads of 64: the pass on tensor cores, the rest on CUDA cores
    (30, 1616, 60, 128, 2, 2, 64, BF, 3, AUTO, PASS), (9, 3200, 500, 16, 14, 2, 64, BF, 4, AUTO, PASS),
    (40, 1616, 60, 1, 8, 8, 64, BF, 0, AUTO, PASS),
    # CUDA cores alone
    (30, 1616, 60, 128, 2, 2, 64, F32, 3, AUTO, PASS), (30, 1616, 60, 33, 6, 2, 128, BF, 3, CORES, PASS),
    (40, 1040, 60, 5, 8, 8, 128, F32, 2, AUTO, PASS), (40, 1040, 60, 1, 8, 8, 64, F32, 0, AUTO, PASS),
    # read by the requests
    (30, 1040, 90, 128, 2, 2, 128, BF, 3, TC, REQUESTS), (30, 1040, 90, 33, 6, 2, 128, BF, 4, TC, REQUESTS),
    (2, 8000, 90, 65, 2, 2, 128, BF, 9, TC, GATHERED), (1, 16000, 40, 4, 8, 2, 128, BF, 0, TC, GATHERED),
    (4, 512, 60, 5, 4, 2, 64, BF, 2, AUTO, CORES_SPLIT), (4, 512, 60, 65, 2, 2, 64, F32, 3, AUTO, CORES_SPLIT),
    (3, 512, 60, 33, 6, 2, 128, BF, 3, CORES, CORES_SPLIT)]


@pytest.mark.parametrize("B,P,own,M,Hq,Hkv,D,dt,width,impl,launches", PREFIX)
def test_prefix_by_path(B, P, own, M, Hq, Hkv, D, dt, width, impl, launches):
    rng = np.random.default_rng(M)
    ctx = P + rng.integers(0, own + 1, B)
    ctx[0] = P  # no key of its own
    st = Step(ctx, M, Hq, Hkv, D, dt, P + M, shared=P // 16, impl=impl)
    st.parent = tree(rng, B, M, width) if width else None
    ref, size = attention64(st)
    run(st, launches, ref, size, prefix=to_dev(st.shared, I32))


PAGES = [  # B, contexts to, pages, M, Hq, Hkv, D, dt, tree's width, impl, launches
    (2, 9000, 300, 128, 2, 2, 128, BF, 3, TC, GATHERED), (1, 9000, 500, 65, 1, 1, 128, BF, 9, TC, GATHERED),
    (3, 5000, 100, 9, 14, 2, 128, BF, 2, TC, GATHERED), (1, 3000, 40, 33, 3, 1, 128, BF, 4, TC, GATHERED),
    (20, 9000, 100, 128, 4, 4, 128, BF, 3, TC, REQUESTS), (70, 3000, 40, 25, 5, 1, 128, BF, 2, TC, REQUESTS),
    (30, 3000, 3, 1, 16, 8, 128, BF, 0, TC, REQUESTS), (2, 300, 1, 2, 2, 1, 128, BF, 0, TC, REQUESTS),
    (3, 9000, 300, 128, 2, 2, 64, BF, 3, AUTO, CORES_SPLIT),
    (20, 9000, 200, 16, 16, 2, 64, BF, 4, AUTO, CORES_SPLIT),
    (1, 30000, 1500, 1, 8, 1, 64, BF, 0, AUTO, CORES_SPLIT),
    (9, 5000, 100, 33, 3, 1, 64, F32, 3, AUTO, CORES_SPLIT),
    (2, 9000, 300, 128, 2, 2, 128, F32, 3, AUTO, CORES_SPLIT)]


@pytest.mark.parametrize("B,most,n,M,Hq,Hkv,D,dt,width,impl,launches", PAGES)
def test_pages_by_path(B, most, n, M, Hq, Hkv, D, dt, width, impl, launches):
    rng = np.random.default_rng(M)
    ctx = rng.integers(0, most + 1, B)
    ctx[0] = most
    st = Step(ctx, M, Hq, Hkv, D, dt, n + M, impl=impl)
    st.parent = tree(rng, B, M, width) if width else None
    lists, cnt = choose(rng, st.ctx, Hkv, n)
    ref, size = attention64(st, lists, cnt)
    run(st, launches, ref, size, pages=to_dev(lists, I32), page_counts=to_dev(cnt, I32))


@pytest.mark.parametrize("dt,D,impl", [(BF, 128, TC), (BF, 64, AUTO), (F32, 128, AUTO)])
def test_scores_that_grow_along_the_prefix(dt, D, impl):
    """Scores that grow far along the prefix, in a pass of its own.  A score's sum of D
    products and its scaling are off by at most (D + 2) 2^-24 of the sum of their absolute
    values (S below, at most over the keys); a log-sum-exp by that, by its sums (a term is
    added to at most some 200 partial sums, each off by 2^-24) and by 2^-21 of the
    exponentials; an output's weights by twice as much, relatively."""
    P, B, M = 3216, 64, 4
    st = Step([P + b for b in range(B)], M, 8, 2, D, dt, 5, shared=P // 16, impl=impl)
    f = lambda x: torch.from_numpy(np.asarray(x, np.float32)).to(dt).double().numpy()  # noqa: E731
    lift = np.zeros((st.nb, 2, 16, 1))
    for j, blk in enumerate(st.shared):
        lift[blk] = (16 * j + np.arange(16)[:, None]) / P
    sign = np.sign(st.q[0, 0, ::4])  # of the first query head of a KV head
    st.k = f(st.k * 0.1 + lift * 6.0 * sign[None, :, None, :])
    st.q = f(st.q * 0.3 + 0.7 * sign.repeat(4, 0))
    st.q[3, 1, 5] = 0
    st.kc = to_dev(st.k, dt)
    ref, size = attention64(st)
    top = np.abs(st.k).max((0, 2)), np.abs(st.kn).max((0, 1))  # [Hkv, D]
    S = (np.abs(st.q) * np.maximum(*top).repeat(4, 0)).sum(-1).max() / D ** 0.5
    d = (D + 2) * 2.0 ** -24 * S + 200 * 2.0 ** -24 + 2.0 ** -21
    st.out = torch.full(st.q.shape, float("nan"), dtype=dt, device="cuda")
    st.lse = torch.full(st.q.shape[:3], float("nan"), device="cuda")
    n = sv.spec_verify_attn(to_dev(st.q, dt), to_dev(st.kn, dt), to_dev(st.vn, dt), st.kc, st.vc,
                            to_dev(st.table, I32), to_dev(st.ctx, I32), None, st.out, st.lse,
                            st.dims, st.ws, prefix=to_dev(st.shared, I32))
    assert n == PASS and sv.device_status(st.ws) == 0
    assert ref[1].max() > 30
    assert np.max(np.abs(st.lse.cpu().numpy() - ref[1])) <= d + 2.0 ** -24 * np.abs(ref[1]).max()
    err = np.abs(st.out.double().cpu().numpy() - ref[0])
    tol = 2 * d * size + 2.0 ** -20
    if dt == BF:  # the probabilities' rounding, and the output's
        tol += 2.0 ** -8 * 1.02 * (size + np.abs(ref[0]))
    assert np.all(err <= tol), float((err / tol).max())
