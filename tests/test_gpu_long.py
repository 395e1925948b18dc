"""GPU parity of the operators over long caches against the CPU oracles: verify
attention behind a shared prefix and over selected pages, bounds and scores of
pages, and their selection; then all of them together in a decoding loop.

Tolerances.  Attention, bf16: the probabilities are rounded to bf16 before
their product with V, so an output is off by at most 2^-8 of sum p |v| (its
fp32 sums, weights and merges of partials by 2^-18 of it more), then rounded by
at most 2^-8 of itself; fp32: scores of 128 terms are off by at most
128 * 2^-24 * max|q||k| * scale < 2e-5 for standard normal data, outputs by about
twice that times max|v| < 5; a log-sum-exp by what its scores are off and 2^-22
of its terms.  Scores of pages: a sum of 2 D products of type-exact inputs in
fp32, so 2 D * 2^-24 of the sum of their absolute values.  Bounds and selections
are exact.
"""
import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import speculative_decoding_verification_19_gb300 as sv  # noqa: E402
from harness import to_dev  # noqa: E402
from oracle import (oracle_kv_commit, oracle_page_bounds, oracle_page_score,  # noqa: E402
                    oracle_page_select, oracle_verify_attn, oracle_verify_attn_pages,
                    oracle_verify_attn_prefix)
from synth import random_tree  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
AUTO, CORES, TC = sv.ATTN_AUTO, sv.ATTN_CUDA_CORES, sv.ATTN_TENSOR_CORES
INVALID, CAPACITY, NONFINITE, BAD_ID = (1 << c for c in (1, 2, 5, 6))


def typed(x, dt):
    """x as numpy fp64 with values of type dt."""
    return torch.from_numpy(np.asarray(x)).to(dt).double().numpy()


class Step:
    """One step's inputs on both sides.  Free blocks hold NaN on the GPU."""

    def __init__(self, ctx, M, Hq, Hkv, D, dt, seed, shared=0, tree=False, impl=0, spare=3,
                 extra_pages=0):
        rng = np.random.default_rng(seed)
        B = len(ctx)
        self.B, self.M, self.Hq, self.Hkv, self.D, self.dt = B, M, Hq, Hkv, D, dt
        self.ctx = np.array(ctx)
        pages = -(-(np.maximum(self.ctx, 0) + M) // 16)
        self.mb = int(pages.max()) + extra_pages
        own = int(np.maximum(0, pages - shared).sum())
        self.nb = own + shared + spare
        ids = rng.permutation(self.nb)
        self.shared = ids[own:own + shared]
        self.table = np.full((B, self.mb), -1, np.int64)
        at = 0
        for b in range(B):
            n = max(0, pages[b] - shared)
            self.table[b, :shared] = self.shared
            self.table[b, shared:shared + n] = ids[at:at + n]
            at += n
        n = lambda *s: typed(rng.standard_normal(s).astype(np.float32), dt)  # noqa: E731
        self.q, self.kn, self.vn = n(B, M, Hq, D), n(B, M, Hkv, D), n(B, M, Hkv, D)
        self.k, self.v = n(self.nb, Hkv, 16, D), n(self.nb, Hkv, 16, D)
        self.parent = (np.stack([random_tree(rng, max(1, M - 1), 2, M) for _ in range(B)])
                       if tree else None)
        self.dims = sv.make_dims(B=B, M=M, Hq=Hq, Hkv=Hkv, D=D, max_blocks=self.mb,
                                 num_blocks=self.nb, kv_dtype=dt, attn_impl=impl)
        self.ws = sv.workspace(self.dims)
        self.kc, self.vc = to_dev(self.k, dt), to_dev(self.v, dt)
        self.rng = rng

    def unused(self, held):
        """NaN in blocks that are not among `held` (ids)."""
        free = np.setdiff1d(np.arange(self.nb), held)
        self.free = torch.from_numpy(free).cuda()
        self.kc[self.free] = float("nan")
        self.vc[self.free] = float("nan")

    def call(self, table=None, ctx=None, **kw):
        q = to_dev(self.q, self.dt)
        self.out = torch.full_like(q, float("nan"))
        self.lse = torch.full(q.shape[:3], float("nan"), device="cuda")
        sv.spec_verify_attn(q, to_dev(self.kn, self.dt), to_dev(self.vn, self.dt), self.kc, self.vc,
                            to_dev(self.table if table is None else table, I32),
                            to_dev(self.ctx if ctx is None else ctx, I32),
                            None if self.parent is None else to_dev(self.parent, I32), self.out,
                            self.lse, self.dims, self.ws, **kw)
        return sv.device_status(self.ws)

    def check(self, ref, sizes, rows=slice(None)):
        o, l = ref[0][rows], ref[1][rows]
        err = np.abs(self.out.double().cpu().numpy()[rows] - o)
        a = sizes[rows]
        tol = 2.0 ** -8 * 1.02 * (a + np.abs(o)) + 2.0 ** -16 if self.dt == BF else 1e-4
        assert np.all(err <= tol), float((err / tol).max())
        assert np.max(np.abs(self.lse.cpu().numpy()[rows] - l)) <= 1e-4

    def check_cache(self, ref):
        for got, want in ((self.kc, ref[2]), (self.vc, ref[3])):
            got, want = got.clone(), to_dev(want, self.dt)
            if hasattr(self, "free"):
                assert torch.isnan(got[self.free]).all()
                got[self.free] = want[self.free] = 0
            assert torch.equal(got, want)


# ------------------------------------------------------------- shared prefix

def prefix_step(ctx, P, *a, **kw):
    st = Step(ctx, *a, shared=P // 16, **kw)
    dirty = st.table.copy()
    dirty[:, :P // 16] = st.rng.choice([-1, 1 << 30], (st.B, P // 16))
    st.unused(st.table[st.table >= 0])
    assert st.call(table=dirty, prefix=to_dev(st.shared, I32)) == 0
    args = (st.q, st.k, st.v, st.table, st.ctx, st.kn)
    ref = oracle_verify_attn_prefix(*args, st.vn, st.shared, parent=st.parent)
    size = oracle_verify_attn_prefix(*args[:2], np.abs(st.v), *args[3:], np.abs(st.vn), st.shared,
                                     parent=st.parent)[0]
    st.check(ref, size)
    st.check_cache(ref)
    return st


PREFIX = [  # ctx, P, M, Hq, Hkv, D, dt, tree, impl
    ([16], 16, 1, 1, 1, 128, BF, False, TC), ([16], 16, 1, 1, 1, 64, F32, False, CORES),
    ([48, 49, 63, 64], 48, 1, 8, 2, 128, BF, False, TC),
    ([130, 128, 300], 128, 5, 14, 2, 128, BF, False, TC),
    ([2000, 2001, 2100], 2000, 9, 8, 2, 128, BF, True, TC),
    ([4096] * 40, 4096, 2, 8, 1, 128, BF, False, TC),         # 640 rows of a head
    ([176, 190], 176, 128, 1, 1, 128, BF, True, TC),          # 128 new rows
    ([352, 380, 352], 352, 16, 16, 2, 128, BF, True, TC),     # 128 rows a KV head
    ([640, 700], 640, 33, 3, 1, 128, BF, False, TC),
    ([48, 49, 63, 64], 48, 1, 8, 2, 128, BF, False, CORES),
    ([2000, 2001, 2100], 2000, 9, 8, 2, 128, BF, True, CORES),
    ([80, 81], 80, 7, 3, 3, 64, BF, False, AUTO),
    ([80, 81], 80, 7, 3, 3, 64, BF, False, CORES),
    ([3008] * 3, 3008, 128, 1, 1, 64, BF, False, AUTO),       # a unit with one tile of rows
    ([1600, 1900, 1616], 1600, 16, 8, 2, 64, BF, True, AUTO),
    ([80, 95], 80, 3, 4, 2, 128, F32, False, AUTO),
    ([1040] * 9, 1040, 16, 2, 1, 128, F32, True, AUTO),
    ([2000, 2005, 2399], 2000, 16, 4, 4, 64, F32, True, AUTO),
    ([33 * 16], 33 * 16, 128, 1, 1, 64, F32, False, AUTO)]


@pytest.mark.parametrize("ctx,P,M,Hq,Hkv,D,dt,tree,impl", PREFIX)
def test_prefix(ctx, P, M, Hq, Hkv, D, dt, tree, impl):
    prefix_step(ctx, P, M, Hq, Hkv, D, dt, P + M, tree=tree, impl=impl)


@pytest.mark.parametrize("ctx,P,M,Hq,Hkv,D,dt,impl", [
    ([12800 + 7 * b for b in range(17)], 12800, 2, 14, 2, 128, BF, TC),     # one pass, 119 rows
    ([8208] * 50, 8208, 1, 8, 1, 128, BF, TC),                              # 400 rows of a head
    ([8000 + b for b in range(60)], 8000, 5, 1, 1, 128, BF, TC),            # a third unit's tile
    ([12816, 12817, 12830, 12900], 12816, 1, 8, 8, 128, BF, TC),            # four rows of a head
    ([14000, 14001, 14030, 14100], 14000, 1, 8, 8, 128, BF, TC),            # as many, a longer prefix
    ([64 + b % 20 for b in range(6500)], 64, 1, 1, 1, 128, BF, TC),         # less than a key tile
    ([4000 + 3 * b for b in range(3)], 4000, 40, 6, 2, 64, BF, AUTO),
    ([16400 + 3 * b for b in range(13)], 16400, 2, 3, 3, 128, F32, AUTO)])
def test_prefix_in_one_pass(ctx, P, M, Hq, Hkv, D, dt, impl):
    """Sizes at which the prefix is read once in a pass of its own."""
    prefix_step(ctx, P, M, Hq, Hkv, D, dt, 4, impl=impl)


@pytest.mark.parametrize("ctx,P,M,Hq,Hkv,D,dt,tree,impl", [
    ([3216 + 5 * b for b in range(24)], 3216, 40, 4, 2, 64, F32, True, AUTO),  # own keys in tiles
    ([1616 + b for b in range(30)], 1616, 3, 9, 3, 128, BF, False, CORES),     # 270 rows of a head
    ([1008 + b % 3 for b in range(40)], 1008, 1, 8, 8, 64, BF, False, CORES),  # a last tile of 48
    ([1040 + 9 * b for b in range(40)], 1040, 33, 2, 2, 128, F32, True, AUTO),
    ([48 + b % 20 for b in range(8200)], 48, 1, 1, 1, 64, F32, False, AUTO)])  # less than a tile
def test_prefix_in_one_pass_on_cuda_cores(ctx, P, M, Hq, Hkv, D, dt, tree, impl):
    prefix_step(ctx, P, M, Hq, Hkv, D, dt, 6, tree=tree, impl=impl)


@pytest.mark.parametrize("impl", [CORES, TC])
def test_prefix_batches_of_many_rows(impl):
    """257 requests, rows that fill tiles unevenly."""
    prefix_step([64 + b % 37 for b in range(257)], 64, 3, 1, 1, 128, BF, 3, impl=impl)


@pytest.mark.parametrize("dt,D,impl", [(BF, 128, TC), (BF, 128, CORES), (F32, 64, AUTO)])
def test_prefix_requests_that_fail(dt, D, impl):
    P = 64
    st = Step([70, 64, 80, 100], 4, 4, 2, D, dt, 9, shared=4, impl=impl, extra_pages=1)
    ctx = np.array([70, 63, -1, 16 * st.mb - 3])  # fine; shorter than the prefix; ended; no room
    before = (st.kc.clone(), st.vc.clone())
    assert st.call(ctx=ctx, prefix=to_dev(st.shared, I32)) == INVALID | CAPACITY
    assert torch.all(st.out[1:] == 0) and torch.all(st.lse[1:] == -float("inf"))
    only = [slice(0, 1)]
    ref = oracle_verify_attn_prefix(st.q[:1], st.k, st.v, st.table[:1], ctx[:1], st.kn[:1],
                                    st.vn[:1], st.shared)
    size = oracle_verify_attn_prefix(st.q[:1], st.k, np.abs(st.v), st.table[:1], ctx[:1],
                                     st.kn[:1], np.abs(st.vn[:1]), st.shared)[0]
    st.check(ref, size, only[0])
    st.check_cache(ref)
    # an entry of the shared table that is no block: nobody runs, nothing is written
    for bad in (-1, st.nb, 2 ** 31 - 1):
        st.kc.copy_(before[0])
        st.vc.copy_(before[1])
        shared = st.shared.copy()
        shared[2] = bad
        assert st.call(prefix=to_dev(shared, I32)) == BAD_ID
        assert torch.all(st.out == 0) and torch.all(st.lse == -float("inf"))
        assert torch.equal(st.kc, before[0]) and torch.equal(st.vc, before[1])
    # one request's own page
    table = st.table.copy()
    table[3, 6] = st.nb
    assert st.call(table=table, prefix=to_dev(st.shared, I32)) == BAD_ID
    assert torch.all(st.out[3] == 0) and torch.all(torch.isfinite(st.lse[:3]))


@pytest.mark.parametrize("dt,D,M,Hq", [(BF, 128, 4, 4), (BF, 64, 2, 6), (F32, 64, 4, 2)])
def test_prefix_in_one_pass_requests_that_fail(dt, D, M, Hq):
    """Failing requests among others where the prefix has a pass of its own."""
    P, B = 3216, 64
    st = Step([P + 3 * b for b in range(B)], M, Hq, 2, D, dt, 9, shared=P // 16, tree=True)
    ctx, table = st.ctx.copy(), st.table.copy()
    ctx[3], ctx[17], ctx[40] = P - 1, -1, 16 * st.mb - M + 1
    table[B - 1, P // 16] = -5
    st.parent[30, 1] = 1
    before = (st.kc.clone(), st.vc.clone())
    assert st.call(table=table, ctx=ctx, prefix=to_dev(st.shared, I32)) == INVALID | CAPACITY | BAD_ID
    bad = np.isin(np.arange(B), [3, 17, 30, 40, B - 1])
    assert torch.all(st.out[torch.from_numpy(bad)] == 0)
    assert torch.all(st.lse[torch.from_numpy(bad)] == -float("inf"))
    live = ~bad
    args = (st.q[live], st.k, st.v, st.table[live], st.ctx[live], st.kn[live])
    ref = oracle_verify_attn(*args, st.vn[live], parent=st.parent[live])
    size = oracle_verify_attn(*args[:2], np.abs(st.v), *args[3:], np.abs(st.vn[live]),
                              parent=st.parent[live])[0]
    keep = torch.from_numpy(live).cuda()
    st.out, st.lse = st.out[keep], st.lse[keep]
    st.check(ref, size)
    st.check_cache(ref)
    shared = st.shared.copy()
    shared[-1] = st.nb
    st.kc.copy_(before[0])
    st.vc.copy_(before[1])
    assert st.call(prefix=to_dev(shared, I32)) & BAD_ID
    assert torch.all(st.out == 0) and torch.all(st.lse == -float("inf"))
    assert torch.equal(st.kc, before[0]) and torch.equal(st.vc, before[1])


@pytest.mark.parametrize("D,impl", [(128, TC), (128, CORES), (64, AUTO)])
def test_attention_scale(D, impl):
    """A scale of the caller's, in every way of reading."""
    for P, B in ((64, 3), (3216, 64)):
        st = Step([P + b for b in range(B)], 4, 8, 2, D, BF, 5, shared=P // 16, impl=impl)
        st.dims.softmax_scale = 0.05
        assert st.call(prefix=to_dev(st.shared, I32)) == 0
        args = (st.q, st.k, st.v, st.table, st.ctx, st.kn)
        ref = oracle_verify_attn(*args, st.vn, scale=0.05)
        size = oracle_verify_attn(*args[:2], np.abs(st.v), *args[3:], np.abs(st.vn), scale=0.05)[0]
        st.check(ref, size)
    pages, cnt = choose(st.rng, st.ctx, 2, 9)
    assert st.call(pages=to_dev(pages, I32), page_counts=to_dev(cnt, I32)) == 0
    ref = oracle_verify_attn_pages(*args, st.vn, pages, cnt, scale=0.05)
    size = oracle_verify_attn_pages(*args[:2], np.abs(st.v), *args[3:], np.abs(st.vn), pages, cnt,
                                    scale=0.05)[0]
    st.check(ref, size)


@pytest.mark.parametrize("dt,D", [(BF, 128), (F32, 64)])
def test_prefix_scores_that_grow(dt, D):
    """Keys whose scores grow along the prefix, far and in steps, so that the
    running maximum moves in every tile, and a row of queries that are zero."""
    P, B = 3216, 64
    st = Step([P + b for b in range(B)], 4, 8, 2, D, dt, 5, shared=P // 16)
    lift = np.zeros((st.nb, 2, 16, 1))
    for j, blk in enumerate(st.shared):
        lift[blk] = (16 * j + np.arange(16)[:, None]) / P
    st.k = typed((st.k * 0.1 + lift * 6.0 * np.sign(st.q[0, 0, ::4])[None, :, None, :]).astype(np.float32), dt)
    st.q = typed((st.q * 0.3 + 0.7 * np.sign(st.q[0, 0, ::4]).repeat(4, 0)).astype(np.float32), dt)
    st.q[3, 1, 5] = 0
    st.kc = to_dev(st.k, dt)
    assert st.call(prefix=to_dev(st.shared, I32)) == 0
    args = (st.q, st.k, st.v, st.table, st.ctx, st.kn)
    ref = oracle_verify_attn(*args, st.vn)
    size = oracle_verify_attn(*args[:2], np.abs(st.v), *args[3:], np.abs(st.vn))[0]
    err = np.abs(st.out.double().cpu().numpy() - ref[0])
    # scores up to s = 6 * 0.7 * 128 / sqrt(128) = 48 and more: fp32 sums of D terms
    # are off by D * 2^-24 of them, and so are the weights, relatively
    s = np.abs(ref[1]).max() + 10
    w = 2 * D * 2.0 ** -24 * s * 4
    tol = (2.0 ** -8 * 1.02 * (size + np.abs(ref[0])) if dt == BF else 0) + w * size + 2.0 ** -16
    assert np.all(err <= tol), float((err / tol).max())
    assert np.max(np.abs(st.lse.cpu().numpy() - ref[1])) <= w + 1e-5


def test_prefix_agrees_with_the_plain_call_and_itself():
    """The same numbers as without the sharing up to roundings, the same bits
    from the same call twice, and without an lse."""
    st = prefix_step([528, 560, 900], 512, 6, 16, 4, 128, BF, 5)
    out, lse = st.out.clone(), st.lse.clone()
    st.call(prefix=to_dev(st.shared, I32))
    assert torch.equal(out, st.out) and torch.equal(lse, st.lse)
    st.call()
    assert torch.allclose(st.out.float(), out.float(), atol=2e-2) and torch.allclose(st.lse, lse, atol=1e-4)
    q = to_dev(st.q, BF)
    sv.spec_verify_attn(q, to_dev(st.kn, BF), to_dev(st.vn, BF), st.kc, st.vc, to_dev(st.table, I32),
                        to_dev(st.ctx, I32), None, st.out, None, st.dims, st.ws,
                        prefix=to_dev(st.shared, I32))
    assert torch.equal(out, st.out)


# ------------------------------------------------------------ selected pages

def choose(rng, ctx, Hkv, n, counts=None):
    pages = np.full((len(ctx), Hkv, n), -1, np.int64)
    cnt = np.zeros(len(ctx), np.int64)
    for b, c in enumerate(ctx):
        F = max(0, c) // 16
        cnt[b] = min(F, n) if counts is None else min(F, counts[b])
        for h in range(Hkv):
            pages[b, h, :cnt[b]] = np.sort(rng.permutation(F)[:cnt[b]])
    return pages, cnt


def pages_step(ctx, n, M, Hq, Hkv, D, dt, counts=None, **kw):
    st = Step(ctx, M, Hq, Hkv, D, dt, n + M, extra_pages=2, **kw)
    pages, cnt = choose(st.rng, ctx, Hkv, n, counts)
    # what no head of a request reads: any entry, NaN in the block
    seen = np.zeros_like(st.table, dtype=bool)
    for b, c in enumerate(ctx):
        seen[b, c // 16:-(-(c + M) // 16)] = True
        for h in range(Hkv):
            seen[b, pages[b, h, :cnt[b]]] = True
    dirty = np.where(seen, st.table, st.rng.choice([-1, 1 << 30], st.table.shape))
    st.unused(st.table[seen])
    junk = pages.copy()  # behind the counts, anything
    junk[pages < 0] = 2 ** 31 - 1
    assert st.call(table=dirty, pages=to_dev(junk, I32), page_counts=to_dev(cnt, I32)) == 0
    args = (st.q, st.k, st.v, st.table, st.ctx, st.kn)
    ref = oracle_verify_attn_pages(*args, st.vn, pages, cnt, parent=st.parent)
    size = oracle_verify_attn_pages(*args[:2], np.abs(st.v), *args[3:], np.abs(st.vn), pages, cnt,
                                    parent=st.parent)[0]
    st.check(ref, size)
    st.check_cache(ref)
    return st


PAGES = [  # ctx, n, M, Hq, Hkv, D, dt, tree, impl, counts
    ([0], 1, 1, 1, 1, 128, BF, False, TC, None), ([0, 5, 16, 31], 1, 1, 8, 2, 128, BF, False, TC, None),
    ([0], 1, 1, 1, 1, 64, F32, False, AUTO, None),
    ([300, 301, 335, 17], 4, 5, 8, 2, 128, BF, False, TC, None),
    ([300, 301, 335, 17], 5, 5, 8, 2, 128, BF, True, CORES, [0, 1, 5, 0]),
    ([1000, 2000, 40, 3], 33, 9, 14, 2, 128, BF, True, TC, None),
    ([5000, 4999], 200, 4, 16, 2, 128, BF, False, TC, [200, 199]),
    ([333] * 40, 7, 2, 8, 1, 128, BF, False, TC, None),
    ([100, 90], 3, 128, 1, 1, 128, BF, True, TC, None),
    ([160, 175], 400, 16, 16, 2, 128, BF, False, TC, None),  # a list longer than the table
    ([80, 81, 15], 2, 7, 3, 3, 64, BF, False, AUTO, None),
    ([600, 900, 64], 12, 16, 8, 2, 64, BF, True, AUTO, None),
    ([80, 95], 3, 3, 4, 2, 128, F32, False, AUTO, None),
    ([700, 2000, 100], 33, 64, 4, 4, 64, F32, True, AUTO, None),
    ([512] * 9, 6, 16, 2, 1, 128, F32, True, AUTO, None)]


@pytest.mark.parametrize("ctx,n,M,Hq,Hkv,D,dt,tree,impl,counts", PAGES)
def test_pages(ctx, n, M, Hq, Hkv, D, dt, tree, impl, counts):
    pages_step(ctx, n, M, Hq, Hkv, D, dt, counts=counts, tree=tree, impl=impl)


@pytest.mark.parametrize("dt,D,impl", [(BF, 128, TC), (BF, 128, CORES), (F32, 64, AUTO)])
def test_pages_lists_that_fail(dt, D, impl):
    """Each request breaks one rule; the first and the last are fine."""
    bad = [[0, 3, 5], [3, 3, 5], [5, 3, 6], [0, 3, 7], [-1, 3, 5], [0, 3, 5], [0, 3, 5], [1, 2, 3]]
    counts = [3, 3, 3, 3, 3, 4, -1, 3]
    B = len(bad)
    st = Step([115] * B, 2, 4, 2, D, dt, 9, impl=impl)
    pages = np.tile(np.array([0, 3, 5]), (B, 2, 1))
    pages[:, 1] = bad  # the second head's lists
    before = (st.kc.clone(), st.vc.clone())
    assert st.call(pages=to_dev(pages, I32), page_counts=to_dev(np.array(counts), I32)) == INVALID
    assert torch.all(st.out[1:-1] == 0) and torch.all(st.lse[1:-1] == -float("inf"))
    for b in (0, B - 1):
        one = slice(b, b + 1)
        args = (st.q[one], st.k, st.v, st.table[one], st.ctx[one], st.kn[one])
        ref = oracle_verify_attn_pages(*args, st.vn[one], pages[one], counts[one])
        size = oracle_verify_attn_pages(*args[:2], np.abs(st.v), *args[3:], np.abs(st.vn[one]),
                                        pages[one], counts[one])[0]
        full = [np.repeat(x, B, 0) for x in (ref[0], ref[1], size)]
        st.check(full[:2], full[2], one)
    kept = torch.from_numpy(st.table[1:-1][st.table[1:-1] >= 0]).cuda()
    assert torch.equal(st.kc[kept], before[0][kept]) and torch.equal(st.vc[kept], before[1][kept])
    # a selected page, and a page of the new rows, that is no block; a length without room
    table, ctx = st.table.copy(), st.ctx.copy()
    table[0, 3], table[1, 7], ctx[2], ctx[3] = st.nb, -1, 16 * st.mb - 1, -5
    good = np.tile(np.array([0, 3, 5]), (B, 2, 1))
    assert st.call(table=table, ctx=ctx, pages=to_dev(good, I32),
                   page_counts=to_dev(np.full(B, 3), I32)) == BAD_ID | CAPACITY
    assert torch.all(st.out[:4] == 0) and torch.all(torch.isfinite(st.lse[4:]))


def test_pages_agree_with_the_plain_call_where_all_are_selected():
    ctx = [520, 64, 1000, 7]
    st = Step(ctx, 5, 8, 2, 128, BF, 4)
    pages, cnt = choose(st.rng, ctx, 2, 64)
    st.call(pages=to_dev(pages, I32), page_counts=to_dev(cnt, I32))
    out, lse = st.out.clone(), st.lse.clone()
    st.call(pages=to_dev(pages, I32), page_counts=to_dev(cnt, I32))
    assert torch.equal(out, st.out) and torch.equal(lse, st.lse)
    st.call()
    assert torch.allclose(st.out.float(), out.float(), atol=2e-2) and torch.allclose(st.lse, lse, atol=1e-4)


# ------------------------------------------------- bounds, scores, selection

@pytest.mark.parametrize("dt,D", [(BF, 128), (BF, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_bounds(dt, D, Hkv):
    ctx = np.array([0, 1, 15, 16, 17, 500, 1000, -1, 640, 77])
    start = np.array([0, 0, 14, 16, 16, 3, 990, 0, 0, 80])  # the last: nothing new
    st = Step(ctx, 1, Hkv, Hkv, D, dt, D + Hkv)
    b0 = typed(st.rng.standard_normal((st.nb, Hkv, 2, D)).astype(np.float32), dt)
    for frm in (start, None):
        bounds = to_dev(b0, dt)
        sv.spec_page_bounds(st.kc, to_dev(st.table, I32), None if frm is None else to_dev(frm, I32),
                            to_dev(ctx, I32), bounds, st.dims, st.ws)
        ref = oracle_page_bounds(st.k, st.table, frm, ctx, b0)
        assert np.array_equal(bounds.double().cpu().numpy(), ref)
    assert sv.device_status(st.ws) == 0


def test_bounds_of_requests_that_fail():
    ctx = np.array([40, 40, 40, 40])
    st = Step(ctx, 1, 2, 2, 128, BF, 1)
    table, frm = st.table.copy(), np.array([0, -1, 0, 0])
    table[2, 1] = st.nb
    call = np.array([40, 40, 40, 16 * st.mb + 1])
    bounds = torch.zeros(st.nb, 2, 2, 128, dtype=BF, device="cuda")
    sv.spec_page_bounds(st.kc, to_dev(table, I32), to_dev(frm, I32), to_dev(call, I32), bounds,
                        st.dims, st.ws)
    assert sv.device_status(st.ws) == INVALID | CAPACITY | BAD_ID
    keep = st.table.copy()
    ref = oracle_page_bounds(st.k, keep[:1], [0], [40], np.zeros(bounds.shape))
    ref = oracle_page_bounds(st.k, keep[2:3, :1], [0], [16], ref)
    ref = oracle_page_bounds(st.k, keep[2:3], [32], [40], ref)
    assert np.array_equal(bounds.double().cpu().numpy(), ref)


SCORE = [(1, 1, 1), (1, 4, 1), (5, 8, 2), (9, 14, 2), (3, 21, 3), (16, 16, 2), (128, 2, 2), (33, 4, 1)]


@pytest.mark.parametrize("dt,D", [(BF, 128), (BF, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("M,Hq,Hkv", SCORE)
def test_score(dt, D, M, Hq, Hkv):
    ctx = np.array([1500, 0, 15, 16, 1024 + 33, -1, 3000])
    st = Step(ctx, M, Hq, Hkv, D, dt, D + M)
    pair = np.sort(st.rng.standard_normal((st.nb, Hkv, 2, D)), axis=2)
    pair[::3] -= 2.0  # both bounds of one sign in places
    pair = typed(pair.astype(np.float32), dt)
    table = st.table.copy()
    for b, c in enumerate(ctx):  # entries behind the whole pages are not read
        table[b, max(0, c) // 16:] = 1 << 30
    bounds = to_dev(pair, dt)
    used = np.concatenate([st.table[b, :max(0, c) // 16] for b, c in enumerate(ctx)])
    bounds[torch.from_numpy(np.setdiff1d(np.arange(st.nb), used)).cuda()] = float("nan")
    scores = torch.full((st.B, Hkv, st.mb), float("nan"), device="cuda")
    sv.spec_page_score(to_dev(st.q, dt), bounds, to_dev(table, I32), to_dev(ctx, I32), scores,
                       st.dims, st.ws)
    assert sv.device_status(st.ws) == 0
    ref, size = oracle_page_score(st.q, pair, st.table, ctx)
    got = scores.double().cpu().numpy()
    there = np.isfinite(ref)
    assert np.all(got[~there] == -np.inf)
    err = np.abs(got[there] - ref[there])
    assert np.all(err <= 2 * D * 2.0 ** -24 * size[there]), err.max()


@pytest.mark.parametrize("dt,D", [(BF, 128), (BF, 64), (F32, 128), (F32, 64)])
def test_score_of_many_requests(dt, D):
    """Enough tiles of 64 pages to fill the GPU, several requests a CTA."""
    B, M, Hq, Hkv = 21, 2, 24, 8
    rng = np.random.default_rng(3)
    ctx = rng.integers(0, 2100, B)
    ctx[:3] = (2099, 0, 1024)
    st = Step(ctx, M, Hq, Hkv, D, dt, 6)
    pair = typed(np.sort(rng.standard_normal((st.nb, Hkv, 2, D)), axis=2).astype(np.float32), dt)
    scores = torch.full((B, Hkv, st.mb), float("nan"), device="cuda")
    sv.spec_page_score(to_dev(st.q, dt), to_dev(pair, dt), to_dev(st.table, I32), to_dev(ctx, I32),
                       scores, st.dims, st.ws)
    assert sv.device_status(st.ws) == 0
    ref, size = oracle_page_score(st.q, pair, st.table, ctx)
    got, there = scores.double().cpu().numpy(), np.isfinite(ref)
    assert np.all(got[~there] == -np.inf)
    assert np.all(np.abs(got[there] - ref[there]) <= 2 * D * 2.0 ** -24 * size[there])


@pytest.mark.parametrize("dt,D", [(BF, 128), (F32, 64)])
def test_score_of_pages_that_fail(dt, D):
    ctx = np.array([1200, 800])
    st = Step(ctx, 2, 4, 2, D, dt, 1)
    pair = typed(np.sort(st.rng.standard_normal((st.nb, 2, 2, D)), axis=2).astype(np.float32), dt)
    table, call = st.table.copy(), np.array([1200, 16 * st.mb + 1])
    table[0, 3], table[0, 70] = -1, st.nb
    scores = torch.full((2, 2, st.mb), float("nan"), device="cuda")
    sv.spec_page_score(to_dev(st.q, dt), to_dev(pair, dt), to_dev(table, I32), to_dev(call, I32),
                       scores, st.dims, st.ws)
    assert sv.device_status(st.ws) == CAPACITY | BAD_ID
    ref, size = oracle_page_score(st.q, pair, st.table, ctx)
    ref[1] = ref[0, :, 3] = ref[0, :, 70] = -np.inf
    got, there = scores.double().cpu().numpy(), np.isfinite(ref)
    assert np.all(got[~there] == -np.inf)
    assert np.all(np.abs(got[there] - ref[there]) <= 2 * D * 2.0 ** -24 * size[there])


def select_check(x, ctx, n, first, last, status=0):
    B, Hkv, mb = x.shape
    dims = sv.make_dims(B=B, M=1, Hq=Hkv, Hkv=Hkv, max_blocks=mb)
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    pages = torch.full((B, Hkv, n), -9, dtype=I32, device="cuda")
    counts = torch.full((B,), -9, dtype=I32, device="cuda")
    sv.spec_page_select(to_dev(x, F32), to_dev(ctx, I32), pages, counts, dims, ws, first=first,
                        last=last)
    assert sv.device_status(ws) == status
    ref, cnt = oracle_page_select(x, ctx, n, first, last)
    assert np.array_equal(counts.cpu().numpy(), cnt)
    assert np.array_equal(pages.cpu().numpy(), ref)


SELECT = [(1, 1, 1, 0, 0), (1, 40, 1, 1, 0), (3, 40, 5, 1, 2), (2, 300, 64, 1, 4), (5, 256, 17, 0, 17),
          (2, 257, 16, 16, 0), (3, 1000, 999, 3, 5), (2, 3000, 100, 0, 0), (2, 9000, 1000, 4, 17),
          (1, 40000, 33, 1, 1), (4, 20, 500, 2, 3), (1, 17000, 12000, 1, 1), (1, 60000, 700, 2, 5)]


@pytest.mark.parametrize("B,mb,n,first,last", SELECT)
@pytest.mark.parametrize("kind", ["normal", "ties", "equal", "close", "wide"])
def test_select(B, mb, n, first, last, kind):
    rng = np.random.default_rng(mb + n)
    x = rng.standard_normal((B, 2, mb)).astype(np.float32)
    if kind == "ties":
        x = np.round(x * 2) / 2 * rng.choice([1, -1], x.shape)  # zeros of both signs among them
    elif kind == "equal":
        x[:] = -3.5
    elif kind == "close":  # neighbouring values: the last digit decides
        x = np.float32(1.5) + rng.integers(0, 300, x.shape).astype(np.float32) * np.float32(2.0 ** -23)
    elif kind == "wide":
        x = (x * 10.0 ** rng.integers(-40, 38, x.shape)).astype(np.float32)
        x[rng.random(x.shape) < 0.3] = -np.inf
        x[0, 0, :: 7] = np.inf
    ctx = rng.integers(0, mb * 16 + 1, B)
    ctx[0] = mb * 16
    select_check(x.astype(np.float32), ctx, n, first, last)


def test_select_special_lengths_and_nan():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 2, 50)).astype(np.float32)
    select_check(x, np.array([-1, 0, 15, 801]), 7, 1, 2, CAPACITY)
    x[2, 1, 10:30] = np.nan
    x[2, 1, 30:45] = -np.inf
    select_check(x, np.array([-1, 0, 800, 800]), 25, 1, 2, NONFINITE)
    x[:, :, 40:] = np.nan  # behind the whole pages: not read
    x[2, 1, 10:30] = 0
    select_check(x, np.array([640, 645, 655, 100]), 25, 1, 2)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dt,D,impl", [(BF, 128, TC), (F32, 64, AUTO)])
def test_decoding_over_selected_pages(dt, D, impl):
    """Steps of a small batch: scores, selection, attention, commit, bounds of what
    was kept; each against its oracle on the GPU's own inputs."""
    B, M, Hq, Hkv, n = 3, 4, 8, 2, 6
    st = Step([300, 47, 161], M, Hq, Hkv, D, dt, 8, impl=impl, extra_pages=4)
    free = np.setdiff1d(np.arange(st.nb), st.table)  # pages for the steps to come
    st.nb += 12
    free = np.concatenate([free, np.arange(st.nb - 12, st.nb)])
    for b in range(B):
        gap = np.nonzero(st.table[b] < 0)[0][:4]
        st.table[b, gap], free = free[:len(gap)], free[len(gap):]
    n_ = lambda *s: typed(st.rng.standard_normal(s).astype(np.float32), dt)  # noqa: E731
    st.k, st.v = n_(st.nb, Hkv, 16, D), n_(st.nb, Hkv, 16, D)
    st.kc, st.vc = to_dev(st.k, dt), to_dev(st.v, dt)
    st.dims = sv.make_dims(B=B, M=M, Hq=Hq, Hkv=Hkv, D=D, max_blocks=st.mb, num_blocks=st.nb,
                           kv_dtype=dt, attn_impl=impl)
    st.ws = sv.workspace(st.dims)
    table, ctx = to_dev(st.table, I32), to_dev(st.ctx, I32)
    bounds = torch.zeros(st.nb, Hkv, 2, D, dtype=dt, device="cuda")
    scores = torch.empty(B, Hkv, st.mb, device="cuda")
    pages = torch.empty(B, Hkv, n, dtype=I32, device="cuda")
    counts, before = torch.empty(B, dtype=I32, device="cuda"), None
    want = np.zeros(bounds.shape)
    for step in range(5):
        sv.spec_page_bounds(st.kc, table, before, ctx, bounds, st.dims, st.ws)
        st.q, st.kn, st.vn = n_(B, M, Hq, D), n_(B, M, Hkv, D), n_(B, M, Hkv, D)
        st.parent = np.stack([random_tree(st.rng, M - 1, 2, M) for _ in range(B)])
        sv.spec_page_score(to_dev(st.q, dt), bounds, table, ctx, scores, st.dims, st.ws)
        sv.spec_page_select(scores, ctx, pages, counts, st.dims, st.ws, first=1, last=2)
        assert st.call(pages=pages, page_counts=counts) == 0
        want = oracle_page_bounds(st.k, st.table, None if before is None else before.cpu().numpy(),
                                  st.ctx, want)
        assert np.array_equal(bounds.double().cpu().numpy(), want)
        ref, size = oracle_page_score(st.q, want, st.table, st.ctx)
        got = scores.double().cpu().numpy()
        there = np.isfinite(ref)
        assert np.all(np.abs(got[there] - ref[there]) <= 2 * D * 2.0 ** -24 * size[there])
        sel, cnt = oracle_page_select(got, st.ctx, n, 1, 2)
        assert np.array_equal(pages.cpu().numpy(), sel) and np.array_equal(counts.cpu().numpy(), cnt)
        args = (st.q, st.k, st.v, st.table, st.ctx, st.kn)
        o = oracle_verify_attn_pages(*args, st.vn, sel, cnt, parent=st.parent)
        a = oracle_verify_attn_pages(*args[:2], np.abs(st.v), *args[3:], np.abs(st.vn), sel, cnt,
                                     parent=st.parent)[0]
        st.check(o, a)
        st.check_cache(o)
        path = np.tile([0, 1, -1, -1], (B, 1))
        acc = np.array([1, 0, 1])
        path[1, 1] = -1
        for b in (0, 2):  # the last child of the root
            path[b, 1] = np.nonzero(st.parent[b] == 0)[0][-1]
        before = ctx.clone()
        sv.kv_commit(st.kc, st.vc, table, before, ctx, to_dev(path, I32), to_dev(acc, I32), st.dims,
                     st.ws)
        st.k, st.v, st.ctx = oracle_kv_commit(o[2], o[3], st.table, st.ctx, path, acc)
        assert np.array_equal(ctx.cpu().numpy(), st.ctx)


@pytest.mark.parametrize("dt,D", [(BF, 128), (BF, 64), (F32, 64)])
def test_prefix_in_one_pass_captured(dt, D):
    """The pass of its own in a graph, the prefix' pages and lengths replaced."""
    P, B = 3216, 64
    st = Step([P + b % 9 for b in range(B)], 2, 4, 2, D, dt, 5, shared=P // 16)
    q, kn, vn = (to_dev(x, dt) for x in (st.q, st.kn, st.vn))
    table, ctx, shared = (to_dev(x, I32) for x in (st.table, st.ctx, st.shared))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_verify_attn(q, kn, vn, st.kc, st.vc, table, ctx, None, out, lse, st.dims, st.ws,
                            prefix=shared)
    for turn in range(2):
        if turn:
            st.shared = st.shared[::-1].copy()
            st.table[:, :P // 16] = st.shared
            shared.copy_(to_dev(st.shared, I32))
            st.ctx = np.minimum(st.ctx, P + 5)
            ctx.copy_(to_dev(st.ctx, I32))
        st.kc.copy_(to_dev(st.k, dt))
        st.vc.copy_(to_dev(st.v, dt))
        g.replay()
        args = (st.q, st.k, st.v, st.table, st.ctx, st.kn)
        ref = oracle_verify_attn(*args, st.vn)
        size = oracle_verify_attn(*args[:2], np.abs(st.v), *args[3:], np.abs(st.vn))[0]
        st.out, st.lse = out, lse
        st.check(ref, size)
        st.check_cache(ref)


@pytest.mark.parametrize("form", ["prefix", "pages"])
@pytest.mark.parametrize("dt,D", [(BF, 128), (F32, 64)])
def test_captured_and_replayed(form, dt, D):
    """One graph, lengths and lists that change between replays."""
    B, M = 3, 3
    st = Step([180, 200, 190], M, 4, 2, D, dt, 3, shared=8)
    q, kn, vn = (to_dev(x, dt) for x in (st.q, st.kn, st.vn))
    table, ctx, shared = (to_dev(x, I32) for x in (st.table, st.ctx, st.shared))
    lists, cnt = choose(st.rng, st.ctx, 2, 6)
    pages, counts = to_dev(lists, I32), to_dev(cnt, I32)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    kw = dict(prefix=shared) if form == "prefix" else dict(pages=pages, page_counts=counts)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_verify_attn(q, kn, vn, st.kc, st.vc, table, ctx, None, out, lse, st.dims, st.ws, **kw)
    # the last time the first request has no page for its new rows: it alone fails
    for c, live in (([180, 200, 190], slice(0, 3)), ([128, 129, 199], slice(0, 3)),
                    ([190, 131, 143], slice(1, 3))):
        st.kc.copy_(to_dev(st.k, dt))
        st.vc.copy_(to_dev(st.v, dt))
        ctx.copy_(torch.tensor(c))
        lists, cnt = choose(st.rng, c, 2, 6)
        pages.copy_(to_dev(lists, I32))
        counts.copy_(to_dev(cnt, I32))
        g.replay()
        assert sv.device_status(st.ws) == (BAD_ID if live.start else 0)
        assert torch.all(out[:live.start] == 0) and torch.all(lse[:live.start] == -float("inf"))
        tabs = (st.table[live], np.array(c)[live], st.kn[live])
        if form == "prefix":
            ref = oracle_verify_attn(st.q[live], st.k, st.v, *tabs, st.vn[live])
            size = oracle_verify_attn(st.q[live], st.k, np.abs(st.v), *tabs, np.abs(st.vn[live]))[0]
        else:
            sel = (lists[live], cnt[live])
            ref = oracle_verify_attn_pages(st.q[live], st.k, st.v, *tabs, st.vn[live], *sel)
            size = oracle_verify_attn_pages(st.q[live], st.k, np.abs(st.v), *tabs,
                                            np.abs(st.vn[live]), *sel)[0]
        st.out, st.lse = out[live], lse[live]
        st.check(ref, size)
        st.check_cache(ref)


def test_waits_that_run_out():
    """A wait limit of 1000 clocks: the calls end, with their results or with the
    status of a wait that gave up, and after the workspace is zeroed they are right."""
    st = Step([3216 + b for b in range(64)], 4, 8, 2, 128, BF, 5, shared=201)
    full = st.dims
    args = (st.q, st.k, st.v, st.table, st.ctx, st.kn)
    ref = oracle_verify_attn(*args, st.vn)
    size = oracle_verify_attn(*args[:2], np.abs(st.v), *args[3:], np.abs(st.vn))[0]
    pair = typed(np.sort(st.rng.standard_normal((st.nb, 2, 2, 128)), axis=2).astype(np.float32), BF)
    scores = torch.empty(64, 2, st.mb, device="cuda")
    want, s = oracle_page_score(st.q, pair, st.table, st.ctx)
    there = np.isfinite(want)
    for limit in (1, 0):
        st.dims = sv.make_dims(B=64, M=4, Hq=8, Hkv=2, D=128, max_blocks=st.mb, num_blocks=st.nb,
                               kv_dtype=BF, wait_limit_kcycles=limit)
        st.ws.zero_()
        status = st.call(prefix=to_dev(st.shared, I32))
        assert status in (0, 1 << 7) and (limit == 1 or status == 0)
        if status == 0:
            st.check(ref, size)
        st.ws.zero_()
        sv.spec_page_score(to_dev(st.q, BF), to_dev(pair, BF), to_dev(st.table, I32),
                           to_dev(st.ctx, I32), scores, st.dims, st.ws)
        status = sv.device_status(st.ws)
        assert status in (0, 1 << 7) and (limit == 1 or status == 0)
        if status == 0:
            got = scores.double().cpu().numpy()
            assert np.all(np.abs(got[there] - want[there]) <= 2 * 128 * 2.0 ** -24 * s[there])
    st.dims = full


def test_calls_on_two_streams():
    """Bounds, scores and selection of two batches side by side share a workspace;
    the attention forms have one each."""
    steps = [Step([900 + 40 * b for b in range(9)], 3, 4, 2, 128, BF, seed, shared=4) for seed in (1, 2)]
    streams = [torch.cuda.Stream() for _ in steps]
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    inputs = [[to_dev(x, BF) for x in (st.q, st.kn, st.vn)] +
              [to_dev(x, I32) for x in (st.table, st.ctx, st.shared)] for st in steps]
    outs = [dict(bounds=torch.zeros(st.nb, 2, 2, 128, dtype=BF, device="cuda"),
                 scores=torch.empty(9, 2, st.mb, device="cuda"),
                 pages=torch.empty(9, 2, 7, dtype=I32, device="cuda"),
                 counts=torch.empty(9, dtype=I32, device="cuda"),
                 out=torch.empty_like(i[0]), lse=torch.empty(9, 3, 4, device="cuda"),
                 out2=torch.empty_like(i[0]), lse2=torch.empty(9, 3, 4, device="cuda"))
            for st, i in zip(steps, inputs)]
    torch.cuda.synchronize()
    for turn in range(5):
        for st, s, i, o in zip(steps, streams, inputs, outs):
            q, kn, vn, table, ctx, shared = i
            sv.spec_page_bounds(st.kc, table, None, ctx, o["bounds"], st.dims, ws, stream=s)
            sv.spec_page_score(q, o["bounds"], table, ctx, o["scores"], st.dims, ws, stream=s)
            sv.spec_page_select(o["scores"], ctx, o["pages"], o["counts"], st.dims, ws, first=1,
                                last=1, stream=s)
            sv.spec_verify_attn(q, kn, vn, st.kc, st.vc, table, ctx, None, o["out"], o["lse"], st.dims,
                                st.ws, pages=o["pages"], page_counts=o["counts"], stream=s)
            sv.spec_verify_attn(q, kn, vn, st.kc, st.vc, table, ctx, None, o["out2"], o["lse2"],
                                st.dims, st.ws, prefix=shared, stream=s)
    torch.cuda.synchronize()
    assert sv.device_status(ws) == 0
    for st, o in zip(steps, outs):
        want = oracle_page_bounds(st.k, st.table, None, st.ctx, np.zeros(o["bounds"].shape))
        assert np.array_equal(o["bounds"].double().cpu().numpy(), want)
        sel, cnt = oracle_page_select(o["scores"].double().cpu().numpy(), st.ctx, 7, 1, 1)
        assert np.array_equal(o["pages"].cpu().numpy(), sel)
        args = (st.q, st.k, st.v, st.table, st.ctx, st.kn)
        sizes = (st.q, st.k, np.abs(st.v), st.table, st.ctx, st.kn)
        st.out, st.lse = o["out"], o["lse"]
        st.check(oracle_verify_attn_pages(*args, st.vn, sel, cnt),
                 oracle_verify_attn_pages(*sizes, np.abs(st.vn), sel, cnt)[0])
        st.out, st.lse = o["out2"], o["lse2"]
        st.check(oracle_verify_attn(*args, st.vn), oracle_verify_attn(*sizes, np.abs(st.vn))[0])


@pytest.mark.parametrize("dt,D,Hkv,blocks", [(BF, 128, 8, 270_000), (F32, 64, 8, 530_000)])
def test_blocks_past_32_bit_offsets(dt, D, Hkv, blocks):
    """The same blocks at the far end of a cache of more than 2^32 values: the same
    bits as in a small cache."""
    P, B, M = 3216, 16, 3
    st = Step([P + 7 * b for b in range(B)], M, 2 * Hkv, Hkv, D, dt, 5, shared=P // 16)
    far = np.arange(st.nb)[::-1] + blocks - st.nb  # block i lives at far[i]
    at = torch.from_numpy(far.copy()).cuda()
    k = torch.empty(blocks, Hkv, 16, D, dtype=dt, device="cuda")
    v = torch.empty(blocks, Hkv, 16, D, dtype=dt, device="cuda")
    assert k.numel() > 2 ** 32
    k[at], v[at] = st.kc, st.vc
    near = dict(k=st.kc, v=st.vc, table=st.table, shared=st.shared, nb=st.nb)
    away = dict(k=k, v=v, table=np.where(st.table >= 0, far[st.table], -1), shared=far[st.shared], nb=blocks)
    lists, cnt = choose(st.rng, st.ctx, Hkv, 20)
    got = []
    for place in (near, away):
        st.kc, st.vc, st.nb = place["k"], place["v"], place["nb"]
        st.dims = sv.make_dims(B=B, M=M, Hq=2 * Hkv, Hkv=Hkv, D=D, max_blocks=st.mb, num_blocks=st.nb,
                               kv_dtype=dt)
        table, ctx = to_dev(place["table"], I32), to_dev(st.ctx, I32)
        bounds = torch.zeros(st.nb, Hkv, 2, D, dtype=dt, device="cuda")
        scores = torch.empty(B, Hkv, st.mb, device="cuda")
        sv.spec_page_bounds(st.kc, table, None, ctx, bounds, st.dims, st.ws)
        sv.spec_page_score(to_dev(st.q, dt), bounds, table, ctx, scores, st.dims, st.ws)
        res = [scores]
        short = to_dev(place["shared"][:9], I32)  # read by the requests; then in a pass of its own
        for kw in (dict(prefix=short), dict(prefix=to_dev(place["shared"], I32)),
                   dict(pages=to_dev(lists, I32), page_counts=to_dev(cnt, I32))):
            assert st.call(table=place["table"], **kw) == 0
            res += [st.out, st.lse]
        used = at if place is away else torch.arange(near["nb"], device="cuda")
        got.append(res + [x[used] for x in (st.kc, st.vc, bounds)])
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_forms_take_turns_on_one_workspace():
    """Every form of the attention, one after another on the same workspace and
    another stream, as a step that mixes layers may."""
    st = Step([180, 200, 190], 3, 4, 2, 128, BF, 3, shared=8)
    lists, cnt = choose(st.rng, st.ctx, 2, 64)  # all pages
    forms = [dict(), dict(prefix=to_dev(st.shared, I32)), dict(window=4000),
             dict(pages=to_dev(lists, I32), page_counts=to_dev(cnt, I32))]
    ref = oracle_verify_attn(st.q, st.k, st.v, st.table, st.ctx, st.kn, st.vn)
    size = oracle_verify_attn(st.q, st.k, np.abs(st.v), st.table, st.ctx, st.kn, np.abs(st.vn))[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for kw in forms + forms[::-1]:
            assert st.call(**kw) == 0
            st.check(ref, size)
    torch.cuda.synchronize()
