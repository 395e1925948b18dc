"""Block tables over a corrupt page state: table and ring entries that are no
block id, against the oracle, bit for bit."""
import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from harness import to_dev  # noqa: E402
from synth import random_tree  # noqa: E402
from test_gpu_step import I32, Pages  # noqa: E402


def corrupt(st, rng, key, n):
    """n entries that the state uses become ids of no block."""
    h = st.h[key].reshape(-1)
    if key == "pool":
        head, count = st.h["pool_state"]
        at = (head + rng.permutation(count)[:n]) % st.nb
    else:
        at = rng.permutation(np.nonzero(h >= 0)[0])[:n]
    h[at] = rng.choice([-1, -5, st.nb, 1 << 30, -(1 << 31)], len(at))
    st.d[key].copy_(to_dev(st.h[key], I32))


@pytest.mark.parametrize("key", ["pool", "block_table"])
@pytest.mark.parametrize("B,nb,longest,window,sinks", [
    (1, 20, 50, 0, 0), (7, 200, 50, 0, 0), (7, 200, 50, 40, 17), (60, 1500, 100, 0, 0),
    (600, 8000, 50, 0, 0), (600, 8000, 50, 30, 20), (1100, 9000, 4, 0, 0)])
def test_ids_of_no_block(key, B, nb, longest, window, sinks):
    """Lives with corrupt entries thrown in; the calls take one CTA (few rows),
    several, and rounds of requests."""
    rng = np.random.default_rng(B + window)
    st = Pages(B, 24, nb, head=nb // 3)
    ctx = np.full(B, -1)
    hit = 0
    for step in range(14):
        n = np.where(ctx < 0, 0, rng.integers(0, longest, B))
        start = np.concatenate([[0], np.cumsum(n)])
        out = st.call(ctx, start, int(start[-1]) + 2, window=window, sinks=sinks)
        hit += bool(out["status"] & 1 << 6)
        assert np.all((out["ok"] == 1) <= (ctx >= 0))
        ctx = np.where(out["ok"] > 0, ctx + rng.integers(0, n + 1), ctx)
        r = rng.random(B)
        ctx = np.where(r < 0.15, -1, np.where((ctx < 0) & (r > 0.3), 0, ctx))
        ctx = np.where(ctx > 24 * 16 - 100, -1, ctx)
        if step % 3 == 1:
            corrupt(st, rng, key, max(1, B // 10))
    assert hit or B == 1
    # with every request ended and the ring's own corrupt entries handed out and
    # dropped, what is left is blocks alone, none of them twice
    for _ in range(2):
        st.call(np.full(B, -1), np.zeros(B + 1, np.int64), 2, window=window, sinks=sinks)
    head, count = st.h["pool_state"]
    free = st.h["pool"][(head + np.arange(count)) % nb]
    good = free[(free >= 0) & (free < nb)]
    assert len(np.unique(good)) == len(good)
    if key == "block_table":
        assert len(good) == count


def test_ids_of_no_block_under_trees():
    rng = np.random.default_rng(5)
    M = 40
    st = Pages(5, 30, 140, M=M)
    ctx = np.array([0, 3, 16, 200, 90])
    for _ in range(5):
        parent = np.stack([random_tree(rng, M - 1, 3, M) for _ in range(5)])
        st.call(ctx, None, 5 * M + 1, parent=parent)
        corrupt(st, rng, "pool", 4)
        corrupt(st, rng, "block_table", 1)
        ctx = ctx + rng.integers(1, 30, 5)
        ctx[rng.integers(0, 5)] = 0


def test_every_id_of_the_ring_corrupt():
    st = Pages(3, 6, 12)
    st.h["pool"][:] = -1
    st.d["pool"].fill_(-1)
    out = st.call(np.array([0, 0, 0]), np.array([0, 20, 20, 40]), 40)
    assert out["ok"].tolist() == [0, 1, 0] and out["pool_state"].tolist() == [4, 8]
    out = st.call(np.array([-1, -1, -1]), np.zeros(4, np.int64), 0)
    assert out["pool_state"].tolist() == [4, 8]
