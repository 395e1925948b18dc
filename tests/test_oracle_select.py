"""The oracles of selected pages and shared prefixes against closed forms and
the verify attention's own oracle, and the Python calls' refusals (no GPU)."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_19_gb300 as sv
from oracle import (oracle_page_bounds, oracle_page_score, oracle_page_select, oracle_verify_attn,
                    oracle_verify_attn_pages, oracle_verify_attn_prefix)

RNG = np.random.default_rng(5)


def cache(nb=9, Hkv=2, D=4):
    return RNG.standard_normal((nb, Hkv, 16, D)), RNG.standard_normal((nb, Hkv, 16, D))


def test_bounds_hold_every_key_and_are_reached():
    k, _ = cache()
    table = np.array([[3, 1, 7], [0, 2, -1]])
    before = np.full((9, 2, 2, 4), 5.0)
    out = oracle_page_bounds(k, table, [16, 0], [40, 20], before)
    assert np.array_equal(out[[3, 4, 5, 6, 8]], before[[3, 4, 5, 6, 8]])  # not met
    for blk, n in ((1, 16), (7, 8), (0, 16), (2, 4)):
        keys = k[blk, :, :n]
        assert np.all(out[blk, :, :1] <= keys) and np.all(out[blk, :, 1:] >= keys)
        assert np.array_equal(out[blk, :, 0], np.min(keys, 1))


def test_a_score_is_never_below_a_product_with_a_key():
    k, _ = cache()
    q = RNG.standard_normal((1, 3, 4, 4))
    table = np.array([[3, 1, 7, 0]])
    bounds = oracle_page_bounds(k, table, None, [60], np.zeros((9, 2, 2, 4)))
    scores, _ = oracle_page_score(q, bounds, table, [60])
    assert np.all(scores[0, :, 3] == -np.inf)
    for p in range(3):
        for h in range(2):
            prod = k[table[0, p], h] @ q[0, :, 2 * h:2 * h + 2].reshape(-1, 4).T
            assert prod.max() <= scores[0, h, p] + 1e-12
    # keys that are all equal: the score is the product
    k[3] = k[3, :, :1]
    bounds = oracle_page_bounds(k, table, None, [16], bounds)
    s, _ = oracle_page_score(q, bounds, table, [16])
    assert np.allclose(s[0, 0, 0], (k[3, 0, 0] @ q[0, :, :2].reshape(-1, 4).T).max())


def test_selection_by_hand():
    x = np.array([[[1.0, 5, 2, 5, 0, 9, 3, -np.inf]]])
    pick = lambda n, f=0, l=0, ctx=128: oracle_page_select(x, [ctx], n, f, l)[0][0, 0].tolist()  # noqa: E731
    assert pick(1) == [5] and pick(2) == [1, 5] and pick(3) == [1, 3, 5]
    assert pick(4, 1, 1) == [0, 1, 5, 7] and pick(2, 0, 2) == [6, 7]
    assert pick(10) == list(range(8)) + [-1, -1] and pick(3, ctx=40) == [0, 1, -1]
    assert oracle_page_select(x, [-1], 3, 0, 0)[1].tolist() == [0]
    x[0, 0, 5] = np.nan
    assert pick(2) == [1, 3] and pick(7) == [0, 1, 2, 3, 4, 6, 7]


@pytest.mark.parametrize("ctx", [0, 5, 16, 47])
def test_all_pages_selected_is_plain_attention(ctx):
    k, v = cache()
    table = np.array([[3, 1, 7, 0]])
    q, kn, vn = (RNG.standard_normal((1, 5, h, 4)) for h in (4, 2, 2))
    parent = np.array([[-1, 0, 0, 1, 2]])
    F = ctx // 16
    pages = np.broadcast_to(np.arange(max(1, F)), (1, 2, max(1, F)))
    a = oracle_verify_attn_pages(q, k, v, table, [ctx], kn, vn, pages, [F], parent=parent)
    b = oracle_verify_attn(q, k, v, table, [ctx], kn, vn, parent=parent)
    for x, y in zip(a, b):
        assert np.allclose(x, y)


def test_prefix_replaces_the_tables_first_pages():
    k, v = cache()
    q, kn, vn = (RNG.standard_normal((2, 3, h, 4)) for h in (4, 2, 2))
    table = np.array([[3, 1, 7, 0], [3, 1, 2, 4]])
    dirty = table.copy()
    dirty[:, :2] = -1
    a = oracle_verify_attn_prefix(q, k, v, dirty, [33, 47], kn, vn, [3, 1])
    b = oracle_verify_attn(q, k, v, table, [33, 47], kn, vn)
    for x, y in zip(a, b):
        assert np.array_equal(x, y)


DIMS = sv.make_dims(B=2, M=3, Hq=4, Hkv=2, D=128, max_blocks=4, num_blocks=9)


@pytest.mark.parametrize("kw", [dict(prefix=1, window=3), dict(pages=1, page_counts=1, window=3),
                                dict(prefix=1, pages=1, page_counts=1), dict(pages=1),
                                dict(page_counts=1), dict(prefix=1, sinks=2)])
def test_forms_of_the_attention_do_not_mix(kw):
    x = torch.zeros(1)
    kw = {k: x if k in ("prefix", "pages", "page_counts") else v for k, v in kw.items()}
    with pytest.raises(ValueError):
        sv.spec_verify_attn(x, x, x, x, x, x, x, None, x, None, DIMS, x, **kw)


def test_tensors_off_the_gpu_are_refused():
    x = torch.zeros(1)
    for call in (lambda: sv.spec_verify_attn(x, x, x, x, x, x, x, None, x, None, DIMS, x, prefix=x),
                 lambda: sv.spec_verify_attn(x, x, x, x, x, x, x, None, x, None, DIMS, x, pages=x,
                                             page_counts=x),
                 lambda: sv.spec_page_bounds(x, x, x, x, x, DIMS, x),
                 lambda: sv.spec_page_score(x, x, x, x, x, DIMS, x),
                 lambda: sv.spec_page_select(x, x, x, x, DIMS, x)):
        with pytest.raises(ValueError):
            call()
