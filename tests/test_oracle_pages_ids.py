"""Block tables over a corrupt page state, by hand: ring and table entries that
are no block id serve no row and spread to no other request."""
import numpy as np
import pytest

from oracle import oracle_block_tables

BAD = [-1, 6, 1 << 30, -(1 << 31)]


def call(ctx, start, table, span, pool, state, rows=None, **kw):
    rows = start[-1] if rows is None else rows
    return oracle_block_tables(np.array(ctx), np.array(start), None, rows,
                               np.array(table, np.int32), np.array(span, np.int32),
                               np.array(pool, np.int32), np.array(state, np.int32),
                               np.full(rows, -9), np.full(rows, -9), 1, **kw)


@pytest.mark.parametrize("bad", BAD)
def test_a_ring_entry_that_is_no_block(bad):
    out = call([0, 0, 0], [0, 16, 48, 60], np.full((3, 3), -1), np.zeros((3, 2)),
               [0, bad, 2, 3, 4, 5], [0, 6])
    assert out["ok"].tolist() == [1, 0, 1] and out["status"] == 1 << 6
    assert out["block_table"].tolist() == [[0, -1, -1], [-1, 2, -1], [3, -1, -1]]
    assert out["slots"][:16].tolist() == list(range(16))
    assert np.all(out["slots"][16:48] == -1) and np.all(out["positions"][16:48] == -1)
    assert out["slots"][48] == 48
    # the request ends: its block goes back, the entry that was none does not
    end = call([16, -1, 12], [0, 0, 0, 0], out["block_table"], out["span"], out["pool"],
               out["pool_state"])
    assert end["pool_state"].tolist() == [4, 3] and end["status"] == 1 << 6
    free = [end["pool"][(4 + i) % 6] for i in range(3)]
    assert free == [4, 5, 2]
    # and all that is left is handed out without another error
    last = call([16, 0, 12], [0, 0, 48, 48], end["block_table"], end["span"], end["pool"],
                end["pool_state"])
    assert last["ok"].all() and last["status"] == 0
    assert last["block_table"][1].tolist() == [4, 5, 2]


@pytest.mark.parametrize("bad", BAD)
def test_a_table_entry_that_is_no_block(bad):
    table, span = [[bad, 1, -1], [2, -1, -1]], [[0, 2], [0, 1]]
    args = table, span, [3, 4, 5, -7, -7, -7], [0, 3]
    # rows on a good page of the request: it runs (the attention checks the rest)
    out = call([17, 3], [0, 2, 4], *args)
    assert out["ok"].tolist() == [1, 1] and out["status"] == 0
    # rows on the bad one do not
    out = call([15, 3], [0, 2, 4], *args)
    assert out["ok"].tolist() == [0, 1] and out["status"] == 1 << 6
    assert out["slots"].tolist() == [-1, -1, 35, 36]
    # given back, it goes nowhere
    out = call([-1, -1], [0, 0, 0], *args)
    assert out["pool"].tolist() == [3, 4, 5, 1, 2, -1] and out["pool_state"].tolist() == [0, 5]
    assert out["status"] == 1 << 6 and np.all(out["block_table"] == -1)
