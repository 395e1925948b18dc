"""Calls on long caches that share a workspace: at the same time where the header allows it,
in turn where it asks for that.

Tolerances as in test_gpu_long.py."""
import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import speculative_decoding_verification_19_gb300 as sv  # noqa: E402
from harness import to_dev  # noqa: E402
from oracle import oracle_page_bounds, oracle_page_score, oracle_page_select  # noqa: E402
from test_gpu_long import BF, F32, I32, Step, choose  # noqa: E402
from test_gpu_long_paths import attention64, tree  # noqa: E402


@pytest.mark.parametrize("dt,D", [(BF, 128), (BF, 64), (F32, 128)])
def test_bounds_scores_and_selections_side_by_side(dt, D):
    """Three batches on three streams, five turns, one workspace of 16 bytes."""
    shapes = [(9, 3, 4, 2), (30, 5, 16, 8), (4, 16, 8, 1)]
    steps = [Step([900 + 140 * b for b in range(B)], M, Hq, Hkv, D, dt, B)
             for B, M, Hq, Hkv in shapes]
    streams = [torch.cuda.Stream() for _ in steps]
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    held = []
    for st in steps:
        held.append(dict(
            q=to_dev(st.q, dt), table=to_dev(st.table, I32), ctx=to_dev(st.ctx, I32),
            bounds=torch.zeros(st.nb, st.Hkv, 2, D, dtype=dt, device="cuda"),
            scores=torch.empty(st.B, st.Hkv, st.mb, device="cuda"),
            pages=torch.empty(st.B, st.Hkv, 17, dtype=I32, device="cuda"),
            counts=torch.empty(st.B, dtype=I32, device="cuda")))
    torch.cuda.synchronize()
    for turn in range(5):
        for st, s, x in zip(steps, streams, held):
            with torch.cuda.stream(s):
                for k in ("bounds", "scores"):
                    x[k].fill_(float("nan"))
                x["counts"].fill_(-3)
            sv.spec_page_bounds(st.kc, x["table"], None, x["ctx"], x["bounds"], st.dims, ws, stream=s)
            sv.spec_page_score(x["q"], x["bounds"], x["table"], x["ctx"], x["scores"], st.dims, ws,
                               stream=s)
            sv.spec_page_select(x["scores"], x["ctx"], x["pages"], x["counts"], st.dims, ws, first=1,
                                last=3, stream=s)
    torch.cuda.synchronize()
    assert sv.device_status(ws) == 0
    for st, x in zip(steps, held):
        want = oracle_page_bounds(st.k, st.table, None, st.ctx, np.full(x["bounds"].shape, np.nan))
        assert np.array_equal(x["bounds"].double().cpu().numpy(), want, equal_nan=True)
        ref, size = oracle_page_score(st.q, want, st.table, st.ctx)
        got, there = x["scores"].double().cpu().numpy(), np.isfinite(ref)
        assert np.all(got[~there] == -np.inf)
        assert np.all(np.abs(got[there] - ref[there]) <= 2 * D * 2.0 ** -24 * size[there])
        sel, cnt = oracle_page_select(got, st.ctx, 17, 1, 3)
        assert np.array_equal(x["pages"].cpu().numpy(), sel)
        assert np.array_equal(x["counts"].cpu().numpy(), cnt)


@pytest.mark.parametrize("dt,D", [(BF, 128), (BF, 64), (F32, 64)])
def test_attention_on_two_streams(dt, D):
    """Both forms, a workspace for each stream: outputs and caches."""
    steps = [Step([900 + 40 * b for b in range(9)], 3, 4, 2, D, dt, seed, shared=4) for seed in (1, 2)]
    streams = [torch.cuda.Stream() for _ in steps]
    lists = [choose(st.rng, st.ctx, 2, 12) for st in steps]
    ins = [[to_dev(x, dt) for x in (st.q, st.kn, st.vn)] +
           [to_dev(x, I32) for x in (st.table, st.ctx, st.shared, *ls)] for st, ls in zip(steps, lists)]
    outs = [[torch.empty_like(i[0]) for _ in range(2)] + [torch.empty(9, 3, 4, device="cuda")
                                                          for _ in range(2)] for i in ins]
    torch.cuda.synchronize()
    for turn in range(5):
        for st, s, i, o in zip(steps, streams, ins, outs):
            q, kn, vn, table, ctx, shared, pages, counts = i
            args = (q, kn, vn, st.kc, st.vc, table, ctx, None)
            sv.spec_verify_attn(*args, o[0], o[2], st.dims, st.ws, prefix=shared, stream=s)
            sv.spec_verify_attn(*args, o[1], o[3], st.dims, st.ws, pages=pages, page_counts=counts,
                                stream=s)
    torch.cuda.synchronize()
    for st, o, (ls, cnt) in zip(steps, outs, lists):
        assert sv.device_status(st.ws) == 0
        for j, (ref, size) in enumerate((attention64(st), attention64(st, ls, cnt))):
            st.out, st.lse = o[j], o[2 + j]
            st.check(ref, size)
            st.check_cache(ref)


def test_batches_of_different_dims_take_turns_on_one_workspace():
    """Prefix (in a pass, and read by the requests), pages, window and plain calls of three
    batches on a workspace of the largest one's size, never zeroed in between."""
    steps = [Step([3216 + 3 * b for b in range(48)], 4, 8, 2, 128, BF, 1, shared=201),
             Step([1040 + 9 * b for b in range(30)], 33, 4, 2, 64, F32, 2, shared=65),
             Step([700, 720], 9, 14, 2, 128, BF, 3, shared=40),
             Step([1616 + 9 * b for b in range(20)], 5, 8, 2, 64, BF, 4, shared=101)]
    room = torch.zeros(max(sv.workspace_size(st.dims) for st in steps), dtype=torch.uint8,
                       device="cuda")
    todo = []
    for st in steps:
        st.parent = tree(st.rng, st.B, st.M, 3)
        st.ws = room
        whole, (lists, cnt) = attention64(st), choose(st.rng, st.ctx, 2, 20)
        some = attention64(st, lists, cnt)
        shared = to_dev(st.shared, I32)
        todo.append([(dict(prefix=shared), whole), (dict(), whole),
                     (dict(pages=to_dev(lists, I32), page_counts=to_dev(cnt, I32)), some),
                     (dict(window=1 << 20), whole), (dict(prefix=shared[:2]), whole)])
    for turn in range(2):
        for j in range(5):
            for i, st in enumerate(steps):
                kw, (ref, size) = todo[i][(j + 2 * i + turn) % 5]
                assert st.call(**kw) == 0
                st.check(ref, size)
                st.check_cache(ref)
