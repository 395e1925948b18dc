"""Queries that are not finite: their pages' scores say so, and so does the selection.

Tolerance of the finite scores as in test_gpu_long.py."""
import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import speculative_decoding_verification_19_gb300 as sv  # noqa: E402
from harness import to_dev  # noqa: E402
from oracle import oracle_page_score, oracle_page_select  # noqa: E402
from test_gpu_long import BF, F32, I32, NONFINITE, Step, typed  # noqa: E402

# bf16: the tensor cores to 128 rows per KV head, CUDA cores beyond
SHAPES = [(3, 1, 4, 2), (3, 5, 14, 2), (2, 33, 4, 1), (2, 128, 2, 1), (20, 2, 16, 8)]


@pytest.mark.parametrize("dt,D", [(BF, 128), (BF, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("B,M,Hq,Hkv", SHAPES)
@pytest.mark.parametrize("bad", [(np.nan,), (np.inf,), (-np.inf,), (np.inf, -np.inf)])
def test_queries_that_are_not_finite(dt, D, B, M, Hq, Hkv, bad):
    st = Step([1500 + 16 * b for b in range(B)], M, Hq, Hkv, D, dt, D + M)
    pair = np.sort(st.rng.standard_normal((st.nb, Hkv, 2, D)), axis=2)
    pair[::3] -= 2.0  # both bounds of one sign in places
    pair = typed(pair.astype(np.float32), dt)
    st.q[1, M // 2, 1, [3, D - 1][:len(bad)]] = bad  # one row of the first KV head
    scores = torch.full((B, Hkv, st.mb), -1.0, device="cuda")
    sv.spec_page_score(to_dev(st.q, dt), to_dev(pair, dt), to_dev(st.table, I32), to_dev(st.ctx, I32),
                       scores, st.dims, st.ws)
    assert sv.device_status(st.ws) == 0
    with np.errstate(invalid="ignore"):
        ref, size = oracle_page_score(st.q, pair, st.table, st.ctx)
    got = scores.double().cpu().numpy()
    there = np.isfinite(ref)
    assert np.array_equal(got[~there], ref[~there], equal_nan=True)
    assert np.all(np.abs(got[there] - ref[there]) <= 2 * D * 2.0 ** -24 * size[there])
    full = int(st.ctx[1]) // 16
    if np.isnan(bad[0]):
        assert np.all(np.isnan(got[1, 0, :full]))
    pages = torch.empty(B, Hkv, 9, dtype=I32, device="cuda")
    counts = torch.empty(B, dtype=I32, device="cuda")
    sv.spec_page_select(scores, to_dev(st.ctx, I32), pages, counts, st.dims, st.ws, first=1, last=2)
    nan = np.isnan(got[1, 0, 1:full - 2]).any()
    assert nan or len(bad) == 1 and not np.isnan(bad[0])
    assert sv.device_status(st.ws) == (NONFINITE if nan else 0)
    assert np.array_equal(pages.cpu().numpy(), oracle_page_select(got, st.ctx, 9, 1, 2)[0])
