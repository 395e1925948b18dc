"""Waits that run out in the calls on long caches.

A limit of a thousand SM clocks, and inputs evicted from L2 so that the first copies take
longer than that (HBM alone answers in some 1500 clocks): the calls return and their status
says so, whatever kernel waits; with the default limit, on a zeroed workspace, the same
call is right again.  Nothing here waits without a limit."""
import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import speculative_decoding_verification_19_gb300 as sv  # noqa: E402
from harness import to_dev  # noqa: E402
from oracle import oracle_page_score  # noqa: E402
from test_gpu_long import BF, I32, Step, choose, typed  # noqa: E402
from test_gpu_long_paths import attention64  # noqa: E402

TIMEOUT = 1 << 7


def limited(st, kcycles):
    """The step's dims with this limit, its workspace zeroed, L2 without its inputs."""
    st.dims = sv.make_dims(B=st.B, M=st.M, Hq=st.Hq, Hkv=st.Hkv, D=st.D, max_blocks=st.mb,
                           num_blocks=st.nb, kv_dtype=st.dt, wait_limit_kcycles=kcycles)
    st.ws.zero_()
    torch.full((96 << 20,), 1.0, device="cuda")
    torch.cuda.synchronize()


@pytest.mark.parametrize("D", [128, 64])
def test_prefix(D):
    """Heads of 64: only the pass has waits; heads of 128: the requests' own part too."""
    st = Step([3216 + b for b in range(64)], 4, 8, 2, D, BF, 5, shared=201)
    ref, size = attention64(st)
    shared = to_dev(st.shared, I32)
    limited(st, 1)
    assert st.call(prefix=shared) == TIMEOUT
    limited(st, 0)
    assert st.call(prefix=shared) == 0
    st.check(ref, size)
    st.check_cache(ref)


@pytest.mark.parametrize("B,n,M", [(1, 500, 65), (3, 100, 9), (20, 100, 9)])
def test_pages(B, n, M):
    """A few requests: the partials are merged by a kernel of their own."""
    st = Step([9000] * B, M, 2, 2, 128, BF, 5)
    lists, cnt = choose(st.rng, st.ctx, 2, n)
    ref, size = attention64(st, lists, cnt)
    kw = dict(pages=to_dev(lists, I32), page_counts=to_dev(cnt, I32))
    limited(st, 1)
    assert st.call(**kw) == TIMEOUT
    limited(st, 0)
    assert st.call(**kw) == 0
    st.check(ref, size)
    st.check_cache(ref)


@pytest.mark.parametrize("D", [128, 64])
def test_scores(D):
    st = Step([3216 + b for b in range(20)], 32, 8, 2, D, BF, 5)
    pair = typed(np.sort(st.rng.standard_normal((st.nb, 2, 2, D)), axis=2).astype(np.float32), BF)
    args = [to_dev(st.q, BF), to_dev(pair, BF), to_dev(st.table, I32), to_dev(st.ctx, I32)]
    scores = torch.empty(20, 2, st.mb, device="cuda")
    limited(st, 1)
    sv.spec_page_score(*args, scores, st.dims, st.ws)
    assert sv.device_status(st.ws) == TIMEOUT
    limited(st, 0)
    sv.spec_page_score(*args, scores, st.dims, st.ws)
    assert sv.device_status(st.ws) == 0
    ref, size = oracle_page_score(st.q, pair, st.table, st.ctx)
    got, there = scores.double().cpu().numpy(), np.isfinite(ref)
    assert np.all(got[~there] == -np.inf)
    assert np.all(np.abs(got[there] - ref[there]) <= 2 * D * 2.0 ** -24 * size[there])
