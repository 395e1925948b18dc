"""The forms of the attention on views keep to the workspace: nothing outside its size is
written, nothing that another call keeps in it is lost, and garbage where their tables and
partials go does no harm.

Tolerances as in test_gpu_long.py."""
import dataclasses

import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import speculative_decoding_verification_19_gb300 as sv  # noqa: E402
from harness import gpu_reject, to_dev  # noqa: E402
from oracle import oracle_verify_attn, oracle_verify_attn_pages  # noqa: E402
from synth import logits_inputs, workload  # noqa: E402
from test_gpu_long import AUTO, BF, CORES, F32, I32, TC, Step, choose  # noqa: E402

# ctx, shared positions, M, Hq, Hkv, D, dt, impl: the prefix in a pass of its own and
# read by the requests, and pages, on every path; few and many rows per KV head
SHAPES = [
    ([3216 + 3 * b for b in range(48)], 3216, 4, 8, 2, 128, BF, TC),
    ([3216 + 3 * b for b in range(48)], 3216, 4, 8, 2, 128, BF, CORES),
    ([1040 + 9 * b for b in range(30)], 1040, 9, 14, 2, 64, BF, AUTO),
    ([1040 + 9 * b for b in range(30)], 1040, 33, 4, 2, 64, F32, AUTO),
    ([1616 + 9 * b for b in range(20)], 1616, 2, 8, 2, 128, F32, AUTO),
    ([700, 710], 640, 36, 2, 2, 128, F32, AUTO),
    ([700], 640, 2, 8, 2, 128, BF, TC)]


def forms(st, lists, cnt):
    return [dict(prefix=to_dev(st.shared, I32)), dict(prefix=to_dev(st.shared[:3], I32)),
            dict(pages=to_dev(lists, I32), page_counts=to_dev(cnt, I32))]


def refs(st, lists, cnt):
    args = (st.q, st.k, st.v, st.table, st.ctx, st.kn)
    sizes = (st.q, st.k, np.abs(st.v), st.table, st.ctx, st.kn)
    whole = oracle_verify_attn(*args, st.vn), oracle_verify_attn(*sizes, np.abs(st.vn))[0]
    some = (oracle_verify_attn_pages(*args, st.vn, lists, cnt),
            oracle_verify_attn_pages(*sizes, np.abs(st.vn), lists, cnt)[0])
    return [whole, whole, some]


@pytest.mark.parametrize("ctx,P,M,Hq,Hkv,D,dt,impl", SHAPES)
def test_views_keep_to_the_workspace(ctx, P, M, Hq, Hkv, D, dt, impl):
    """The exact size between guard bytes; everything behind the counters that are zero
    between calls filled with ones before each call (no block id, NaN partials)."""
    st = Step(ctx, M, Hq, Hkv, D, dt, 5, shared=P // 16, impl=impl)
    lists, cnt = choose(st.rng, st.ctx, Hkv, 20)
    n, guard = sv.workspace_size(st.dims), 1 << 20
    room = torch.zeros(n + 2 * guard, dtype=torch.uint8, device="cuda")
    room[:guard] = room[guard + n:] = 0xAB
    st.ws = room[guard:guard + n]
    for kw, (ref, size) in zip(forms(st, lists, cnt), refs(st, lists, cnt)):
        st.ws[256:] = 0xFF
        assert st.call(**kw) == 0
        st.check(ref, size)
        st.check_cache(ref)
        assert torch.all(room[:guard] == 0xAB) and torch.all(room[guard + n:] == 0xAB)


@pytest.mark.parametrize("dt,D,impl", [(BF, 128, TC), (BF, 128, CORES), (F32, 64, AUTO)])
def test_views_between_reject_samples(dt, D, impl):
    """Reject-samples before, between and after the forms on one workspace: the same
    decisions as on a workspace of their own, so their counters are untouched."""
    B, P = 48, 3216
    wl = dataclasses.replace(workload("tiny_chain"), B=B, V=5000, Hq=8, Hkv=2, D=D,
                             dtype="bf16" if dt == BF else "f32")
    lg = logits_inputs(wl, seed=3)
    st = Step([P + 3 * b for b in range(B)], wl.M, 8, 2, D, dt, 5, shared=P // 16, impl=impl)
    st.dims = sv.make_dims(B=B, M=wl.M, Hq=8, Hkv=2, D=D, max_blocks=st.mb, num_blocks=st.nb,
                           V=wl.V, kv_dtype=dt, logits_dtype=dt, attn_impl=impl)
    lists, cnt = choose(st.rng, st.ctx, 2, 20)
    want = gpu_reject(wl, lg, 11, 5, dims=st.dims)
    st.ws = sv.workspace(st.dims)

    def sample():
        got = gpu_reject(wl, lg, 11, 5, dims=st.dims, ws=st.ws)
        assert all(np.array_equal(got[k], want[k], equal_nan=True) for k in
                   ("out_tokens", "path", "accepted_len", "probe"))

    for kw, (ref, size) in zip(forms(st, lists, cnt), refs(st, lists, cnt)):
        sample()
        assert st.call(**kw) == 0
        st.check(ref, size)
    sample()
