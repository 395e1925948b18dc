"""What calls share: one workspace among calls of different dims."""
import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import speculative_decoding_verification_19_gb300 as sv  # noqa: E402
from harness import to_dev  # noqa: E402
from synth import kv_inputs_host, workload  # noqa: E402
from test_gpu_step import BF, I32, Pages  # noqa: E402


def attention(M, B, impl, ws=None, window=200):
    """Dims, and the call's outputs on a workspace."""
    wl = workload("chain_gqa_128k").scaled(gamma=M - 1, Hq=8, Hkv=2)
    kv = kv_inputs_host(wl, seed=M, B=B, ctx=np.linspace(0, 900, B).astype(int))
    dims = sv.make_dims(B=B, M=M, Hq=8, Hkv=2, D=128, max_blocks=kv["max_blocks"],
                        num_blocks=kv["num_blocks"], attn_impl=impl)
    if ws is None:
        ws = sv.workspace(dims)
    q, kn, vn, kc, vc = (to_dev(kv[k], BF) for k in ("q", "k_new", "v_new", "k_cache", "v_cache"))
    out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:3], float("nan"), device="cuda")
    sv.spec_verify_attn(q, kn, vn, kc, vc, to_dev(kv["block_table"], I32),
                        to_dev(kv["ctx_lens"], I32), None, out, lse, dims, ws, window=window, sinks=3)
    assert sv.device_status(ws) == 0
    return dims, out, lse


@pytest.mark.parametrize("impl", [sv.ATTN_TENSOR_CORES, sv.ATTN_CUDA_CORES])
def test_one_workspace_for_calls_of_different_dims(impl):
    """Attention of six rows and of one row a request, and block tables over
    several CTAs, take turns on one workspace."""
    cases = [(6, 40), (1, 5), (3, 17)]
    want = {c: attention(*c, impl) for c in cases}
    st = Pages(40, 700, 20000)
    size = max([sv.workspace_size(d) for d, _, _ in want.values()] + [st.ws.numel()])
    st.ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    ctx = np.zeros(40, np.int64)
    n = np.full(40, 300)
    n[3], n[7] = 0, 1
    start = np.concatenate([[0], np.cumsum(n)])
    for step in range(6):
        for c in cases:
            _, out, lse = attention(*c, impl, ws=st.ws)
            assert torch.equal(out, want[c][1]) and torch.equal(lse, want[c][2])
            # 11102 rows: several CTAs; lengths grow, and some requests end
            got = st.call(ctx, start, int(start[-1]) + 1)
            assert got["ok"].sum() == (ctx >= 0).sum()
            ctx = np.where(ctx < 0, 0, ctx + n)
            ctx[step % 3::5] = -1
