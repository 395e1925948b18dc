"""Elements of a head past rot_dim do not turn: without a norm their bits stay as
they are, infinities, NaN and zeros of both signs among them, and with one an
infinity or NaN spoils its own head alone.
"""
import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import speculative_decoding_verification_19_gb300 as sv  # noqa: E402
from harness import to_dev  # noqa: E402
from oracle import oracle_norm_rope  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 0), (64, 16), (128, 48), (128, 112)])
@pytest.mark.parametrize("norm", [False, True])
def test_elements_that_do_not_turn(dt, interleaved, D, rot, norm):
    rows, Hq, Hkv = 40, 5, 1
    g = torch.Generator(device="cuda").manual_seed(D + rot)
    x = torch.randn(rows, Hq + Hkv, D, device="cuda", generator=g).to(dt)
    special = torch.tensor([float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 3e38],
                           device="cuda").to(dt)
    at = torch.randint(rot, D, (rows,), generator=g, device="cuda")
    head = torch.randint(0, Hq + Hkv, (rows,), generator=g, device="cuda")
    row = torch.arange(rows, device="cuda")
    x[row, head, at] = special[row % 6]
    w = (torch.rand(D, device="cuda", generator=g) + 0.5).to(dt) if norm else None
    pos = torch.randint(0, 100000, (rows,), generator=g, device="cuda", dtype=I32)
    f = 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
    dims = sv.make_dims(B=1, M=1, Hq=Hq, Hkv=Hkv, D=D, kv_dtype=dt)
    ws = sv.workspace(dims)
    qo = torch.empty(rows, Hq, D, device="cuda", dtype=dt)
    ko = torch.empty(rows, Hkv, D, device="cuda", dtype=dt)
    sv.spec_qk_norm_rope(x[:, :Hq].contiguous(), x[:, Hq:].contiguous(), None, w, w, pos,
                         to_dev(f, torch.float64) if rot else None, qo, ko, dims, ws,
                         interleaved=interleaved)
    assert sv.device_status(ws) == 0
    got = torch.cat([qo, ko], 1)
    if not norm:
        bits = torch.int16 if dt == BF else I32
        nan = x[..., rot:].isnan()  # a NaN stays one, whatever its bits
        same = got[..., rot:].contiguous().view(bits) == x[..., rot:].contiguous().view(bits)
        assert torch.equal(got[..., rot:].isnan(), nan) and bool((same | nan).all())
    # the turned part (without a norm) and every other head are as without them
    clean = torch.ones(rows, Hq + Hkv, dtype=torch.bool, device="cuda")
    clean[row, head] = False
    ref = oracle_norm_rope(torch.where(torch.isfinite(x), x, 0).double().cpu().numpy(),
                           None if w is None else w.double().cpu().numpy(), pos.cpu().numpy(), f,
                           interleaved)
    part = slice(0, D if norm else rot)
    keep = clean if norm else torch.ones_like(clean)
    a, b = got[keep][..., part].double().cpu().numpy(), ref[keep.cpu().numpy()][..., part]
    # fp32 throughout: a pair's error is below 2^-20 of its length, the angle off by
    # position * 2^-50; one rounding to bf16, 2^-8 (standard normal values: below 8,
    # times a weight below 1.5, a pair below 17)
    tol = 17 * (2.0 ** -20 + 1e5 * 2.0 ** -50)
    assert np.all(np.abs(a - b) <= tol + (2.0 ** -8 * (np.abs(b) + tol) if dt == BF else 0))
