"""How near spec_sample's weights and probabilities are to the definition's.

Tolerances.  A weight is off by at most 2^-28.9 of its value: the exponent's
rest r, up to 2^-6 and a little, is rounded to fp32 (2^-30 in log2 units), and
so are the last product and sum of the series for 2^r - 1 (2^-31 each) and the
table's low word, 2^-25, goes without its product with the series (2^-31.5).
The first CTA's list holds weights to 2^-41 of the largest one, 3584 of them at
most (2^-29.2 of their sum); sums add 2^-40.  A probability is a weight over a
sum of weights, so it is off by at most twice 2^-28.9 and 2^-29.2, and rounded
once (2^-24).
"""
import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import speculative_decoding_verification_19_gb300 as sv  # noqa: E402

F32, I32 = torch.float32, torch.int32
PROB = 2.0 ** -24 + 2 * 2.0 ** -28.9 + 2.0 ** -29.2


def draw(x, T, u, **kw):
    tok = torch.empty(len(x), dtype=I32, device="cuda")
    prob = torch.empty(len(x), device="cuda")
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    sv.spec_sample(x, T, u, tok, prob, ws, **kw)
    assert sv.device_status(ws) == 0
    return tok.long(), prob.double()


@pytest.mark.parametrize("n,V,k,min_p", [
    (4000, 60, 0, 1e-6),     # the exact draw over a row's runs
    (4000, 60, 40, 0.0),     # the list, compared pairwise
    (1500, 3000, 600, 0.0),  # the list, by selects
    (300, 9000, 5000, 0.0),  # a select over the cluster, then the exact draw
    (500, 20000, 30, 0.01)])
def test_probabilities_are_rounded_once(n, V, k, min_p):
    g = torch.Generator(device="cuda").manual_seed(V + k)
    x = torch.randn(n, V, device="cuda", generator=g) * 2
    T = torch.rand(n, device="cuda", generator=g) * 1.5 + 0.5
    u = torch.rand(n, device="cuda", generator=g)
    kw = dict(min_p=torch.full((n,), min_p, device="cuda"))
    if k:
        kw["top_k"] = torch.full((n,), k, dtype=I32, device="cuda")
    tok, prob = draw(x, T, u, **kw)
    w = torch.exp((x.double() - x.double().amax(1, keepdim=True)) / T.double()[:, None])
    if k:
        w = torch.where(x >= x.topk(k, dim=1)[0][:, -1:], w, 0)
    w = torch.where(w >= float(np.float32(min_p)), w, 0)
    p = w.gather(1, tok[:, None])[:, 0] / w.sum(1)
    err = ((prob - p).abs() / p).max().item()
    assert err <= PROB, err * 2 ** 24


@pytest.mark.parametrize("path", ["plain", "runs", "list"])
def test_tokens_beside_a_step(path):
    """Two tokens and a uniform number next to the step between them, on either
    side: the definition's token wherever it is more than 2^-28 away."""
    rng = np.random.default_rng(40)
    n = 20000
    x = np.zeros((n, 2 if path != "list" else 3), np.float32)
    x[:, 0] = -rng.uniform(0, 5, n)
    x[:, 2:] = -300.0
    T = rng.choice([0.3, 0.7, 1.0, 1.7], n).astype(np.float32)
    first = np.exp(x[:, 0].astype(np.longdouble) / T.astype(np.longdouble))
    step = first / (1 + first)
    near = step.astype(np.float32)
    kw = {}
    if path == "runs":
        kw["min_p"] = torch.full((n,), 1e-20, device="cuda")
    if path == "list":
        kw["top_k"] = torch.full((n,), 2, dtype=I32, device="cuda")
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    sure = 0
    for u in (np.nextafter(near, np.float32(0)), near, np.nextafter(near, np.float32(1))):
        u = np.minimum(u, np.float32(1 - 2.0 ** -24))
        tok, _ = draw(dev(x), dev(T), dev(u), **kw)
        want = (step <= u.astype(np.longdouble)).astype(np.int64)  # the first with C > u Z
        clear = np.abs(step - u.astype(np.longdouble)) > 2.0 ** -28
        assert np.array_equal(tok.cpu().numpy()[clear], want[clear])
        sure += clear.mean()
    # of the three sides; a count of the inputs alone (steps below 2^-4 have their
    # neighbours within 2^-28): 1.342
    assert sure > 1.3
