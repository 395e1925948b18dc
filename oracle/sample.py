"""One token per row from given uniforms, fp64 on the CPU.

The law of a row is the one of the verify walk (softmax at the request's
temperature, restricted by top-k and then top-p), restricted further to the
tokens of at least min_p times the largest probability; the token is drawn by
inverse CDF in vocabulary order, and temperature 0 is greedy.  min-p is not in
the pages; reading: it comes after top-k and top-p, relative to the largest
probability, as the restrictions before it keep the largest token.
"""
from __future__ import annotations

import numpy as np

from .reject_sample import filter_order, softmax_rows


def oracle_sample(logits, temperature, uniform, top_k=None, top_p=None, min_p=None):
    """Returns a dict: tokens, prob, and margin (how far u stands from the
    nearest step of the CDF and, relative, the filters' cuts from theirs);
    rows that fail have token -1, and status holds their code."""
    n, V = logits.shape
    tokens = np.full(n, -1, dtype=np.int64)
    prob = np.zeros(n)
    margin = np.full(n, np.inf)
    status = np.zeros(n, dtype=np.int64)
    tiny = np.finfo(np.float32).tiny
    for r in range(n):
        T, u = float(temperature[r]), float(uniform[r])
        k = 0 if top_k is None else int(top_k[r])
        t = 1.0 if top_p is None else float(top_p[r])
        mp = 0.0 if min_p is None else float(min_p[r])
        z = np.asarray(logits[r], dtype=np.float64)
        good_T = T == 0.0 or (tiny <= T <= np.finfo(np.float32).max)
        if not (good_T and 0 <= u < 1 and k >= 0 and 0 < t <= 1 and 0 <= mp <= 1):
            status[r] = 1
            continue
        if np.isnan(z).any() or (z == np.inf).any() or z.max() == -np.inf:
            status[r] = 5
            continue
        if T == 0.0:
            tokens[r], prob[r] = int(np.argmax(z)), 1.0
            continue
        law = softmax_rows(z[None], T)[0]
        if (0 < k < V) or t < 1.0:
            order = filter_order(z)[:k or None]
            mass = np.cumsum(law[order])
            if t < 1.0:
                cut = int(np.searchsorted(mass, t * mass[-1]))
                near = mass[max(0, cut - 1):cut + 1]
                margin[r] = np.min(np.abs(near / mass[-1] - t))
                order = order[:cut + 1]
            kept = np.zeros(V, dtype=bool)
            kept[order] = True
            law = np.where(kept, law, 0.0)
        if mp > 0.0:
            ratio = law / law.max()
            inside = ratio[ratio > 0]
            if mp < 1.0:
                margin[r] = min(margin[r], np.min(np.abs(inside / mp - 1.0)))
            law = np.where(ratio >= mp, law, 0.0)
        c = np.cumsum(law)
        i = int(np.searchsorted(c, u * c[-1], side="right"))
        tokens[r], prob[r] = i, law[i] / c[-1]
        lower = c[i - 1] if i else -np.inf
        margin[r] = min(margin[r], (c[i] - u * c[-1]) / c[-1],
                        np.inf if u == 0.0 else (u * c[-1] - lower) / c[-1])
    return dict(tokens=tokens, prob=prob, margin=margin, status=status)
