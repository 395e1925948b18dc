"""Selected pages of a long cache, fp64 on the CPU.

Bounds of a page's keys (least and largest value of every coordinate), the
largest score that a key between them can have with any query that reads the
KV head, the pages that are then read, and verify attention over those: of
the cached positions a row sees the ones in its KV head's selected pages and
the ones in the last, partial page (page 1 §2.1: every row sees what precedes
it; here less of it).

Also the verify attention of requests that begin with the same pages: the
result is that of the requests' whole tables.
"""
from __future__ import annotations

import numpy as np

from .attention import ancestors_or_self, oracle_kv_append, oracle_verify_attn


def oracle_page_bounds(k_cache, block_table, from_lens, ctx_lens, bounds, block=16):
    """bounds [num_blocks, Hkv, 2, D] with the pages that a request has from
    position from_lens on, up to ctx_lens, brought up to date (a copy)."""
    out = np.array(bounds, dtype=np.float64)
    for b in range(len(ctx_lens)):
        start = 0 if from_lens is None else int(from_lens[b])
        for p in range(start // block, -(-int(ctx_lens[b]) // block)):
            n = min(block, int(ctx_lens[b]) - p * block)
            keys = np.asarray(k_cache[block_table[b, p], :, :n], dtype=np.float64)
            out[block_table[b, p], :, 0] = keys.min(1)
            out[block_table[b, p], :, 1] = keys.max(1)
    return out


def oracle_page_score(q, bounds, block_table, ctx_lens, block=16):
    """(scores [B, Hkv, max_blocks], the sum of |products| of the largest row)."""
    q = np.asarray(q, dtype=np.float64)
    B, M, Hq, D = q.shape
    Hkv = bounds.shape[1]
    scores = np.full((B, Hkv, block_table.shape[1]), -np.inf)
    size = np.zeros_like(scores)
    for b in range(B):
        for p in range(max(0, int(ctx_lens[b])) // block):
            pair = np.asarray(bounds[block_table[b, p]], dtype=np.float64)
            for h in range(Hkv):
                rows = q[b].reshape(M, Hkv, Hq // Hkv, D)[:, h].reshape(-1, 1, D)
                best = np.maximum(rows * pair[h, 0], rows * pair[h, 1])[:, 0]
                scores[b, h, p] = best.sum(-1).max()
                size[b, h, p] = (np.abs(rows) * np.abs(pair[h]).max(0)).sum(-1).max()
    return scores, size


def oracle_page_select(scores, ctx_lens, n_pages, first, last, block=16):
    """(pages [B, Hkv, n_pages], counts [B]): one page after another."""
    B, Hkv, mb = scores.shape
    pages = np.full((B, Hkv, n_pages), -1, np.int64)
    counts = np.zeros(B, np.int64)
    for b in range(B):
        c = int(ctx_lens[b])
        full = c // block if 0 < c <= mb * block else 0
        counts[b] = min(full, n_pages)
        for h in range(Hkv):
            x = np.asarray(scores[b, h, :full], dtype=np.float64)
            key = np.where(np.isnan(x), -np.inf, x)
            left = list(range(full))
            if full > n_pages:
                must = set(range(first)) | set(range(full - last, full))
                # NaN after -inf, then the lower page first
                rest = sorted((p for p in left if p not in must),
                              key=lambda p: (-key[p], np.isnan(x[p]), p))
                left = sorted(must | set(rest[:n_pages - len(must)]))
            pages[b, h, :len(left)] = left
    return pages, counts


def oracle_verify_attn_pages(q, k_cache, v_cache, block_table, ctx_lens, k_new, v_new, pages,
                             counts, parent=None, scale=None, block=16):
    """(out, lse, k_after, v_after): one row, one KV head, one key at a time."""
    q = np.asarray(q, dtype=np.float64)
    B, M, Hq, D = q.shape
    Hkv = k_new.shape[2]
    group = Hq // Hkv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out, lse = np.zeros((B, M, Hq, D)), np.zeros((B, M, Hq))
    for b in range(B):
        ctx = int(ctx_lens[b])
        par = None if parent is None else np.asarray(parent[b])
        for h in range(Hkv):
            seen = [t for p in pages[b, h, :counts[b]] for t in range(p * block, (p + 1) * block)]
            seen += list(range(ctx // block * block, ctx))
            seen = np.array(seen, dtype=np.int64)
            blk = block_table[b, seen // block]
            K0 = np.asarray(k_cache[blk, h, seen % block], dtype=np.float64)
            V0 = np.asarray(v_cache[blk, h, seen % block], dtype=np.float64)
            for i in range(M):
                path = ancestors_or_self(par, i)
                K = np.concatenate([K0, np.asarray(k_new[b, path, h], dtype=np.float64)])
                V = np.concatenate([V0, np.asarray(v_new[b, path, h], dtype=np.float64)])
                for g in range(h * group, (h + 1) * group):
                    s = K @ q[b, i, g] * scale
                    w = np.exp(s - s.max())
                    out[b, i, g] = w @ V / w.sum()
                    lse[b, i, g] = s.max() + np.log(w.sum())
    kc, vc = oracle_kv_append(k_cache, v_cache, block_table, ctx_lens, k_new, v_new, block)
    return out, lse, kc, vc


def oracle_verify_attn_prefix(q, k_cache, v_cache, block_table, ctx_lens, k_new, v_new, prefix,
                              parent=None, scale=None, block=16):
    """Verify attention where every request's first pages are those of `prefix`."""
    table = np.array(block_table)
    table[:, :len(prefix)] = np.asarray(prefix)[None, :]
    return oracle_verify_attn(q, k_cache, v_cache, table, ctx_lens, k_new, v_new, parent=parent,
                              scale=scale, block=block)
