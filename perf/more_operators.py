"""Operators of verify steps over long caches, as a measuring program calls them.

Five operators of two ways to read less of a long paged cache.  The first
serves batches whose requests begin alike:

  prefix  verify attention of requests that share a long prefix: its keys and
          values are read once for the whole batch

the others, in the order in which a step meets them, let each KV head of a
request read a few of its pages only:

  bounds  the least and largest value of every coordinate of a page's keys, for
          the pages that the last step filled
  score   how large a score a page's keys can have with any query of the step
  select  the pages of each request and KV head to be read: the first and the
          last ones and those with the largest scores
  pages   verify attention over the selected pages and the newest positions

`run` computes them in plain torch operations where `own` is false, and calls
this repository's package where it is true.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
DEV = "cuda"


def _types(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # four requests that decode behind a short common instruction: latency
        dict(name="prefix_decode_4", op="prefix", B=4, M=1, Hq=32, Hkv=8, D=128, prefix=2048,
             suf_lo=0, suf_hi=64, tree=0, dtype="bf16"),
        # trees behind a common prompt whose last page is odd, 32-bit values,
        # heads of 64
        dict(name="prefix_tree_f32", op="prefix", B=16, M=16, Hq=8, Hkv=8, D=64, prefix=2000,
             suf_lo=0, suf_hi=400, tree=4, dtype="f32"),
        # many continuations of one long document, each with its own chain
        dict(name="prefix_chain_64", op="prefix", B=64, M=5, Hq=64, Hkv=8, D=128, prefix=32768,
             suf_lo=0, suf_hi=1024, tree=0, dtype="bf16"),
        # one verify step of a batch: one or two pages a request
        dict(name="bounds_step_64", op="bounds", B=64, Hkv=8, D=128, kind="step", ctx_lo=2048,
             ctx_hi=32768, rows=6, dtype="bf16"),
        # after a prefill: every page of the prompts
        dict(name="bounds_build_16", op="bounds", B=16, Hkv=8, D=128, kind="build", ctx_lo=2000,
             ctx_hi=32768, rows=0, dtype="bf16"),
        # plain decoding of one request at a long context
        dict(name="score_decode_1", op="score", B=1, M=1, Hq=32, Hkv=8, D=128, ctx_lo=32000,
             ctx_hi=32768, dtype="bf16"),
        # the chains of a batch
        dict(name="score_chain_64", op="score", B=64, M=5, Hq=64, Hkv=8, D=128, ctx_lo=4096,
             ctx_hi=32768, dtype="bf16"),
        # one request: latency
        dict(name="select_1", op="select", B=1, Hkv=8, ctx_lo=32000, ctx_hi=32768, n_pages=64,
             first=1, last=4, ties=False),
        # a large batch at mixed lengths, with equal scores among a row's
        dict(name="select_128", op="select", B=128, Hkv=8, ctx_lo=1000, ctx_hi=131072, n_pages=255,
             first=4, last=17, ties=True),
        # plain decoding of one request over 64 of its 2000 pages
        dict(name="pages_decode_1", op="pages", B=1, M=1, Hq=32, Hkv=8, D=128, ctx_lo=32000,
             ctx_hi=32768, n_pages=64, tree=0, dtype="bf16"),
        # 64-node trees, 32-bit values, heads of 64, short contexts among them
        dict(name="pages_tree_f32", op="pages", B=8, M=64, Hq=8, Hkv=8, D=64, ctx_lo=100,
             ctx_hi=4096, n_pages=33, tree=4, dtype="f32"),
        # the chains of a large batch at long contexts
        dict(name="pages_chain_64", op="pages", B=64, M=5, Hq=64, Hkv=8, D=128, ctx_lo=1024,
             ctx_hi=32768, n_pages=256, tree=0, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefix", "bounds", "score", "select", "pages"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128, 128])
    if op == "bounds":
        B, kind = _log(rng, 1, 64), rng.choice(["step", "build"])
        hi = _log(rng, 20, 32768 if kind == "step" else max(64, min(32768, 300_000 // B)))
        return dict(op=op, B=B, Hkv=Hkv, D=D, kind=kind, ctx_lo=rng.randint(1, hi), ctx_hi=hi,
                    rows=_log(rng, 1, 64) if kind == "step" else 0, dtype=dtype)
    if op == "select":
        B, hi = _log(rng, 1, 128), _log(rng, 1000, 131072)
        # the longest requests have a choice, short ones may hold fewer pages
        n = _log(rng, 2, min(512, hi // 64))
        first = rng.randint(0, min(n - 1, 6))
        return dict(op=op, B=B, Hkv=Hkv, ctx_lo=rng.randint(0 if B > 4 else hi // 2, hi), ctx_hi=hi,
                    n_pages=n, first=first, last=rng.randint(0, min(n - 1 - first, 20)),
                    ties=rng.random() < 0.4)
    group = rng.choice([1, 2, 4, 7, 8])
    M = rng.choice([1, _log(rng, 1, 128 // group)])
    small = dtype == "f32" or D == 64
    c = dict(op=op, M=M, Hq=Hkv * group, Hkv=Hkv, D=D, dtype=dtype)
    if op == "score":
        return c | dict(B=_log(rng, 1, 16 if small else 64), ctx_lo=rng.randint(0, 2000),
                        ctx_hi=_log(rng, 2001, 16384 if small else 32768))
    c["tree"] = rng.choice([0, 0, 3]) if M > 2 else 0
    if op == "pages":
        return c | dict(B=_log(rng, 1, 16 if small else 64), ctx_lo=rng.randint(0, 2000),
                        ctx_hi=_log(rng, 2001, 32768), n_pages=_log(rng, 1, 256))
    c["B"] = _log(rng, 1, 32 if small else 64)
    rows = c["B"] * M * c["Hq"]
    most = min(32768, (20_000_000 if small else 600_000_000) // rows)
    return c | dict(prefix=BLOCK * _log(rng, 1, max(1, most // BLOCK)),
                    suf_lo=rng.choice([0, 1, 16]), suf_hi=_log(rng, 17, 1024))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2 + 1)
    rng = np.random.default_rng([int(seed), 78])
    s = {"prefix": _prepare_prefix, "bounds": _prepare_bounds, "score": _prepare_score,
         "select": _prepare_select, "pages": _prepare_pages}[case["op"]](case, rng, g)
    s["case"] = case
    if own:  # the dims and the workspace that a program keeps
        import speculative_decoding_verification_19_gb300 as sv
        s["sv"] = sv
        c = dict(M=1, Hq=case["Hkv"], D=128, dtype="bf16") | case
        s["dims"] = sv.make_dims(B=c["B"], M=c["M"], Hq=c["Hq"], Hkv=c["Hkv"], D=c["D"],
                                 max_blocks=s["max_blocks"], num_blocks=s["num_blocks"],
                                 kv_dtype=_types(c))
        s["ws"] = sv.workspace(s["dims"])
    return s


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


def _normal(g, dt, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dt)


def _tree(case, rng):
    if not case["tree"]:
        return None
    B, M = case["B"], case["M"]
    n = np.arange(M)[None, :]
    parent = np.maximum(0, n - 1 - rng.integers(0, case["tree"], (B, M)))
    parent[:, 0] = -1
    return _i32(parent)


def _new_rows(case, g):
    """Queries, new keys and values, and the outputs' buffers of a step."""
    B, M, Hq, Hkv, D = (case[x] for x in ("B", "M", "Hq", "Hkv", "D"))
    dt = _types(case)
    return dict(q=_normal(g, dt, B, M, Hq, D), k_new=_normal(g, dt, B, M, Hkv, D),
                v_new=_normal(g, dt, B, M, Hkv, D),
                out=torch.empty(B, M, Hq, D, dtype=dt, device=DEV),
                lse=torch.empty(B, M, Hq, dtype=torch.float32, device=DEV))


def _tables(ctx, mb, rng):
    """Block tables of requests that hold all their pages, and the size of a cache
    that would do for the longest."""
    pages = -(-ctx // BLOCK)
    held = np.arange(mb)[None, :] < pages[:, None]
    nb = held.size + 3
    table = np.full(held.shape, -1, dtype=np.int64)
    table[held] = rng.permutation(nb)[:int(held.sum())]
    return table, nb


def _prepare_prefix(case, rng, g):
    B, M, Hkv, D, dt = case["B"], case["M"], case["Hkv"], case["D"], _types(case)
    pp = case["prefix"] // BLOCK
    ctx = case["prefix"] + rng.integers(case["suf_lo"], case["suf_hi"] + 1, B)
    mb = -(-(case["prefix"] + case["suf_hi"] + M) // BLOCK)
    # the requests' own pages, then the shared ones in every table
    own_table, nb_own = _tables(ctx + M - case["prefix"], mb - pp, rng)
    shared = rng.permutation(pp) + nb_own
    table = np.concatenate([np.repeat(shared[None, :], B, 0), own_table], 1)
    nb = nb_own + pp
    return _new_rows(case, g) | dict(
        k_cache=_normal(g, dt, nb, Hkv, BLOCK, D), v_cache=_normal(g, dt, nb, Hkv, BLOCK, D),
        table=_i32(table), shared=_i32(shared), ctx=_i32(ctx), parent=_tree(case, rng),
        num_blocks=nb, max_blocks=mb)


def _prepare_bounds(case, rng, g):
    B, Hkv, D, dt = case["B"], case["Hkv"], case["D"], _types(case)
    ctx = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, B)
    start = np.zeros(B, dtype=np.int64)
    if case["kind"] == "step":  # the last step kept some of its rows
        start = np.maximum(0, ctx - rng.integers(1, case["rows"] + 1, B))
    mb = -(-case["ctx_hi"] // BLOCK)
    if case["kind"] == "step":  # a cache of its own size is not needed: few pages are met
        nb = B * (2 + case["rows"] // BLOCK + 1) + 3
        table = np.full((B, mb), -1, dtype=np.int64)
        page = np.arange(mb)[None, :]
        held = (page >= (start // BLOCK)[:, None]) & (page < (-(-ctx // BLOCK))[:, None])
        table[held] = rng.permutation(nb)[:int(held.sum())]
    else:
        table, nb = _tables(ctx, mb, rng)
    return dict(k_cache=_normal(g, dt, nb, Hkv, BLOCK, D), table=_i32(table), start=_i32(start),
                ctx=_i32(ctx), bounds=torch.zeros(nb, Hkv, 2, D, dtype=dt, device=DEV),
                num_blocks=nb, max_blocks=mb)


def _prepare_score(case, rng, g):
    B, M, Hq, Hkv, D, dt = (*(case[x] for x in ("B", "M", "Hq", "Hkv", "D")), _types(case))
    ctx = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, B)
    mb = -(-(case["ctx_hi"] + M) // BLOCK)
    table, nb = _tables(ctx, mb, rng)
    # 16 normal values lie between about -1.8 and 1.8
    pair = _normal(g, torch.float32, nb, Hkv, 2, D) * 0.5
    pair += 1.77 * torch.tensor([-1.0, 1.0], device=DEV)[:, None]
    bounds = torch.sort(pair, dim=2)[0].to(dt)
    return dict(q=_normal(g, dt, B, M, Hq, D), bounds=bounds, table=_i32(table), ctx=_i32(ctx),
                scores=torch.empty(B, Hkv, mb, dtype=torch.float32, device=DEV),
                num_blocks=nb, max_blocks=mb)


def _prepare_select(case, rng, g):
    B, Hkv, n = case["B"], case["Hkv"], case["n_pages"]
    ctx = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, B)
    mb = max(1, -(-(case["ctx_hi"] + 8) // BLOCK))
    scores = _normal(g, torch.float32, B, Hkv, mb) * 12 + 140
    if case["ties"]:
        scores = torch.round(scores)
    full = _i32(ctx // BLOCK)
    scores[(torch.arange(mb, device=DEV) >= full[:, None])[:, None].expand(B, Hkv, mb)] = -math.inf
    return dict(scores=scores, ctx=_i32(ctx),
                pages=torch.empty(B, Hkv, n, dtype=torch.int32, device=DEV),
                counts=torch.empty(B, dtype=torch.int32, device=DEV), num_blocks=1, max_blocks=mb)


def _prepare_pages(case, rng, g):
    B, M, Hkv, D, n, dt = (*(case[x] for x in ("B", "M", "Hkv", "D", "n_pages")), _types(case))
    ctx = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, B)
    mb = -(-(case["ctx_hi"] + M) // BLOCK)
    table, nb = _tables(ctx + M, mb, rng)
    # a choice for every request and KV head: a random set of its full pages
    full, F = ctx // BLOCK, max(1, case["ctx_hi"] // BLOCK)
    counts = np.minimum(full, n)
    key = torch.rand(B, Hkv, F, generator=g, device=DEV)
    key = torch.where(torch.arange(F, device=DEV) < _i32(full)[:, None, None], key, 2.0)
    pick = torch.sort(key, dim=-1)[1][..., :n]
    pick = torch.nn.functional.pad(pick, (0, n - pick.shape[-1]))
    on = torch.arange(n, device=DEV) < _i32(counts)[:, None, None]
    pick = torch.sort(torch.where(on, pick, F), dim=-1)[0]
    pages = torch.where(on, pick, -1).to(torch.int32).contiguous()
    return _new_rows(case, g) | dict(
        k_cache=_normal(g, dt, nb, Hkv, BLOCK, D), v_cache=_normal(g, dt, nb, Hkv, BLOCK, D),
        table=_i32(table), ctx=_i32(ctx), parent=_tree(case, rng), pages=pages,
        counts=_i32(counts), num_blocks=nb, max_blocks=mb)


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if op == "prefix" or op == "pages":
        if own:
            kw = (dict(prefix=s["shared"]) if op == "prefix" else
                  dict(pages=s["pages"], page_counts=s["counts"]))
            s["sv"].spec_verify_attn(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"],
                                     s["table"], s["ctx"], s["parent"], s["out"], s["lse"],
                                     s["dims"], s["ws"], **kw)
        elif op == "prefix":
            _plain_prefix(s, case)
        else:
            _plain_pages(s, case)
        return {k: s[k] for k in ("out", "lse", "k_cache", "v_cache")}
    if op == "bounds":
        if own:
            s["sv"].spec_page_bounds(s["k_cache"], s["table"], s["start"], s["ctx"], s["bounds"],
                                     s["dims"], s["ws"])
        else:
            _plain_bounds(s, case)
        return {"bounds": s["bounds"]}
    if op == "score":
        if own:
            s["sv"].spec_page_score(s["q"], s["bounds"], s["table"], s["ctx"], s["scores"],
                                    s["dims"], s["ws"])
        else:
            _plain_score(s, case)
        return {"scores": s["scores"]}
    if own:
        s["sv"].spec_page_select(s["scores"], s["ctx"], s["pages"], s["counts"], s["dims"], s["ws"],
                                 first=case["first"], last=case["last"])
    else:
        _plain_select(s, case)
    return {"pages": s["pages"], "counts": s["counts"]}


def _append(s, case):
    """The new rows into the cache, and the rest of the last page cleared."""
    B, M, ctx = case["B"], case["M"], s["ctx"].long()
    end = (ctx + M + BLOCK - 1) // BLOCK * BLOCK
    at = ctx[:, None] + torch.arange(M + BLOCK - 1, device=DEV)
    at = torch.where(at < end[:, None], at, ctx[:, None])  # past the page: the first row again
    src = (at - ctx[:, None]).clamp(max=M)
    pick = torch.arange(B, device=DEV)[:, None]
    blk = s["table"].long().gather(1, at // BLOCK)
    pad = torch.nn.functional.pad
    s["k_cache"][blk, :, at % BLOCK] = pad(s["k_new"], (0, 0, 0, 0, 0, 1))[pick, src]
    s["v_cache"][blk, :, at % BLOCK] = pad(s["v_new"], (0, 0, 0, 0, 0, 1))[pick, src]


def _see_tail(s, case, pos):
    """[B, M, P]: whether row i sees position pos[b, j], a cached one or a new one
    of its own path (-1: none)."""
    B, M, ctx = case["B"], case["M"], s["ctx"].long()
    node = torch.arange(M, device=DEV)
    if s["parent"] is None:
        anc = (node[None, :] <= node[:, None]).expand(B, M, M)
    else:
        step = (s["parent"][:, :, None] == node).double() + torch.eye(M, device=DEV).double()
        anc = torch.linalg.matrix_power(step, M) > 0.5
    new = pos >= ctx[:, None]
    k_node = (pos - ctx[:, None]).clamp(0, M - 1)
    see = ~new[:, None, :] | anc.gather(2, k_node[:, None, :].expand(B, M, pos.shape[1]))
    return see & (pos >= 0)[:, None, :]


def _grouped(x, Hkv):
    """[B, M, Hq, D] as [B, Hkv, M * group, D] in 32 bits."""
    B, M, Hq, D = x.shape
    g = Hq // Hkv
    return x.float().view(B, M, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, M * g, D)


def _finish(s, case, parts):
    """Softmax over all parts: pairs of scores [B, Hkv, M * group, P] and a
    function that multiplies weights with the part's values."""
    B, M, Hq, Hkv, D = (case[x] for x in ("B", "M", "Hq", "Hkv", "D"))
    m = torch.stack([sc.amax(-1) for sc, _ in parts]).amax(0)[..., None]
    z, o = 0, 0
    for sc, times in parts:
        e = torch.exp(sc - m)
        z = z + e.sum(-1, keepdim=True)
        o = o + times(e)
    g = Hq // Hkv
    o = (o / z).view(B, Hkv, M, g, D).permute(0, 2, 1, 3, 4)
    s["out"].copy_(o.reshape(B, M, Hq, D))
    s["lse"].copy_((m + z.log()).view(B, Hkv, M, g).permute(0, 2, 1, 3).reshape(B, M, Hq))


def _plain_prefix(s, case):
    B, M, Hq, Hkv, D, P = (case[x] for x in ("B", "M", "Hq", "Hkv", "D", "prefix"))
    R = M * Hq // Hkv
    ctx, table = s["ctx"].long(), s["table"].long()
    _append(s, case)
    q = _grouped(s["q"], Hkv) / math.sqrt(D)
    # the prefix: all rows of the batch against its keys
    sh = s["shared"].long()
    K = s["k_cache"][sh].float().transpose(0, 1).reshape(Hkv, P, D)
    V = s["v_cache"][sh].float().transpose(0, 1).reshape(Hkv, P, D)
    rows = q.transpose(0, 1).reshape(Hkv, B * R, D)
    sc = torch.matmul(rows, K.transpose(1, 2)).view(Hkv, B, R, P).transpose(0, 1)

    def of_prefix(e):
        o = torch.matmul(e.transpose(0, 1).reshape(Hkv, B * R, P), V)
        return o.view(Hkv, B, R, D).transpose(0, 1)

    # what each request has of its own
    S = case["suf_hi"] + M
    pos = (P + torch.arange(S, device=DEV)).expand(B, S)
    pos = torch.where(pos < (ctx + M)[:, None], pos, -1)
    see = _see_tail(s, case, pos)
    p = pos.clamp(min=P)
    blk = table.gather(1, p // BLOCK).clamp(min=0)
    Ko = s["k_cache"][blk, :, p % BLOCK].float().transpose(1, 2)
    Vo = s["v_cache"][blk, :, p % BLOCK].float().transpose(1, 2)
    so = torch.matmul(q, Ko.transpose(2, 3)).view(B, Hkv, M, Hq // Hkv, S)
    so = so.masked_fill(~see[:, None, :, None, :], -math.inf).view(B, Hkv, R, S)
    _finish(s, case, [(sc, of_prefix), (so, lambda e: torch.matmul(e, Vo))])


def _plain_pages(s, case):
    B, M, Hq, Hkv, D, n = (case[x] for x in ("B", "M", "Hq", "Hkv", "D", "n_pages"))
    g = Hq // Hkv
    ctx, table = s["ctx"].long(), s["table"].long()
    _append(s, case)
    q = _grouped(s["q"], Hkv) / math.sqrt(D)
    # the selected pages of each KV head
    on = torch.arange(n, device=DEV) < s["counts"].long()[:, None]
    page = torch.where(on[:, None, :], s["pages"].long(), 0)
    blk = table[:, None, :].expand(B, Hkv, table.shape[1]).gather(2, page).clamp(min=0)
    head = torch.arange(Hkv, device=DEV)[None, :, None]
    K = s["k_cache"][blk, head].float().reshape(B, Hkv, n * BLOCK, D)
    V = s["v_cache"][blk, head].float().reshape(B, Hkv, n * BLOCK, D)
    sc = torch.matmul(q, K.transpose(2, 3))
    sc = sc.masked_fill(~on.repeat_interleave(BLOCK, 1)[:, None, None, :], -math.inf)
    # from the first position of the last page of the context on
    S = BLOCK - 1 + M
    pos = (ctx // BLOCK * BLOCK)[:, None] + torch.arange(S, device=DEV)
    pos = torch.where(pos < (ctx + M)[:, None], pos, -1)
    see = _see_tail(s, case, pos)
    p = torch.where(pos >= 0, pos, ctx[:, None])
    tb = table.gather(1, p // BLOCK)
    Ko = s["k_cache"][tb, :, p % BLOCK].float().transpose(1, 2)
    Vo = s["v_cache"][tb, :, p % BLOCK].float().transpose(1, 2)
    so = torch.matmul(q, Ko.transpose(2, 3)).view(B, Hkv, M, g, S)
    so = so.masked_fill(~see[:, None, :, None, :], -math.inf).view(B, Hkv, M * g, S)
    _finish(s, case, [(sc, lambda e: torch.matmul(e, V)), (so, lambda e: torch.matmul(e, Vo))])


def _plain_bounds(s, case):
    ctx, start, table = s["ctx"].long(), s["start"].long(), s["table"].long()
    mb = table.shape[1]
    # pages that a request may have to do, from its first one on
    n = -(-case["rows"] // BLOCK) + 1 if case["kind"] == "step" else mb
    page = (start // BLOCK)[:, None] + torch.arange(n, device=DEV)
    todo = page * BLOCK < ctx[:, None]
    blk = table.gather(1, page.clamp(max=mb - 1))[todo]
    length = (ctx[:, None] - page * BLOCK).clamp(max=BLOCK)[todo]
    keys = s["k_cache"][blk].float()  # [pages, Hkv, 16, D]
    hide = (torch.arange(BLOCK, device=DEV) >= length[:, None])[:, None, :, None]
    lo = keys.masked_fill(hide, math.inf).amin(2)
    hi = keys.masked_fill(hide, -math.inf).amax(2)
    s["bounds"][blk] = torch.stack([lo, hi], 2).to(s["bounds"].dtype)


def _plain_score(s, case):
    B, Hkv, mb = s["scores"].shape
    q = _grouped(s["q"], Hkv)
    pair = s["bounds"][s["table"].long().clamp(min=0)].float()  # [B, mb, Hkv, 2, D]
    lo, hi = pair[:, :, :, 0].permute(0, 2, 3, 1), pair[:, :, :, 1].permute(0, 2, 3, 1)
    sc = torch.matmul(q.clamp(min=0), hi) + torch.matmul(q.clamp(max=0), lo)
    full = torch.arange(mb, device=DEV) < (s["ctx"].long() // BLOCK)[:, None]
    s["scores"].copy_(torch.where(full[:, None, :], sc.amax(2), -math.inf))


def _plain_select(s, case):
    B, Hkv, mb = s["scores"].shape
    n = case["n_pages"]
    full = (s["ctx"].long() // BLOCK)[:, None, None]
    page = torch.arange(mb, device=DEV)
    there = (page < full).expand(B, Hkv, mb)
    kept = there & ((page < case["first"]) | (page >= full - case["last"]))
    # kept pages first, then by score, the lower page first among equal ones
    order = torch.sort(s["scores"], dim=-1, descending=True, stable=True)[1]
    rank = kept.gather(2, order).int() * 2 + there.gather(2, order).int()
    order = order.gather(2, torch.sort(rank, dim=-1, descending=True, stable=True)[1])
    order = torch.nn.functional.pad(order[..., :n], (0, max(0, n - mb)))
    count = full.clamp(max=n)
    on = torch.arange(n, device=DEV) < count
    pick = torch.sort(torch.where(on, order, mb), dim=-1)[0]
    s["pages"].copy_(torch.where(on, pick, -1))
    s["counts"].copy_(count[:, 0, 0])


# --------------------------------------------------------------------------
# work and exact values
# --------------------------------------------------------------------------

def _mean_min(lo, hi, most):
    """Mean of min(x, most) over whole x from lo to hi."""
    below = max(0, min(hi, most) - lo + 1)
    return (below * (lo + min(hi, most)) / 2 + max(0, hi - max(lo, most + 1) + 1) * most) / (hi - lo + 1)


def work(case):
    op, e = case["op"], 2 if case.get("dtype") == "bf16" else 4
    B, Hkv = case["B"], case["Hkv"]
    mean = (case.get("ctx_lo", 0) + case.get("ctx_hi", 0)) / 2
    if op == "select":
        F = mean / BLOCK
        return dict(bytes=B * Hkv * 4 * (F + case["n_pages"]) + 8 * B, flops=2 * B * Hkv * F)
    D = case["D"]
    if op == "bounds":
        tokens = B * (mean if case["kind"] == "build" else (case["rows"] + 1) / 2 + 8)
        return dict(bytes=tokens * Hkv * D * e * (1 + 2 / BLOCK) + 12 * B, flops=2 * tokens * Hkv * D)
    M, Hq = case["M"], case["Hq"]
    if op == "score":
        P = B * mean / BLOCK
        return dict(bytes=P * Hkv * 2 * D * e + B * M * Hq * D * e + P * 4 + P * Hkv * 4,
                    flops=4 * P * M * Hq * D)
    # queries, outputs, new rows and their place in the cache
    b = 2 * B * M * Hq * D * e + 4 * B * M * Hkv * D * e + 4 * B * M * Hq
    if op == "prefix":
        P, suf = case["prefix"], B * (case["suf_lo"] + case["suf_hi"]) / 2
        return dict(bytes=b + 2 * (P + suf) * Hkv * D * e,
                    flops=4 * Hq * M * D * (B * P + suf + B * M / 2))
    keys = B * (BLOCK * _mean_min(case["ctx_lo"] // BLOCK, case["ctx_hi"] // BLOCK, case["n_pages"]) + 7.5)
    return dict(bytes=b + 2 * keys * Hkv * D * e + 4 * B * Hkv * case["n_pages"],
                flops=4 * Hq * M * D * (keys + B * M / 2))


def exact(case, seed):
    op = case["op"]
    if op == "select":
        return None  # whole numbers only
    s = prepare(case, seed)
    if op == "bounds":
        return _exact_bounds(s, case)
    return _exact_score(s, case) if op == "score" else _exact_attn(s, case)


def _exact_attn(s, case):
    """One request after another, over the keys that each KV head sees."""
    B, M, Hq, Hkv, D = (case[x] for x in ("B", "M", "Hq", "Hkv", "D"))
    ctx, table = s["ctx"].tolist(), s["table"].cpu().numpy()
    parents = None if s["parent"] is None else s["parent"].tolist()
    lists = s["pages"].cpu().numpy() if case["op"] == "pages" else None
    out = torch.empty(B, M, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, M, Hq, dtype=torch.float64, device=DEV)
    for b in range(B):
        c = ctx[b]
        see = np.zeros((M, M), dtype=bool)
        for i in range(M):
            k = i
            while k >= 0:
                see[i, k] = True
                k = k - 1 if parents is None else parents[b][k]
        hide = torch.from_numpy(~see).to(DEV)
        for h in range(Hkv):
            if lists is None:
                cached = np.arange(c)
            else:
                chosen = lists[b, h][lists[b, h] >= 0]
                cached = (chosen[:, None] * BLOCK + np.arange(BLOCK)).reshape(-1)
                cached = np.concatenate([cached, np.arange(c // BLOCK * BLOCK, c)])
            at = cached.astype(np.int64)
            blk = torch.from_numpy(table[b][at // BLOCK].astype(np.int64)).to(DEV)
            off = torch.from_numpy(at % BLOCK).to(DEV)
            K = torch.cat([s["k_cache"][blk, h, off], s["k_new"][b, :, h]]).double()
            V = torch.cat([s["v_cache"][blk, h, off], s["v_new"][b, :, h]]).double()
            q = s["q"][b].double().view(M, Hkv, Hq // Hkv, D)[:, h]
            sc = torch.einsum("mgd,pd->gmp", q, K) * D ** -0.5
            sc[:, :, len(at):].masked_fill_(hide, -math.inf)
            hs = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            lse[b, :, hs] = torch.logsumexp(sc, -1).T
            out[b, :, hs] = torch.einsum("gmp,pd->mgd", torch.softmax(sc, -1), V)
    return {"out": out, "lse": lse, "k_cache": None, "v_cache": None}


def _exact_bounds(s, case):
    """Page after page of each request, all its keys at once."""
    out = s["bounds"].double()
    ctx, start, table = s["ctx"].tolist(), s["start"].tolist(), s["table"].tolist()
    for b, c in enumerate(ctx):
        if start[b] >= c:
            continue
        p0, whole = start[b] // BLOCK, c // BLOCK
        ids = torch.tensor(table[b][p0:whole], dtype=torch.int64, device=DEV)
        keys = s["k_cache"][ids].double()
        out[ids] = torch.stack([torch.min(keys, 2)[0], torch.max(keys, 2)[0]], 2)
        if c % BLOCK:
            keys = s["k_cache"][table[b][whole], :, :c % BLOCK].double()
            out[table[b][whole]] = torch.stack([torch.min(keys, 1)[0], torch.max(keys, 1)[0]], 1)
    return {"bounds": out}


def _exact_score(s, case):
    """For each request and query the larger of the two products, coordinate by
    coordinate."""
    B, M, Hq, Hkv, D = (case[x] for x in ("B", "M", "Hq", "Hkv", "D"))
    out = torch.full(s["scores"].shape, -math.inf, dtype=torch.float64, device=DEV)
    for b, c in enumerate(s["ctx"].tolist()):
        F = c // BLOCK
        pair = s["bounds"][s["table"][b, :F].long()].double()  # [F, Hkv, 2, D]
        q = s["q"][b].double().view(M, Hkv, Hq // Hkv, D)
        for h in range(Hkv):
            mid = (pair[:, h, 0] + pair[:, h, 1]) / 2
            half = (pair[:, h, 1] - pair[:, h, 0]) / 2
            rows = q[:, h].reshape(-1, D)
            out[b, h, :F] = (mid @ rows.T + half @ rows.abs().T).amax(1)
    return {"scores": out}
