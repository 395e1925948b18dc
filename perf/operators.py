"""Operators that run around the verify step, as a measuring program calls them.

Four operators of one serving step, in the order in which a step meets them:

  pages      block tables, slot maps and positions of the new rows, built from
             the requests' lengths (pages taken from and returned to a ring of
             free ones)
  rope       RMS norm of every query and key head with the position rotation,
             written to dense rows and, where slots are given, to the paged cache
  attn       verify attention with a sliding window and sink tokens
  sample     temperature, top-k, top-p and min-p sampling from given uniforms

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
        # one verify step of a small batch: a page now and then, and the slots
        # of six rows a request (the latency of a step that moves little)
        dict(name="pages_step_8", op="pages", B=8, max_blocks=160, kind="step", M=6, ctx_lo=2048,
             ctx_hi=2048, window=0, sinks=0, chunk=0, budget=0, short=False),
        # continuous batching: new requests prefill, others decode one token,
        # some have ended and return their pages
        dict(name="pages_ragged_512", op="pages", B=512, max_blocks=2049, kind="mixed", M=1,
             ctx_lo=1024, ctx_hi=16384, window=0, sinks=0, chunk=4096, budget=65536,
             short=False),
        # one decoded token of one request: latency
        dict(name="rope_decode_1", op="rope", rows=1, pad=0, Hq=32, Hkv=8, D=128, rot=128,
             interleaved=False, dtype="bf16", cache=False, norm=True, pos_hi=8192, strided=True),
        # the verify rows of a batch of trees, 32-bit values, half of each head
        # rotated in interleaved pairs, a padded batch
        dict(name="rope_f32_993", op="rope", rows=993, pad=31, Hq=32, Hkv=32, D=64, rot=32,
             interleaved=True, dtype="f32", cache=False, norm=True, pos_hi=4160, strided=False),
        # a prefill chunk with its keys and values written into the cache
        dict(name="rope_prefill_16384", op="rope", rows=16384, pad=0, Hq=64, Hkv=8, D=128, rot=128,
             interleaved=False, dtype="bf16", cache=True, norm=True, pos_hi=131072, strided=True),
        # plain decoding of one request at a long context
        dict(name="attn_decode_1", op="attn", B=1, M=1, Hq=32, Hkv=8, D=128, ctx_lo=32000,
             ctx_hi=32768, window=1024, sinks=4, tree=0, dtype="bf16"),
        # chains of a mixed batch, some contexts inside the window
        dict(name="attn_chain_32", op="attn", B=32, M=9, Hq=32, Hkv=8, D=128, ctx_lo=1, ctx_hi=8192,
             window=2048, sinks=16, tree=0, dtype="bf16"),
        # 64-node trees, 32-bit values, heads of 64
        dict(name="attn_tree_f32", op="attn", B=8, M=64, Hq=8, Hkv=8, D=64, ctx_lo=500, ctx_hi=4096,
             window=500, sinks=5, tree=4, dtype="f32"),
        # the largest batch: long contexts, wide groups of query heads
        dict(name="attn_chain_128", op="attn", B=128, M=5, Hq=64, Hkv=8, D=128, ctx_lo=4096,
             ctx_hi=32768, window=4096, sinks=4, tree=0, dtype="bf16"),
        # the token of one request, all filters on: latency
        dict(name="sample_1", op="sample", rows=1, V=32000, dtype="bf16", filters=True, greedy=False),
        # a batch of plain decoding with each request's own filters, 32-bit
        # logits, rows that start at odd places
        dict(name="sample_f32_33", op="sample", rows=33, V=32001, dtype="f32", filters=True,
             greedy=True),
        # the draft rows of a large batch, temperature only
        dict(name="sample_640", op="sample", rows=640, V=152064, dtype="bf16", filters=False,
             greedy=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "rope", "attn", "sample"])
    if op == "pages":
        kind = rng.choice(["step", "mixed"])
        ctx_hi = _log(rng, 64, 30000)
        M = _log(rng, 1, 64) if kind == "step" else 1
        chunk = _log(rng, 1, 2048) if kind == "mixed" else 0
        window, B = rng.choice([0, _log(rng, 16, 4096)]), _log(rng, 1, 512)
        return dict(op=op, B=B, max_blocks=-(-(ctx_hi + max(M, chunk)) // BLOCK) + 1,
                    kind=kind, M=M, ctx_lo=rng.randint(1, ctx_hi), ctx_hi=ctx_hi, window=window,
                    sinks=rng.randint(0, 70) if window else 0, chunk=chunk,
                    budget=B + _log(rng, 1, 60000) if chunk else 0,
                    short=rng.random() < 0.25)
    if op == "rope":
        dtype = rng.choice(["bf16", "f32"])
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        cache = rng.random() < 0.4
        return dict(op=op, rows=_log(rng, 1, 8192), pad=rng.choice([0, rng.randint(1, 40)]),
                    Hq=Hkv * rng.choice([1, 4, 5, 8]), Hkv=Hkv, D=D,
                    rot=rng.choice([D, D, D // 2, 16]), interleaved=rng.random() < 0.4,
                    dtype=dtype, cache=cache, norm=rng.random() < 0.8,
                    pos_hi=_log(rng, 16, 1 << 20), strided=rng.random() < 0.5)
    if op == "attn":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        Hkv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 7, 8])
        M = rng.choice([1, _log(rng, 1, 128 // group)])
        small = dtype == "f32"
        return dict(op=op, B=_log(rng, 1, 16 if small else 64), M=M, Hq=Hkv * group, Hkv=Hkv,
                    D=rng.choice([64, 128]) if small else 128, ctx_lo=rng.randint(0, 2000),
                    ctx_hi=_log(rng, 2001, 16384), window=_log(rng, 1, 4096),
                    sinks=rng.choice([0, 1, 4, 64, 100]),
                    tree=rng.choice([0, 0, 3]) if M > 2 else 0, dtype=dtype)
    V = _log(rng, 100, 152064)
    return dict(op=op, rows=_log(rng, 1, max(1, min(512, 24_000_000 // V))), V=V,
                dtype=rng.choice(["bf16", "f32"]), filters=rng.random() < 0.7,
                greedy=rng.random() < 0.3)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2 + 1)
    rng = np.random.default_rng([int(seed), 77])
    s = {"pages": _prepare_pages, "rope": _prepare_rope, "attn": _prepare_attn,
         "sample": _prepare_sample}[case["op"]](case, rng, g)
    s["case"] = case
    if own:  # the dims and the workspace that a program keeps
        import speculative_decoding_verification_19_gb300 as sv
        s["sv"] = sv
        c = dict(B=1, M=1, Hq=1, Hkv=1, D=128, dtype="bf16") | case
        s["dims"] = sv.make_dims(B=c["B"], M=c["M"], Hq=c["Hq"], Hkv=c["Hkv"], D=c["D"],
                                 max_blocks=s.get("max_blocks", 1), num_blocks=s.get("num_blocks", 1),
                                 kv_dtype=_types(c))
        s["ws"] = sv.workspace(s["dims"])
    return s


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


def _prepare_pages(case, rng, g):
    B, mb, W, M = case["B"], case["max_blocks"], case["window"], case["M"]
    sink_pages = -(-case["sinks"] // BLOCK) if W else 0
    ctx0 = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, B)  # before the last step
    if case["kind"] == "step":
        # the last step appended M rows and kept some of them
        hi = -(-(ctx0 + M) // BLOCK)
        ctx = ctx0 + rng.integers(1, M + 1, B)
        ctx = np.minimum(ctx, mb * BLOCK - M)
        n = np.full(B, M)
    else:
        kind = rng.random(B)
        new, ended = kind < 0.25, kind > 0.9
        hi = np.where(new, 0, -(-ctx0 // BLOCK))
        ctx = np.where(new, 0, np.where(ended, -1, ctx0))
        n = np.where(new, rng.integers(1, case["chunk"] + 1, B), np.where(ended, 0, 1))
        # what the step's token budget leaves: later requests wait with 0 rows
        n = np.diff(np.minimum(np.cumsum(np.concatenate([[0], n])), case["budget"]))
    lo = np.where(hi > 0, np.maximum(0, ctx0 - W + 1) // BLOCK, 0) if W else np.zeros(B, np.int64)
    page = np.arange(mb)[None, :]
    held = (page < hi[:, None]) & ((page < sink_pages) | (page >= lo[:, None]))
    n_held = int(held.sum())
    need = int(np.maximum(0, -(-(np.maximum(ctx, 0) + n) // BLOCK) - hi).sum())
    budget = B * M if case["kind"] == "step" else case["budget"]
    num_blocks = B * (-(-(case["ctx_hi"] + M) // BLOCK) + 2) + budget // BLOCK
    free = need // 2 if case["short"] else num_blocks - n_held
    perm = rng.permutation(num_blocks)
    table = np.full((B, mb), -1, dtype=np.int64)
    table[held] = perm[:n_held]
    pool = np.full(num_blocks, -1, dtype=np.int64)
    head = int(rng.integers(num_blocks))
    pool[(head + np.arange(free)) % num_blocks] = perm[n_held:n_held + free]
    start = np.concatenate([[0], np.cumsum(n)])
    rows = budget + 5  # a few padding rows
    # the program's page state lives in one buffer: tables, spans, ring, ring state
    parts = [table.reshape(-1), np.stack([lo, hi], 1).reshape(-1), pool, [head, free]]
    init = _i32(np.concatenate(parts))
    s = dict(init=init, buf=torch.empty_like(init), num_blocks=num_blocks, max_blocks=mb,
             ctx=_i32(ctx), row_start=None if case["kind"] == "step" else _i32(start),
             slots=torch.full((rows,), -7, dtype=torch.int64, device=DEV),
             positions=torch.full((rows,), -7, dtype=torch.int32, device=DEV),
             ok=torch.empty(B, dtype=torch.int32, device=DEV))
    a, b, c = B * mb, B * mb + 2 * B, B * mb + 2 * B + num_blocks
    buf = s["buf"]
    s.update(table=buf[:a].view(B, mb), span=buf[a:b].view(B, 2), pool=buf[b:c], state=buf[c:])
    return s


def _prepare_rope(case, rng, g):
    N, Hq, Hkv, D, dt = case["rows"] + case["pad"], case["Hq"], case["Hkv"], case["D"], _types(case)
    # one projection's output, cut into queries, keys and values (strided views)
    # or three tensors of their own
    H = Hq + 2 * Hkv
    qkv = (torch.randn(N, H, D, generator=g, device=DEV) * 1.7).to(dt)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not case["strided"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    s = dict(q=q, k=k, v=v, q_weight=None, k_weight=None)
    if case["norm"]:
        s["q_weight"] = (1 + 0.3 * torch.randn(D, generator=g, device=DEV)).to(dt)
        s["k_weight"] = (1 + 0.3 * torch.randn(D, generator=g, device=DEV)).to(dt)
    pos = rng.integers(0, case["pos_hi"], N)
    pos[case["rows"]:] = -1  # the padding of a batch
    s["positions"] = _i32(pos)
    half = case["rot"] // 2
    s["inv_freq"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
    s["q_out"] = torch.empty(N, Hq, D, dtype=dt, device=DEV)
    s["k_out"] = torch.empty(N, Hkv, D, dtype=dt, device=DEV)
    s["slots"] = s["k_cache"] = s["v_cache"] = None
    s["num_blocks"] = 1
    if case["cache"]:
        nb = s["num_blocks"] = -(-N // BLOCK) + 7
        slots = rng.permutation(nb)[np.arange(N) // BLOCK] * BLOCK + np.arange(N) % BLOCK
        slots[case["rows"]:] = -1
        s["slots"] = torch.from_numpy(slots.astype(np.int64)).to(DEV)
        s["k_cache"] = torch.randn(nb, Hkv, BLOCK, D, generator=g, device=DEV).to(dt)
        s["v_cache"] = torch.randn(nb, Hkv, BLOCK, D, generator=g, device=DEV).to(dt)
    return s


def _prepare_attn(case, rng, g):
    B, M, Hq, Hkv, D = (case[x] for x in ("B", "M", "Hq", "Hkv", "D"))
    W, dt = case["window"], _types(case)
    ctx = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, B)
    hi = -(-(ctx + M) // BLOCK)
    lo = np.maximum(0, ctx - W + 1) // BLOCK
    mb = -(-(case["ctx_hi"] + M) // BLOCK)
    page = np.arange(mb)[None, :]
    # pages outside the window and the sinks have been given back
    held = (page < hi[:, None]) & ((page < -(-case["sinks"] // BLOCK)) | (page >= lo[:, None]))
    nb = 3 + B * min(mb, -(-case["sinks"] // BLOCK) + (W + M) // BLOCK + 2)
    table = np.full((B, mb), -1, dtype=np.int64)
    table[held] = rng.permutation(nb)[:int(held.sum())]
    parent = None
    if case["tree"]:
        n = np.arange(M)[None, :]
        parent = np.maximum(0, n - 1 - rng.integers(0, case["tree"], (B, M)))
        parent[:, 0] = -1
        parent = _i32(parent)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dt)

    return dict(q=normal(B, M, Hq, D), k_new=normal(B, M, Hkv, D), v_new=normal(B, M, Hkv, D),
                k_cache=normal(nb, Hkv, BLOCK, D), v_cache=normal(nb, Hkv, BLOCK, D),
                table=_i32(table), ctx=_i32(ctx), parent=parent, num_blocks=nb, max_blocks=mb,
                out=torch.empty(B, M, Hq, D, dtype=dt, device=DEV),
                lse=torch.empty(B, M, Hq, dtype=torch.float32, device=DEV))


def _prepare_sample(case, rng, g):
    n, V = case["rows"], case["V"]
    logits = (torch.randn(n, V, generator=g, device=DEV) * 3).to(_types(case))
    T = rng.uniform(0.5, 1.2, n)
    if case["greedy"]:
        T[rng.random(n) < 0.2] = 0.0
    f32 = lambda x: torch.from_numpy(np.asarray(x, dtype=np.float32)).to(DEV)  # noqa: E731
    s = dict(logits=logits, temperature=f32(T), uniform=f32(rng.integers(0, 1 << 24, n) / (1 << 24)),
             top_k=None, top_p=None, min_p=None,
             tokens=torch.empty(n, dtype=torch.int32, device=DEV),
             prob=torch.empty(n, dtype=torch.float32, device=DEV))
    if case["filters"]:
        # each request's own choice; a filter that is off has its neutral value
        on = rng.random((3, n)) < 0.6
        s["top_k"] = _i32(np.where(on[0], rng.choice([1, 20, 50, 200, 1000], n), 0))
        s["top_p"] = f32(np.where(on[1], rng.uniform(0.5, 0.99, n), 1.0))
        s["min_p"] = f32(np.where(on[2], rng.uniform(0.001, 0.2, n), 0.0))
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if op == "pages":
        s["buf"].copy_(s["init"])  # the page state before the step
        if own:
            s["sv"].spec_block_tables(s["ctx"], s["row_start"], None, s["table"], s["span"],
                                      s["pool"], s["state"], s["slots"], s["positions"], s["ok"],
                                      s["dims"], s["ws"], window=case["window"],
                                      sinks=case["sinks"])
        else:
            _plain_pages(s, case)
        return {k: s[k] for k in ("table", "span", "pool", "state", "slots", "positions", "ok")}
    if op == "rope":
        if own:
            s["sv"].spec_qk_norm_rope(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"],
                                      s["positions"], s["inv_freq"], s["q_out"], s["k_out"],
                                      s["dims"], s["ws"], eps=1e-6,
                                      interleaved=case["interleaved"], slots=s["slots"],
                                      k_cache=s["k_cache"], v_cache=s["v_cache"])
        else:
            _plain_rope(s, case)
        return {k: s[k] for k in ("q_out", "k_out", "k_cache", "v_cache")}
    if op == "attn":
        if own:
            s["sv"].spec_verify_attn(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"],
                                     s["table"], s["ctx"], s["parent"], s["out"], s["lse"],
                                     s["dims"], s["ws"], window=case["window"],
                                     sinks=case["sinks"])
        else:
            _plain_attn(s, case)
        return {k: s[k] for k in ("out", "lse", "k_cache", "v_cache")}
    if own:
        s["sv"].spec_sample(s["logits"], s["temperature"], s["uniform"], s["tokens"], s["prob"],
                            s["ws"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    else:
        _plain_sample(s)
    return {"tokens": s["tokens"], "prob": s["prob"]}


def _plain_pages(s, case):
    table, span, pool, state = s["table"], s["span"].long(), s["pool"], s["state"].long()
    B, mb = table.shape
    nb, W = pool.numel(), case["window"]
    ctx = s["ctx"].long()
    live = ctx >= 0
    if s["row_start"] is None:
        start = torch.arange(B + 1, device=DEV) * case["M"]
    else:
        start = s["row_start"].long()
    n = torch.where(live, start[1:] - start[:-1], 0)
    sp = -(-case["sinks"] // BLOCK) if W else 0
    lo, hi = span[:, 0], span[:, 1]
    hi2 = torch.where(live, (ctx + n + BLOCK - 1) // BLOCK, 0)
    lo2 = torch.where(live, (ctx - W + 1).clamp(min=0) // BLOCK, 0) if W else torch.zeros_like(hi)
    page = torch.arange(mb, device=DEV)
    held = (page < hi[:, None]) & ((page < sp) | (page >= lo[:, None]))
    want = (page < hi2[:, None]) & ((page < sp) | (page >= lo2[:, None]))
    take, give = want & ~held, held & ~want
    # requests that the ring has pages for, in order
    need = take.sum(1)
    head, count = state[0], state[1]
    ok = (need == 0) | (need.cumsum(0) <= count)
    take &= ok[:, None]
    taken = take.sum()
    t_rank = take.reshape(-1).cumsum(0).reshape(B, mb) - 1
    g_rank = give.reshape(-1).cumsum(0).reshape(B, mb) - 1
    ids = pool[(head + t_rank) % nb]
    where = torch.where(give, (head + count + g_rank) % nb, nb)
    grown = torch.cat([pool, pool.new_zeros(1)]).scatter_(
        0, where.reshape(-1), torch.where(give, table, 0).reshape(-1))
    # nb collects what is not given back
    pool.copy_(grown[:nb])
    table.copy_(torch.where(take, ids, torch.where(give, -1, table)))
    s["span"].copy_(torch.stack([lo2, torch.where(ok, hi2, torch.minimum(hi, hi2))], 1))
    s["state"].copy_(torch.stack([(head + taken) % nb, count - taken + give.sum()]))
    s["ok"].copy_(ok & live)
    # slots and positions of the rows; rows behind the last request stay
    rows = s["slots"].numel()
    r = torch.arange(rows, device=DEV)
    b = torch.searchsorted(start, r, right=True) - 1
    inside = b < B
    b = b.clamp(max=B - 1)
    pos = ctx[b] + r - start[b]
    good = inside & (ok & live)[b]
    pos = torch.where(good, pos, -1)
    p = pos.clamp(min=0)
    slot = table[b, p // BLOCK].long() * BLOCK + p % BLOCK
    s["slots"].copy_(torch.where(inside, torch.where(good, slot, -1), s["slots"]))
    s["positions"].copy_(torch.where(inside, pos, s["positions"]))


def _norm_rotate(x, w, pos, inv_freq, rot, interleaved, t):
    """Norm and rotation of x [N, H, D] in type t (angles in 64 bits)."""
    x = x.to(t)
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.to(t)
    ang = pos.clamp(min=0).double()[:, None] * inv_freq
    c, sn = ang.cos().to(t)[:, None], ang.sin().to(t)[:, None]
    half = rot // 2
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    x = torch.cat([turned, x[..., rot:]], -1)
    return torch.where((pos < 0)[:, None, None], 0, x)


def _plain_rope(s, case):
    args = (s["positions"], s["inv_freq"], case["rot"], case["interleaved"], torch.float32)
    s["q_out"].copy_(_norm_rotate(s["q"], s["q_weight"], *args))
    s["k_out"].copy_(_norm_rotate(s["k"], s["k_weight"], *args))
    if s["slots"] is not None:
        n = case["rows"]  # the padding rows have no slot
        slot = s["slots"][:n]
        s["k_cache"][slot // BLOCK, :, slot % BLOCK] = s["k_out"][:n]
        s["v_cache"][slot // BLOCK, :, slot % BLOCK] = s["v"][:n]


def _plain_attn(s, case):
    q, ctx, M, W, S = s["q"], s["ctx"].long(), case["M"], case["window"], case["sinks"]
    B, D, Hkv = case["B"], case["D"], case["Hkv"]
    group = case["Hq"] // Hkv
    kc, vc, table = s["k_cache"], s["v_cache"], s["table"].long()
    node = torch.arange(M, device=DEV)
    # append, and clear the rest of the last page
    end = (ctx + M + BLOCK - 1) // BLOCK * BLOCK
    at = ctx[:, None] + torch.arange(M + BLOCK - 1, device=DEV)
    at = torch.where(at < end[:, None], at, ctx[:, None])  # past the page: the first row again
    src = (at - ctx[:, None]).clamp(max=M)
    pick = torch.arange(B, device=DEV)[:, None]
    blk = table.gather(1, at // BLOCK)
    pad = torch.nn.functional.pad
    kc[blk, :, at % BLOCK] = pad(s["k_new"], (0, 0, 0, 0, 0, 1))[pick, src]
    vc[blk, :, at % BLOCK] = pad(s["v_new"], (0, 0, 0, 0, 0, 1))[pick, src]
    # ancestors-or-self and depths of the new rows
    if s["parent"] is None:
        anc = (node[None, :] <= node[:, None]).expand(B, M, M)
    else:
        step = (s["parent"][:, :, None] == node).double() + torch.eye(M, device=DEV).double()
        anc = torch.linalg.matrix_power(step, M) > 0.5
    depth = anc.sum(-1) - 1
    # the positions that any row of the request may see: sinks, then the window
    w0 = torch.clamp(ctx - W + 1, min=S)
    P = S + min(W, case["ctx_hi"] + 1) + M - 1
    j = torch.arange(P, device=DEV)
    pos = torch.where(j < S, j, w0[:, None] + j - S)
    pos = torch.where(pos < (ctx + M)[:, None], pos, -1)
    p = pos.clamp(min=0)
    new = p >= ctx[:, None]
    k_node = (p - ctx[:, None]).clamp(0, M - 1)
    k_pos = torch.where(new, ctx[:, None] + depth.gather(1, k_node), p)
    q_pos = ctx[:, None] + depth
    see = (k_pos[:, None, :] < S) | (k_pos[:, None, :] > q_pos[:, :, None] - W)
    see &= ~new[:, None, :] | anc.gather(2, k_node[:, None, :].expand(B, M, P))
    see &= (pos >= 0)[:, None, :]
    blk = table.gather(1, p // BLOCK).clamp(min=0)
    K = kc[blk, :, p % BLOCK].float()  # [B, P, Hkv, D]
    V = vc[blk, :, p % BLOCK].float()
    qf = q.float().view(B, M, Hkv, group, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, M * group, D)
    sc = torch.matmul(qf, K.permute(0, 2, 3, 1)) / math.sqrt(D)
    sc = sc.view(B, Hkv, M, group, P).masked_fill(~see[:, None, :, None, :], -math.inf)
    m = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - m)
    z = e.sum(-1, keepdim=True)
    o = torch.matmul((e / z).view(B, Hkv, M * group, P), V.transpose(1, 2))
    s["out"].copy_(o.view(B, Hkv, M, group, D).permute(0, 2, 1, 3, 4).reshape(q.shape))
    s["lse"].copy_((m + z.log())[..., 0].permute(0, 2, 1, 3).reshape(B, M, case["Hq"]))


def _plain_sample(s):
    x = s["logits"].double()
    n, V = x.shape
    T = s["temperature"].double()[:, None]
    top = x.amax(-1, keepdim=True)
    w = torch.exp((x - top) / torch.where(T > 0, T, 1.0))
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        k = torch.where(k > 0, k, V)
        order = torch.sort(x, dim=-1, descending=True, stable=True)[1]
        ws = w.gather(1, order)
        ws = torch.where(torch.arange(V, device=DEV) < k, ws, 0)
        cum = ws.cumsum(-1)
        keep = (ws > 0) & (cum - ws < s["top_p"].double()[:, None] * cum[:, -1:])
        keep = torch.zeros_like(keep).scatter_(1, order, keep)
        w = torch.where(keep & (w >= s["min_p"].double()[:, None]), w, 0)
    at = torch.arange(V, device=DEV)
    first = torch.where(x == top, at, V).amin(-1)
    cdf = w.cumsum(-1)
    tok = (cdf <= s["uniform"].double()[:, None] * cdf[:, -1:]).sum(-1)
    p = (w.gather(1, tok[:, None]) / cdf[:, -1:])[:, 0]
    greedy = T[:, 0] == 0
    s["tokens"].copy_(torch.where(greedy, first, tok))
    s["prob"].copy_(torch.where(greedy, 1.0, p))


# --------------------------------------------------------------------------
# work and exact values
# --------------------------------------------------------------------------

def work(case):
    op, e = case["op"], 2 if case.get("dtype") == "bf16" else 4
    if op == "pages":
        B, sp = case["B"], 8
        if case["kind"] == "step":
            rows, moved = B * case["M"], B * case["M"] / BLOCK
        else:
            rows = min(case["budget"], B * (0.25 * case["chunk"] / 2 + 0.65))
            moved = rows / BLOCK + 0.1 * B * (case["ctx_lo"] + case["ctx_hi"]) / 2 / BLOCK
        # lengths, spans and verdicts; ids of moved pages in and out; slots and positions
        return dict(bytes=B * (4 + 4 + 2 * sp + 4) + moved * 8 + rows * 12, flops=0)
    if op == "rope":
        rows, D = case["rows"], case["D"]
        H = case["Hq"] + case["Hkv"]
        b = 2 * rows * H * D * e + rows * 4 + case["rot"] * 4 + case["pad"] * H * D * e
        if case["cache"]:
            b += rows * case["Hkv"] * D * e * 3 + rows * 8
        return dict(bytes=b, flops=8 * rows * H * D)
    if op == "attn":
        B, M, Hq, Hkv, D = (case[x] for x in ("B", "M", "Hq", "Hkv", "D"))
        lo, hi, vis = case["ctx_lo"], case["ctx_hi"], case["window"] + case["sinks"]
        # mean of min(ctx, window + sinks) over the contexts
        below = max(0, min(hi, vis) - lo + 1)
        mean = (below * (lo + min(hi, vis)) / 2 + max(0, hi - max(lo, vis + 1) + 1) * vis) / (hi - lo + 1)
        keys = B * Hkv * mean
        b = 2 * keys * D * e + 2 * B * M * Hq * D * e + 4 * B * M * Hkv * D * e + 4 * B * M * Hq
        return dict(bytes=b, flops=4 * (Hq // Hkv) * M * D * (keys + B * Hkv * M / 2))
    return dict(bytes=case["rows"] * (case["V"] * e + 4 * 6), flops=4 * case["rows"] * case["V"])


def exact(case, seed):
    op = case["op"]
    if op == "pages":
        return None  # whole numbers only
    s = prepare(case, seed)
    if op == "rope":
        return _exact_rope(s, case)
    return _exact_attn(s, case) if op == "attn" else _exact_sample(s)


def _exact_rope(s, case):
    """Every pair as a complex number times the turn's own."""
    rot, half = case["rot"], case["rot"] // 2
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       s["positions"].double()[:, None] * s["inv_freq"])[:, None]
    out = {}
    for name, x, w in (("q_out", s["q"], s["q_weight"]), ("k_out", s["k"], s["k_weight"])):
        y = x.double()
        if w is not None:
            y = y / (y.square().sum(-1, keepdim=True) / case["D"] + 1e-6).sqrt() * w.double()
        first = slice(0, rot, 2) if case["interleaved"] else slice(0, half)
        second = slice(1, rot, 2) if case["interleaved"] else slice(half, rot)
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        y[case["rows"]:] = 0
        out[name] = y
    out["k_cache"] = out["v_cache"] = None
    if case["cache"]:
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        rows = torch.arange(case["rows"], device=DEV)
        b, o = s["slots"][rows] // BLOCK, s["slots"][rows] % BLOCK
        kc[b, :, o] = out["k_out"][rows]
        vc[b, :, o] = s["v"][rows].double()
        out["k_cache"], out["v_cache"] = kc, vc
    return out


def _exact_attn(s, case):
    """One request after another, over the keys that it can see."""
    B, M, D, W, S = case["B"], case["M"], case["D"], case["window"], case["sinks"]
    Hq, Hkv = case["Hq"], case["Hkv"]
    ctx, table = s["ctx"].tolist(), s["table"].cpu().numpy()
    parents = None if s["parent"] is None else s["parent"].tolist()
    out = torch.empty(B, M, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, M, Hq, dtype=torch.float64, device=DEV)
    for b in range(B):
        c = ctx[b]
        cached = [t for t in range(c) if t < S or t > c - W]
        at = torch.tensor(cached, dtype=torch.int64)
        blk = torch.from_numpy(table[b][at.numpy() // BLOCK].astype(np.int64)).to(DEV)
        off = (at % BLOCK).to(DEV)
        K = torch.cat([s["k_cache"][blk, :, off], s["k_new"][b]]).double()
        V = torch.cat([s["v_cache"][blk, :, off], s["v_new"][b]]).double()
        paths = []
        for i in range(M):
            up = [i]
            while up[-1] != 0:
                up.append(up[-1] - 1 if parents is None else parents[b][up[-1]])
            paths.append(up[::-1])
        where = np.array(cached, dtype=np.int64)
        see = np.zeros((M, len(cached) + M), dtype=bool)
        for i in range(M):
            at_i = c + len(paths[i]) - 1
            see[i, :len(cached)] = (where < S) | (where > at_i - W)
            for d, k in enumerate(paths[i]):
                see[i, len(cached) + k] = c + d < S or c + d > at_i - W
        hide = torch.from_numpy(~see).to(DEV)
        q = s["q"][b].double().view(M, Hkv, Hq // Hkv, D)
        sc = torch.einsum("mhgd,phd->hgmp", q, K) * D ** -0.5
        sc = sc.masked_fill(hide, -math.inf)
        lse[b] = torch.logsumexp(sc, -1).permute(2, 0, 1).reshape(M, Hq)
        out[b] = torch.einsum("hgmp,phd->mhgd", torch.softmax(sc, -1), V).reshape(M, Hq, D)
    return {"out": out, "lse": lse, "k_cache": None, "v_cache": None}


def _exact_sample(s):
    """The probability of the drawn token, row by row on the host."""
    x = s["logits"].double().cpu().numpy()
    T, u = (s[k].double().cpu().numpy() for k in ("temperature", "uniform"))
    filt = None if s["top_k"] is None else [s[k].cpu().numpy() for k in ("top_k", "top_p", "min_p")]
    prob = np.ones(len(x))
    for r in range(len(x)):
        if T[r] == 0:
            continue
        p = np.exp((x[r] - x[r].max()) / T[r])
        if filt is not None:
            k, t, mp = int(filt[0][r]), float(filt[1][r]), float(filt[2][r])
            order = np.argsort(-x[r], kind="stable")[:k or None]
            c = np.cumsum(p[order])
            order = order[:int(np.searchsorted(c, t * c[-1])) + 1]
            order = np.sort(order[p[order] >= mp])
            p = p[order]
        c = np.cumsum(p)
        i = int(np.searchsorted(c, u[r] * c[-1], side="right"))
        prob[r] = p[i] / c[-1]
    return {"tokens": None, "prob": torch.from_numpy(prob)}
