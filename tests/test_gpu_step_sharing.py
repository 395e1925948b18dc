"""What calls share: one workspace among calls of different dims, and the
kernels' settings among host threads."""
import threading

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


def in_threads(jobs, rounds):
    """Each job (prepare, call, result) on a thread and a stream of its own, all
    at once; a call's result is the one it has alone."""
    want = []
    for prepare, call, result in jobs:
        state = prepare()
        call(state, None)
        torch.cuda.synchronize()
        want.append((state, [t.clone() for t in result(state)]))
    gate, errors = threading.Barrier(len(jobs)), []

    def run(job, state, expect):
        stream = torch.cuda.Stream()
        try:
            gate.wait()
            for _ in range(rounds):
                job[1](state, stream)
            stream.synchronize()
            for a, b in zip(job[2](state), expect):
                assert torch.equal(a, b)
        except Exception as e:  # told to the thread that asserts
            errors.append(repr(e))

    threads = [threading.Thread(target=run, args=(j, *w)) for j, w in zip(jobs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_sampling_from_several_host_threads():
    """Vocabularies and batches whose kernels ask for different amounts of
    shared memory: no thread's call makes another's fail."""
    def job(n, V, **filters):
        def prepare():
            g = torch.Generator(device="cuda").manual_seed(V)
            s = dict(x=torch.randn(n, V, device="cuda", generator=g).to(BF),
                     T=torch.ones(n, device="cuda"), u=torch.rand(n, device="cuda", generator=g),
                     tok=torch.empty(n, dtype=I32, device="cuda"), prob=torch.empty(n, device="cuda"),
                     ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
            s["kw"] = {k: torch.full((n,), v, device="cuda", dtype=I32 if k == "top_k" else None)
                       for k, v in filters.items()}
            return s

        def call(s, stream):
            sv.spec_sample(s["x"], s["T"], s["u"], s["tok"], s["prob"], s["ws"], stream=stream,
                           **s["kw"])

        return prepare, call, lambda s: (s["tok"], s["prob"])

    in_threads([job(2, 152064, top_k=50), job(2, 2000, top_k=50), job(200, 32000, top_k=40),
                job(3, 300000, top_p=0.5)], 400)
    in_threads([job(700, 20000), job(700, 152064), job(620, 9000)], 60)


def test_cuda_core_attention_from_several_host_threads():
    def job(M, window):
        wl = workload("tiny_chain").scaled(gamma=M - 1, Hq=2, Hkv=2, D=64)
        kv = kv_inputs_host(wl, seed=M, B=2, ctx=np.array([40, 200]))
        f32 = torch.float32
        dims = sv.make_dims(B=2, M=M, Hq=2, Hkv=2, D=64, max_blocks=kv["max_blocks"],
                            num_blocks=kv["num_blocks"], kv_dtype=f32)

        def prepare():
            s = {k: to_dev(kv[k], f32) for k in ("q", "k_new", "v_new", "k_cache", "v_cache")}
            s.update(table=to_dev(kv["block_table"], I32), ctx=to_dev(kv["ctx_lens"], I32),
                     out=torch.empty_like(s["q"]), lse=torch.empty(2, M, 2, device="cuda"),
                     ws=sv.workspace(dims))
            return s

        def call(s, stream):
            sv.spec_verify_attn(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"],
                                s["table"], s["ctx"], None, s["out"], s["lse"], dims, s["ws"],
                                stream=stream, window=window)

        return prepare, call, lambda s: (s["out"], s["lse"])

    in_threads([job(65, None), job(128, None), job(66, None), job(90, 50)], 300)


def test_tensors_without_memory_are_refused():
    """A tensor that only stands for others (inside vmap) has no address."""
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    one, tok = torch.ones(2, device="cuda"), torch.zeros(2, dtype=I32, device="cuda")

    def call(x):
        sv.spec_sample(x, one, one * 0.5, tok, None, ws)
        return x

    with pytest.raises((RuntimeError, ValueError)):
        torch.func.vmap(call)(torch.zeros(3, 2, 64, device="cuda"))
    call(torch.zeros(2, 64, device="cuda"))
    assert sv.device_status(ws) == 0
