"""Binding of libspecverify.so (argument marshalling only): ctypes, and for the
step operators the native checks of csrc/binding.cpp.

Every function here takes torch tensors that already live on the GPU,
passes their device pointers, sizes and the current CUDA stream to the C ABI
declared in include/spec_verify.h, and raises SpecError on a non-zero status.
No step of the verify path runs in Python.  If the shared library is missing
the import fails loudly: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libspecverify.so")

SPEC_BF16, SPEC_F32 = 0, 1
STATUS_NAMES = {
    0: "SPEC_OK", 1: "SPEC_ERR_INVALID_ARG", 2: "SPEC_ERR_CAPACITY",
    3: "SPEC_ERR_UNSUPPORTED", 4: "SPEC_ERR_CUDA", 5: "SPEC_ERR_NONFINITE",
    6: "SPEC_ERR_DEVICE_BOUNDS", 7: "SPEC_ERR_TIMEOUT",
}
ATTN_AUTO, ATTN_CUDA_CORES, ATTN_TENSOR_CORES = 0, 1, 2
REJECT_AUTO, REJECT_STAGED, REJECT_FUSED = 0, 1, 2

# every symbol the header declares
EXPORTS = (
    "spec_workspace_size", "spec_workspace_init", "spec_get_device_status",
    "spec_verify_attn", "spec_reject_sample", "spec_reject_sample_filtered", "kv_commit",
    "spec_philox_block", "spec_lm_head", "spec_reject_sample_lm_head",
    "spec_status_string", "spec_last_launch_count", "spec_reject_sample_noalloc",
    "spec_ctrl_default_config", "spec_ctrl_init", "spec_ctrl_update", "spec_ctrl_metrics",
    "spec_step_stats",
    "spec_verify_attn_window", "spec_block_tables", "spec_qk_norm_rope", "spec_sample",
    "spec_verify_attn_prefix", "spec_verify_attn_pages", "spec_page_bounds", "spec_page_score",
    "spec_page_select",
)


class SpecError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(code, code)}")
        self.code = code


class SpecDims(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("M", ctypes.c_int32), ("Hq", ctypes.c_int32),
        ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32), ("block", ctypes.c_int32),
        ("max_blocks", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
        ("V", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
        ("logits_dtype", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
        ("attn_impl", ctypes.c_int32), ("reject_impl", ctypes.c_int32),
        ("wait_limit_kcycles", ctypes.c_int32),
    ]


_lib = None
_binding = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(LIB_PATH)
    vp, sz, i32, u64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_uint64
    pd = ctypes.POINTER(SpecDims)
    L.spec_workspace_size.argtypes = [pd]
    L.spec_workspace_size.restype = sz
    L.spec_workspace_init.argtypes = [vp, sz, vp]
    L.spec_workspace_init.restype = i32
    L.spec_get_device_status.argtypes = [vp, vp, ctypes.POINTER(i32), i32]
    L.spec_get_device_status.restype = i32
    L.spec_verify_attn.argtypes = [vp] * 10 + [pd, vp, sz, vp]
    L.spec_verify_attn.restype = i32
    L.spec_reject_sample.argtypes = [vp, vp, vp, vp, vp, u64, u64, u64, vp, vp, vp,
                                     vp, pd, vp, sz, vp]
    L.spec_reject_sample.restype = i32
    L.spec_reject_sample_filtered.argtypes = [vp, vp, vp, vp, vp, vp, vp, u64, u64, u64, vp,
                                              vp, vp, vp, pd, vp, sz, vp]
    L.spec_reject_sample_filtered.restype = i32
    L.spec_lm_head.argtypes = [vp, vp, i32, i32, i32, vp, vp, sz, vp]
    L.spec_lm_head.restype = i32
    L.spec_reject_sample_lm_head.argtypes = [vp, vp, i32, vp, vp, i32, vp, vp, vp, vp, vp, u64,
                                             u64, u64, vp, vp, vp, vp, pd, vp, sz, vp]
    L.spec_reject_sample_lm_head.restype = i32
    L.spec_reject_sample_noalloc.argtypes = [vp, vp, vp, vp, vp, u64, u64, u64, vp, vp,
                                             vp, vp, pd, vp]
    L.spec_reject_sample_noalloc.restype = i32
    L.kv_commit.argtypes = [vp] * 7 + [pd, vp, sz, vp]
    L.kv_commit.restype = i32
    f32, i64 = ctypes.c_float, ctypes.c_int64
    L.spec_verify_attn_window.argtypes = [vp] * 8 + [i32, i32, vp, vp, pd, vp, sz, vp]
    L.spec_verify_attn_window.restype = i32
    L.spec_block_tables.argtypes = [vp, vp, vp, i32, i32, i32] + [vp] * 7 + [pd, vp, sz, vp]
    L.spec_block_tables.restype = i32
    L.spec_qk_norm_rope.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, f32, vp, vp, i32, i32, i32,
                                    vp, vp, vp, vp, vp, pd, vp, sz, vp]
    L.spec_qk_norm_rope.restype = i32
    L.spec_sample.argtypes = [vp, i64, i32, i32, i32] + [vp] * 7 + [vp, sz, vp]
    L.spec_sample.restype = i32
    L.spec_verify_attn_prefix.argtypes = [vp] * 9 + [i32, vp, vp, pd, vp, sz, vp]
    L.spec_verify_attn_prefix.restype = i32
    L.spec_verify_attn_pages.argtypes = [vp] * 10 + [i32, vp, vp, pd, vp, sz, vp]
    L.spec_verify_attn_pages.restype = i32
    L.spec_page_bounds.argtypes = [vp] * 5 + [pd, vp, sz, vp]
    L.spec_page_bounds.restype = i32
    L.spec_page_score.argtypes = [vp] * 5 + [pd, vp, sz, vp]
    L.spec_page_score.restype = i32
    L.spec_page_select.argtypes = [vp, vp, i32, i32, i32, vp, vp, pd, vp, sz, vp]
    L.spec_page_select.restype = i32
    L.spec_philox_block.argtypes = [ctypes.POINTER(u64)] * 3
    L.spec_philox_block.restype = None
    L.spec_status_string.argtypes = [i32]
    L.spec_status_string.restype = ctypes.c_char_p
    L.spec_last_launch_count.argtypes = []
    L.spec_last_launch_count.restype = i32
    _lib = L
    return L


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn: str, code: int):
    if code != 0:
        raise SpecError(fn, code)


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return SPEC_BF16
    if dt == torch.float32:
        return SPEC_F32
    raise ValueError(f"unsupported dtype {dt}")


def make_dims(B, M, Hq=1, Hkv=1, D=128, max_blocks=1, num_blocks=1, V=1,
              kv_dtype=torch.bfloat16, logits_dtype=torch.bfloat16,
              softmax_scale=0.0, block=16, attn_impl=0, reject_impl=0,
              wait_limit_kcycles=0) -> SpecDims:
    return SpecDims(B, M, Hq, Hkv, D, block, max_blocks, num_blocks, V,
                    dtype_code(kv_dtype), dtype_code(logits_dtype),
                    float(softmax_scale), int(attn_impl), int(reject_impl),
                    int(wait_limit_kcycles))


def workspace_size(dims: SpecDims) -> int:
    return int(lib().spec_workspace_size(ctypes.byref(dims)))


def workspace(dims: SpecDims, device="cuda", stream=None) -> torch.Tensor:
    """A zero-initialised device workspace for calls with these dims."""
    n = workspace_size(dims)
    if n == 0:
        raise SpecError("spec_workspace_size", 1)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    _check("spec_workspace_init",
           lib().spec_workspace_init(_ptr(ws), n, _stream(stream)))
    return ws


def device_status(ws: torch.Tensor, clear: bool = True, stream=None) -> int:
    """Bitmask of spec_status codes raised on the device (syncs the stream)."""
    out = ctypes.c_int32(0)
    _check("spec_get_device_status",
           lib().spec_get_device_status(_ptr(ws), _stream(stream), ctypes.byref(out),
                                        1 if clear else 0))
    return int(out.value)


def _bind():
    """The native argument checks of the step operators (raises if they have
    not been built)."""
    global _binding
    if _binding is None:
        lib()
        from . import _specbind
        _binding = _specbind
    return _binding


def _done(fn: str, result: int) -> int:
    if result < 0:
        raise SpecError(fn, -result)
    return result


def spec_verify_attn(q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens,
                     parent, out, lse, dims: SpecDims, ws, stream=None, window=None,
                     sinks=0, prefix=None, pages=None, page_counts=None) -> int:
    """spec_verify_attn; with a window (and sinks) spec_verify_attn_window, with
    `prefix` (block ids of the pages that all requests begin with, [n] int32)
    spec_verify_attn_prefix, with `pages` and `page_counts` (a selection by
    spec_page_select) spec_verify_attn_pages; one of the three at most.  A
    window of None or 0 is none, as in spec_block_tables."""
    windowed = window is not None and window != 0
    if sinks and not windowed:
        raise ValueError("sinks: a window is wanted with them")
    if (pages is None) != (page_counts is None):
        raise ValueError("pages and page_counts: both are wanted, or neither")
    if windowed + (prefix is not None) + (pages is not None) > 1:
        raise ValueError("window, prefix and pages: one of them at most")
    st = None if stream is None else stream.cuda_stream
    args = (q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, parent, out, lse, dims, ws)
    if windowed:
        return _done("spec_verify_attn_window",
                     _bind().verify_attn_window(*args, window, sinks, st))
    if prefix is not None:
        return _done("spec_verify_attn_prefix", _bind().verify_attn_prefix(*args, prefix, st))
    if pages is not None:
        return _done("spec_verify_attn_pages",
                     _bind().verify_attn_pages(*args, pages, page_counts, st))
    code = lib().spec_verify_attn(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
        _ptr(block_table), _ptr(ctx_lens), _ptr(parent), _ptr(out), _ptr(lse),
        ctypes.byref(dims), _ptr(ws), ws.numel(), _stream(stream))
    _check("spec_verify_attn", code)
    return lib().spec_last_launch_count()


def spec_reject_sample(target_logits, draft_logits, tokens, parent, temperature,
                       seed, offset, out_tokens, path, accepted_len, probe,
                       dims: SpecDims, ws, b_base=0, stream=None, top_k=None,
                       top_p=None) -> int:
    """spec_reject_sample; with top_k and / or top_p ([B] int32 / float32
    device tensors) spec_reject_sample_filtered."""
    if top_k is None and top_p is None:
        code = lib().spec_reject_sample(
            _ptr(target_logits), _ptr(draft_logits), _ptr(tokens), _ptr(parent),
            _ptr(temperature), int(seed) % (1 << 64), int(offset) % (1 << 64),
            int(b_base) % (1 << 64), _ptr(out_tokens), _ptr(path), _ptr(accepted_len),
            _ptr(probe), ctypes.byref(dims), _ptr(ws), ws.numel(), _stream(stream))
        _check("spec_reject_sample", code)
    else:
        code = lib().spec_reject_sample_filtered(
            _ptr(target_logits), _ptr(draft_logits), _ptr(tokens), _ptr(parent),
            _ptr(temperature), _ptr(top_k), _ptr(top_p), int(seed) % (1 << 64),
            int(offset) % (1 << 64), int(b_base) % (1 << 64), _ptr(out_tokens), _ptr(path),
            _ptr(accepted_len), _ptr(probe), ctypes.byref(dims), _ptr(ws), ws.numel(),
            _stream(stream))
        _check("spec_reject_sample_filtered", code)
    return lib().spec_last_launch_count()


def spec_block_tables(ctx_lens, row_start, parent, block_table, span, pool, pool_state, slots,
                      positions, ok, dims: SpecDims, ws, window=0, sinks=0, stream=None) -> int:
    """Block tables, slot map and positions of a step's new rows from the
    requests' lengths; pages come from and go back to a ring of free ids
    (block_table, span, pool and pool_state are updated in place).  A window of
    None or 0 is none: every page is held."""
    window = 0 if window is None else window
    return _done("spec_block_tables", _bind().block_tables(
        ctx_lens, row_start, parent, block_table, span, pool, pool_state, slots, positions, ok, dims,
        ws, window, sinks, None if stream is None else stream.cuda_stream))


def spec_page_bounds(k_cache, block_table, from_lens, ctx_lens, bounds, dims: SpecDims, ws,
                     stream=None) -> int:
    """Least and largest coordinates of the keys of every page from position
    from_lens (None: 0) to ctx_lens, to bounds [num_blocks, Hkv, 2, D]."""
    return _done("spec_page_bounds", _bind().page_bounds(
        k_cache, block_table, from_lens, ctx_lens, bounds, dims, ws,
        None if stream is None else stream.cuda_stream))


def spec_page_score(q, bounds, block_table, ctx_lens, scores, dims: SpecDims, ws,
                    stream=None) -> int:
    """How large a score the keys of each whole page can have with any query
    that reads the KV head, to scores [B, Hkv, max_blocks]."""
    return _done("spec_page_score", _bind().page_score(
        q, bounds, block_table, ctx_lens, scores, dims, ws,
        None if stream is None else stream.cuda_stream))


def spec_page_select(scores, ctx_lens, pages, page_counts, dims: SpecDims, ws, first=0, last=0,
                     stream=None) -> int:
    """The pages of each request and KV head to be read: the `first` and the
    `last` whole ones and those of largest score, pages.shape[2] together."""
    return _done("spec_page_select", _bind().page_select(
        scores, ctx_lens, pages, page_counts, dims, ws, first, last,
        None if stream is None else stream.cuda_stream))


def spec_qk_norm_rope(q, k, v, q_weight, k_weight, positions, inv_freq, q_out, k_out,
                      dims: SpecDims, ws, eps=1e-6, interleaved=False, slots=None, k_cache=None,
                      v_cache=None, stream=None) -> int:
    """RMS norm of every query and key head and the position rotation
    (2 * len(inv_freq) values of each head turn); with slots, the keys and
    values also go to the paged cache (a prefill; a verify step passes none, as
    spec_verify_attn appends its rows itself)."""
    return _done("spec_qk_norm_rope", _bind().qk_norm_rope(
        q, k, v, q_weight, k_weight, positions, inv_freq, q_out, k_out, dims, ws, eps, interleaved,
        slots, k_cache, v_cache, None if stream is None else stream.cuda_stream))


def spec_sample(logits, temperature, uniform, out_tokens, out_prob, ws, top_k=None, top_p=None,
                min_p=None, stream=None) -> int:
    """One token per row of logits [rows, V] (any row stride) from given
    uniforms, with temperature, top-k, top-p and min-p.  Drafts that the verify
    tests are drawn without min-p, which its laws do not have."""
    return _done("spec_sample", _bind().sample(
        logits, temperature, uniform, out_tokens, out_prob, ws, top_k, top_p, min_p,
        None if stream is None else stream.cuda_stream))


def spec_lm_head(hidden, weight, logits, ws, stream=None) -> int:
    """logits [rows, V] = hidden [rows, H] @ weight [V, H]^T (bf16)."""
    rows, H = hidden.shape
    V = weight.shape[0]
    code = lib().spec_lm_head(_ptr(hidden), _ptr(weight), rows, H, V, _ptr(logits), _ptr(ws),
                              ws.numel(), _stream(stream))
    _check("spec_lm_head", code)
    return lib().spec_last_launch_count()


def spec_reject_sample_lm_head(hidden_target, weight_target, hidden_draft, weight_draft,
                               target_logits, draft_logits, tokens, parent, temperature, seed,
                               offset, out_tokens, path, accepted_len, probe, dims: SpecDims, ws,
                               b_base=0, stream=None) -> int:
    """The target and draft LM heads with the verify decisions (the
    statistics formed in the LM heads' epilogue)."""
    code = lib().spec_reject_sample_lm_head(
        _ptr(hidden_target), _ptr(weight_target), hidden_target.shape[-1], _ptr(hidden_draft),
        _ptr(weight_draft), hidden_draft.shape[-1], _ptr(target_logits), _ptr(draft_logits),
        _ptr(tokens), _ptr(parent), _ptr(temperature), int(seed) % (1 << 64),
        int(offset) % (1 << 64), int(b_base) % (1 << 64), _ptr(out_tokens), _ptr(path),
        _ptr(accepted_len), _ptr(probe), ctypes.byref(dims), _ptr(ws), ws.numel(),
        _stream(stream))
    _check("spec_reject_sample_lm_head", code)
    return lib().spec_last_launch_count()


def spec_reject_sample_noalloc(target_logits, draft_logits, tokens, parent,
                               temperature, seed, offset, out_tokens, path,
                               accepted_len, probe, dims: SpecDims, b_base=0,
                               stream=None) -> None:
    """spec_reject_sample without a workspace, for callers that cannot
    allocate device memory; its scratch is a fixed 1 MiB array inside the
    library shared by every call, so overlapping calls race."""
    code = lib().spec_reject_sample_noalloc(
        _ptr(target_logits), _ptr(draft_logits), _ptr(tokens), _ptr(parent),
        _ptr(temperature), int(seed) % (1 << 64), int(offset) % (1 << 64),
        int(b_base) % (1 << 64), _ptr(out_tokens), _ptr(path), _ptr(accepted_len),
        _ptr(probe), ctypes.byref(dims), _stream(stream))
    _check("spec_reject_sample_noalloc", code)


def kv_commit(k_cache, v_cache, block_table, ctx_lens, new_ctx_lens, path,
              accepted_len, dims: SpecDims, ws, stream=None) -> int:
    code = lib().kv_commit(
        _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens),
        _ptr(new_ctx_lens), _ptr(path), _ptr(accepted_len), ctypes.byref(dims),
        _ptr(ws), ws.numel(), _stream(stream))
    _check("kv_commit", code)
    return lib().spec_last_launch_count()


def philox_block(key, counter):
    """Host-side Philox4x64-10 block of the library (for known-answer tests)."""
    K = (ctypes.c_uint64 * 2)(*[int(k) % (1 << 64) for k in key])
    C = (ctypes.c_uint64 * 4)(*[int(c) % (1 << 64) for c in counter])
    O = (ctypes.c_uint64 * 4)()
    lib().spec_philox_block(K, C, O)
    return [int(x) for x in O]
