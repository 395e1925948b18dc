"""The workspace's size beside the forms of the attention on views: what they keep lies
where calls without a view have partials, and a call without a view does with what it
needs itself (no GPU: no call here gets past its checks)."""
import ctypes

import pytest
import torch

import speculative_decoding_verification_19_gb300 as sv
from speculative_decoding_verification_19_gb300 import build as sv_build

P = ctypes.c_void_p(4096)  # an address that no refused call looks at
INVALID, UNSUPPORTED = 1, 3
F32 = torch.float32

# dims, bytes that the calls without a view need, bytes that those on views add at most
SIZES = [
    (dict(B=128, M=5, Hq=64, Hkv=8, max_blocks=2049), 190620672, 0),
    (dict(B=256, M=16, Hq=64, Hkv=8, max_blocks=2049), 1218894080, 0),
    (dict(B=64, M=9, V=32000), 4533504, 256),  # no attention: a table of one page a request
    (dict(B=1, M=5, Hq=32, Hkv=8, max_blocks=260), 5530880, 8 * 260 * 4 + 256),  # a table
    (dict(B=8, M=8, Hq=32, Hkv=8, max_blocks=130), 9789440, 64 * 130 * 4 + 256),
    (dict(B=1, M=8, Hq=1, Hkv=1, D=64, max_blocks=1900, kv_dtype=F32), 1156096, 0),
    # single tokens behind up to 32768 positions: a pass' 168 partials of 256 rows
    (dict(B=64, M=1, Hq=32, Hkv=8, max_blocks=2049), 9664768, 168 * 256 * 132 * 4 + 512),
    # 456 partials of 64 rows of 64 fp32 values
    (dict(B=8, M=64, Hq=8, Hkv=8, D=64, max_blocks=260, kv_dtype=F32), 18266368,
     456 * 64 * 68 * 4 + 1024)]


@pytest.fixture(scope="module")
def lib():
    sv_build.build()
    return sv.lib()


@pytest.mark.parametrize("kw,plain,more", SIZES)
def test_size(lib, kw, plain, more):
    n = sv.workspace_size(sv.make_dims(**kw))
    assert plain <= n <= plain + more


def plain_call(L, d, size):
    return L.spec_verify_attn(P, P, P, P, P, P, P, None, P, None, ctypes.byref(d), P, size, None)


def prefix_call(L, d, size):
    return L.spec_verify_attn_prefix(P, P, P, P, P, P, P, None, P, 16, P, None, ctypes.byref(d), P,
                                     size, None)


@pytest.mark.parametrize("kw,plain", [(k, n) for k, n, _ in SIZES])
def test_calls_without_a_view_need_no_room_for_one(lib, kw, plain):
    d = sv.make_dims(**kw)
    d.attn_impl = 9  # refused in any case
    assert plain_call(lib, d, plain - 1) == INVALID
    d.attn_impl, d.kv_dtype = sv.ATTN_TENSOR_CORES, 1  # fp32: not on tensor cores
    assert plain_call(lib, d, plain) == UNSUPPORTED


@pytest.mark.parametrize("kw,plain", [(k, n) for k, n, _ in SIZES if k.get("max_blocks", 1) > 1])
def test_calls_on_views_need_all_of_it(lib, kw, plain):
    d = sv.make_dims(**kw)
    n = sv.workspace_size(d)
    assert prefix_call(lib, d, n - 1) == INVALID
    d.attn_impl = sv.ATTN_TENSOR_CORES
    d.D = 64  # not on tensor cores
    assert prefix_call(lib, d, 1 << 40) == UNSUPPORTED


@pytest.mark.parametrize("kw,n", [
    (dict(D=0), 90880), (dict(D=-1), 78592), (dict(Hq=3, Hkv=2), 858624), (dict(Hkv=0), 40960),
    (dict(Hq=1 << 25, M=128), None), (dict(D=-1, Hq=40, Hkv=1, kv_dtype=F32), None),
    (dict(B=2**31 - 1, Hq=2**31 - 1, Hkv=2**31 - 1, max_blocks=2**31 - 1), None)])
def test_sizes_of_dims_that_calls_refuse(lib, kw, n):
    """A size, and no more: nothing is divided by what they multiply to."""
    got = sv.workspace_size(sv.make_dims(**(dict(B=2, M=3, Hq=4, Hkv=2, max_blocks=40) | kw)))
    assert n is None or got == n


def test_groups_past_32_bits_are_refused(lib):
    d = sv.make_dims(B=2, M=128, Hq=1 << 25, Hkv=1, max_blocks=40)  # 2^32 rows per KV head
    assert plain_call(lib, d, 2**64 - 1) == UNSUPPORTED
    assert prefix_call(lib, d, 2**64 - 1) == UNSUPPORTED
