"""What the C ABI's calls on shared prefixes and selected pages refuse before
anything is launched (no GPU: no call here gets past its checks)."""
import ctypes

import pytest

import speculative_decoding_verification_19_gb300 as sv
from speculative_decoding_verification_19_gb300 import build as sv_build

P = ctypes.c_void_p(4096)  # an address that no refused call looks at
BIG = 1 << 40
INVALID, UNSUPPORTED = 1, 3


@pytest.fixture(scope="module")
def lib():
    sv_build.build()
    return sv.lib()


def dims(**kw):
    return sv.make_dims(**(dict(B=2, M=3, Hq=4, Hkv=2, D=128, max_blocks=4, num_blocks=9) | kw))


def prefix(L, d=None, n=32, table=P, q=P, ws=P, size=BIG):
    return L.spec_verify_attn_prefix(q, P, P, P, P, P, P, None, table, n, P, None,
                                     ctypes.byref(d or dims()), ws, size, None)


def pages(L, d=None, n=2, sel=P, counts=P, out=P):
    return L.spec_verify_attn_pages(P, P, P, P, P, P, P, None, sel, counts, n, out, None,
                                    ctypes.byref(d or dims()), P, BIG, None)


def select(L, n=4, first=0, last=0, scores=P, d=None, ws=P, size=16):
    return L.spec_page_select(scores, P, n, first, last, P, P, ctypes.byref(d or dims()), ws, size,
                              None)


def bounds(L, d=None, k=P, b=P, ws=P, size=16):
    return L.spec_page_bounds(k, P, None, P, b, ctypes.byref(d or dims()), ws, size, None)


def score(L, d=None, q=P, s=P, ws=P, size=16):
    return L.spec_page_score(q, P, P, P, s, ctypes.byref(d or dims()), ws, size, None)


@pytest.mark.parametrize("n", [0, -16, 8, 17, 64, 80, 1 << 30])
def test_prefix_lengths(lib, n):
    assert prefix(lib, n=n) == INVALID


def test_prefix_arguments(lib):
    assert prefix(lib, table=None) == INVALID and prefix(lib, q=None) == INVALID
    assert prefix(lib, q=ctypes.c_void_p(4098)) == INVALID
    assert prefix(lib, ws=None) == INVALID and prefix(lib, size=64) == INVALID
    assert prefix(lib, d=dims(M=33, Hq=8)) == UNSUPPORTED  # 132 rows per KV head
    assert prefix(lib, d=dims(D=96)) == UNSUPPORTED
    assert prefix(lib, d=dims(max_blocks=1 << 27)) == UNSUPPORTED  # positions past 2^30
    assert lib.spec_last_launch_count() == 0


def test_pages_arguments(lib):
    assert pages(lib, n=0) == INVALID and pages(lib, n=-1) == INVALID
    assert pages(lib, sel=None) == INVALID and pages(lib, counts=None) == INVALID
    assert pages(lib, out=None) == INVALID
    assert pages(lib, d=dims(M=128, Hq=4)) == UNSUPPORTED
    assert pages(lib, d=dims(max_blocks=1 << 27)) == UNSUPPORTED


@pytest.mark.parametrize("n,first,last", [(0, 0, 0), (-3, 0, 0), (4, -1, 0), (4, 0, -1), (4, 3, 2),
                                          (4, 2**31 - 1, 2**31 - 1)])
def test_selection_counts(lib, n, first, last):
    assert select(lib, n, first, last) == INVALID


def test_page_calls_arguments(lib):
    for call in (select, bounds, score):
        assert call(lib, ws=None) == INVALID and call(lib, size=15) == INVALID
        assert call(lib, ws=ctypes.c_void_p(4104)) == INVALID
        assert call(lib, d=dims(B=1 << 16)) == UNSUPPORTED
        assert call(lib, d=dims(max_blocks=0)) == INVALID
        assert call(lib, d=dims(Hq=3)) == INVALID
    assert select(lib, scores=None) == INVALID
    assert bounds(lib, k=None) == INVALID and bounds(lib, b=None) == INVALID
    assert bounds(lib, b=ctypes.c_void_p(4104)) == INVALID
    assert score(lib, q=None) == INVALID and score(lib, s=None) == INVALID
    assert score(lib, q=ctypes.c_void_p(4104)) == INVALID


@pytest.mark.parametrize("scale", [-0.1, float("nan"), float("inf")])
def test_scales(lib, scale):
    assert prefix(lib, d=dims(softmax_scale=scale)) == INVALID
    assert pages(lib, d=dims(softmax_scale=scale)) == INVALID


def test_lists_past_32_bit_counts(lib):
    assert select(lib, (1 << 30) + 1) == UNSUPPORTED and pages(lib, n=(1 << 30) + 1) == UNSUPPORTED
    wide = dims(Hq=1 << 12, Hkv=1 << 12, max_blocks=1 << 19, M=1)
    assert pages(lib, d=wide) == UNSUPPORTED and prefix(lib, d=wide) == UNSUPPORTED


def test_workspace_has_room_for_a_prefix(lib):
    # partials of the prefix: at least a slot of every 256 rows of a KV head
    d = dims(B=128, M=5, Hq=64, Hkv=8, max_blocks=2049)
    assert sv.workspace_size(d) >= 8 * 20 * 256 * 132 * 4
