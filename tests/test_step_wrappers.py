"""The Python calls' own handling of arguments, without a GPU: a model without a
window passes the same value (None or 0) to the block tables and the attention."""
import pytest
import torch

import speculative_decoding_verification_19_gb300 as sv
from speculative_decoding_verification_19_gb300 import _native

DIMS = sv.make_dims(B=2, M=3, Hq=4, Hkv=2, D=128, max_blocks=4, num_blocks=9)


class Library:
    """Records the entry point that a call reaches."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def reached(monkeypatch):
    rec = Library()
    monkeypatch.setattr(_native, "lib", lambda: rec)
    monkeypatch.setattr(_native, "_bind", lambda: rec)
    monkeypatch.setattr(_native, "_ptr", lambda t: None)
    monkeypatch.setattr(_native, "_stream", lambda s: None)
    return rec


def attention(**kw):
    x = torch.zeros(1)
    return sv.spec_verify_attn(x, x, x, x, x, x, x, None, x, None, DIMS, x, **kw)


@pytest.mark.parametrize("kw", [{}, dict(window=None), dict(window=0), dict(window=0, sinks=0)])
def test_no_window(reached, kw):
    attention(**kw)
    assert reached.calls[0][0] == "spec_verify_attn"


def test_a_window(reached):
    attention(window=7, sinks=2)
    (name, args), = reached.calls
    assert name == "verify_attn_window" and args[12:14] == (7, 2)


@pytest.mark.parametrize("window", [None, 0])
def test_sinks_without_a_window_are_refused(reached, window):
    with pytest.raises(ValueError):
        attention(window=window, sinks=4)
    assert not reached.calls


@pytest.mark.parametrize("window,passed", [(None, 0), (0, 0), (9, 9)])
def test_block_tables_without_a_window(reached, window, passed):
    x = torch.zeros(1)
    sv.spec_block_tables(x, None, None, x, x, x, x, x, x, None, DIMS, x, window=window)
    (name, args), = reached.calls
    assert name == "block_tables" and args[12] == passed
