"""Kernels that start before their predecessor on the stream has ended
(programmatic dependent launch) take no restrict-qualified inputs.

Such a kernel waits (pdl_wait) before it reads what the predecessor writes.  A
load through a restrict-qualified pointer to constant data may be moved above
the wait, or be served by the read-only path, and then sees the memory from
before the write.  Any call of a step may stand before any other, so the rule
holds for every input of every kernel that waits: block tables and slots come
from spec_block_tables, queries, keys and cache rows from spec_qk_norm_rope,
tokens from spec_sample, logits from spec_lm_head, lengths from kv_commit.
For the same reason nothing is read by an explicit load of the read-only path.
Checked in the source: a race shows on a GPU by luck alone.
"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_verification_19_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def closing(text, at, pair):
    """Index behind the bracket that closes the one at `at`."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i + 1
    raise AssertionError("unbalanced")


def kernels(path):
    """(name, parameters, body) of every kernel defined in a file."""
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"__global__\s+void\b", text):
        at = m.end()
        bounds = re.match(r"\s*__launch_bounds__\s*\(", text[at:])
        if bounds:
            at = closing(text, at + bounds.end() - 1, "()")
        name = re.match(r"\s*(\w+)\s*\(", text[at:])
        stop = closing(text, at + name.end() - 1, "()")
        if text[stop:].lstrip()[0] != "{":
            continue  # a declaration
        brace = text.index("{", stop)
        yield name[1], text[at + name.end():stop - 1], text[brace:closing(text, brace, "{}")]


@pytest.mark.parametrize("path", SOURCES + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))),
                         ids=os.path.basename)
def test_no_loads_of_the_read_only_path(path):
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"__ldg\b|ld\.global\.nc", text)


def test_the_kernels_are_found():
    found = {k[0]: "pdl_wait()" in k[2] for path in SOURCES for k in kernels(path)}
    assert found["kv_append_kernel"] and found["attn_tc_kernel"] and found["rs_tree_walk_kernel"]
    assert not found["attn_split_kernel"] and len(found) >= 20


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_waiting_kernels_take_no_restricted_inputs(path):
    for name, params, body in kernels(path):
        if "pdl_wait()" not in body:
            continue
        for p in params.split(","):
            if "__restrict__" in p:
                assert "const" not in p and not re.search(r"[kv]_cache", p), (name, p.strip())
