"""Windowed attention on the CUDA cores at every number of rows per KV head that
has an instance of its own, up to 128, in both types and head sizes; trees to
128 nodes (both words of a row's mask).

Tolerances as in test_gpu_step.py: bf16 2^-8 of sum p |v| and of the output
(the CUDA cores round the output alone), fp32 1e-4.
"""
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import speculative_decoding_verification_19_gb300 as sv  # noqa: E402
from synth import workload  # noqa: E402
from test_gpu_step import window_case  # noqa: E402

CTX = [0, 3, 31, 64, 129, 500]


@pytest.mark.parametrize("name", ["chain_gqa_128k", "tiny_chain"])  # bf16, fp32
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("M,group", [(1, 1), (8, 1), (9, 1), (4, 4), (17, 1), (4, 8), (11, 3), (64, 1),
                                     (9, 7), (65, 1), (32, 4), (128, 1)])
def test_rows_per_head(name, D, M, group):
    wl = workload(name).scaled(gamma=M - 1, Hq=2 * group, Hkv=2, D=D)
    for window, sinks, tree in ((20, 3, False), (100, 80, True)):
        window_case(wl, CTX, window, sinks, tree, seed=M + group, impl=sv.ATTN_CUDA_CORES)


@pytest.mark.parametrize("name,D", [("chain_gqa_128k", 64), ("tiny_chain", 64), ("tiny_chain", 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (31, 32), (33, 31), (64, 5), (4000, 0)])
def test_windows_on_wide_trees(name, D, window, sinks):
    """What the kernel choice takes by itself: fp32, and bf16 heads of 64."""
    wl = workload(name).scaled(gamma=69, Hq=1, Hkv=1, D=D)
    window_case(wl, CTX, window, sinks, True, seed=window, impl=0)


def test_bf16_heads_of_64_over_long_contexts():
    wl = workload("chain_gqa_128k").scaled(gamma=4, Hq=8, Hkv=2, D=64)
    window_case(wl, [9000, 20, 12345], 4096, 100, False, seed=3, impl=0)
    window_case(wl, [9000, 20, 12345], 300, 0, True, seed=4, impl=0)
