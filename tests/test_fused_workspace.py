"""Workspace sizes of the fused operators: one sized for the most tokens serves every smaller call (no GPU)."""
import pytest

import weight_only_int4_linear_b200 as w4
from weight_only_int4_linear_b200 import build as w4build

TOKENS = [1, 2, 4, 5, 8, 9, 16, 17, 64, 65, 128, 129, 256, 257, 4096]  # both sides of every change of kernel or tile
WEIGHTS = [(16, 1024), (10240, 8192), (152064, 1024), (8192, 28672), (4096, 11008)]


@pytest.fixture(scope="module")
def lib():
    w4build.build()
    return w4.load()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", WEIGHTS)
def test_sizes_do_not_fall_with_more_tokens(lib, N, K, group):
    for size in (w4.fused_workspace_bytes, w4.dx_workspace_bytes):
        last = 0
        for M in TOKENS:
            b = size(M, N, K, group)
            assert b >= last, (M, b, last)
            last = b
