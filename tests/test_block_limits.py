"""Sizes at the ends of what the block operators accept, on the host (no GPU
needed: nothing here reaches a launch)."""

import os

import pytest


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_101_amd import kda
    if not os.path.exists(kda.LIBRARY):
        from gated_delta_rule_101_amd.build_lib import build_library
        build_library()
    return kda


@pytest.mark.parametrize("B,T,D,W", [(131072, 1, 4194301, 4), (65536, 1, 8388607, 4), (1 << 16, 1, (1 << 24) - 257, 2),
                                     ((1 << 24) - 1, 1, 1 << 15, 3), (1, (1 << 24) - 1, (1 << 16) - 1, 4), (3, 2, 7, 4)])
def test_conv_workspace_of_the_largest_sizes(kda, B, T, D, W):
    """dw and dbias of every run of up to 256 tokens: a size, for any that is accepted."""
    n = kda.load_library().kda_short_conv_bwd_workspace_bytes(B, T, D, W)
    row = 4 * D * (W + 1)
    assert n % (B * row) == 0 and -(-T // 256) <= n // (B * row) <= -(-T // 4)
