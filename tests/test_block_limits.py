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


def _addresses(n):
    """Far enough apart for any size here; never dereferenced."""
    return [(i + 1) << 48 for i in range(n)]


@pytest.mark.parametrize("B,D", [(4096, (1 << 20) + 1), (131072, 4194298), (1 << 20, (1 << 19) - 8)])
def test_conv_grids_past_the_launch_limit_are_refused(kda, B, D):
    """2^32 threads or more, as many tokens wide as the type and the channels allow."""
    lib, st = kda.load_library(), kda
    p = _addresses(7)
    for dtype in (st.KDA_F32, st.KDA_BF16):
        assert lib.kda_short_conv_fwd(*p, B, 1, D, 4, 1, dtype, None) == st.KDA_ERR_UNSUPPORTED
        assert lib.kda_short_conv_step(*p[:5], B, D, 4, 1, dtype, None) == st.KDA_ERR_UNSUPPORTED
        assert lib.kda_short_conv_bwd(*_addresses(12), lib.kda_short_conv_bwd_workspace_bytes(B, 1, D, 4), B, 1, D, 4,
                                      1, dtype, None) == st.KDA_ERR_UNSUPPORTED


@pytest.mark.parametrize("B,T,D,N,G", [(1 << 23, 1, 2, 1, 2), (1 << 20, 1, 1024, 4, 1), (1 << 18, 40, 64, 64, 64)])
def test_scan_grids_past_the_launch_limit_are_refused(kda, B, T, D, N, G):
    lib, st = kda.load_library(), kda
    size = (B, T, D, N, G)
    for dtype in (st.KDA_F32, st.KDA_BF16):
        assert lib.kda_selective_scan_fwd(*_addresses(13), lib.kda_selective_scan_fwd_workspace_bytes(*size), *size, 1,
                                          dtype, None) == st.KDA_ERR_UNSUPPORTED
        assert lib.kda_selective_scan_bwd(*_addresses(22), lib.kda_selective_scan_bwd_workspace_bytes(*size), *size, 1,
                                          dtype, None) == st.KDA_ERR_UNSUPPORTED


def test_scan_step_and_joins_past_the_launch_limit_are_refused(kda):
    lib, st = kda.load_library(), kda
    # 16 lanes a channel of four sequences
    assert lib.kda_selective_scan_step(*_addresses(10), 1 << 16, 1 << 14, 64, 1, 1, st.KDA_BF16, None) == \
        st.KDA_ERR_UNSUPPORTED
    # the gradients' own grid fits; the one over sequences, channels and states in two directions does not
    size = (8192, 32, 4096, 64, 1)
    assert lib.kda_selective_scan_bwd(*_addresses(22), lib.kda_selective_scan_bwd_workspace_bytes(*size), *size, 1,
                                      st.KDA_BF16, None) == st.KDA_ERR_UNSUPPORTED
    # nor does the sum of the rows of B and C here
    size = (1 << 14, 1 << 14, 64, 64, 1)
    assert lib.kda_selective_scan_bwd(*_addresses(22), lib.kda_selective_scan_bwd_workspace_bytes(*size), *size, 1,
                                      st.KDA_BF16, None) == st.KDA_ERR_UNSUPPORTED
