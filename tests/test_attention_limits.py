"""Sizes at the ends of what the cache attention accepts, on the host (no GPU needed: nothing here reaches a launch)."""

import os

import pytest


@pytest.fixture(scope="module")
def st():
    from gated_delta_rule_101_amd import kda
    if not os.path.exists(kda.LIBRARY):
        from gated_delta_rule_101_amd.build_lib import build_library
        build_library()
    return kda


@pytest.mark.parametrize("N,B,Hq,Hk,D,page,per", [(6, 3, 8, 2, 128, 64, 4), (6, 3, 8, 2, 256, 64, 400), (1, 1, 65535, 1, 256, 16, 9),
                                                  (3000, 7, 32, 8, 128, 16, 1 << 20), (32767, 1, 65535, 1, 64, 16, 1)])
def test_more_rows_than_there_are(st, N, B, Hq, Hk, D, page, per):
    """The longest sequence has no more rows than the call: a larger number chooses as that does."""
    ws = st.load_library().kda_cache_attention_workspace_bytes
    want = ws(N, B, Hq, Hk, D, page, per, N)
    for most in (N + 1, 1 << 20, 1 << 29, 1 << 30, 3 << 29, 2 ** 31 - 1):
        assert ws(N, B, Hq, Hk, D, page, per, most) == want, most
    assert ws(N, B, Hq, Hk, D, page, per, 0) == ws(N, B, Hq, Hk, D, page, per, 1)


@pytest.mark.parametrize("B,N,Hq,Hk,page,per", [
    (11863283, 1 << 16, 32767, 32767, 128, (1 << 24) - 3),   # sequences' blocks past 2^63 units: a negative number
    ((1 << 24) - 1, 1 << 16, 32767, 32767, 128, (1 << 24) - 3), ((1 << 24) - 1, (1 << 24) - 1, 100, 1, 16, 1 << 26),
    (1, 1 << 15, 32767, 32767, 16, 1 << 26)])
def test_lines_past_any_length_are_refused(st, B, N, Hq, Hk, page, per):
    lib = st.load_library()
    p = [(i + 1) << 58 for i in range(11)]                   # apart enough for any size here; never dereferenced
    for most in (1, 2 ** 31 - 1):
        need = lib.kda_cache_attention_workspace_bytes(N, B, Hq, Hk, 256, page, per, most)
        assert 0 <= need < 1 << 40
        # float32 rows of 256 channels have a line whatever their number is
        assert lib.kda_cache_attention(*p, need, N, B, Hq, Hk, 256, 9, page, per, most, 0.1, st.KDA_CODE_E4M3, st.KDA_F32,
                                       None) == st.KDA_ERR_UNSUPPORTED
