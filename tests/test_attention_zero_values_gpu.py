"""Attention over pages whose values are all zero, which an append leaves with scale 0."""

import math

import pytest
import torch

import attention_reference as ref
from test_attention_gpu import BF16, F32, INT8, check_attention, close, gen, kda  # noqa: F401

pytestmark = pytest.mark.gpu


def climbing(new, dtype, above, ordinary):
    """One sequence of 32 pages of 64 tokens and 128 heads, so that a wave walks several tiles of a row: the scores
    of pages 20 .. 31 stand `above` over those of pages 0 .. 19, in units of the exponent (base 2).  Values are zero
    but for those of the last `ordinary` pages."""
    H, D, page, pages = 128, 64, 64, 32
    g = gen(new)
    kc = torch.zeros(pages, H, page, D, dtype=torch.int8)
    kc[..., 0] = 64
    ks = torch.full((pages, H), math.log(2) / 64)
    ks[20:] *= 1 + above
    v = torch.randn(pages, H, page, D, generator=g)
    v[:pages - ordinary] = 0
    vc, vs = ref.fill(v, INT8, True)
    q = torch.zeros(new, H, D, dtype=dtype)
    q[..., 0] = 1
    return (q, [kc, vc, ks, vs], torch.arange(pages).int()[None], torch.tensor([page * pages]).int(),
            torch.tensor([0, new]).int())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [1, 40, 130])
@pytest.mark.parametrize("ordinary", [0, 3])
def test_maxima_that_climb_over_zero_values(kda, new, dtype, ordinary):  # noqa: F811
    """Weights stay finite as float16 where the maximum grows by just less than what leaves the base as it is."""
    for above in (1.0, 1.9996, 1.9999, 2.0, 3.0):
        x = climbing(new, dtype, above, ordinary)
        o, _ = check_attention(kda, *x, f"above {above}", most=new, scale=1.0)
        assert ordinary or not o.any()
