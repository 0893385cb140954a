"""Attention over pages whose key scale is not finite, with codes that are not zero: the rows that see their tokens are
NaN, whatever the signs of the products, and the others as they are without."""

import math

import pytest
import torch

from test_attention_gpu import BF16, E4M3, F32, INT8, gen, kda  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,dtype", [(INT8, BF16), (E4M3, F32)])
@pytest.mark.parametrize("new", [1, 20, 40, 150])
@pytest.mark.parametrize("scale", [math.inf, -math.inf, math.nan])
def test_key_scales_that_are_not_finite(kda, new, kind, dtype, scale):  # noqa: F811
    D, page, total, Hk = 64, 16, 400, 2
    pages = total // page
    g = gen(new)
    sign = torch.ones(pages, 1, 1, 1)
    sign[::3] = -1                                            # products of either sign
    kc = (sign * torch.randint(1, 100, (pages, Hk, page, D), generator=g)).to(kind)
    vc = torch.randint(-100, 100, (pages, Hk, D, page), generator=g).to(kind)
    ks, vs = 0.001 + torch.rand((2, pages, Hk), generator=g) * 0.01
    q = torch.rand((new, 4, D), generator=g).to(dtype)
    args = [kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), torch.arange(pages).int().cuda()[None], torch.tensor([total]).int().cuda()]
    kw = dict(q_start=torch.tensor([0, new]).int().cuda(), max_queries=new, want_lse=True)
    for sign in (1, -1):
        x = sign * q.cuda()
        clean, clean_lse = kda.kda_cache_attention(x, *args, **kw)
        assert torch.isfinite(clean).all() and torch.isfinite(clean_lse).all()
        for p in (0, 3, pages - 1):
            bad = ks.clone()
            bad[p, 0] = scale
            o, lse = kda.kda_cache_attention(x, *args[:2], bad.cuda(), *args[3:], **kw)
            sees = torch.zeros((new, 4), dtype=torch.bool)
            sees[:, :2] = (total - new + torch.arange(new) >= p * page)[:, None]     # heads 0 and 1 read key head 0
            assert torch.equal(torch.isnan(o).all(-1).cpu(), sees) and torch.equal(torch.isnan(lse).cpu(), sees), (sign, p)
            # the same products and sums, but for the base of their exponents: weights are rounded once more, in
            # float16 (bfloat16 rows: 2^-11 each, on values up to 1.1) or two parts of it (2^-22), then the outputs
            same, near = ~sees.cuda(), ((2.0 ** -7, 2.0 ** -10) if dtype is BF16 else (2.0 ** -22, 2.0 ** -20))
            x0, y0 = o[same].float(), clean[same].float()
            assert ((x0 - y0).abs() <= near[0] * y0.abs() + 1.2 * near[1]).all(), (sign, p)
            x0, y0 = lse[same], clean_lse[same]                # sums of 400 terms
            assert ((x0 - y0).abs() <= 2.0 ** -22 * y0.abs() + 2.0 ** -15).all(), (sign, p)
        # all of them
        o, lse = kda.kda_cache_attention(x, *args[:2], torch.full_like(args[2], scale), *args[3:], **kw)
        assert torch.isnan(o).all() and torch.isnan(lse).all()
