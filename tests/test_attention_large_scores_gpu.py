"""Attention whose scores are large numbers, up to 2^33 with steps of 2^17 and more between them: each row is the value of
its largest score, to the roundings of the value and of the one weight."""

import math

import pytest
import torch

from attention_reference import HALF
from test_attention_gpu import BF16, E4M3, F32, INT8, close, gen, kda  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,G,Hk,D,dtype", [
    (1, 4, 2, 64, BF16), (9, 1, 1, 128, F32), (50, 1, 2, 64, BF16), (60, 2, 40, 64, F32), (33, 1, 2, 256, F32),
    (200, 2, 1, 128, BF16), (150, 2, 1, 64, F32), (90, 2, 1, 256, BF16)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("low", [2.0 ** 14, 1.7 * 2.0 ** 16, 2.0 ** 19])
def test_scores_far_apart(kda, rows, G, Hk, D, dtype, sign, low):  # noqa: F811
    page, pages = 64, 10
    total = page * pages - 13
    g = gen(rows)
    kc = torch.zeros(pages, Hk, page, D, dtype=torch.int8)
    kc[..., 0] = (64 + torch.arange(page)).to(torch.int8)       # places climb inside a page and from page to page
    ks = (low * 2.0 ** torch.arange(pages))[:, None].expand(pages, Hk).contiguous()
    vc = torch.randint(-127, 128, (pages, Hk, D, page), generator=g).to(torch.int8)
    vs = 0.01 + torch.rand((pages, Hk), generator=g)
    q = torch.zeros(rows, G * Hk, D, dtype=dtype)
    q[..., 0] = sign
    o, lse = kda.kda_cache_attention(*[t.cuda() for t in (q, kc, vc, ks, vs)], torch.arange(pages).int()[None].cuda(),
                                     torch.tensor([total]).int().cuda(), q_start=torch.tensor([0, rows]).int().cuda(),
                                     max_queries=rows, scale=1.0, want_lse=True)
    at = total - rows + torch.arange(rows) if sign > 0 else torch.zeros(rows).long()
    head = torch.arange(G * Hk) // G
    v = vc.double()[at // page][:, head, :, :].gather(3, (at % page)[:, None, None, None].expand(rows, G * Hk, D, 1))[..., 0]
    v = v * vs.double()[at // page][:, head][..., None]
    # logarithms of value scales are off by less than 2^-20 (below 8), weights by 2^-11 (two parts: 2^-22)
    part = 2.0 ** -11 if dtype is BF16 else 2.0 ** -22
    close(o, v, (HALF[dtype] + part + 2.0 ** -18) * v.abs() + 1e-30, "out")
    z = sign * (64 + at % page).double() * low * 2.0 ** (at // page).double()
    z = z[:, None].expand(rows, G * Hk)
    close(lse, z, 2.0 ** -21 * z.abs(), "lse")
