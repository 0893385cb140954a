"""Attention with row starts that count the call's rows many times over: nothing outside the buffers is read or written
(how the line of units is cut is tests/test_attention_line.py), and the next call is right."""

import pytest
import torch

from test_attention_gpu import BF16, E4M3, check_attention, gen, kda, layer  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,N,Hq,Hk,page,per,most", [
    (4096, 4096, 64, 8, 64, 512, 1),             # the kernel for few queries: 1.7e10 units
    (400, 50000, 1, 1, 128, 15000, 129),         # the one for many: 2.3e9
    (200, 300, 4, 2, 64, 40, 3)])                # few enough to be done
def test_row_starts_that_alternate(kda, B, N, Hq, Hk, page, per, most):  # noqa: F811
    D, pages = 64, 3
    g = gen(B)
    kc = torch.randint(-128, 128, (pages, Hk, page, D), generator=g).to(torch.int8).cuda()
    vc = torch.randint(-128, 128, (pages, Hk, D, page), generator=g).to(torch.int8).cuda()
    ks, vs = torch.rand((2, pages, Hk), generator=g).cuda()
    q = torch.randn((N, Hq, D), generator=g).to(BF16).cuda()
    table = torch.randint(0, pages, (B, per), generator=g).int().cuda()
    context = torch.full((B,), page * per, dtype=torch.int32, device="cuda")
    starts = (torch.arange(B + 1) % 2 * N).int().cuda()
    need = kda.kda_cache_attention_workspace_bytes(N, B, Hq, Hk, D, page, per, most)
    ws = torch.full((need + 4096,), 7, dtype=torch.uint8, device="cuda")
    room = torch.full((N + 64, Hq, D), 7.0, dtype=BF16, device="cuda")
    kda.kda_cache_attention(q, kc, vc, ks, vs, table, context, q_start=starts, max_queries=most, out=room[32:N + 32],
                            workspace=ws[:need])
    torch.cuda.synchronize()
    assert (ws[need:] == 7).all() and (room[:32] == 7).all() and (room[N + 32:] == 7).all()
    assert torch.isfinite(room).all()
    x = layer([300, 200, 100], [3] * 3, 4, 2, 64, 32, E4M3, BF16, 49)
    check_attention(kda, *x, "after", most=3)
