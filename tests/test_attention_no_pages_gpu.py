"""Attention over a cache of no pages, by each kernel that a table and its rows may choose: nothing is seen, whatever
the table and the lengths say, and the workspace is the chosen kernel's."""

import math

import pytest
import torch

from test_attention_gpu import BF16, E4M3, F32, kda  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,new,Hq,Hk,D,page,per,dtype", [
    (300, 32, 8, 8, 64, 64, 30, BF16),      # more than 16384 units by the table: the kernel for many rows, no workspace
    (300, 32, 8, 8, 64, 64, 1, BF16),       # fewer: the one for few
    (1, 1, 4, 1, 128, 16, 5000, F32), (3, 50, 4, 1, 128, 128, 4000, F32), (2, 600, 2, 2, 256, 32, 20, BF16),
    (70, 20, 2, 1, 256, 16, 900, F32)])
def test_no_pages(kda, B, new, Hq, Hk, D, page, per, dtype):  # noqa: F811
    N = B * new
    q = torch.randn((N, Hq, D), device="cuda").to(dtype)
    kc = torch.empty((0, Hk, page, D), dtype=E4M3, device="cuda")
    vc = torch.empty((0, Hk, D, page), dtype=E4M3, device="cuda")
    s = torch.empty((0, Hk), device="cuda")
    table = torch.zeros((B, per), dtype=torch.int32, device="cuda")
    context = torch.full((B,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    starts = (torch.arange(B + 1) * new).int().cuda()
    need = kda.kda_cache_attention_workspace_bytes(N, B, Hq, Hk, D, page, per, new)
    ws = torch.full((need + 4096,), 7, dtype=torch.uint8, device="cuda")
    o, lse = kda.kda_cache_attention(q, kc, vc, s, s, table, context, q_start=starts, max_queries=new, want_lse=True,
                                     workspace=ws[:need])
    assert not o.any() and (lse == -math.inf).all() and (ws[need:] == 7).all()
