"""Attention over pages whose value scales lie far apart, held to the size of what each row itself sees: neither a page
that a row does not see nor one that has no weight in it may take bits from it."""

import math

import pytest
import torch

from attention_reference import HALF
from test_attention_gpu import BF16, E4M3, F32, INT8, close, gen, kda  # noqa: F401

pytestmark = pytest.mark.gpu


def exact(q, kc, vc, ks, vs, table, context, starts, scale):
    """(out, tolerance) in float64 on the CPU.  Tolerances are relative to a row's own sum of weight x |value|."""
    N, Hq, D = q.shape
    _, Hk, page, _ = kc.shape
    out, tol = torch.zeros(N, Hq, D).double(), torch.zeros(N, Hq, D).double()
    bf = q.dtype is BF16
    for b in range(table.shape[0]):
        r0, r1, ctx = int(starts[b]), int(starts[b + 1]), int(context[b])
        ids = table[b, :-(-ctx // page)].long()
        pos = ctx - (r1 - r0) + torch.arange(r1 - r0)
        seen = torch.arange(ctx)[None] <= pos[:, None]
        for hq in range(Hq):
            h = hq * Hk // Hq
            K = (kc[ids, h].double() * ks[ids, h].double()[:, None, None]).reshape(-1, D)[:ctx]
            code = vc[ids, h].double().transpose(1, 2).reshape(-1, D)[:ctx]
            size = vs[ids, h].double().repeat_interleave(page)[:ctx]
            z = scale * (q[r0:r1, hq].double() @ K.t())
            L = (abs(scale) * (q[r0:r1, hq].double().abs() @ K.abs().t()) * seen).amax(1, keepdim=True)
            w = torch.softmax(z.masked_fill(~seen, -math.inf), 1).nan_to_num(0)       # rows that see nothing
            y, A = w @ (code * size[:, None]), w @ (code.abs() * size[:, None])
            # scores as in attention_reference; exponents: eight roundings at the size of scores and logarithms of
            # scales, in base 2; weights as float16 (two parts): 2^-11 (2^-21), and half of a subnormal's step, 2^-25,
            # where the row's largest weight x scale stands at 2^12 or above
            dz = (D + 24) * 2.0 ** -24 * L + (0 if bf else 2.0 ** -21) * L + 2.0 ** -20
            far = (L / math.log(2) + size.log2().abs().max() + 16) * 8 * math.log(2) * 2.0 ** -24
            rel = (2.0 ** -11 if bf else 2.0 ** -21) + 2 * dz + far + (ctx / 8 + 64) * 2.0 ** -24
            lost = 2.0 ** -37 * (w * size).amax(1, keepdim=True) * (seen.double() @ code.abs())
            out[r0:r1, hq] = y
            tol[r0:r1, hq] = HALF[q.dtype] * y.abs() + rel * A + lost + 1e-36
    return out, tol


def inputs(sizes, new, G, Hk, D, page, kind, dtype, seed, lean):
    """One sequence of a page for each of `sizes`, its value scale; lean: what the page's scores stand above 0."""
    g = gen(seed)
    pages = len(sizes)
    top = 100 if kind is INT8 else 240
    kc = torch.randint(-10, 11, (pages, Hk, page, D), generator=g).float()
    kc[..., 0] = 100
    ks = torch.tensor(lean)[:, None].expand(pages, Hk) / 100
    ks = torch.where(ks.abs() < 0.001, 0.001, ks)            # the sign goes with the codes
    kc[..., 0] *= torch.sign(ks)[..., None]
    vc = torch.randint(-top, top + 1, (pages, Hk, D, page), generator=g).float()
    q = (torch.randn(new, G * Hk, D, generator=g) * 0.02).to(dtype)
    q[..., 0] = 1
    vs = torch.tensor(sizes, dtype=torch.float32)[:, None].expand(pages, Hk).contiguous()
    return q, kc.to(kind), vc.to(kind), ks.abs().float().contiguous(), vs, torch.arange(pages).int()[None]


def check(kda, x, context, new, what):  # noqa: F811
    q, kc, vc, ks, vs, table = x
    context, starts = torch.tensor([context]).int(), torch.tensor([0, new]).int()
    want, tol = exact(q, kc, vc, ks, vs, table, context, starts, 1.0)
    o = kda.kda_cache_attention(*[t.cuda() for t in (q, kc, vc, ks, vs, table, context)], q_start=starts.cuda(), max_queries=new,
                                scale=1.0)
    close(o, want, tol, what)


KERNELS = [  # rows, G, Hk, D, dtype: few rows, blocks of 16, lines and blocks of 64 and 128 rows
    (1, 4, 2, 64, BF16), (9, 1, 1, 128, F32), (50, 1, 2, 64, BF16), (60, 2, 40, 64, F32), (33, 1, 2, 256, F32),
    (200, 2, 1, 128, BF16), (150, 2, 1, 64, F32), (90, 2, 1, 256, BF16)]


@pytest.mark.parametrize("rows,G,Hk,D,dtype", KERNELS)
@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_pages_without_weight(kda, rows, G, Hk, D, dtype, kind):  # noqa: F811
    """A page of large values, far below in its scores, among pages of small ones: first, in the middle, last."""
    for power in (-20, -33, -45, -60, -90):
        for at in (0, 2, 11):
            sizes, lean = [2.0 ** power] * 16, [2.0] * 16
            sizes[at], lean[at] = 1.0, -120.0
            check(kda, inputs(sizes, rows, G, Hk, D, 32, kind, dtype, 40 + at, lean), 16 * 32 - 5, rows, f"2^{power} at {at}")


@pytest.mark.parametrize("rows,G,Hk,D,dtype", KERNELS)
@pytest.mark.parametrize("step", [20, -20, 9])
def test_pages_that_later_rows_see(kda, rows, G, Hk, D, dtype, step):  # noqa: F811
    """Values that grow (or shrink) by 2^step a page of 16 tokens: a row before the step does not see it, though the
    tile and the block that it is worked on in hold both.  All rows are the sequence's own, from its first token."""
    pages = max(1, -(-rows // 16))
    half = pages // 2
    sizes = [2.0 ** max(-100, min(90, step * (p - half))) for p in range(pages)]
    check(kda, inputs(sizes, rows, G, Hk, D, 16, INT8, dtype, 41, [1.0] * pages), rows, rows, f"step {step}")


@pytest.mark.parametrize("rows,G,Hk,D,dtype", KERNELS)
def test_large_values_tiles_later(kda, rows, G, Hk, D, dtype):  # noqa: F811
    """The last rows see one page of large values, several tiles behind the first rows' places."""
    pages = 6 + -(-rows // 64)
    sizes = [2.0 ** -50] * (pages - 1) + [8.0]
    check(kda, inputs(sizes, rows, G, Hk, D, 64, E4M3, dtype, 42, [1.0] * pages), 64 * pages - 20, rows, "later")


@pytest.mark.parametrize("rows,G,Hk,D,dtype", KERNELS)
def test_weights_that_balance_scales(kda, rows, G, Hk, D, dtype):  # noqa: F811
    """Pages whose weights fall as their values grow: each adds about as much."""
    pages = 12
    lean = [-6.0 * p for p in range(pages)]
    sizes = [math.exp(6.0 * p - 30) for p in range(pages)]
    check(kda, inputs(sizes, rows, G, Hk, D, 16, INT8, dtype, 43, lean), 16 * pages, rows, "balance")
