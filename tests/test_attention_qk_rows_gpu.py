"""Query and key norm: rows of no token without a rotation."""

import math

import pytest
import torch

import attention_reference as ref
from test_attention_gpu import BF16, F32, close, cpu, gen, kda, qk_inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D,eps", [(BF16, 128, 1e-6), (F32, 64, 0.0), (F32, 6, 1e-6), (BF16, 90, 0.0)])
@pytest.mark.parametrize("table", [False, True])
def test_rows_of_no_token_without_rotation(kda, dtype, D, eps, table):  # noqa: F811
    """Negative positions mark them, whether there is no table or one that turns no channel; the others may be any."""
    T, Hq, Hk = 21, 3, 2
    q, k, wq, wk, _, _ = qk_inputs(T, Hq, Hk, D, 0, dtype, False, D)
    g = gen(D)
    dq, dk = (torch.randn(t.shape, generator=g).to(dtype).cuda() for t in (q, k))
    pos = torch.randint(0, 2 ** 31 - 1, (T,), generator=g).int()
    pos[4:9], pos[20] = -1, -2 ** 31
    gone = (pos < 0).cuda()
    for t in (q, k, dq, dk):
        t[gone] = math.nan
    kw = dict(positions=pos.cuda(), rotary=torch.empty((3, 0), device="cuda") if table else None)
    y = kda.kda_qk_norm_rope_fwd(q, k, wq, wk, eps, **kw)
    r = kda.kda_qk_norm_rope_bwd(dq, dk, q, k, wq, wk, eps, **kw)
    keep = ~gone
    for i, (n, x, w, dy) in enumerate((("q", q, wq, dq), ("k", k, wk, dk))):
        assert not y[i][gone].any() and not r["d" + n][gone].any()
        x, dy = x[keep], dy[keep]
        want, tol = ref.qk_fwd(*cpu(x, w), eps, None, None, False)
        close(y[i][keep], want, tol, n)
        dx, tol, dw, wtol = ref.qk_bwd(*cpu(dy, x, w), eps, None, None, False)
        close(r["d" + n][keep], dx, tol, "d" + n)
        close(r[f"d{n}_weight"], dw, wtol, f"d{n}_weight")


def test_a_table_needs_positions(kda):  # noqa: F811
    q, k, _, _, _, table = qk_inputs(5, 2, 1, 64, 64, F32, False, 1)
    with pytest.raises(ValueError):
        kda.kda_qk_norm_rope_fwd(q, k, rotary=table)


@pytest.mark.parametrize("T,D,R,dtype", [(2500, 90, 30, BF16), (2500, 90, 90, F32), (2500, 250, 250, F32)])
def test_gradients_by_elements_over_many_workgroups(kda, T, D, R, dtype):  # noqa: F811
    """Rows whose channels fit no wider access, in more workgroups than such rows had."""
    q, k, wq, wk, pos, table = qk_inputs(T, 6, 2, D, R, dtype, False, D)
    pos = pos % (3 * T)                                       # none beyond the table: the weights' sums stay finite
    g = gen(T)
    dq, dk = (torch.randn(t.shape, generator=g).to(dtype).cuda() for t in (q, k))
    r = kda.kda_qk_norm_rope_bwd(dq, dk, q, k, wq, wk, 1e-6, positions=pos, rotary=table)
    for n, x, w, dy in (("q", q, wq, dq), ("k", k, wk, dk)):
        dx, tol, dw, wtol = ref.qk_bwd(*cpu(dy, x, w), 1e-6, *cpu(pos, table), False)
        close(r["d" + n], dx, tol, "d" + n)
        close(r[f"d{n}_weight"], dw, wtol, f"d{n}_weight")
