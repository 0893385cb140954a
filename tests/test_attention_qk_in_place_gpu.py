"""Gradients of the query and key norm written over the forward's inputs."""

import pytest
import torch

from test_attention_gpu import BF16, F32, gen, kda, qk_inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,Hq,Hk,D,R,dtype", [(37, 4, 2, 128, 64, BF16), (5000, 9, 3, 64, 64, F32), (300, 3, 2, 90, 30, BF16),
                                               (1, 32, 8, 128, 128, F32)])
def test_gradients_over_their_inputs(kda, T, Hq, Hk, D, R, dtype):  # noqa: F811
    q, k, wq, wk, pos, table = qk_inputs(T, Hq, Hk, D, R, dtype, True, 7)
    g = gen(8)
    dq, dk = (torch.randn(t.shape, generator=g).to(dtype).cuda() for t in (q, k))
    kw = dict(positions=pos, rotary=table)
    want = kda.kda_qk_norm_rope_bwd(dq, dk, q, k, wq, wk, **kw)
    around = q._base.clone()
    r = kda.kda_qk_norm_rope_bwd(dq, dk, q, k, wq, wk, dq=q, dk=k, **kw)
    assert r["dq"] is q and r["dk"] is k
    for n in want:
        assert torch.equal(torch.nan_to_num(r[n].float()), torch.nan_to_num(want[n].float())), n
    v0 = 8 + (Hq + Hk) * D
    assert torch.equal(q._base[:, :8], around[:, :8]) and torch.equal(q._base[:, v0:], around[:, v0:])
