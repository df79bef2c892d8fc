"""GPU: gradients of the attention over selected rows where keys are not finite."""
import numpy as np
import pytest

from attend_oracle import attend as oracle_attend
from attend_oracle import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hk():
    import exact_top_token_gb300 as hk

    hk.build()
    hk.load()
    return hk


def values(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("n", [2, 200])  # a query's rows split over CTAs, and not
@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 64), (8, 2, 64), (16, 1, 128), (20, 1, 128), (64, 1, 64),
                                      (100, 1, 128)])
def test_gradients_of_rows_with_scores_of_minus_infinity(hk, Hq, Hkv, d, n):
    """Keys of -inf in one column make scores of -inf: the row's weight is 0, its dk and dv are 0
    and the other rows' are as without it. (dq of that column alone is 0 times infinity.)"""
    import torch

    k, L = 300, 400
    g = torch.Generator(device="cuda").manual_seed(Hq)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g).bfloat16()

    q, kk, vv, grad = normal(n, Hq, d), normal(L, Hkv, d), normal(L, Hkv, d), normal(n, Hq, d)
    q[..., 0] = 1.0
    low = torch.rand(L, device="cuda", generator=g) < 0.3
    kk[low, :, 0] = -float("inf")
    idx = torch.rand(n, L, device="cuda", generator=g).argsort(1)[:, :k].int().contiguous()
    idx[:, 5::19] = -1
    idx[0] = torch.where(low[idx[0].clamp(min=0).long()], idx[0], -1)  # no other row
    keep = torch.arange(0, n, 41, device="cuda")
    other = torch.ones(n, dtype=torch.bool, device="cuda")
    other[keep] = False
    grad[other] = 0
    out, lse = hk.attend(q, kk, vv, idx, out_dtype=torch.float32)
    dq, dk, dv = hk.attend_backward(q, kk, vv, idx, out, lse, grad)
    seen = torch.where(low[idx.clamp(min=0).long()], -1, idx)
    finite = kk.clone()
    finite[low, :, 0] = 0
    r = oracle_attend(values(q[keep]), values(finite), values(vv), seen[keep].cpu().numpy(), d ** -0.5, 24,
                      values(grad[keep]))
    check("dk", dk.cpu().numpy(), r["dk"], r["tol_dk"])
    check("dv", dv.cpu().numpy(), r["dv"], r["tol_dv"])
    check("dq", dq[keep][..., 1:].cpu().numpy(), r["dq"][..., 1:], r["tol_dq"][..., 1:])
