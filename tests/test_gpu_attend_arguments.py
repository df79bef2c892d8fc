"""GPU: arguments of the attention over selected rows and of its gradients that the plain calls
leave at their defaults: scales, strides, repeated rows, a bf16 result."""
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


@pytest.fixture(scope="module")
def dev():
    import torch

    return torch.device("cuda", 0)


def values(t):
    return t.float().cpu().numpy().astype(np.float64)


def make(torch, dev, n, Hq, Hkv, d, k, L, seed):
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=g).bfloat16()

    idx = torch.rand(n, L, device=dev, generator=g).argsort(1)[:, :k].int().contiguous()
    idx[:, 3::17] = -1
    return normal(n, Hq, d), normal(L, Hkv, d), normal(L, Hkv, d), idx, normal(n, Hq, d)


def verify(hk, torch, q, k, v, idx, grad, scale):
    """Forward and gradients at a scale of either sign: -scale is scale of -q."""
    out, lse = hk.attend(q, k, v, idx, out_dtype=torch.float32, scale=scale)
    got = (out, lse) + hk.attend_backward(q, k, v, idx, out, lse, grad, scale=scale)
    sign = -1.0 if scale < 0 else 1.0
    r = oracle_attend(sign * values(q), values(k), values(v), idx.cpu().numpy(), abs(scale), 24,
                      values(grad))
    r["dq"] = sign * r["dq"]
    for name, x in zip(("out", "lse", "dq", "dk", "dv"), got):
        check(name, x.cpu().numpy(), r[name], r["tol_" + name])


@pytest.mark.parametrize("scale", [-0.3, 0.3, -0.02])
@pytest.mark.parametrize("n,Hq,Hkv,d,k", [(1, 8, 2, 64, 70), (6, 20, 1, 128, 300), (90, 40, 2, 64, 150)])
def test_scales_of_either_sign(hk, dev, n, Hq, Hkv, d, k, scale):
    import torch

    verify(hk, torch, *make(torch, dev, n, Hq, Hkv, d, k, 400, n + k), scale)


@pytest.mark.parametrize("Hq,Hkv,d", [(16, 4, 64), (20, 1, 128)])
@pytest.mark.parametrize("n", [3, 200])
def test_gradients_of_strided_queries_and_interleaved_rows(hk, dev, n, Hq, Hkv, d):
    """q inside a wider projection; k and v rows of one [L, 2, Hkv, d] tensor."""
    import torch

    q, k, v, idx, grad = make(torch, dev, n, Hq + 8, Hkv, d, 90, 300, 7)
    kv = torch.stack([k, v], 1)
    verify(hk, torch, q[:, 4:4 + Hq], kv[:, 0], kv[:, 1], idx, grad[:, :Hq].contiguous(), d ** -0.5)


def test_gradients_of_repeated_rows_add_up(hk, dev):
    import torch

    q, k, v, idx, grad = make(torch, dev, 5, 12, 2, 64, 150, 200, 9)
    idx[:, 75:150] = idx[:, :75]
    idx[1] = 7                      # one row alone, many times
    idx[2, ::2] = 11
    verify(hk, torch, q, k, v, idx, grad, 64 ** -0.5)


def test_key_gradients_from_a_bf16_result(hk, dev):
    """out in bf16 changes a row's ds by p times at most 2^-8 |grad| . |out|, and dk by the sum
    of that times |q|."""
    import torch

    n, Hq, d, L = 5, 24, 128, 300
    q, k, v, idx, grad = make(torch, dev, n, Hq, 1, d, 100, L, 53)
    out, lse = hk.attend(q, k, v, idx, out_dtype=torch.float32)
    full = hk.attend_backward(q, k, v, idx, out, lse, grad)
    half = hk.attend_backward(q, k, v, idx, out.bfloat16(), lse, grad)
    scale = d ** -0.5
    s = torch.einsum("thd,ld->thl", q.double(), k[:, 0].double()) * scale
    seen = torch.zeros(n, L + 1, dtype=torch.bool, device=dev)
    seen.scatter_(1, torch.where(idx < 0, L, idx).long(), True)
    p = torch.softmax(s.masked_fill(~seen[:, None, :L], -float("inf")), -1)
    shift = 2.0 ** -8 * (grad.double().abs() * out.double().abs()).sum(-1)
    most = scale * torch.einsum("thl,th,thd->ld", p, shift, q.double().abs())
    moved = (full[1] - half[1])[:, 0].double().abs()
    assert bool((moved <= most * (1 + 1e-4) + 1e-5).all())
    assert float(moved.max()) > 1e-4  # (the row sum is used)
