"""GPU: attention over selected rows where scores are not ordinary, against the 64-bit
formulas of attend_oracle.py."""
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


def values(t, scale=None):
    x = t.float().cpu().numpy().astype(np.float64)
    return x if scale is None else x * scale.cpu().numpy().astype(np.float64)[..., None]


@pytest.mark.parametrize("n", [1, 200])  # items split over a cluster, and not
@pytest.mark.parametrize("cache,Hq,d,out_dtype", [
    ("bf16", 4, 64, "bfloat16"), ("bf16", 20, 128, "bfloat16"), ("bf16", 100, 128, "bfloat16"),
    ("bf16", 20, 256, "bfloat16"), ("bf16", 4, 128, "float32"), ("bf16", 20, 64, "float32"),
    ("e4m3", 4, 64, "bfloat16"), ("e4m3", 20, 128, "bfloat16"), ("e4m3", 20, 128, "float32")])
@pytest.mark.parametrize("where", ["first tile", "first tiles", "last tiles", "scattered", "all"])
def test_scores_of_minus_infinity(hk, dev, where, cache, Hq, d, out_dtype, n):
    """Rows whose score is -inf weigh nothing, wherever they stand in the list; where all
    are, the result is that of no row."""
    import torch

    k = L = 900
    g = torch.Generator(device=dev).manual_seed(d + Hq)
    q = torch.randn(n, Hq, d, device=dev, generator=g).abs().bfloat16()  # (so that no score is +inf)
    kk, vv = (torch.randn(L, 1, d, device=dev, generator=g) for _ in range(2))
    low = torch.zeros(L, dtype=torch.bool, device=dev)
    if where == "first tile":
        low[:128] = True
    elif where == "first tiles":
        low[:500] = True
    elif where == "last tiles":
        low[500:] = True
    elif where == "scattered":
        low[::3] = True
    else:
        low[:] = True
    kw = {}
    if cache == "bf16":
        kk, vv = kk.bfloat16(), vv.bfloat16()
        kk[low, :, 0] = -float("inf")
    else:
        kk[low] = -kk[low].abs() - 0.1
        kk, vv = (kk * 16).to(torch.float8_e4m3fn), (vv * 16).to(torch.float8_e4m3fn)
        kw = dict(k_scale=torch.full((L, 1), 0.0625, device=dev),
                  v_scale=torch.full((L, 1), 0.0625, device=dev))
        kw["k_scale"][low] = float("inf")
    idx = torch.arange(L, device=dev, dtype=torch.int32).expand(n, k).contiguous()
    idx[:, 7::31] = -1
    dt = getattr(torch, out_dtype)
    out, lse = hk.attend(q, kk, vv, idx, out_dtype=dt, **kw)
    # the rows of weight zero left out
    seen = torch.where(low[idx.clamp(min=0).long()], -1, idx)
    fk = values(kk.float(), None if cache == "bf16" else torch.full((L, 1), 0.0625))
    fk[low.cpu().numpy()] = 0.0
    sample = torch.arange(0, n, 67, device=dev)
    r = oracle_attend(values(q[sample]), fk, values(vv, kw.get("v_scale")), seen[sample].cpu().numpy(),
                      d ** -0.5, 8 if dt == torch.bfloat16 else 24)
    check("out", out[sample].float().cpu().numpy(), r["out"], r["tol_out"])
    check("lse", lse[sample].cpu().numpy(), r["lse"], r["tol_lse"])
    if where == "all":
        assert bool((out == 0).all()) and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("n", [1, 200])
@pytest.mark.parametrize("Hq,d,out_dtype", [(4, 64, "bfloat16"), (20, 128, "bfloat16"),
                                            (100, 128, "bfloat16"), (20, 128, "float32")])
@pytest.mark.parametrize("rows", [(0, 1), (5, 6), (0, 128), (400, 401), (384, 512), (0, 900)])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_a_selected_row_that_is_not_a_number_shows(hk, dev, what, rows, Hq, d, out_dtype, n):
    """A score of NaN or +inf makes its head's result and log-sum-exp NaN, wherever it stands."""
    import torch

    k = L = 900
    g = torch.Generator(device=dev).manual_seed(d + Hq)
    q = torch.randn(n, Hq, d, device=dev, generator=g).abs().bfloat16()
    kk, vv = (torch.randn(L, 1, d, device=dev, generator=g).bfloat16() for _ in range(2))
    kk[rows[0]:rows[1], :, 0] = float(what)
    idx = torch.arange(L, device=dev, dtype=torch.int32).expand(n, k).contiguous()
    out, lse = hk.attend(q, kk, vv, idx, out_dtype=getattr(torch, out_dtype))
    assert bool(torch.isnan(out.float()).all())
    assert not bool(torch.isfinite(lse).any())
    if what == "nan":
        assert bool(torch.isnan(lse).all())
