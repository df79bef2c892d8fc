"""GPU: the example's frequency table is stretched, and the factor that goes with the table is
on queries and keys alike, in serving and in training."""
import importlib.util
import os

import numpy as np
import pytest

from attend_oracle import attend as oracle_attend
from attend_oracle import check

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import exact_top_token_gb300 as hk

    hk.build()
    spec = importlib.util.spec_from_file_location("sparse_attention",
                                                  os.path.join(ROOT, "examples", "sparse_attention.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rotated(layer, x, pos, sign=1):
    """The rotation of the first half of each row by the layer's table and factor, in 64 bits."""
    f = layer.freq.cpu().numpy().astype(np.float64)
    a = np.asarray(pos, dtype=np.float64)[:, None] * f[None] * sign
    c, s = np.cos(a)[:, None] * layer.mscale, np.sin(a)[:, None] * layer.mscale
    y, h = np.array(x, dtype=np.float64), len(f)
    x1, x2 = y[..., :h].copy(), y[..., h:2 * h].copy()
    y[..., :h], y[..., h:2 * h] = x1 * c - x2 * s, x1 * s + x2 * c
    return y


def values(t):
    return t.float().cpu().numpy().astype(np.float64)


def test_cached_keys_carry_the_factor(example):
    import exact_top_token_gb300 as hk

    layer = example.Layer(300, 64, heads=8, cache_heads=2, index_heads=4)
    assert layer.mscale > 1.1
    state = layer.gen.get_state()
    pos = layer.append(300).cpu().numpy()
    layer.gen.set_state(state)
    for cache, heads in ((layer.index_keys, 1), (layer.keys, 2)):
        want = rotated(layer, values(layer._rows(300, heads)), pos)
        got = values(hk.cache_read(cache.codes, cache.scale))
        # the nearest code, 1 / 16 of a value or half the smallest step, and a bf16 rounding
        step = values(cache.scale)[..., None] * 2.0 ** -10
        assert np.all(np.abs(got - want) <= np.maximum(np.abs(want) / 16, step) * 1.01 +
                      np.abs(want) * 2.0 ** -8)


def test_training_step_against_the_formulas(example):
    import torch

    import exact_top_token_gb300 as hk

    layer = example.Layer(260, 48, heads=8, cache_heads=2, index_heads=4)
    layer.append(240)
    positions = layer.append(20)
    _, _, idx = layer.forward(positions)
    state = layer.gen.get_state()
    got = [values(t) for t in layer.train_step(positions, idx)]
    layer.gen.set_state(state)
    n, L = 20, 260
    x_q, x_k, v, grad = layer._rows(n, 8), layer._rows(L, 2), layer._rows(L, 2), layer._rows(n, 8)
    pos, rows = positions.cpu().numpy(), np.arange(L)
    at = torch.arange(L, dtype=torch.int32, device="cuda")
    # (rounded to bf16 as the layer's are)
    q = hk.rope(x_q, positions, layer.freq, mscale=layer.mscale)
    k = hk.rope(x_k, at, layer.freq, mscale=layer.mscale)
    for t, x, p in ((q, x_q, pos), (k, x_k, rows)):
        want = rotated(layer, values(x), p)
        assert np.all(np.abs(values(t) - want) <= np.abs(want) * 2.0 ** -8 + 1e-5)
    r = oracle_attend(values(q), values(k), values(v), idx.cpu().numpy(), 128 ** -0.5, 24, values(grad))
    check("out", got[0], r["out"], r["tol_out"])
    check("dv", got[3], r["dv"], r["tol_dv"])
    for name, x, p in (("dq", got[1], pos), ("dk", got[2], rows)):
        # through the rotation: a pair's bounds add up, and 18 ulp of its magnitude
        tol, h = r["tol_" + name] + 18 * 2.0 ** -24 * np.abs(r[name]), 32
        pair = tol[..., :h] + tol[..., h:2 * h]
        tol = np.concatenate([layer.mscale * pair, layer.mscale * pair, tol[..., 2 * h:]], -1)
        check(name, x, rotated(layer, r[name], p, sign=-1), tol)
