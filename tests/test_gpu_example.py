"""GPU: the sparse-attention example end to end on a small context, its attention checked
against the formula on what its own caches hold."""
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


def test_prompt_tokens_and_training_step(example):
    import torch

    import exact_top_token_gb300 as hk

    layer = example.Layer(600, 64, heads=8, cache_heads=2, index_heads=4)
    layer.append(500)
    positions = layer.append(20)
    out, lse, idx = layer.forward(positions)
    # every query's rows lie before it, once each
    got = idx.cpu().numpy()
    for t, p in enumerate(positions.tolist()):
        assert got[t].max() <= p and got[t].min() >= 0 and len(set(got[t])) == 64
    # the attention on the caches' contents, with the queries drawn again from the same state
    state = example.Layer(600, 64, heads=8, cache_heads=2, index_heads=4)
    state.append(500)
    state.append(20)
    state._rows(20, 4)
    torch.rand(20, 4, device="cuda", generator=state.gen)
    q = hk.rope(state._rows(20, 8), positions, state.freq, mscale=state.mscale)
    k = hk.cache_read(layer.keys.codes, layer.keys.scale, dtype=torch.float32)
    v = hk.cache_read(layer.values.codes, layer.values.scale, dtype=torch.float32)
    r = oracle_attend(*(x.float().cpu().numpy().astype(np.float64) for x in (q, k, v)), got,
                      128 ** -0.5, 8)
    check("out", out.float().cpu().numpy(), r["out"], r["tol_out"])
    check("lse", lse.cpu().numpy(), r["lse"], r["tol_lse"])
    # one token at a time
    for _ in range(3):
        out, _, last = layer.forward(layer.append(1))
        assert out.shape == (1, 8, 128) and torch.isfinite(out.float()).all()
    for g in layer.train_step(positions, idx):
        assert torch.isfinite(g).all() and float(g.abs().max()) > 0
