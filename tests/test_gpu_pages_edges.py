"""Attention over a cache in pages (GPU) at the edges of what its entry point takes, against the
formula in 64 bits with the bounds of tests/pages_oracle.py: contexts that begin with rows that
are not there, both kernels."""
import numpy as np
import pytest
import torch

import exact_top_token_gb300 as hk
from test_gpu_pages_attend import Case as AnyCase
from test_gpu_pages_attend import cuda
from test_gpu_pages_tokens import Case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    hk.build()


@pytest.mark.parametrize("d,P", [(64, 16), (64, 128), (128, 16), (128, 128)])
@pytest.mark.parametrize("gone", [128, 256, 384])
def test_contexts_whose_first_rows_are_not_there(gone, d, P):
    """Whole tiles of entries of -1 in front, and one in the middle: what follows them counts. So
    many contexts that a multiprocessor has several tiles of each."""
    g = np.random.default_rng(gone + P)
    lengths = [400, 9000, 385] + g.integers(500, 1000, 180).tolist()
    c = Case([(x, 1) for x in lengths], Hq=8, Hkv=2, d=d, P=P, seed=gone + P, single=True)
    c.table[1:, :gone // P] = -1
    c.table[0, 128 // P:256 // P] = -1
    out, lse = check(c)
    assert torch.isfinite(lse).all() and (out != 0).any(-1).all()
    e = AnyCase([(700, 40), (900, 1), (385, 385)], Hq=8, Hkv=2, d=d, P=P, seed=gone + P)
    e.table[:, :gone // P] = -1
    e.run()


@pytest.mark.parametrize("d", [64, 128])
def test_heads_whose_first_scores_are_minus_infinity(d):
    """Of heads on one cache head some have no score above -inf in the first two tiles, the
    others do."""
    g = np.random.default_rng(d)
    lengths = [2000] + g.integers(300, 900, 300).tolist()
    c = Case([(x, 1) for x in lengths], Hq=6, Hkv=1, d=d, P=16, seed=d, single=True)
    c.k &= 0x7F                                    # codes >= 0
    c.k[c.k == 0x7F] = 1
    c.k[:, :, :, 0] = 0x38
    c.q = (c.q.abs() * 2.0 ** -64).bfloat16()
    c.q[:, ::2] = -(2.0 ** 126)
    c.ks[:] = 2.0 ** -120
    c.ks[c.table[:, :16]] = 2.0 ** 60
    out, lse = check(c)
    assert torch.isfinite(lse).all() and (out[:, ::2] != 0).any(-1).all()
