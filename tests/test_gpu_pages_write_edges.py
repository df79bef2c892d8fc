"""Rows written into pages (GPU) at the edges of what the entry point takes, against the definition
in 64 bits."""
import numpy as np
import pytest
import torch

import exact_top_token_gb300 as hk
from test_gpu_pages_write import Case, cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    hk.build()


@pytest.mark.parametrize("B", [1, 256, 257, 600])
@pytest.mark.parametrize("H", [1, 20])
def test_every_sequence_is_reported_on(B, H):
    """A length or an offset out of range in the last of many sequences, which may have no row."""
    c = Case([(20, 1)] * B, H=H, d=64, P=16, seed=B)
    c.run()
    for last, lengths in ((B, c.lengths[:-1] + [33]), (B, c.lengths[:-1] + [-1]), (B + 3, c.lengths),
                          (B - 2, c.lengths), (B - 1, c.lengths[:-1] + [33])):
        pages = cuda(c.codes, torch.uint8).view(torch.float8_e4m3fn)
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        hk.page_write(c.x.cuda(), pages, cuda(c.scale, torch.float32), cuda(c.table), cuda(lengths),
                      cuda(list(range(B)) + [last]), status=word)
        assert word.item() == hk.DEV_BAD_POSITION, (last, lengths[-1])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,P", [(64, 16), (64, 128), (64, 256), (128, 64), (128, 128), (128, 256),
                                 (256, 16), (256, 32), (256, 64), (256, 256)])
def test_rotation_of_pages_of_any_size(d, P, dtype, interleaved):
    """Pages whose rows stay in a block's registers, and larger ones, whose angles are made a part
    of the rows after the other, for every head."""
    first, rot = (0, d) if interleaved else (d // 4, d // 2)
    c = Case([(3 * P + 5, 2 * P + 1), (P, P), (2 * P - 1, 3), (1, 1)], H=3, d=d, P=P, seed=P + d, dtype=dtype)
    freq, _ = hk.rope_frequencies(rot)
    cu = c.offsets()
    pos = np.concatenate([np.arange(l - (cu[b + 1] - cu[b]), l) for b, l in enumerate(c.lengths)])
    for given in (False, True):
        kw = dict(inv_freq=freq, first=first, interleaved=interleaved)
        if given:
            pos = np.random.default_rng(2).integers(0, 1 << 20, len(pos))
            kw["positions"] = cuda(pos)
        x = c.x.double().numpy()
        a = pos[:, None, None] * freq.double().cpu().numpy()
        i = np.arange(rot // 2)
        p, q = (first + 2 * i, first + 2 * i + 1) if interleaved else (first + i, first + i + rot // 2)
        y = x.copy()
        y[..., p] = x[..., p] * np.cos(a) - x[..., q] * np.sin(a)
        y[..., q] = x[..., p] * np.sin(a) + x[..., q] * np.cos(a)
        # cos and sin are off by 1.3 x 2^-24, and three roundings of fp32
        c.run(y, tol_y=6 * 2.0 ** -24 * 2 * np.abs(x).max(), **kw)
