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
