"""GPU: rotary angles at every position."""
import numpy as np
import pytest

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


@pytest.mark.parametrize("low,high", [(0, 1 << 10), (1 << 10, 1 << 19), (1 << 19, 1 << 20),
                                      (1 << 20, 1 << 21), (1 << 21, 1 << 22), (1 << 22, 1 << 24)])
@pytest.mark.parametrize("d", [64, 48])  # both row kernels
def test_angles_at_every_position(hk, dev, d, low, high):
    """cos and sin themselves, from rows of ones and zeros, with frequencies just below 1, where
    the angles are largest. Bound: the angle goes through four roundings of values below 1
    (2^-25 each), the series through about two more: 3 x 2^-24 in all."""
    import torch

    n, half = 1 << 16, 16
    g = np.random.default_rng(low + d)
    pos = g.integers(low, high, size=n).astype(np.int32)
    pos[:2] = [low, high - 1]
    freq = np.concatenate([[1.0], 1.0 - g.random(half - 1) * 0.3]).astype(np.float32)
    x = torch.zeros(n, 1, d, device=dev)
    x[..., :half] = 1.0
    y = hk.rope(x, torch.from_numpy(pos).to(dev), torch.from_numpy(freq).to(dev))
    angle = pos.astype(np.float64)[:, None] * freq.astype(np.float64)[None]
    got = y[:, 0, :2 * half].cpu().numpy().astype(np.float64)
    worst = max(np.abs(got[:, :half] - np.cos(angle)).max(), np.abs(got[:, half:] - np.sin(angle)).max())
    assert worst <= 3 * 2.0 ** -24, f"{worst:.3g}"
