"""GPU: rotary angles at every position, and positions of rows that are not written."""
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


@pytest.mark.parametrize("d", [64, 128, 256, 48])  # rows in lanes, and a warp a row
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_of_rows_not_written_do_not_matter(hk, dev, d, cache, interleaved):
    """A padded batch (slot -1, position -1) reports nothing; a slot out of range reports the
    slot alone; the rows written and the report are the same for every width."""
    import torch

    n, H, L = 37, 2, 60
    g = torch.Generator(device=dev).manual_seed(d)
    x = torch.randn(n, H, d, device=dev, generator=g).bfloat16()
    pos = torch.randint(0, 5000, (n,), device=dev, generator=g, dtype=torch.int32)
    slots = torch.randperm(L, device=dev, generator=g)[:n].int()
    freq, _ = hk.rope_frequencies(32, device=dev)

    def write(slots, pos):
        if cache == "e4m3":
            codes = torch.zeros(L, H, d, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
            scale = torch.full((L, H), 3.0, device=dev)
        else:
            codes, scale = torch.zeros(L, H, d, device=dev, dtype=torch.bfloat16), None
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        hk.cache_write(x, codes, scale, slots=slots, positions=pos, inv_freq=freq,
                       interleaved=interleaved, status=st)
        return codes.view(torch.uint8), scale, int(st.item())

    skipped = torch.zeros(n, dtype=torch.bool, device=dev)
    skipped[[0, 5, 6, 20, n - 1]] = True
    slots[skipped] = -1
    want = write(slots, pos)
    assert want[2] == 0
    pos[skipped] = torch.tensor([-1, 1 << 24, -7, 1 << 30, -1], dtype=torch.int32, device=dev)
    got = write(slots, pos)
    assert got[2] == 0
    assert torch.equal(got[0], want[0]) and (cache == "bf16" or torch.equal(got[1], want[1]))
    slots[5] = L                                   # no slot: reported, its position not
    assert write(slots, pos)[2] == hk.DEV_BAD_INDEX
    slots[5] = -1
    pos[1] = -1                                    # a row that is written
    nan = hk.DEV_NONFINITE if cache == "e4m3" else 0
    assert write(slots, pos)[2] == hk.DEV_BAD_POSITION | nan
