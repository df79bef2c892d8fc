"""GPU: rotary positions and cache rows (written, quantised, read back) against
64-bit formulas, through the public entry points."""
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


def rope64(x, pos, freq, first, interleaved, mscale, inverse):
    """The rotation in 64 bits, and |x1| + |x2| of each element's pair (0 outside)."""
    r = 2 * len(freq)
    a = pos.astype(np.float64)[:, None] * freq.astype(np.float64)[None]
    c, s = np.cos(a)[:, None] * mscale, np.sin(a)[:, None] * mscale * (-1 if inverse else 1)
    i = np.arange(r // 2)
    j1, j2 = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    j1, j2 = j1 + first, j2 + first
    x = x.astype(np.float64)
    y, m = x.copy(), np.zeros_like(x)
    y[..., j1] = x[..., j1] * c - x[..., j2] * s
    y[..., j2] = x[..., j1] * s + x[..., j2] * c
    m[..., j1] = m[..., j2] = np.abs(x[..., j1]) + np.abs(x[..., j2])
    return y, m


def tolerance(y, m, mscale, bf16):
    """Angle (2^-22: its reduction and the rounding of hi + lo), cos / sin and their factor
    (2 ulp each), two products and a sum: 12 ulp of fp32 of the pair's magnitude, then the
    result's own rounding."""
    return 12 * 2.0 ** -24 * mscale * m * 1.5 + (2.0 ** -8 if bf16 else 2.0 ** -23) * np.abs(y)


def inputs(torch, dev, n, H, d, rot, dtype, top, seed=0):
    g = np.random.default_rng(seed)
    x = torch.from_numpy(g.standard_normal((n, H, d), dtype=np.float32)).to(dev).to(dtype)
    pos = g.integers(0, top, size=n).astype(np.int32)
    pos[: min(n, 3)] = [0, top - 1, 1][: min(n, 3)]
    return x, torch.from_numpy(pos).to(dev)


ROPE = [
    # n, H, d, rot, first, top
    (1, 1, 64, 64, 0, 10),
    (5, 3, 128, 64, 64, 1 << 20),
    (33, 64, 128, 128, 0, 1 << 20),
    (7, 8, 256, 64, 0, 1 << 24),
    (129, 2, 24, 16, 8, 5000),
    (3, 5, 1024, 48, 320, 100000),
    (1000, 1, 128, 32, 40, 1 << 17),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n,H,d,rot,first,top", ROPE)
def test_rope(hk, dev, n, H, d, rot, first, top, dtype, interleaved):
    import torch

    dt = getattr(torch, dtype)
    x, pos = inputs(torch, dev, n, H, d, rot, dt, top, seed=n)
    freq, _ = hk.rope_frequencies(rot, 50000.0, device=dev)
    for inverse in (False, True):
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        y = hk.rope(x, pos, freq, first=first, interleaved=interleaved, mscale=1.25,
                    inverse=inverse, status=st)
        want, m = rope64(x.float().cpu().numpy(), pos.cpu().numpy(), freq.cpu().numpy(), first,
                         interleaved, 1.25, inverse)
        err = np.abs(y.float().cpu().numpy() - want)
        assert np.all(err <= tolerance(want, m, 1.25, dt == torch.bfloat16))
        outside = np.ones(d, bool)
        outside[first:first + rot] = False
        outside = torch.from_numpy(outside).to(dev)
        assert torch.equal(y[..., outside], x[..., outside])  # copied, not scaled
        assert int(st.item()) == 0


def test_rope_gradient_is_the_inverse(hk, dev):
    """<rope(x), g> = <x, rope(g, inverse)>, and the inverse undoes the rotation."""
    import torch

    x, pos = inputs(torch, dev, 50, 4, 128, 64, torch.float32, 1 << 20, seed=2)
    g, _ = inputs(torch, dev, 50, 4, 128, 64, torch.float32, 1 << 20, seed=3)
    freq, m = hk.rope_frequencies(64, scaling="parts", factor=8.0, original_context=4096, device=dev)
    y = hk.rope(x, pos, freq, first=32, mscale=m)
    b = hk.rope(g, pos, freq, first=32, mscale=m, inverse=True)
    left, right = (y.double() * g).sum(), (x.double() * b).sum()
    scale = (y.double() * g).abs().sum()
    assert abs(left - right) <= 1e-6 * scale
    back = hk.rope(hk.rope(x, pos, freq), pos, freq, inverse=True)
    # two rotations of 18 ulp each
    assert (back - x).abs().max() <= 2 * 18 * 2.0 ** -24 * 2 * x.abs().max()


def test_rope_strides_in_place_and_streams(hk, dev):
    import torch

    n, H, d = 21, 6, 64
    wide = torch.randn(n, H + 3, d, device=dev).bfloat16()
    pos = torch.arange(n, device=dev, dtype=torch.int32) * 1000
    freq, _ = hk.rope_frequencies(64, device=dev)
    view = wide[:, 1:1 + H]
    want = hk.rope(view.contiguous(), pos, freq)
    assert torch.equal(hk.rope(view, pos, freq), want)
    across = torch.randn(H, n, d, device=dev).bfloat16().transpose(0, 1)  # heads outermost
    assert torch.equal(hk.rope(across, pos, freq), hk.rope(across.contiguous(), pos, freq))
    keep = wide.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = hk.rope(view, pos, freq, out=view, stream=side)
    side.synchronize()
    assert got.data_ptr() == view.data_ptr() and torch.equal(view, want)
    assert torch.equal(wide[:, 0], keep[:, 0]) and torch.equal(wide[:, 1 + H:], keep[:, 1 + H:])
    assert hk.rope(view[:0], pos[:0], freq).shape == (0, H, d)
    two = torch.randn(n, d, device=dev)
    assert torch.equal(hk.rope(two, pos, freq), hk.rope(two[:, None], pos, freq)[:, 0])


def test_bad_positions_are_reported(hk, dev):
    import torch

    x = torch.randn(4, 2, 64, device=dev)
    freq, _ = hk.rope_frequencies(32, device=dev)
    pos = torch.tensor([5, -1, 1 << 24, (1 << 24) - 1], dtype=torch.int32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    y = hk.rope(x, pos, freq, status=st)
    assert int(st.item()) == hk.DEV_BAD_POSITION
    assert torch.isnan(y[1:3, :, :32]).all() and torch.equal(y[1:3, :, 32:], x[1:3, :, 32:])
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all()


# ---- cache rows ---------------------------------------------------------------------

def quantised(torch, x):
    """Codes and scales of fp32 rows by the definition, with numpy's IEEE divisions (torch
    multiplies by the reciprocal of a scalar divisor on the GPU)."""
    v = x.cpu().numpy()
    amax = np.abs(v).max(-1)
    scale = np.where(amax > 0, np.maximum(amax / np.float32(448), np.float32(2.0 ** -126)),
                     np.float32(1.0)).astype(np.float32)
    codes = torch.from_numpy(v / scale[..., None]).to(torch.float8_e4m3fn)
    return codes.to(x.device), torch.from_numpy(scale).to(x.device)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n,H,d,L", [(1, 1, 64, 1), (6, 1, 128, 9000), (37, 3, 256, 40),
                                     (1001, 8, 128, 1001), (5, 2, 1024, 7), (9, 2, 16, 20)])
def test_quantised_rows_bit_for_bit(hk, dev, n, H, d, L, dtype):
    import torch

    x, _ = inputs(torch, dev, n, H, d, 16, getattr(torch, dtype), 10, seed=n + d)
    x[0] = 0                              # a row of zeros
    if n > 4:
        x[1] *= 1e-30
        x[2] *= 1e30
        x[3] = torch.finfo(torch.float32).tiny / 64 if dtype == "float32" else 1e-39
        x[4, :, 1:] = 0                   # one element alone
    slots = torch.randperm(L, device=dev)[:n].int()
    codes = torch.full((L, H, d), 0x11, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scale = torch.full((L, H), 5.0, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    hk.cache_write(x, codes, scale, slots=slots, status=st)
    wc, ws = quantised(torch, x.float())
    assert int(st.item()) == 0
    assert torch.equal(scale[slots.long()], ws)
    assert torch.equal(codes.view(torch.uint8)[slots.long()], wc.view(torch.uint8))
    rest = torch.ones(L, dtype=torch.bool, device=dev)
    rest[slots.long()] = False            # no other row is touched
    assert torch.all(codes.view(torch.uint8)[rest] == 0x11) and torch.all(scale[rest] == 5.0)
    for out in (torch.bfloat16, torch.float32):
        back = hk.cache_read(codes, scale, slots=slots, dtype=out)
        assert torch.equal(back, (wc.float() * ws[..., None]).to(out))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,H,d,rot,first", [(3, 1, 128, 64, 0), (50, 4, 128, 64, 64),
                                             (300, 1, 64, 64, 0), (17, 3, 256, 48, 40)])
def test_rotated_and_quantised(hk, dev, n, H, d, rot, first, interleaved):
    """A code is the nearest one: |code scale - y| <= |y| / 16 (half a step of 3 mantissa
    bits), or half a subnormal step 2^-10 scale, past the rotation's own error."""
    import torch

    x, pos = inputs(torch, dev, n, H, d, rot, torch.bfloat16, 1 << 20, seed=n)
    freq, _ = hk.rope_frequencies(rot, device=dev)
    codes = torch.zeros(n, H, d, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scale = torch.zeros(n, H, device=dev)
    hk.cache_write(x, codes, scale, positions=pos, inv_freq=freq, first=first,
                   interleaved=interleaved, mscale=1.1)
    y, m = rope64(x.float().cpu().numpy(), pos.cpu().numpy(), freq.cpu().numpy(), first,
                  interleaved, 1.1, False)
    tol = tolerance(y, m, 1.1, False)
    s = scale.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(s * 448 - np.abs(y).max(-1)) <= tol.max(-1) + 2.0 ** -22 * 448 * s)
    got = codes.float().cpu().numpy().astype(np.float64) * s[..., None]
    assert np.all(np.abs(got - y) <= np.maximum(np.abs(y) / 16, 2.0 ** -10 * s[..., None]) * (1 + 1e-5) + 2 * tol)
    # a bf16 cache takes the same values rounded once
    plain = torch.zeros(n, H, d, device=dev, dtype=torch.bfloat16)
    hk.cache_write(x, plain, positions=pos, inv_freq=freq, first=first, interleaved=interleaved,
                   mscale=1.1)
    assert torch.equal(plain, hk.rope(x, pos, freq, first=first, interleaved=interleaved, mscale=1.1))


def test_slots_skipped_and_out_of_range(hk, dev):
    import torch

    x = torch.randn(5, 2, 64, device=dev)
    codes = torch.zeros(8, 2, 64, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scale = torch.full((8, 2), 3.0, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    slots = torch.tensor([7, -1, 0, -1, 3], dtype=torch.int32, device=dev)
    hk.cache_write(x, codes, scale, slots=slots, status=st)
    assert int(st.item()) == 0
    assert torch.equal(scale[[1, 2, 4, 5, 6]], torch.full((5, 2), 3.0, device=dev))
    slots[1] = 8
    hk.cache_write(x, codes, scale, slots=slots, status=st)
    assert int(st.item()) == hk.DEV_BAD_INDEX
    st.zero_()
    back = hk.cache_read(codes, scale, slots=torch.tensor([7, -1, 3], dtype=torch.int32, device=dev),
                         status=st)
    assert int(st.item()) == 0 and torch.all(back[1] == 0)
    back = hk.cache_read(codes, scale, slots=torch.tensor([7, -5, 8], dtype=torch.int32, device=dev),
                         status=st)
    assert int(st.item()) == hk.DEV_BAD_INDEX
    assert torch.isnan(back[1:]).all() and torch.isfinite(back[0].float()).all()
    whole = hk.cache_read(codes, scale, dtype=torch.float32)
    assert torch.equal(whole, codes.float() * scale[..., None])


def test_values_that_are_not_finite(hk, dev):
    import torch

    x = torch.randn(4, 1, 64, device=dev)
    want, ws = quantised(torch, x)
    x[1, 0, 5] = float("nan")
    x[2, 0, 6] = float("inf")
    x[3] = float("-inf")
    codes = torch.zeros(4, 1, 64, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scale = torch.zeros(4, 1, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    hk.cache_write(x, codes, scale, status=st)
    assert int(st.item()) == hk.DEV_NONFINITE
    assert torch.isfinite(scale).all() and (scale > 0).all()
    f = codes.float()
    assert torch.equal(f[0], want.float()[0]) and torch.isnan(f[1, 0, 5]) and torch.isnan(f[2, 0, 6])
    assert int(torch.isnan(f).sum()) == 2 + 64 and float(scale[3, 0]) == 1.0


def test_strided_rows_and_two_dimensions(hk, dev):
    import torch

    wide = torch.randn(12, 5, 128, device=dev).bfloat16()
    a = torch.zeros(12, 2, 128, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
    b, sa, sb = a.clone(), torch.zeros(12, 2, device=dev), torch.zeros(12, 2, device=dev)
    hk.cache_write(wide[:, 2:4], a, sa)
    hk.cache_write(wide[:, 2:4].contiguous(), b, sb)
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(sa, sb)
    c, sc = a[:, 0].contiguous().view(torch.uint8).zero_().view(torch.float8_e4m3fn), sa[:, 0].contiguous()
    hk.cache_write(wide[:, 2], c, sc)
    assert torch.equal(c.view(torch.uint8), a[:, 0].view(torch.uint8)) and torch.equal(sc, sa[:, 0])


def test_offsets_past_32_bits(hk, dev):
    import torch

    L, d = (1 << 25) + 3, 128
    cache = torch.zeros(L, 1, d, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scale = torch.ones(L, 1, device=dev)
    x = torch.randn(2, 1, d, device=dev)
    slots = torch.tensor([L - 1, L - 3], dtype=torch.int32, device=dev)
    hk.cache_write(x, cache, scale, slots=slots)
    wc, ws = quantised(torch, x)
    assert torch.equal(hk.cache_read(cache, scale, slots=slots, dtype=torch.float32),
                       wc.float() * ws[..., None])


def test_written_rows_are_what_select_takes(hk, dev):
    """Queries and keys rotated and quantised here, selected and replayed: the scores are those
    of the dequantised values."""
    import torch

    n, H, d, L, k = 16, 4, 128, 700, 64
    g = torch.Generator(device=dev).manual_seed(0)
    q, key = torch.randn(n, H, d, device=dev, generator=g), torch.randn(L, d, device=dev, generator=g)
    freq, _ = hk.rope_frequencies(64, device=dev)
    qc = torch.zeros(n, H, d, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
    kc = torch.zeros(L, d, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
    qs, ks = torch.zeros(n, H, device=dev), torch.zeros(L, device=dev)
    pos = torch.arange(L - n, L, device=dev, dtype=torch.int32)
    hk.cache_write(q, qc, qs, positions=pos, inv_freq=freq)
    hk.cache_write(key, kc, ks, positions=torch.arange(L, device=dev, dtype=torch.int32), inv_freq=freq)
    w = torch.rand(n, H, device=dev, generator=g)
    idx, sc, _ = hk.select(qc, kc, w, pos, k, q_scale=qs, k_scale=ks)
    qd, kd = hk.cache_read(qc, qs, dtype=torch.float32), hk.cache_read(kc, ks, dtype=torch.float32)
    s = (torch.relu(torch.einsum("nhd,ld->nhl", qd.double(), kd.double())) * w[..., None].double()).sum(1)
    s = s.masked_fill(torch.arange(L, device=dev)[None] > pos[:, None], -float("inf"))
    want = s.topk(k, 1).values
    assert torch.all((sc.double() - want).abs() <= 1e-3 * want.abs().clamp(min=1e-3))


def test_refusals(hk, dev):
    import torch

    x = torch.randn(4, 2, 64, device=dev)
    pos = torch.zeros(4, dtype=torch.int32, device=dev)
    freq, _ = hk.rope_frequencies(32, device=dev)
    e4 = torch.zeros(4, 2, 64, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
    sc = torch.ones(4, 2, device=dev)
    with pytest.raises(TypeError):
        hk.rope(x.half(), pos, freq)
    with pytest.raises(TypeError):
        hk.rope(x, pos.long(), freq)
    with pytest.raises(ValueError):
        hk.rope(x, pos[:2], freq)
    with pytest.raises(ValueError):
        hk.rope(x[..., ::2], pos, freq)
    with pytest.raises(ValueError):
        hk.rope(x, pos, freq, out=torch.empty(4, 2, 32, device=dev))
    with pytest.raises(ValueError):
        hk.rope(x.cpu(), pos, freq)
    for first, f, status in ((40, freq, 1), (4, freq, 2), (-8, freq, 1), (0, freq[:5].contiguous(), 2)):
        with pytest.raises(hk.HytopkError) as e:
            hk.rope(x, pos, f, first=first)
        assert e.value.status == status
    with pytest.raises(hk.HytopkError) as e:
        hk.rope(torch.randn(4, 2, 68, device=dev)[..., 2:66], pos, freq)
    assert e.value.status == 5
    with pytest.raises(ValueError):
        hk.cache_write(x, e4)                        # scales missing
    with pytest.raises(ValueError):
        hk.cache_write(x, x.bfloat16(), sc)          # scales of a bf16 cache
    with pytest.raises(TypeError):
        hk.cache_write(x, x.clone())
    with pytest.raises(ValueError):
        hk.cache_write(x[:, :1], e4, sc)
    with pytest.raises(ValueError):
        hk.cache_write(x, e4, sc, positions=pos)
    with pytest.raises(TypeError):
        hk.cache_write(x, e4, sc, slots=pos.long())
    with pytest.raises(hk.HytopkError) as e:
        hk.cache_write(torch.randn(5, 2, 64, device=dev), e4, sc)  # more rows than the cache
    assert e.value.status == 1
    with pytest.raises(TypeError):
        hk.cache_read(e4, sc, dtype=torch.float16)
    with pytest.raises(ValueError):
        hk.cache_read(e4)
    with pytest.raises(ValueError):
        hk.cache_write(x, e4[:, :, :32], sc)
