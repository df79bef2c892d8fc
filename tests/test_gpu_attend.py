"""GPU: attention over selected rows and its gradients against the 64-bit
formulas, through the public entry points, with bounds derived in
attend_oracle.py."""
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


def rows_of(g, n, L, k, holes=0.05):
    idx = g.integers(0, L, size=(n, k)).astype(np.int32)
    if L >= k:
        for t in range(n):
            idx[t] = g.choice(L, size=k, replace=False)
    idx[g.random((n, k)) < holes] = -1
    return idx


def make(torch, dev, n, Hq, Hkv, d, k, L, cache="bf16", seed=0, qmul=1.5):
    g = np.random.default_rng(seed)
    q = torch.from_numpy(g.standard_normal((n, Hq, d), dtype=np.float32) * qmul).to(dev).bfloat16()
    kk = torch.from_numpy(g.standard_normal((L, Hkv, d), dtype=np.float32)).to(dev)
    vv = torch.from_numpy(g.standard_normal((L, Hkv, d), dtype=np.float32)).to(dev)
    idx = torch.from_numpy(rows_of(g, n, L, k)).to(dev)
    if cache == "bf16":
        return q, kk.bfloat16(), vv.bfloat16(), idx, {}
    sk = torch.from_numpy(np.exp2(g.uniform(-7, -5, size=(L, Hkv))).astype(np.float32)).to(dev)
    sv = torch.from_numpy(np.exp2(g.uniform(-9, -3, size=(L, Hkv))).astype(np.float32)).to(dev)
    return (q, (kk / sk[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn),
            (vv / sv[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn), idx,
            dict(k_scale=sk, v_scale=sv))


def values(t, scale=None):
    x = t.float().cpu().numpy().astype(np.float64)
    return x if scale is None else x * scale.cpu().numpy().astype(np.float64)[..., None]


def reference(q, k, v, idx, kw, scale, bits, grad=None):
    return oracle_attend(values(q), values(k, kw.get("k_scale")), values(v, kw.get("v_scale")),
                         idx.cpu().numpy(), scale, bits, None if grad is None else values(grad))


def verify(hk, torch, q, k, v, idx, kw, out_dtype, scale=None, **more):
    scale_used = q.shape[2] ** -0.5 if scale is None else scale
    status = torch.zeros(1, dtype=torch.int32, device=q.device)
    out, lse = hk.attend(q, k, v, idx, out_dtype=out_dtype, scale=scale, status=status, **kw, **more)
    bits = 8 if out_dtype == torch.bfloat16 else 24
    r = reference(q, k, v, idx, kw, scale_used, bits)
    check("out", out.float().cpu().numpy(), r["out"], r["tol_out"])
    check("lse", lse.cpu().numpy(), r["lse"], r["tol_lse"])
    return out, lse, int(status.item())


SHAPES = [
    # n, Hq, Hkv, d, k, L
    (1, 1, 1, 64, 1, 1),
    (1, 64, 1, 128, 2048, 5000),
    (1, 128, 1, 128, 333, 1000),
    (2, 16, 2, 256, 63, 200),
    (3, 32, 8, 64, 64, 300),
    (5, 7, 1, 128, 65, 130),
    (4, 128, 1, 64, 129, 500),
    (9, 40, 8, 128, 200, 777),
    (2, 65, 1, 256, 190, 400),
    (170, 4, 2, 64, 127, 256),
    (330, 2, 1, 128, 66, 90),
    (40, 33, 1, 128, 700, 2000),
]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,Hq,Hkv,d,k,L", SHAPES)
def test_attend_bf16_result(hk, dev, n, Hq, Hkv, d, k, L, cache):
    import torch

    q, kk, vv, idx, kw = make(torch, dev, n, Hq, Hkv, d, k, L, cache, seed=n + k)
    _, _, st = verify(hk, torch, q, kk, vv, idx, kw, torch.bfloat16)
    assert st == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,Hq,Hkv,d,k,L", [s for s in SHAPES if s[3] != 256])
def test_attend_f32_result(hk, dev, n, Hq, Hkv, d, k, L, cache):
    import torch

    q, kk, vv, idx, kw = make(torch, dev, n, Hq, Hkv, d, k, L, cache, seed=n + k + 1)
    verify(hk, torch, q, kk, vv, idx, kw, torch.float32)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,d", [(12, 1, 64), (50, 1, 64), (12, 1, 128), (50, 1, 128), (100, 1, 128),
                                      (12, 1, 256), (50, 1, 256), (100, 1, 256), (4, 2, 256)])
def test_many_items_of_several_tiles(hk, dev, Hq, Hkv, d, cache):
    """Several items per CTA, each of several tiles, in every instance of the engine: what is
    kept from item to item (buffers, phases, references) and no bounded wait giving up."""
    import torch

    n, k, L = 500, 300, 400
    q, kk, vv, idx, kw = make(torch, dev, n, Hq, Hkv, d, k, L, cache, seed=d + Hq)
    types = [torch.bfloat16] if d == 256 else [torch.bfloat16, torch.float32]
    sample = torch.arange(0, n, 29, device=dev)
    for dt in types:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        out, lse = hk.attend(q, kk, vv, idx, out_dtype=dt, status=status, **kw)
        assert int(status.item()) == 0
        r = reference(q[sample], kk, vv, idx[sample], kw, d ** -0.5, 8 if dt == torch.bfloat16 else 24)
        check("out", out[sample].float().cpu().numpy(), r["out"], r["tol_out"])
        check("lse", lse[sample].cpu().numpy(), r["lse"], r["tol_lse"])


@pytest.mark.parametrize("out_dtype", ["bfloat16", "float32"])
def test_large_scores_and_late_maxima(hk, dev, out_dtype):
    """Scores of several hundred, growing along the list: the running maximum moves at
    almost every tile, by more than any fixed slack."""
    import torch

    n, Hq, d, k, L = 3, 20, 128, 640, 640
    q, kk, vv, idx, kw = make(torch, dev, n, Hq, 1, d, k, L, seed=5, qmul=4.0)
    ramp = torch.linspace(0.0, 12.0, L, device=dev)[:, None, None]
    kk = (kk.float() * ramp).bfloat16()
    order = torch.arange(L, device=dev, dtype=torch.int32)
    idx = torch.stack([order, order.flip(0), torch.roll(order, 300)]).contiguous()
    verify(hk, torch, q, kk, vv, idx, kw, getattr(torch, out_dtype))


@pytest.mark.parametrize("n", [1, 200])  # items split over a cluster, and not
@pytest.mark.parametrize("Hq,d,out_dtype", [(20, 64, "bfloat16"), (20, 128, "bfloat16"),
                                            (100, 128, "bfloat16"), (20, 256, "bfloat16"),
                                            (20, 128, "float32")])
@pytest.mark.parametrize("what", ["scores", "wide", "rising", "falling", "zero first", "tiny"])
def test_e4m3_scales_far_apart(hk, dev, Hq, d, out_dtype, n, what):
    """Scores that grow by hundreds along the list, and row scales of V that differ by up to
    2^120, rise or fall along the list, are zero (the row still counts in the sum) or are the
    smallest that there are."""
    import torch

    k, L = 640, 640
    q, kk, vv, idx, kw = make(torch, dev, n, Hq, 1, d, k, L, "e4m3", seed=d + Hq, qmul=3.0)
    order = torch.arange(L, device=dev, dtype=torch.int32)
    idx = order.expand(n, k).contiguous()
    idx[:, 5::17] = -1
    sv, sk = kw["v_scale"], kw["k_scale"]
    up = torch.linspace(-60.0, 60.0, L, device=dev)[:, None]
    if what == "scores":
        sk *= torch.linspace(0.0, 60.0, L, device=dev)[:, None]
        sk[0] = sk[1]
    elif what == "wide":
        sv.copy_(torch.exp2(up[torch.randperm(L, device=dev)]))
    elif what == "rising":
        sv.copy_(torch.exp2(up))
    elif what == "falling":
        sv.copy_(torch.exp2(-up))
    elif what == "zero first":
        sv[:200] = 0.0
        sv[300:310] = 0.0
    else:
        sv.fill_(2.0 ** -126)
    dt = getattr(torch, out_dtype)
    sample = torch.arange(0, n, 67, device=dev)
    out, lse = hk.attend(q, kk, vv, idx, out_dtype=dt, **kw)
    r = reference(q[sample], kk, vv, idx[sample], kw, d ** -0.5, 8 if dt == torch.bfloat16 else 24)
    check("out", out[sample].float().cpu().numpy(), r["out"], r["tol_out"])
    check("lse", lse[sample].cpu().numpy(), r["lse"], r["tol_lse"])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,d", [(12, 64), (50, 128), (100, 128), (12, 256)])
def test_heads_do_not_touch_each_other(hk, dev, Hq, d, cache):
    """One head 2^40 times the others and one 2^-40 times; then infinities in one head."""
    import torch

    n, k, L = 3, 200, 300
    q, kk, vv, idx, kw = make(torch, dev, n, Hq, 1, d, k, L, cache, seed=d)
    q[:, 3] *= 2.0 ** 40
    q[:, 5] *= 2.0 ** -40
    q[:, 7] = 0.0
    verify(hk, torch, q, kk, vv, idx, kw, torch.bfloat16)
    r = reference(q, kk, vv, idx, kw, d ** -0.5, 8)
    q[:, 7, ::9] = float("inf")
    out, lse = hk.attend(q, kk, vv, idx, **kw)
    keep = [h for h in range(Hq) if h != 7]
    check("out", out[:, keep].float().cpu().numpy(), r["out"][:, keep], r["tol_out"][:, keep])
    check("lse", lse[:, keep].cpu().numpy(), r["lse"][:, keep], r["tol_lse"][:, keep])


def test_empty_rows_holes_and_bad_indices(hk, dev):
    import torch

    n, Hq, Hkv, d, k, L = 6, 8, 2, 128, 300, 400
    q, kk, vv, idx, kw = make(torch, dev, n, Hq, Hkv, d, k, L, seed=9)
    idx[0] = -1                       # nothing selected
    idx[1, :-1] = -1                  # only the last entry of a ragged tile
    idx[2, 64:192] = -1               # whole tiles of nothing
    idx[3, ::2] = -1
    out, lse, st = verify(hk, torch, q, kk, vv, idx, kw, torch.bfloat16)
    assert st == 0
    assert torch.all(out[0] == 0) and torch.all(lse[0] == -float("inf"))
    idx[4, 5] = L                     # counts as no row, and is reported
    idx[5, 7] = -2
    _, _, st = verify(hk, torch, q, kk, vv, idx, kw, torch.bfloat16)
    assert st == hk.DEV_BAD_INDEX


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_values_of_rows_not_selected_do_not_matter(hk, dev, cache):
    """NaN and infinities in every row that is not selected, row 0 among them (the
    row a masked entry could fall back to), and in the scales of those rows."""
    import torch

    n, Hq, d, k, L = 4, 16, 128, 100, 600
    q, kk, vv, idx, kw = make(torch, dev, n, Hq, 1, d, k, L, cache, seed=11)
    idx = idx.clamp(min=-1)
    idx[idx == 0] = -1
    used = torch.zeros(L, dtype=torch.bool, device=dev)
    used[idx[idx >= 0].long()] = True
    if cache == "bf16":
        kk[~used] = float("nan")
        vv[~used] = float("inf")
    else:
        kk.view(torch.uint8)[~used] = 0x7F
        vv.view(torch.uint8)[~used] = 0xFF
        kw["k_scale"][~used] = float("nan")
        kw["v_scale"][~used] = float("inf")
    clean_k, clean_v = kk.clone(), vv.clone()
    ckw = {a: b.clone() for a, b in kw.items()}
    clean_k.view(torch.uint8)[~used] = 0
    clean_v.view(torch.uint8)[~used] = 0
    for s in ckw.values():
        s[~used] = 1.0
    for dt in (torch.bfloat16, torch.float32):
        a = hk.attend(q, kk, vv, idx, out_dtype=dt, **kw)
        b = hk.attend(q, clean_k, clean_v, idx, out_dtype=dt, **ckw)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    r = reference(q, clean_k, clean_v, idx, ckw, d ** -0.5, 24)
    check("out", a[0].cpu().numpy(), r["out"], r["tol_out"])


def test_duplicates_count_as_often_as_they_are_listed(hk, dev):
    import torch

    q, kk, vv, idx, kw = make(torch, dev, 3, 12, 1, 64, 150, 200, seed=13)
    idx[:, 75:150] = idx[:, :75]
    verify(hk, torch, q, kk, vv, idx, kw, torch.float32)


def test_strided_queries_and_interleaved_cache(hk, dev):
    """q inside a wider projection; k and v rows of one [L, 2, Hkv, d] cache."""
    import torch

    n, Hq, Hkv, d, k, L = 7, 16, 4, 64, 90, 300
    g = torch.Generator(device=dev).manual_seed(3)
    wide = torch.randn(n, Hq + 8, d, device=dev, generator=g).bfloat16()
    kv = torch.randn(L, 2, Hkv, d, device=dev, generator=g).bfloat16()
    idx = torch.from_numpy(rows_of(np.random.default_rng(1), n, L, k)).to(dev)
    verify(hk, torch, wide[:, 4:4 + Hq], kv[:, 0], kv[:, 1], idx, {}, torch.bfloat16)
    verify(hk, torch, wide[:, 4:4 + Hq], kv[:, 0], kv[:, 0], idx, {}, torch.float32)


def test_two_dimensional_cache_and_scale(hk, dev):
    import torch

    q, kk, vv, idx, kw = make(torch, dev, 2, 3, 1, 128, 40, 50, "e4m3", seed=17)
    a = hk.attend(q, kk, vv, idx, scale=0.3, **kw)
    b = hk.attend(q, kk[:, 0], vv[:, 0], idx, scale=0.3, k_scale=kw["k_scale"][:, 0].contiguous(),
                  v_scale=kw["v_scale"][:, 0].contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    verify(hk, torch, q, kk, vv, idx, kw, torch.bfloat16, scale=0.3)
    # a negative scale reverses the order of the scores; zero makes them equal
    verify(hk, torch, q, kk, vv, idx, kw, torch.float32, scale=0.0)


def test_offsets_past_32_bits(hk, dev):
    """Rows beyond 2^32 bytes (and 2^31 elements) of a long cache."""
    import torch

    L, d, n, Hq, k = (1 << 24) + 4097, 128, 2, 16, 200
    cache = torch.zeros(L, 1, d, device=dev, dtype=torch.bfloat16)
    g = torch.Generator(device=dev).manual_seed(4)
    tail = torch.randn(4096, 1, d, device=dev, generator=g).bfloat16()
    cache[L - 4096:] = tail
    q = torch.randn(n, Hq, d, device=dev, generator=g).bfloat16()
    idx = torch.randint(0, 4096, (n, k), device=dev, generator=g, dtype=torch.int32)
    want = hk.attend(q, tail, tail, idx, out_dtype=torch.float32)
    got = hk.attend(q, cache, cache, idx + (L - 4096), out_dtype=torch.float32)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_no_queries_and_given_outputs(hk, dev):
    import torch

    q, kk, vv, idx, kw = make(torch, dev, 4, 8, 2, 64, 70, 100, seed=19)
    out, lse = hk.attend(q[:0], kk, vv, idx[:0])
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
    buf = torch.full((4, 8, 64), 7.0, device=dev, dtype=torch.bfloat16)
    out, _ = hk.attend(q, kk, vv, idx, out=buf)
    assert out is buf
    assert torch.equal(buf, hk.attend(q, kk, vv, idx)[0])


def test_another_stream_and_repeat(hk, dev):
    """On a side stream, and the same bits every time."""
    import torch

    q, kk, vv, idx, kw = make(torch, dev, 20, 32, 1, 128, 500, 900, seed=21)
    want = hk.attend(q, kk, vv, idx)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(5):
            got = hk.attend(q, kk, vv, idx)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_a_stream_given_explicitly(hk, dev):
    """stream=: the same bits, and memory of a dropped result is not used anew while the
    call still writes it."""
    import torch

    q, kk, vv, idx, kw = make(torch, dev, 600, 32, 1, 128, 900, 900, seed=22)
    want = hk.attend(q, kk, vv, idx)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = hk.attend(q, kk, vv, idx, stream=side)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    del got
    for _ in range(10):
        side.wait_stream(torch.cuda.current_stream())
        hk.attend(q, kk, vv, idx, stream=side)  # dropped at once
        marks = torch.full_like(want[0], 7.0)
        torch.cuda.synchronize()
        assert bool((marks == 7.0).all())


def test_captured_in_a_graph(hk, dev):
    import torch

    q, kk, vv, idx, kw = make(torch, dev, 2, 64, 1, 128, 700, 900, seed=23)
    out = torch.empty(2, 64, 128, device=dev, dtype=torch.bfloat16)
    hk.attend(q, kk, vv, idx, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hk.attend(q, kk, vv, idx, out=out)
    q.copy_(q.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, hk.attend(q, kk, vv, idx)[0])


# ---- gradients ----------------------------------------------------------------------

BACKWARD = [
    (1, 1, 1, 64, 1, 1),
    (2, 8, 2, 64, 63, 100),
    (3, 16, 1, 128, 130, 200),
    (4, 64, 1, 128, 200, 300),
    (3, 128, 1, 128, 100, 150),
    (5, 65, 1, 64, 65, 80),
    (160, 6, 3, 128, 40, 64),
    (2, 128, 1, 64, 257, 400),
    (7, 20, 4, 128, 300, 1000),
]


@pytest.mark.parametrize("n,Hq,Hkv,d,k,L", BACKWARD)
def test_gradients(hk, dev, n, Hq, Hkv, d, k, L):
    import torch

    q, kk, vv, idx, kw = make(torch, dev, n, Hq, Hkv, d, k, L, seed=31 + n)
    if n > 2:
        idx[1] = -1
    grad = torch.randn(n, Hq, d, device=dev, generator=torch.Generator(device=dev).manual_seed(n)).bfloat16()
    out, lse = hk.attend(q, kk, vv, idx, out_dtype=torch.float32)
    dq, dk, dv = hk.attend_backward(q, kk, vv, idx, out, lse, grad)
    r = reference(q, kk, vv, idx, kw, d ** -0.5, 24, grad)
    for name, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        check(name, got.cpu().numpy(), r[name], r["tol_" + name])


@pytest.mark.parametrize("n,Hq,Hkv,d", [(1, 8, 1, 64), (2, 20, 1, 128), (10, 16, 4, 64),
                                        (20, 12, 2, 128), (70, 40, 1, 128)])
def test_gradients_of_few_queries_with_many_rows(hk, dev, n, Hq, Hkv, d):
    """Several CTAs share a query's rows and add up its dq; new tensors and given ones."""
    import torch

    k, L = 1700, 2500
    q, kk, vv, idx, kw = make(torch, dev, n, Hq, Hkv, d, k, L, seed=41 + n)
    if n > 2:
        idx[1] = -1
        idx[2, 100:1500] = -1  # shares with no row at all
    grad = torch.randn(n, Hq, d, device=dev, generator=torch.Generator(device=dev).manual_seed(n)).bfloat16()
    out, lse = hk.attend(q, kk, vv, idx, out_dtype=torch.float32)
    r = reference(q, kk, vv, idx, kw, d ** -0.5, 24, grad)
    dk0, dv0 = torch.zeros(L, Hkv, d, device=dev), torch.zeros(L, Hkv, d, device=dev)
    for given in ({}, dict(dk=dk0, dv=dv0)):
        got = hk.attend_backward(q, kk, vv, idx, out, lse, grad, **given)
        for name, x in zip(("dq", "dk", "dv"), got):
            check(name, x.cpu().numpy(), r[name], r["tol_" + name])


@pytest.mark.parametrize("Hq,d", [(12, 64), (50, 64), (12, 128), (100, 128)])
def test_gradients_of_many_items_of_several_tiles(hk, dev, Hq, d):
    import torch

    n, k, L = 400, 650, 700
    q, kk, vv, idx, kw = make(torch, dev, n, Hq, 1, d, k, L, seed=d + Hq)
    keep = torch.arange(0, n, 57, device=dev)
    grad = torch.zeros(n, Hq, d, device=dev, dtype=torch.bfloat16)  # the others' rows add nothing
    g = torch.Generator(device=dev).manual_seed(3)
    grad[keep] = torch.randn(len(keep), Hq, d, device=dev, generator=g).bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = hk.attend(q, kk, vv, idx, out_dtype=torch.float32)
    dq, dk, dv = hk.attend_backward(q, kk, vv, idx, out, lse, grad, status=status)
    assert int(status.item()) == 0
    r = reference(q[keep], kk, vv, idx[keep], kw, d ** -0.5, 24, grad[keep])
    check("dq", dq[keep].cpu().numpy(), r["dq"], r["tol_dq"])
    check("dk", dk.cpu().numpy(), r["dk"], r["tol_dk"])
    check("dv", dv.cpu().numpy(), r["dv"], r["tol_dv"])


def test_gradients_against_differences(hk, dev):
    """The directional derivative of sum(out * grad) by central differences in 64 bits
    (the oracle's forward alone), along random directions of q, k and v."""
    import torch

    n, Hq, Hkv, d, k, L = 3, 6, 2, 64, 50, 70
    q, kk, vv, idx, kw = make(torch, dev, n, Hq, Hkv, d, k, L, seed=41)
    grad = torch.randn(n, Hq, d, device=dev, generator=torch.Generator(device=dev).manual_seed(1)).bfloat16()
    out, lse = hk.attend(q, kk, vv, idx, out_dtype=torch.float32)
    got = [x.cpu().numpy().astype(np.float64) for x in
           hk.attend_backward(q, kk, vv, idx, out, lse, grad)]
    base = [values(q), values(kk), values(vv)]
    r = reference(q, kk, vv, idx, kw, d ** -0.5, 24, grad)
    gv, ids, g = values(grad), idx.cpu().numpy(), np.random.default_rng(2)
    eps = 1e-4
    for i in range(3):
        u = g.standard_normal(base[i].shape)

        def loss(sign):
            x = list(base)
            x[i] = base[i] + sign * eps * u
            return (oracle_attend(*x, ids, d ** -0.5)["out"] * gv).sum()

        want = (loss(1) - loss(-1)) / (2 * eps)
        # the gradients' own bounds, and eps^2 times third derivatives (scores move by about
        # eps |q| along a unit of u: a few eps, hence 100 eps^2 of the summed magnitudes)
        bound = (r[("tol_dq", "tol_dk", "tol_dv")[i]] * np.abs(u)).sum()
        assert abs((got[i] * u).sum() - want) <= bound + 100 * eps ** 2 * np.abs(got[i] * u).sum()


def test_gradients_are_added_and_bad_indices_reported(hk, dev):
    import torch

    n, Hq, Hkv, d, k, L = 4, 8, 1, 128, 90, 200
    q, kk, vv, idx, kw = make(torch, dev, n, Hq, Hkv, d, k, L, seed=43)
    grad = torch.ones(n, Hq, d, device=dev, dtype=torch.bfloat16)
    out, lse = hk.attend(q, kk, vv, idx, out_dtype=torch.float32)
    dq, dk, dv = hk.attend_backward(q, kk, vv, idx, out, lse, grad)
    dk2, dv2 = torch.full_like(dk, 3.0), torch.full_like(dv, -2.0)
    idx2 = idx.clone()
    idx2[idx2 == -1] = L + 5  # counts as no row all the same
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    dq2, a, b = hk.attend_backward(q, kk, vv, idx2, out, lse, grad, dk=dk2, dv=dv2, status=st)
    assert a is dk2 and b is dv2
    assert int(st.item()) == hk.DEV_BAD_INDEX
    r = reference(q, kk, vv, idx, kw, d ** -0.5, 24, grad)
    check("dq", dq2.cpu().numpy(), r["dq"], r["tol_dq"])
    # 2^-21: rounding of sums of magnitude 3 and more
    check("dk", dk2.cpu().numpy(), r["dk"] + 3.0, r["tol_dk"] + 2.0 ** -20)
    check("dv", dv2.cpu().numpy(), r["dv"] - 2.0, r["tol_dv"] + 2.0 ** -20)


def test_gradients_ignore_rows_not_selected(hk, dev):
    import torch

    n, Hq, d, k, L = 3, 8, 64, 70, 300
    q, kk, vv, idx, kw = make(torch, dev, n, Hq, 1, d, k, L, seed=47)
    idx[idx == 0] = -1
    used = torch.zeros(L, dtype=torch.bool, device=dev)
    used[idx[idx >= 0].long()] = True
    ck, cv = kk.clone(), vv.clone()
    kk[~used] = float("nan")
    vv[~used] = float("inf")
    ck[~used] = 0
    cv[~used] = 0
    grad = torch.ones(n, Hq, d, device=dev, dtype=torch.bfloat16)
    out, lse = hk.attend(q, kk, vv, idx, out_dtype=torch.float32)
    dq, dk, dv = hk.attend_backward(q, kk, vv, idx, out, lse, grad)
    assert torch.all(dk[~used] == 0) and torch.all(dv[~used] == 0)
    r = reference(q, ck, cv, idx, kw, d ** -0.5, 24, grad)
    for name, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        check(name, got.cpu().numpy(), r[name], r["tol_" + name])


def test_gradients_from_a_bf16_result(hk, dev):
    """out in bf16 only changes the row sum grad . out, by at most 2^-8 |grad| . |out|."""
    import torch

    n, Hq, d, k, L = 5, 24, 128, 100, 300
    q, kk, vv, idx, kw = make(torch, dev, n, Hq, 1, d, k, L, seed=53)
    grad = torch.randn(n, Hq, d, device=dev, generator=torch.Generator(device=dev).manual_seed(5)).bfloat16()
    out, lse = hk.attend(q, kk, vv, idx, out_dtype=torch.float32)
    full = hk.attend_backward(q, kk, vv, idx, out, lse, grad)
    half = hk.attend_backward(q, kk, vv, idx, out.bfloat16(), lse, grad)
    # ds changes by p * 2^-8 |grad| . |out|, the same for every row of a head
    shift = 2.0 ** -8 * (grad.double().abs() * out.double().abs()).sum(-1)
    kmax = kk.double().abs().amax()
    assert torch.all((full[0] - half[0]).abs().amax(-1) <= d ** -0.5 * shift * kmax + 1e-5)
    assert torch.allclose(full[2], half[2], rtol=1e-4, atol=1e-5)  # dv does not use out


# ---- refusals -----------------------------------------------------------------------

def test_refusals(hk, dev):
    import torch

    q, kk, vv, idx, kw = make(torch, dev, 2, 8, 2, 64, 20, 50, seed=61)
    bad = [
        (TypeError, dict(q=q.float())),
        (TypeError, dict(k=kk.float(), v=vv.float())),
        (ValueError, dict(v=vv[:40])),
        (ValueError, dict(k=kk.to(torch.float8_e4m3fn), v=vv.to(torch.float8_e4m3fn))),
        (ValueError, dict(k_scale=torch.ones(50, 2, device=dev), v_scale=torch.ones(50, 2, device=dev))),
        (TypeError, dict(idx=idx.long())),
        (ValueError, dict(idx=idx[:1])),
        (ValueError, dict(idx=idx[:, ::2])),
        (ValueError, dict(q=q[:, :, ::2])),
        (ValueError, dict(q=q[:, ::2])),
        (ValueError, dict(q=q.cpu())),
        (TypeError, dict(out_dtype=torch.float16)),
        (hk.HytopkError, dict(q=q[:, :7].contiguous())),  # 7 heads over 2 cache heads
    ]
    for error, change in bad:
        args = dict(q=q, k=kk, v=vv, idx=idx)
        args.update(change)
        with pytest.raises(error):
            hk.attend(**args)
    with pytest.raises(hk.HytopkError) as e:  # d not supported
        hk.attend(torch.zeros(1, 1, 96, device=dev).bfloat16(), torch.zeros(4, 1, 96, device=dev).bfloat16(),
                  torch.zeros(4, 1, 96, device=dev).bfloat16(), torch.zeros(1, 4, dtype=torch.int32, device=dev))
    assert e.value.status == 2
    out, lse = hk.attend(q, kk, vv, idx, out_dtype=torch.float32)
    with pytest.raises(TypeError):
        hk.attend_backward(q, kk, vv, idx, out, lse, out)
    with pytest.raises(TypeError):
        hk.attend_backward(q, kk.to(torch.float8_e4m3fn), vv.to(torch.float8_e4m3fn), idx, out, lse,
                           out.bfloat16())
    with pytest.raises(ValueError):
        hk.attend_backward(q, kk, vv, idx, out, lse[:1], out.bfloat16())
