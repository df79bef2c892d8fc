"""The operators around a selection without a GPU: host-side argument checks of
the C entry points and the rotary frequency tables."""
import ctypes
import math

import pytest

import exact_top_token_gb300 as hk

P = ctypes.c_void_p
FAKE = P(1 << 20)  # never dereferenced: every case fails a host check (or has no rows)


@pytest.fixture(scope="module")
def lib():
    hk.build()
    return hk.load()


def rope_args(**kw):
    r = dict(positions=1 << 20, inv_freq=1 << 20, rot=64, first=0, interleaved=0, inverse=0,
             mscale=1.0)
    r.update(kw)
    return ctypes.byref(hk.RopeParams(**r))


def test_rope_checks(lib):
    def call(rope=rope_args(), **kw):
        a = dict(x=FAKE, xr=128, xh=64, type=0, n=4, H=2, d=64, out=FAKE, orow=128, oh=64)
        a.update(kw)
        return lib.hytopk_rope(a["x"], a["xr"], a["xh"], a["type"], a["n"], a["H"], a["d"], rope,
                               a["out"], a["orow"], a["oh"], None, None)

    assert call(rope=None) == 1
    assert call(x=None) == 1
    assert call(out=None) == 1
    assert call(n=-1) == 1
    assert call(H=0) == 1
    assert call(type=1) == 1
    assert call(d=60) == 2
    assert call(d=2048) == 2
    assert call(rope=rope_args(rot=24)) == 2
    assert call(rope=rope_args(rot=0)) == 1
    assert call(rope=rope_args(rot=48, first=4)) == 2
    assert call(rope=rope_args(rot=64, first=8)) == 1
    assert call(rope=rope_args(first=-8)) == 1
    assert call(rope=rope_args(positions=0)) == 1
    assert call(rope=rope_args(inv_freq=0)) == 1
    assert call(rope=rope_args(positions=(1 << 20) + 2)) == 5
    assert call(x=P((1 << 20) + 8)) == 5
    assert call(xr=132, out=P(1 << 21)) == 5
    assert call(oh=68, out=P(1 << 21)) == 5
    assert call(xr=256) == 1  # in place with other strides
    assert call(n=0, x=None, out=None) == 0


def test_cache_checks(lib):
    def write(**kw):
        a = dict(x=FAKE, xr=128, xh=64, type=0, n=4, H=2, d=64, rope=None, slots=None, cache=FAKE,
                 ct=1, cs=FAKE, L=100)
        a.update(kw)
        return lib.hytopk_cache_write(a["x"], a["xr"], a["xh"], a["type"], a["n"], a["H"], a["d"],
                                      a["rope"], a["slots"], a["cache"], a["ct"], a["cs"], a["L"],
                                      None, None)

    assert write(x=None) == 1
    assert write(cache=None) == 1
    assert write(cs=None) == 1
    assert write(ct=0) == 1      # bf16 takes no scales
    assert write(ct=2, cs=None) == 1
    assert write(type=1) == 1
    assert write(L=0) == 1
    assert write(L=3) == 1       # no slots and more rows than the cache
    assert write(d=72) == 2      # e4m3 rows of whole 16 bytes
    assert write(rope=rope_args(rot=40)) == 2
    assert write(cache=P((1 << 20) + 8)) == 5
    assert write(cs=P((1 << 20) + 2)) == 5
    assert write(slots=P((1 << 20) + 2)) == 5
    assert write(n=0, x=None) == 0

    def read(**kw):
        a = dict(cache=FAKE, ct=1, cs=FAKE, L=100, slots=FAKE, n=4, H=2, d=64, out=FAKE, ot=0)
        a.update(kw)
        return lib.hytopk_cache_read(a["cache"], a["ct"], a["cs"], a["L"], a["slots"], a["n"],
                                     a["H"], a["d"], a["out"], a["ot"], None, None)

    assert read(cache=None) == 1
    assert read(cs=None) == 1
    assert read(ct=0) == 1
    assert read(ct=2) == 1
    assert read(ot=1) == 1
    assert read(out=None) == 1
    assert read(slots=None, n=101) == 1
    assert read(d=72) == 2
    assert read(out=P((1 << 20) + 4)) == 5
    assert read(n=0, cache=None, out=None) == 0


def test_attend_checks(lib):
    def call(**kw):
        a = dict(q=FAKE, qr=512, k=FAKE, kr=128, ks=None, v=FAKE, vr=128, vs=None, idx=FAKE, n=4,
                 L=100, Hq=8, Hkv=2, d=64, k_top=10, ct=0, out=FAKE, ot=0, lse=FAKE)
        a.update(kw)
        return lib.hytopk_attend(a["q"], a["qr"], a["k"], a["kr"], a["ks"], a["v"], a["vr"],
                                 a["vs"], a["idx"], a["n"], a["L"], a["Hq"], a["Hkv"], a["d"],
                                 a["k_top"], a["ct"], 0.125, a["out"], a["ot"], a["lse"], None,
                                 None)

    for name in ("q", "k", "v", "idx", "out"):
        assert call(**{name: None}) == 1, name
    assert call(n=-1) == 1
    assert call(L=0) == 1
    assert call(Hkv=0) == 1
    assert call(Hkv=3) == 1
    assert call(k_top=0) == 1
    assert call(k_top=16385) == 2
    assert call(Hq=258) == 2      # 129 heads on one cache head
    assert call(d=96) == 2
    assert call(d=256, ot=2) == 2
    assert call(ct=2) == 1
    assert call(ot=1) == 1
    assert call(ct=1) == 1        # scales missing
    assert call(ks=FAKE, vs=FAKE) == 1
    assert call(ct=1, ks=FAKE) == 1
    assert call(q=P((1 << 20) + 8)) == 5
    assert call(qr=516) == 5
    assert call(kr=132) == 5
    assert call(kr=-128) == 1
    assert call(vr=-128) == 1
    assert call(kr=1 << 31) == 2  # a row of 4 GiB
    assert call(vr=1 << 31) == 2
    assert call(ct=1, ks=FAKE, vs=FAKE, vr=136) == 5
    assert call(n=0, q=None, out=None) == 0


def test_attend_backward_checks(lib):
    def call(**kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, idx=FAKE, out=FAKE, ot=2, lse=FAKE, grad=FAKE, n=4, L=100,
                 Hq=8, Hkv=2, d=64, k_top=10, dq=FAKE, dk=FAKE, dv=FAKE, add=1, kr=128, vr=128)
        a.update(kw)
        return lib.hytopk_attend_backward(a["q"], 512, a["k"], a["kr"], a["v"], a["vr"], a["idx"], a["out"],
                                          a["ot"], a["lse"], a["grad"], a["n"], a["L"], a["Hq"],
                                          a["Hkv"], a["d"], a["k_top"], 0.125, a["dq"], a["dk"],
                                          a["dv"], a["add"], None, None)

    for name in ("q", "k", "v", "idx", "out", "lse", "grad", "dq", "dk", "dv"):
        assert call(**{name: None}) == 1, name
    assert call(d=256) == 2
    assert call(ot=1) == 1
    assert call(Hkv=5) == 1
    assert call(kr=-128) == 1
    assert call(vr=1 << 31) == 2
    assert call(Hq=1 << 24, Hkv=1 << 24, n=1) == 2  # a gradient row of 4 GiB
    assert call(dk=P((1 << 20) + 4)) == 5
    assert call(grad=P((1 << 20) + 2)) == 5
    assert call(n=0, q=None) == 0


def test_entry_points_refuse_what_is_no_cuda_tensor(lib):
    import torch

    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    pos, f, idx = torch.zeros(2, dtype=torch.int32), torch.ones(32), torch.zeros(2, 4, dtype=torch.int32)
    calls = [lambda a: hk.rope(a, pos, f), lambda a: hk.cache_write(a, x), lambda a: hk.cache_read(a),
             lambda a: hk.attend(a, x, x, idx), lambda a: hk.attend_backward(a, x, x, idx, x, f, x)]
    for call in calls:
        with pytest.raises(ValueError):
            call(x)                     # not on a GPU
        with pytest.raises(TypeError):
            call([1, 2])                # no tensor
        with pytest.raises(TypeError):
            call(None)
    with pytest.raises(TypeError):
        hk.rope(x)
    with pytest.raises(TypeError):
        hk.attend(x, x, x, idx, no_such_argument=1)


def test_frequency_tables():
    def table(*a, **kw):
        f, m = hk.rope_frequencies(*a, device="cpu", **kw)
        return f.double().tolist(), m

    plain, m = table(64)
    assert m == 1.0 and len(plain) == 32 and plain[0] == 1.0
    assert plain[16] == pytest.approx(1e-2, rel=1e-6)
    lin, _ = table(64, scaling="linear", factor=4.0)
    assert lin == pytest.approx([f / 4 for f in plain], rel=1e-6)
    raised, _ = table(64, scaling="base", factor=4.0)
    assert raised[0] == 1.0 and raised[-1] == pytest.approx(plain[-1] / 4, rel=1e-6)
    parts, m = table(64, scaling="parts", factor=4.0, original_context=4096)
    assert m == pytest.approx(0.1 * math.log(4.0) + 1.0)
    for f, p in zip(plain, parts):
        turns = 4096 * f / (2 * math.pi)
        if turns >= 32:
            assert p == pytest.approx(f, rel=1e-6)
        elif turns <= 1:
            assert p == pytest.approx(f / 4, rel=1e-6)
        else:
            assert f / 4 <= p <= f
    for bad in (dict(rot=7), dict(rot=64, base=0.0), dict(rot=64, factor=0.5),
                dict(rot=64, scaling="parts", factor=2.0), dict(rot=64, scaling="other"),
                dict(rot=2, scaling="base", factor=2.0)):
        rot = bad.pop("rot")
        with pytest.raises(ValueError):
            hk.rope_frequencies(rot, bad.pop("base", 1e4), device="cpu", **bad)
