"""The cache in pages without a GPU: host-side argument checks of the C entry points, and of
the Python module on tensors that only claim a device."""
import ctypes
import math
import os
import subprocess
import sys

import pytest

import exact_top_token_gb300 as hk
from test_operators_binding import FAKE_RUNTIME, PRELUDE, ROOT

P = ctypes.c_void_p
AT = 1 << 20
FAKE = P(AT)  # never dereferenced: every case fails a host check (or has nothing to do)
OK, INVALID, UNSUPPORTED, SMALL, MISALIGNED = 0, 1, 2, 3, 5


@pytest.fixture(scope="module")
def lib():
    hk.build()
    return hk.load()


def paged(**kw):
    s = dict(table=AT, lengths=AT, cu_q=AT, B=4, columns=8, N=100, P=16)
    s.update(kw)
    return ctypes.byref(hk.Paged(**s))


# what is wrong with the sequences of a call, for both operators that take them
SEQUENCES = [
    (None, INVALID),
    (dict(B=-1), INVALID),
    (dict(columns=0), INVALID),
    (dict(N=0), INVALID),
    (dict(table=0), INVALID),
    (dict(lengths=0), INVALID),
    (dict(cu_q=0), INVALID),  # (nine rows, four sequences)
    (dict(P=0), UNSUPPORTED),
    (dict(P=8), UNSUPPORTED),
    (dict(P=48), UNSUPPORTED),
    (dict(P=512), UNSUPPORTED),
    (dict(columns=1 << 23, P=256), UNSUPPORTED),  # 2^31 rows of a context
    (dict(table=AT + 2), MISALIGNED),
    (dict(lengths=AT + 1), MISALIGNED),
    (dict(cu_q=AT + 2), MISALIGNED),
]


def attend(lib, s=None, **kw):
    a = dict(q=FAKE, qr=1024, kp=FAKE, ks=FAKE, vp=FAKE, vs=FAKE, n=9, Hq=8, Hkv=2, d=128,
             scale=0.1, out=FAKE, lse=FAKE, ws=FAKE, wb=1 << 40)
    a.update(kw)
    return lib.hytopk_attend_pages(a["q"], a["qr"], a["kp"], a["ks"], a["vp"], a["vs"],
                                   paged() if s is None else s, a["n"], a["Hq"], a["Hkv"], a["d"],
                                   a["scale"], a["out"], a["lse"], a["ws"], a["wb"], None, None)


def write(lib, s=None, **kw):
    a = dict(x=FAKE, xr=256, xh=128, type=0, n=9, H=2, d=128, rope=None, pages=FAKE, scale=FAKE)
    a.update(kw)
    return lib.hytopk_page_write(a["x"], a["xr"], a["xh"], a["type"], a["n"], a["H"], a["d"],
                                 a["rope"], a["pages"], a["scale"], paged() if s is None else s,
                                 None, None)


@pytest.mark.parametrize("fields,status", SEQUENCES, ids=lambda v: str(v))
def test_sequences(lib, fields, status):
    s = P(None) if fields is None else paged(**fields)
    assert attend(lib, s) == status
    assert write(lib, s) == status


def test_attend(lib):
    assert attend(lib, n=-1) == INVALID
    for kw in (dict(Hkv=0), dict(Hq=0), dict(Hq=9), dict(Hq=1, Hkv=2), dict(scale=math.nan),
               dict(scale=-math.inf)):
        assert attend(lib, **kw) == INVALID, kw
    for kw in (dict(Hq=258), dict(d=96), dict(d=256), dict(n=1 << 28)):
        assert attend(lib, **kw) == UNSUPPORTED, kw
    assert attend(lib, paged(N=(1 << 27) - 1, P=16)) == UNSUPPORTED  # rows of the pool
    for name in ("q", "kp", "vp", "ks", "vs", "out", "ws"):
        assert attend(lib, **{name: None}) == INVALID, name
    for name in ("q", "kp", "vp", "out"):
        assert attend(lib, **{name: P(AT + 8)}) == MISALIGNED, name
    for name in ("ks", "vs", "lse"):
        assert attend(lib, **{name: P(AT + 2)}) == MISALIGNED, name
    assert attend(lib, ws=P(AT + 128)) == MISALIGNED
    assert attend(lib, qr=1028) == MISALIGNED
    need = lib.hytopk_attend_pages_workspace_size(9, 8, 2, 128)
    assert need > 0 and attend(lib, wb=need - 1) == SMALL
    # nothing to do
    assert attend(lib, n=0, q=None, out=None) == OK
    assert attend(lib, paged(B=0, table=0, lengths=0), q=None, out=None) == OK


def test_attend_workspace(lib):
    size = lib.hytopk_attend_pages_workspace_size
    # no item has more than a block of 128 rows, or some may
    assert 0 < size(32, 8, 2, 128) < size(33, 8, 2, 128) == size(1 << 20, 8, 2, 128)
    assert size(32, 8, 2, 64) < size(32, 8, 2, 128)
    for bad in ((-1, 8, 2, 128), (4, 8, 0, 128), (4, 9, 2, 128), (4, 1, 2, 128), (4, 258, 2, 128),
                (4, 8, 2, 96)):
        assert size(*bad) == 0, bad


def test_write(lib):
    def rope(**kw):
        r = dict(positions=0, inv_freq=AT, rot=64, first=0, interleaved=0, inverse=0, mscale=1.0)
        r.update(kw)
        return ctypes.byref(hk.RopeParams(**r))

    assert write(lib, n=-1) == INVALID
    assert write(lib, H=0) == INVALID
    assert write(lib, type=1) == INVALID
    for d in (32, 96, 192, 512):
        assert write(lib, d=d) == UNSUPPORTED
    assert write(lib, n=1 << 30) == UNSUPPORTED
    for name in ("x", "pages", "scale"):
        assert write(lib, **{name: None}) == INVALID, name
    assert write(lib, rope=rope(inv_freq=0)) == INVALID
    assert write(lib, rope=rope(rot=0)) == INVALID
    assert write(lib, rope=rope(first=-8)) == INVALID
    assert write(lib, rope=rope(rot=128, first=8)) == INVALID
    assert write(lib, rope=rope(rot=24)) == UNSUPPORTED
    assert write(lib, rope=rope(first=4)) == UNSUPPORTED
    assert write(lib, rope=rope(positions=AT + 2)) == MISALIGNED
    assert write(lib, rope=rope(inv_freq=AT + 2)) == MISALIGNED
    assert write(lib, x=P(AT + 8)) == MISALIGNED
    assert write(lib, xr=260) == MISALIGNED  # of 16-bit elements
    assert write(lib, xh=132) == MISALIGNED
    assert write(lib, pages=P(AT + 8)) == MISALIGNED
    assert write(lib, scale=P(AT + 2)) == MISALIGNED
    assert write(lib, n=0, x=None) == OK
    assert write(lib, paged(B=0, table=0, lengths=0), x=None) == OK


POOL = dict(table=FAKE, lengths=FAKE, refs=FAKE, B=4, columns=8, N=100, P=16)


def calls_of(lib):
    """name -> call(**changes) of the operators on a pool's bookkeeping"""
    def pool(a):
        return [a[k] for k in ("table", "lengths", "refs", "B", "columns", "N", "P")]

    def fork(**kw):
        a = dict(POOL, src=FAKE, dst=FAKE, count=2) | kw
        return lib.hytopk_page_fork(*pool(a), a["src"], a["dst"], a["count"], None, None)

    def free(**kw):
        a = dict(POOL, rows=FAKE, count=2) | kw
        return lib.hytopk_page_free(*pool(a), a["rows"], a["count"], None, None)

    def grow(**kw):
        a = dict(POOL, add=FAKE, src=FAKE, dst=FAKE, ws=FAKE, wb=1 << 40) | kw
        return lib.hytopk_page_grow(*pool(a), a["add"], a["src"], a["dst"], a["ws"], a["wb"], None,
                                    None)

    def compact(**kw):
        a = dict(POOL, src=FAKE, dst=FAKE, ws=FAKE, wb=1 << 40) | kw
        return lib.hytopk_page_compact(*pool(a), a["src"], a["dst"], a["ws"], a["wb"], None, None)

    return dict(fork=fork, free=free, grow=grow, compact=compact)


@pytest.mark.parametrize("name", ["fork", "free", "grow", "compact"])
def test_pool(lib, name):
    call = calls_of(lib)[name]
    assert call(B=-1) == INVALID
    assert call(columns=0) == INVALID
    assert call(N=0) == INVALID
    for rows in (0, 8, 48, 512):
        assert call(P=rows) == UNSUPPORTED, rows
    assert call(columns=1 << 23, P=256) == UNSUPPORTED
    for k in ("table", "lengths", "refs"):
        assert call(**{k: None}) == INVALID, k
        assert call(**{k: P(AT + 2)}) == MISALIGNED, k
    others = dict(fork=("src", "dst"), free=("rows",), grow=("add", "src", "dst"),
                  compact=("src", "dst"))[name]
    for k in others:
        assert call(**{k: None}) == INVALID, k
        assert call(**{k: P(AT + 2)}) == MISALIGNED, k
    if name in ("fork", "free"):
        assert call(count=-1) == INVALID
        assert call(count=0, **{k: None for k in others}) == OK
    else:
        need = lib.hytopk_page_workspace_size(100)
        assert need >= 400 and lib.hytopk_page_workspace_size(0) == 0
        assert call(wb=need - 1) == SMALL
        assert call(ws=None) == INVALID
        assert call(ws=P(AT + 64)) == MISALIGNED
    if name == "grow":
        assert call(B=0, table=None, lengths=None, add=None) == OK


def test_copy(lib):
    def copy(**kw):
        a = dict(kp=FAKE, ks=FAKE, vp=FAKE, vs=FAKE, N=100, bytes=4096, H=2, src=FAKE, dst=FAKE,
                 count=3) | kw
        return lib.hytopk_page_copy(a["kp"], a["ks"], a["vp"], a["vs"], a["N"], a["bytes"], a["H"],
                                    a["src"], a["dst"], a["count"], None, None)

    for kw in (dict(N=0), dict(H=0), dict(bytes=0), dict(bytes=-16), dict(count=-1)):
        assert copy(**kw) == INVALID, kw
    assert copy(bytes=4104) == UNSUPPORTED
    for k in ("kp", "ks", "src", "dst"):
        assert copy(**{k: None}) == INVALID, k
    assert copy(vp=None) == INVALID  # one without the other
    assert copy(vs=None) == INVALID
    for k in ("kp", "vp"):
        assert copy(**{k: P(AT + 8)}) == MISALIGNED, k
    for k in ("ks", "vs", "src", "dst"):
        assert copy(**{k: P(AT + 2)}) == MISALIGNED, k
    assert copy(count=0, kp=None, src=None) == OK


# ---- the Python module ------------------------------------------------------------------

PAGES = PRELUDE + """
@ctypes.CFUNCTYPE(ctypes.c_size_t, *([ctypes.c_void_p] * 4))
def size(*a):
    return 256


sizes = ctypes.cast(size, ctypes.c_void_p).value
hk._operators().init_pages(sizes, address, address, sizes, *[address] * 5)
i32, f32, e4m3 = (dict(dtype=t) for t in (torch.int32, torch.float32, torch.float8_e4m3fn))
N, P, H, d, B, columns, n = 10, 16, 2, 64, 3, 4, 7
pages, scale = Claims(N, P, H, d, **e4m3), Claims(N, H, **f32)
table, lengths, refs, cu = Claims(B, columns, **i32), Claims(B, **i32), Claims(N, **i32), Claims(B + 1, **i32)
x, q = Claims(n, H, d), Claims(n, 4 * H, d)
out, lse = Claims(n, 4 * H, d), Claims(n, 4 * H, **f32)
some, add = Claims(2, **i32), Claims(B, **i32)
kw = dict(stream=Stream())


def refused(f, *a, error=ValueError, **k):
    try:
        f(*a, **{**kw, **k})
    except error:
        assert not calls, calls
        return
    raise SystemExit(f"no {error}: {a} {k}")


def write(x=x, pages=pages, scale=scale, table=table, lengths=lengths, cu=cu, **k):
    return hk.page_write(x, pages, scale, table, lengths, cu, **{**kw, **k})


def attend(q=q, k=pages, v=pages, ks=scale, vs=scale, table=table, lengths=lengths, cu=cu, **o):
    return hk.attend_pages(q, k, v, ks, vs, table, lengths, cu, **{**kw, "out": out, "lse": lse, **o})
"""


def child(code, env=None):
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", PAGES + code], cwd=ROOT, text=True,
                       capture_output=True, timeout=300, env=env)
    assert r.returncode == 0, f"exit code {r.returncode}\n{r.stdout}\n{r.stderr}"


def test_module_refuses_shapes():
    hk.build()
    child("""
both = (ValueError, TypeError)
for f in (write, attend):
    for bad in (dict(table=Claims(B, **i32)), dict(table=Claims(B, columns, **f32)),
                dict(lengths=Claims(B + 1, **i32)), dict(lengths=Claims(B, dtype=torch.int64)),
                dict(cu=Claims(B, **i32)), dict(cu=Claims(B + 1, **f32)),
                dict(table=Claims(B, columns, device="cuda:0", **i32)),
                dict(lengths=Claims(B, device="cuda:0", **i32)),
                dict(cu=Claims(B + 1, device="cpu", **i32)), dict(table=3), dict(lengths=None)):
        refused(f, error=both, **bad)
for bad in (dict(x=Claims(n, d)), dict(x=Claims(n, H + 1, d)), dict(x=Claims(n, H, 2 * d)),
            dict(x=Claims(n, H, d, dtype=torch.float16)), dict(x=Claims(n, H, d, device="cuda:0")),
            dict(pages=Claims(N, P, H, d)), dict(pages=Claims(N, P, d, **e4m3)),
            dict(scale=Claims(N, **f32)), dict(scale=Claims(N, H)), dict(scale=Claims(N, H + 1, **f32)),
            dict(scale=None), dict(inv_freq=Claims(32, 2, **f32)), dict(inv_freq=Claims(32)),
            dict(inv_freq=Claims(32, **f32), positions=Claims(n + 1, **i32)),
            dict(positions=Claims(n, **i32))):
    refused(write, error=both, **bad)
for bad in (dict(q=Claims(n, d)), dict(q=Claims(n, 8, 2 * d)),
            dict(q=Claims(n, 8, d, **f32)), dict(v=Claims(N + 1, P, H, d, **e4m3)),
            dict(k=Claims(N, P, H, d)), dict(vs=Claims(N, H + 1, **f32)),
            dict(ks=None), dict(out=Claims(n, 8, d, **f32)), dict(out=Claims(n + 1, 8, d)),
            dict(lse=Claims(n, 8)), dict(lse=Claims(n, 7, **f32)),
            dict(out=Claims(n, 8, d, device="cuda:0"))):
    refused(attend, error=both, **bad)
pool = (table, lengths, refs)
for f, rest in ((hk.page_fork, (some, some)), (hk.page_free, (some,)), (hk.page_grow, (add,)),
                (hk.page_compact, ())):
    for i, bad in ((0, Claims(B, **i32)), (0, Claims(B, columns, **f32)), (1, Claims(B + 1, **i32)),
                   (1, Claims(B, **f32)), (2, Claims(N, 1, **i32)), (2, Claims(N, dtype=torch.int64)),
                   (2, Claims(N, device="cuda:0", **i32))):
        a = list(pool)
        a[i] = bad
        refused(f, *a, *rest, page=P, error=both)
refused(hk.page_fork, *pool, some, Claims(3, **i32), page=P, error=both)
refused(hk.page_fork, *pool, some, Claims(2, **f32), page=P, error=both)
refused(hk.page_free, *pool, Claims(2, 2, **i32), page=P, error=both)
refused(hk.page_grow, *pool, Claims(B + 1, **i32), page=P, error=both)
for bad in ((pages, Claims(N, P, H, 2 * d, **e4m3), scale, scale), (pages, pages, scale, None),
            (pages, None, scale, scale), (pages, pages, Claims(N, **f32), scale)):
    refused(hk.page_copy, *bad, some, some, error=both)
refused(hk.page_copy, pages, pages, scale, scale, some, Claims(3, **i32), error=both)
""")


def test_the_tensors_device_is_current_in_every_call(tmp_path):
    """Tensors on device 1 while device 0 is current: the library is called with device 1
    current, and device 0 is current afterwards, after refusals too."""
    hk.build()
    source, so = tmp_path / "runtime.c", tmp_path / "libcuda.so.1"
    source.write_text(FAKE_RUNTIME)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(so), str(source)], check=True)
    env = dict(os.environ, LD_PRELOAD=str(so), LD_LIBRARY_PATH=os.pathsep.join(
        [str(tmp_path)] + [p for p in (os.environ.get("LD_LIBRARY_PATH"),) if p]))
    child("""
runtime, status = ctypes.CDLL(None), 0


@ctypes.CFUNCTYPE(ctypes.c_int, *([ctypes.c_void_p] * 13))
def entry(*a):
    calls.append(runtime.current_device())
    return status


address = ctypes.cast(entry, ctypes.c_void_p).value
hk._operators().init_pages(sizes, address, address, sizes, *[address] * 5)
pool = (table, lengths, refs)
every = [lambda: write(stream=None), lambda: write(inv_freq=Claims(32, **f32), stream=None),
         lambda: hk.page_fork(*pool, some, some, page=P), lambda: hk.page_free(*pool, some, page=P),
         lambda: hk.page_copy(pages, pages, scale, scale, some, some),
         lambda: hk.page_copy(pages, None, scale, None, some, some, **kw), write,
         lambda: hk.page_fork(*pool, some, some, page=P, **kw)]
for status in (0, 1):
    for f in every:
        try:
            f()
            assert status == 0
        except hk.HytopkError:
            assert status == 1
        assert runtime.current_device() == 0
assert calls == [1] * (2 * len(every)), calls
""", env)


def test_tensors_without_memory_raise():
    """Inside a vmap a tensor has no pointer to give: an exception, at whichever argument."""
    hk.build()
    child("""
def vmapped(f, a):
    try:
        torch.func.vmap(f)(a)
    except RuntimeError:
        assert not calls
        return
    raise SystemExit("no exception")

vmapped(lambda b: write(x=b), Claims(3, n, H, d))
vmapped(lambda b: write(pages=b), Claims(3, N, P, H, d, **e4m3))
vmapped(lambda b: write(lengths=b), Claims(3, B, **i32))
vmapped(lambda b: attend(q=b), Claims(3, n, 4 * H, d))
vmapped(lambda b: attend(out=b), Claims(3, n, 4 * H, d))
vmapped(lambda b: attend(ks=b), Claims(3, N, H, **f32))
vmapped(lambda b: hk.page_free(b, lengths, refs, some, page=P, **kw), Claims(3, B, columns, **i32))
vmapped(lambda b: hk.page_copy(b, pages, scale, scale, some, some, **kw), Claims(3, N, P, H, d, **e4m3))
""")
