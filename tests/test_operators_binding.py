"""The operators' Python module where it meets torch, without a GPU: tensors that only
claim a device, and a library whose entry points only count their calls."""
import os
import subprocess
import sys

import pytest

import exact_top_token_gb300 as hk

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# `Claims` says it is a tensor on a device and holds no memory; `calls` counts what reaches
# the library (its entry points are replaced).
PRELUDE = """
import ctypes
import torch
import exact_top_token_gb300 as hk


class Claims(torch.Tensor):
    @staticmethod
    def __new__(cls, *shape, dtype=torch.bfloat16, device="cuda:1"):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype,
                                                   device=torch.device(device))

    @classmethod
    def __torch_dispatch__(cls, f, types, args=(), kw=None):
        raise RuntimeError(f"dispatch of {f}")


class Stream:
    cuda_stream = 5


calls = []


@ctypes.CFUNCTYPE(ctypes.c_int, *([ctypes.c_void_p] * 13))
def entry(*a):
    calls.append(a)
    return 0


address = ctypes.cast(entry, ctypes.c_void_p).value
hk._operators().init(hk.HytopkError, torch.OutOfMemoryError, *[address] * 5)
x, out = Claims(4, 2, 64), Claims(4, 2, 64)
pos, freq = Claims(4, dtype=torch.int32), Claims(32, dtype=torch.float32)
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    hk.build()


def child(code, env=None):
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", PRELUDE + code], cwd=ROOT, text=True,
                       capture_output=True, timeout=300, env=env)
    assert r.returncode == 0, f"exit code {r.returncode}\n{r.stdout}\n{r.stderr}"
    return r.stdout


def test_tensors_without_memory_raise():
    """Inside a vmap a tensor has no pointer to give: an exception, at whichever argument."""
    child("""
def refused(f, *a):
    try:
        torch.func.vmap(f)(*a)
    except RuntimeError:
        return
    raise SystemExit("no exception")

many = Claims(3, 4, 2, 64)
refused(lambda b: hk.rope(b, pos, freq, out=out, stream=Stream()), many)
refused(lambda b: hk.rope(x, pos, freq, out=b, stream=Stream()), many)
refused(lambda b: hk.cache_write(x, b, positions=pos, inv_freq=freq, stream=Stream()), many)
refused(lambda b: hk.cache_write(b, x, positions=pos, inv_freq=freq, stream=Stream()), many)
assert not calls
""")


# Two devices that only remember which of them is current.
FAKE_RUNTIME = """
static int current = 0;
int cudaGetDeviceCount(int* n) { *n = 2; return 0; }
int cudaGetDevice(int* d) { *d = current; return 0; }
int cudaSetDevice(int d) { current = d; return 0; }
int cudaDeviceGetStreamPriorityRange(int* low, int* high) { *low = 0; *high = -5; return 0; }
int cuDevicePrimaryCtxGetState(int d, unsigned* flags, int* active) {
  *flags = 0;
  *active = 1;
  return 0;
}
int current_device(void) { return current; }
"""


def test_the_tensors_device_is_current_in_every_call(tmp_path):
    """Tensors on device 1 while device 0 is current: the library is called with device 1
    current, and device 0 is current afterwards, after refusals too."""
    source, lib = tmp_path / "runtime.c", tmp_path / "libcuda.so.1"
    source.write_text(FAKE_RUNTIME)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(lib), str(source)], check=True)
    env = dict(os.environ, LD_PRELOAD=str(lib), LD_LIBRARY_PATH=os.pathsep.join(
        [str(tmp_path)] + [p for p in (os.environ.get("LD_LIBRARY_PATH"),) if p]))
    got = child("""
runtime, seen, status = ctypes.CDLL(None), [], 0


@ctypes.CFUNCTYPE(ctypes.c_int, *([ctypes.c_void_p] * 13))
def entry(*a):
    seen.append(runtime.current_device())
    return status


address = ctypes.cast(entry, ctypes.c_void_p).value
hk._operators().init(hk.HytopkError, torch.OutOfMemoryError, *[address] * 5)
f32 = dict(dtype=torch.float32)
cache, scale = Claims(9, 2, 64, dtype=torch.float8_e4m3fn), Claims(9, 2, **f32)
idx, rows = Claims(4, 3, dtype=torch.int32), Claims(9, 2, 64)
for st in (None, Stream()):
    hk.cache_write(x, cache, scale, stream=st)
    if st is None:  # (a result is recorded with a stream given: not these tensors)
        hk.rope(x, pos, freq, out=x)
        hk.cache_read(cache, scale, out=rows, dtype=torch.bfloat16)
    assert runtime.current_device() == 0
    status = 1
    try:
        hk.cache_write(x, cache, scale, stream=st)
    except hk.HytopkError:
        pass
    status = 0
    assert runtime.current_device() == 0
assert set(seen) == {1}, seen
print(len(seen))
""", env)
    assert int(got) == 6
