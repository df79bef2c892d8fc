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


def child(code):
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", PRELUDE + code], cwd=ROOT, text=True,
                       capture_output=True, timeout=300)
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
