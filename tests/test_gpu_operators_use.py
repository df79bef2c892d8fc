"""GPU: the operators around a selection as programs use them: inside function transforms, on
streams of their own, one after another on the same memory."""
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


def test_inside_a_vmap_every_call_raises(hk, dev):
    """The tensors that a vmap hands on have no pointer; none of them reaches the library."""
    import torch

    x = torch.randn(3, 4, 2, 64, device=dev).bfloat16()
    pos = torch.zeros(4, dtype=torch.int32, device=dev)
    freq, _ = hk.rope_frequencies(64, device=dev)
    idx = torch.zeros(4, 3, dtype=torch.int32, device=dev)
    plain, out = x[0], torch.empty(4, 2, 64, device=dev, dtype=torch.bfloat16)
    for f in (lambda b: hk.rope(b, pos, freq), lambda b: hk.rope(b, pos, freq, out=out),
              lambda b: hk.rope(plain, pos, freq, out=b), lambda b: hk.cache_write(b, out),
              lambda b: hk.cache_write(plain, b), lambda b: hk.cache_read(b),
              lambda b: hk.attend(b, plain, plain, idx), lambda b: hk.attend(plain, b, b, idx),
              lambda b: hk.attend(plain, plain, plain, idx, out=b)):
        with pytest.raises(RuntimeError):
            torch.func.vmap(f)(x)
    assert torch.isfinite(hk.rope(plain, pos, freq).float()).all()
