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


def calls_that_allocate(hk, dev):
    """name, call(**kw) -> tensors, for every entry point that makes its results."""
    import torch

    g = torch.Generator(device=dev).manual_seed(5)
    n, Hq, d, k, L = 64, 16, 128, 100, 300

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=g).bfloat16()

    q, kk, vv, grad = normal(n, Hq, d), normal(L, 1, d), normal(L, 1, d), normal(n, Hq, d)
    idx = torch.randint(0, L, (n, k), device=dev, generator=g, dtype=torch.int32)
    pos = torch.arange(n, device=dev, dtype=torch.int32)
    freq, _ = hk.rope_frequencies(64, device=dev)
    out, lse = hk.attend(q, kk, vv, idx, out_dtype=torch.float32)
    buf = torch.empty_like(q)
    # (additions in no order: gradients repeat only up to the last bits, so one head and one
    # query per row, where a row of dk or dv takes a single addition)
    own_rows = torch.arange(n, device=dev, dtype=torch.int32)[:, None].contiguous()
    out1, lse1 = hk.attend(q[:, :1], kk, vv, own_rows, out_dtype=torch.float32)
    grad1 = grad[:, :1].contiguous()
    torch.cuda.synchronize()
    return [
        ("rope", lambda **kw: (hk.rope(q, pos, freq, **kw),)),
        ("cache_read", lambda **kw: (hk.cache_read(kk, dtype=torch.float32, **kw),)),
        ("attend", lambda **kw: hk.attend(q, kk, vv, idx, **kw)),
        ("attend, out given", lambda **kw: hk.attend(q, kk, vv, idx, out=buf, **kw)[1:]),
        ("attend_backward", lambda **kw: hk.attend_backward(
            q[:, :1], kk, vv, own_rows, out1, lse1, grad1, **kw)),
    ]


def test_results_on_a_given_stream_take_none_of_the_callers_memory(hk, dev):
    """Blocks that were freed while the caller's stream still has to read them: a call on
    another stream, which waits for nothing, leaves them alone."""
    import torch

    side = torch.cuda.Stream()
    for name, call in calls_that_allocate(hk, dev):
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        for _ in range(3):
            old = [torch.full_like(t, 7.0) for t in want]
            where = {t.data_ptr() for t in old}
            torch.cuda.synchronize()
            torch.cuda._sleep(20_000_000)            # some 10 ms, then the reads
            kept = [t.clone() for t in old]
            del old
            got = call(stream=side)
            side.synchronize()
            assert not where & {t.data_ptr() for t in got}, name
            for a, b in zip(got, want):
                assert torch.equal(a, b), name
            torch.cuda.synchronize()
            assert all(bool((t == 7.0).all()) for t in kept), name


def test_results_of_a_given_stream_may_be_dropped_while_the_caller_reads_them(hk, dev):
    import torch

    side = torch.cuda.Stream()
    for name, call in calls_that_allocate(hk, dev):
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        got = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        where = {t.data_ptr() for t in got}
        torch.cuda._sleep(20_000_000)
        kept = [t.clone() for t in got]              # waits behind the sleep
        del got
        more = call(stream=side)
        with torch.cuda.stream(side):
            junk = [torch.full_like(t, 7.0) for t in want]
        assert not where & {t.data_ptr() for t in list(more) + junk}, name
        torch.cuda.synchronize()
        for a, b in zip(kept, want):
            assert torch.equal(a, b), name


def test_given_tensors_written_on_a_given_stream_may_be_dropped(hk, dev):
    """out=, dk= and dv= of the caller's memory stay taken until the given stream has written
    them."""
    import torch

    x = torch.randn(64, 16, 128, device=dev).bfloat16()
    pos = torch.arange(64, device=dev, dtype=torch.int32)
    freq, _ = hk.rope_frequencies(64, device=dev)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = torch.empty_like(x)
    at = out.data_ptr()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    hk.rope(x, pos, freq, out=out, stream=side)
    del out
    marks = torch.full_like(x, 7.0)
    assert marks.data_ptr() != at
    torch.cuda.synchronize()
    assert bool((marks == 7.0).all())


@pytest.mark.parametrize("n", [2, 40])
def test_calls_in_a_row_read_what_the_last_ones_wrote(hk, dev, n):
    """Queries, cache rows, scales, results and log-sum-exps in the same places step after
    step, each call launched while the ones before still run: the same bits as with a wait
    after every call."""
    import torch

    g = torch.Generator(device=dev).manual_seed(n)
    steps, d, L, k = 100, 128, 256, 6
    x = torch.randn(steps, n, 1, d, device=dev, generator=g).bfloat16()
    y = torch.randn(steps, n, 1, d, device=dev, generator=g).bfloat16()
    grad = torch.randn(steps, n, 1, d, device=dev, generator=g).bfloat16()
    # rows of its own for every query, so that a gradient's row takes one addition
    idx = torch.arange(n * k, device=dev, dtype=torch.int32).view(n, k)
    idx = idx if n * k <= L else (idx % L).contiguous()
    slots = torch.randperm(L, device=dev, generator=g)[:n].int()
    pos = torch.arange(n, device=dev, dtype=torch.int32)
    freq, _ = hk.rope_frequencies(64, device=dev)

    def run(wait):
        def now():
            if wait:
                torch.cuda.synchronize()

        codes = torch.zeros(L, 1, d, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
        scale = torch.ones(L, 1, device=dev)
        plain = torch.zeros(L, 1, d, device=dev, dtype=torch.bfloat16)
        q, out = torch.zeros_like(x[0]), torch.zeros(n, 1, d, device=dev)
        results = [torch.empty(steps, n, 1, d, device=dev) for _ in range(2)]
        kept = []
        torch.cuda.synchronize()
        for i in range(steps):
            hk.rope(x[i], pos, freq, out=q), now()
            hk.cache_write(y[i], codes, scale, slots=slots, positions=pos, inv_freq=freq), now()
            hk.cache_read(codes, scale, slots=slots, out=results[0][i]), now()
            hk.cache_write(x[i], plain, slots=slots), now()
            hk.attend(q, codes, codes, idx, k_scale=scale, v_scale=scale, out=results[1][i]), now()
            _, lse = hk.attend(q, plain, plain, idx, out=out)
            now()
            dq, dk, dv = hk.attend_backward(q, plain, plain, idx, out, lse, grad[i])
            now()
            kept.append((lse, dq, dk, dv) if n * k <= L else (lse, dq))
        torch.cuda.synchronize()
        return results + [t for one in kept for t in one]

    want = run(True)
    for _ in range(5):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)
