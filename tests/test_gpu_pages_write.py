"""Rows written into pages (GPU): codes and page scales against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import exact_top_token_gb300 as hk
import pages_oracle as po

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    hk.build()


def cuda(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda()


class Case:
    def __init__(self, seqs, H=2, d=64, P=16, seed=0, dtype=torch.bfloat16, single=False, size=1.0):
        g = np.random.default_rng(seed)
        self.H, self.d, self.P = H, d, P
        self.lengths = [s[0] for s in seqs]
        new = [s[1] for s in seqs]
        self.cu = None if single else np.concatenate([[0], np.cumsum(new)]).tolist()
        n = sum(new)
        held = [po.pages_of(x, P) for x in self.lengths]
        N = sum(held) + 2
        order = g.permutation(N)
        self.table = np.full((len(seqs), max(held + [1])), -1, dtype=np.int64)
        at = 0
        for b, k in enumerate(held):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.codes = (g.integers(0, 0x7F, (N, P, H, d)) | (g.integers(0, 2, (N, P, H, d)) << 7)).astype(np.uint8)
        # of old pages some scales are larger than the new rows need, some smaller
        self.scale = (2.0 ** g.uniform(-14, 2, (N, H))).astype(np.float32)
        self.x = (torch.from_numpy(g.standard_normal((n, H, d)) * size)).to(dtype)
        self.first_new = [b_len - m for b_len, m in zip(self.lengths, new)]

    def offsets(self):
        return list(range(len(self.lengths) + 1)) if self.cu is None else self.cu

    def expected(self, y):
        """codes before rounding [N, P, H, d] (NaN: a code as it was), scales; y: the rows rotated"""
        want = np.full(self.codes.shape, np.nan)
        scale = self.scale.astype(np.float64)
        cu = self.offsets()
        for b, length in enumerate(self.lengths):
            lo, hi = cu[b], cu[b + 1]
            start = max(length - (hi - lo), 0)
            if hi == lo or length <= start:
                continue
            for column in range(start // self.P, po.pages_of(length, self.P)):
                page = self.table[b, column]
                if not 0 <= page < len(self.codes):
                    continue
                first, end = max(start, column * self.P), min(length, (column + 1) * self.P)
                part = y[hi - length + first:hi - length + end]
                amax = np.abs(part).max((0, 2))
                fresh = np.where(amax > 0, np.maximum(amax / 448.0, 2.0 ** -126), 0.0)
                kept = first - column * self.P
                new = np.maximum(fresh, scale[page]) if kept else fresh
                new = np.where(new > 0, new, 1.0)
                if kept:
                    old = po.VALUES[self.codes[page, :kept]] * (scale[page] / new)[:, None]
                    grew = new > scale[page]
                    want[page, :kept][:, grew] = old[:, grew]
                want[page, kept:kept + end - first] = part / new[:, None]
                scale[page] = new
        return want, scale

    def run(self, y=None, tol_y=0.0, status=0, **kw):
        pages, scale = cuda(self.codes, torch.uint8).view(E4M3), cuda(self.scale, torch.float32)
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        args = dict(x=self.x.cuda(), table=cuda(self.table), lengths=cuda(self.lengths),
                    cu_q=None if self.cu is None else cuda(self.cu))
        args.update(kw)
        got = hk.page_write(args.pop("x"), pages, scale, args.pop("table"), args.pop("lengths"),
                            args.pop("cu_q"), status=word, **args)
        assert got is pages
        torch.cuda.synchronize()
        assert word.item() == status
        self.compare(pages, scale, self.x.double().numpy() if y is None else y, tol_y)

    def compare(self, pages, scale, y, tol_y=0.0):
        want, s = self.expected(y)
        got_s = scale.double().cpu().numpy()
        # amax / 448 rounded once; of rotated rows amax is off by tol_y
        assert (np.abs(got_s - s) <= s * 2.0 ** -24 + tol_y / 448.0).all()
        codes = pages.view(torch.uint8).cpu().numpy()
        kept = np.isnan(want)
        assert np.array_equal(codes[kept], self.codes[kept])
        value = po.VALUES[codes[~kept]]
        want = want[~kept]
        # half a step of e4m3 (2^-4 of the value, 2^-10 below 2^-6), and what the scale and the
        # quotient are off by (three roundings of fp32)
        where = np.broadcast_to((tol_y / s)[:, None, :, None], codes.shape)[~kept]
        tol = np.maximum(np.abs(want) * 2.0 ** -4, 2.0 ** -10) + np.abs(want) * 2.0 ** -21 + 2 * where
        assert (np.abs(value - want) <= tol).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_at_page_ends(d, P, dtype):
    Case([(1, 1), (P, 1), (P, P), (P + 1, 1), (P + 1, 2), (2 * P + 3, P + 5), (0, 0), (5, 3),
          (3 * P, 2 * P)], H=3, d=d, P=P, seed=P + d, dtype=dtype).run()


@pytest.mark.parametrize("H", [1, 5, 8, 17])
def test_heads(H):
    Case([(100, 7), (40, 40), (300, 130)], H=H, d=128, P=32, seed=H).run()


def test_single_rows():
    Case([(x, 1) for x in (1, 15, 16, 17, 200, 31)], H=8, d=128, P=16, seed=3, single=True).run()


def test_many_sequences():
    g = np.random.default_rng(1)
    Case([(int(x), int(min(x, g.integers(0, 5)))) for x in g.integers(0, 90, 700)], H=2, d=64, P=16,
         seed=4).run()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("first,rot", [(0, 64), (64, 64), (0, 128), (8, 48)])
@pytest.mark.parametrize("given", [False, True])
def test_rotation(interleaved, first, rot, given):
    c = Case([(130, 70), (64, 1), (33, 33)], H=3, d=128, P=64, seed=rot + first)
    freq, m = hk.rope_frequencies(rot, factor=4.0, original_context=4096, scaling="parts")
    cu = c.offsets()
    pos = np.concatenate([np.arange(l - (cu[b + 1] - cu[b]), l) for b, l in enumerate(c.lengths)])
    kw = dict(inv_freq=freq, first=first, interleaved=interleaved, mscale=m)
    if given:
        pos = np.random.default_rng(2).integers(0, 1 << 20, len(pos))
        kw["positions"] = cuda(pos)
    x = c.x.double().numpy()
    a = pos[:, None, None] * freq.double().cpu().numpy()
    i = np.arange(rot // 2)
    p, q = (first + 2 * i, first + 2 * i + 1) if interleaved else (first + i, first + i + rot // 2)
    y = x.copy()
    y[..., p] = m * (x[..., p] * np.cos(a) - x[..., q] * np.sin(a))
    y[..., q] = m * (x[..., p] * np.sin(a) + x[..., q] * np.cos(a))
    # cos and sin are off by 1.3 x 2^-24, and three roundings of fp32
    c.run(y, tol_y=6 * 2.0 ** -24 * m * 2 * np.abs(x).max(), **kw)


def test_zeros_and_tiny_rows():
    c = Case([(20, 20), (40, 30), (17, 1)], H=2, d=64, P=16, seed=5, dtype=torch.float32)
    c.x[:, 0] = 0.0
    c.x[:, 1] *= 2.0 ** -130
    c.run()


def test_values_that_are_not_finite():
    c = Case([(40, 40), (20, 4)], H=2, d=64, P=16, seed=6, dtype=torch.float32)
    c.x[3, 0, 5], c.x[20, 1, 7], c.x[42, 1, 0] = float("nan"), float("inf"), -float("inf")
    y = c.x.double().numpy().copy()
    odd = ~np.isfinite(y)
    y[odd] = 0.0
    pages, scale = cuda(c.codes, torch.uint8).view(E4M3), cuda(c.scale, torch.float32)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    hk.page_write(c.x.cuda(), pages, scale, cuda(c.table), cuda(c.lengths), cuda(c.cu), status=word)
    assert word.item() == hk.DEV_NONFINITE
    codes = pages.view(torch.uint8)
    for b, j, h, e in ((0, 3, 0, 5), (0, 20, 1, 7), (1, 18, 1, 0)):
        at = (c.table[b, j // 16], j % 16, h, e)
        assert codes[at].item() & 0x7F == 0x7F
        codes[at] = 0
    c.compare(codes.view(E4M3), scale, y)


def test_old_scales_that_are_no_scales():
    for value in (0.0, -1.0, float("nan"), float("inf")):
        c = Case([(20, 4), (40, 2)], H=2, d=64, P=16, seed=7)
        page = c.table[0, 1 if 16 <= 16 else 0]            # rows 16 .. 19: all new
        c.scale[page, 0] = value
        c.run(y=c.x.double().numpy())                      # no earlier rows: not looked at
        c = Case([(20, 2), (40, 2)], H=2, d=64, P=16, seed=7)
        page = c.table[0, 1]                               # rows 16, 17 earlier
        c.scale[page, 0] = value
        pages, scale = cuda(c.codes, torch.uint8).view(E4M3), cuda(c.scale, torch.float32)
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        hk.page_write(c.x.cuda(), pages, scale, cuda(c.table), cuda(c.lengths), cuda(c.cu), status=word)
        assert word.item() == hk.DEV_BAD_SCALE
        codes = pages.view(torch.uint8).cpu().numpy()
        assert (codes[page, :2, 0] & 0x7F == 0x7F).all()
        x = c.x.double().numpy()[:2, 0]
        want = np.abs(x).max() / 448.0
        assert abs(scale[page, 0].item() - want) <= want * 2.0 ** -24
        assert np.array_equal(codes[page, 4:], c.codes[page, 4:])


def test_rows_that_have_no_page():
    c = Case([(40, 40), (20, 4), (64, 1)], H=2, d=64, P=16, seed=8)
    c.table[0, 1] = -1
    c.run()
    c.table[1, 1] = 10 ** 6
    c.table[2, 3] = -9
    c.run(status=hk.DEV_BAD_INDEX)


def test_more_rows_than_context_and_padding():
    c = Case([(40, 40), (20, 4)], H=2, d=64, P=16, seed=9)
    c.lengths = [30, 20]                                   # the first 10 rows are before it
    c.run()
    c = Case([(40, 40), (20, 4)], H=2, d=64, P=16, seed=9)
    c.x = torch.cat([c.x, torch.full((5, 2, 64), float("nan")).bfloat16()])
    c.run()


def test_offsets_and_lengths_out_of_range():
    c = Case([(40, 10), (48, 4)], H=2, d=64, P=16, seed=10)
    c.run(lengths=cuda([40, 10 ** 9]), status=hk.DEV_BAD_POSITION)
    pages, scale = cuda(c.codes, torch.uint8).view(E4M3), cuda(c.scale, torch.float32)
    for cu, lengths in (([0, 10, 99], [40, 48]), ([-3, 10, 14], [40, 48]), ([0, 12, 10], [40, 48]),
                        ([0, 10, 14], [-1, 48])):
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        hk.page_write(c.x.cuda(), pages, scale, cuda(c.table), cuda(lengths), cuda(cu), status=word)
        assert word.item() == hk.DEV_BAD_POSITION


def test_bad_positions_of_rows():
    c = Case([(20, 20)], H=1, d=64, P=16, seed=11)
    freq, _ = hk.rope_frequencies(32)
    pos = np.arange(20)
    pos[4] = 1 << 24
    pages, scale = cuda(c.codes, torch.uint8).view(E4M3), cuda(c.scale, torch.float32)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    hk.page_write(c.x.cuda(), pages, scale, cuda(c.table), cuda(c.lengths), cuda(c.cu), inv_freq=freq,
                  positions=cuda(pos), status=word)
    assert word.item() == hk.DEV_BAD_POSITION | hk.DEV_NONFINITE
    codes = pages.view(torch.uint8)[c.table[0, 0], 4, 0]
    assert (codes[:32] & 0x7F == 0x7F).all() and not (codes[32:] & 0x7F == 0x7F).any()


def test_strided_rows():
    c = Case([(130, 70), (64, 1)], H=3, d=64, P=32, seed=12)
    wide = torch.randn(71, 2, 5, 64, device="cuda").bfloat16()
    wide[:, 1, 1:4] = c.x.cuda()
    c.run(x=wide[:, 1, 1:4])


def test_appended_row_by_row():
    """A context written token by token: what comes back is within the roundings of every
    requantisation of its page."""
    P, H, d, L = 32, 2, 64, 70
    x = torch.randn(L, H, d, device="cuda") * torch.linspace(0.1, 3.0, L, device="cuda")[:, None, None]
    pages = torch.zeros(5, P, H, d, dtype=torch.uint8, device="cuda").view(E4M3)
    scale = torch.zeros(5, H, device="cuda")
    table = cuda([[4, 0, 2]])
    for t in range(L):
        hk.page_write(x[t:t + 1], pages, scale, table, cuda([t + 1]))
    got = (pages.float() * scale[:, None, :, None])[[4, 0, 2]].flatten(0, 1)[:L]
    # every rounding: half a step of the value it has, and at most P of them a page; the largest
    # of a page bounds a step below the normal range
    top = scale[[4, 0, 2]].repeat_interleave(P, 0)[:L, :, None]
    assert ((got - x).abs() <= P * (x.abs() * 2.0 ** -4 + top * 2.0 ** -10) * 2).all()
    assert ((got - x).abs().mean() / x.abs().mean()) < 2.0 ** -3


def test_graph_and_streams():
    c = Case([(100, 1), (64, 1), (17, 1)], H=4, d=128, P=16, seed=13, single=True)
    args = [c.x.cuda(), cuda(c.codes, torch.uint8).view(E4M3), cuda(c.scale, torch.float32),
            cuda(c.table), cuda(c.lengths)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    hk.page_write(*args, stream=s)
    s.synchronize()
    c.compare(args[1], args[2], c.x.double().numpy())
    args[1].view(torch.uint8).copy_(cuda(c.codes, torch.uint8))
    args[2].copy_(cuda(c.scale, torch.float32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hk.page_write(*args)
    graph.replay()
    torch.cuda.synchronize()
    c.compare(args[1], args[2], c.x.double().numpy())
