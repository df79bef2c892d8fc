"""Attention over a cache in pages (GPU) at the edges of what its entry point takes, against the
formula in 64 bits with the bounds of tests/pages_oracle.py: contexts that begin with rows that
are not there, both kernels."""
import numpy as np
import pytest
import torch

import exact_top_token_gb300 as hk
import pages_oracle as po
from test_gpu_pages_attend import Case as AnyCase
from test_gpu_pages_attend import cuda
from test_gpu_pages_tokens import Case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    hk.build()


@pytest.mark.parametrize("d,P", [(64, 16), (64, 128), (128, 16), (128, 128)])
@pytest.mark.parametrize("gone", [128, 256, 384])
def test_contexts_whose_first_rows_are_not_there(gone, d, P):
    """Whole tiles of entries of -1 in front, and one in the middle: what follows them counts. So
    many contexts that a multiprocessor has several tiles of each."""
    g = np.random.default_rng(gone + P)
    lengths = [400, 9000, 385] + g.integers(500, 1000, 180).tolist()
    c = Case([(x, 1) for x in lengths], Hq=8, Hkv=2, d=d, P=P, seed=gone + P, single=True)
    c.table[1:, :gone // P] = -1
    c.table[0, 128 // P:256 // P] = -1
    out, lse = check(c)
    assert torch.isfinite(lse).all() and (out != 0).any(-1).all()
    e = AnyCase([(700, 40), (900, 1), (385, 385)], Hq=8, Hkv=2, d=d, P=P, seed=gone + P)
    e.table[:, :gone // P] = -1
    e.run()


@pytest.mark.parametrize("d", [64, 128])
def test_heads_whose_first_scores_are_minus_infinity(d):
    """Of heads on one cache head some have no score above -inf in the first two tiles, the
    others do."""
    g = np.random.default_rng(d)
    lengths = [2000] + g.integers(300, 900, 300).tolist()
    c = Case([(x, 1) for x in lengths], Hq=6, Hkv=1, d=d, P=16, seed=d, single=True)
    c.k &= 0x7F                                    # codes >= 0
    c.k[c.k == 0x7F] = 1
    c.k[:, :, :, 0] = 0x38
    c.q = (c.q.abs() * 2.0 ** -64).bfloat16()
    c.q[:, ::2] = -(2.0 ** 126)
    c.ks[:] = 2.0 ** -120
    c.ks[c.table[:, :16]] = 2.0 ** 60
    out, lse = check(c)
    assert torch.isfinite(lse).all() and (out[:, ::2] != 0).any(-1).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [(100, 128), (257, 384)])
def test_codes_of_nan_stay_in_their_sequences(lengths, d):
    """Single tokens that see a NaN code of v, of an odd number of tiles, between pieces of
    prompts of two blocks of rows, in no order, a dozen of both for each multiprocessor: NaN in
    the column of those tokens, and nowhere else."""
    g = np.random.default_rng(d)
    G, P, B, N = 32, 128, 1800, 8
    piece = g.random(B) < 0.4                          # (8 rows, twice those of a block)
    new = np.where(piece, 8, 1)
    length = np.where(piece, 300, g.integers(lengths[0], lengths[1] + 1, B))
    tile = (length[:, None] + P - 1) // P > np.arange(3)
    table = np.where(tile, g.integers(0, N, (B, 3)), -1)
    # the last page of a token's context has a NaN code in one column, a page for each column
    pages, last = N + d, (length - 1) // P
    column = g.integers(0, d, B)
    tokens = np.nonzero(~piece)[0]
    table[tokens, last[tokens]] = N + column[tokens]
    v = torch.full((pages, P, 1, d), 0x30, dtype=torch.uint8, device="cuda")
    at = torch.arange(d, device="cuda")
    v[N + at, 0, 0, at] = 0x7F
    k = torch.full_like(v, 0x31)
    q = torch.randn(int(new.sum()), G, d, device="cuda").bfloat16()
    one = torch.ones(pages, 1, device="cuda")
    cu = np.concatenate([[0], np.cumsum(new)])
    want = torch.zeros(int(new.sum()), G, d, dtype=torch.bool, device="cuda")
    want[cuda(cu[:-1][tokens], torch.int64), :, cuda(column[tokens], torch.int64)] = True
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(3):
        out, lse = hk.attend_pages(q, k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), one, one,
                                   cuda(table), cuda(length), cuda(cu), status=word)
        assert word.item() == 0
        assert torch.equal(torch.isnan(out), want)
        assert torch.isfinite(lse).all()


@pytest.mark.parametrize("rows", [1, 2])
def test_a_context_of_almost_2_31_rows(rows):
    """Of which only the last page is there; the row behind the context holds NaN codes."""
    P, d, columns = 16, 64, (1 << 27) - 1
    length = columns * P - 1
    table = torch.full((1, columns), -1, dtype=torch.int32, device="cuda")
    table[0, -1] = 2
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randint(0x20, 0x40, (4, P, 1, d), dtype=torch.uint8, device="cuda", generator=g)
    v = torch.randint(0x20, 0x40, (4, P, 1, d), dtype=torch.uint8, device="cuda", generator=g)
    k[:, 15] = v[:, 15] = 0x7F
    one = torch.ones(4, 1, device="cuda")
    q = torch.randn(rows, 4, d, device="cuda", generator=g).bfloat16()
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = None if rows == 1 else cuda([0, rows])
    out, lse = hk.attend_pages(q, k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), one, one,
                               table, cuda([length]), cu, status=word)
    assert word.item() == 0
    for i in range(rows):
        there = 15 - (rows - 1 - i)
        K, V = (t[2, :there, 0].view(torch.float8_e4m3fn).double() for t in (k, v))
        s = q[i].double() @ K.T / 8
        want = torch.softmax(s, -1) @ V
        # the result's rounding, f16 weights, and fp32 scores below 2^6
        assert ((out[i].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -10) * want.abs()).all()
        assert ((lse[i].double() - torch.logsumexp(s, -1)).abs() <= 2.0 ** -16).all()


# ---- scales of v far apart, scores far from 0 -------------------------------------------------

def tight(c, equal=False):
    """out, lse and bounds as tests/pages_oracle.py has them, but for weights that f16 holds as
    subnormal numbers: each is off by 2^-27 (twice rounded) of the largest weight times its scale of
    v, whatever the other scales are. `equal`: scores that matter are the same number, so that
    their rounding falls out of the weights."""
    q, k, v = c.q.double().numpy(), c.k, c.v
    n, Hq, d = q.shape
    G = Hq // c.Hkv
    out, lse = np.zeros((n, Hq, d)), np.full((n, Hq), -np.inf)
    t_out, t_lse = np.zeros((n, Hq, d)), np.zeros((n, Hq))
    for b, length in enumerate(c.lengths):
        lo, hi = (b, b + 1) if c.cu is None else (c.cu[b], c.cu[b + 1])
        K, sk, there = po.context(k, c.ks.astype(np.float64), c.table[b], length)
        V, sv, _ = po.context(v, c.vs.astype(np.float64), c.table[b], length)
        for t in range(lo, hi):
            rows = np.nonzero(there[:length - (hi - lo) + t - lo + 1])[0]
            for h in range(Hq):
                hk = h // G
                size = sk[rows, hk] * abs(c.scale)
                s = (K[rows, hk] @ q[t, h]) * sk[rows, hk] * c.scale
                top = s.max()
                e = np.exp(s - top)
                z = e.sum()
                val = V[rows, hk] * sv[rows, hk][:, None]
                o = e @ val / z
                delta = (d / 16 + 16) * po.U32 * ((np.abs(K[rows, hk]) @ np.abs(q[t, h])) * size).max() + \
                    2.0 ** -20 + 2.0 ** -21 * np.abs(s).max()
                out[t, h], lse[t, h] = o, top + np.log(z)
                share = 2.0 ** -20 if equal else 2 * delta
                small = (e / z * sv[rows, hk]).max()
                t_out[t, h] = (share + 2.0 ** -11 + (rows.size / 16 + 16) * po.U32) * (e / z @ np.abs(val)) + \
                    2.0 ** -27 * small * np.abs(V[rows, hk]).sum(0) + 2.0 ** -8 * np.abs(o)
                t_lse[t, h] = 2 * delta + 2.0 ** -21 * abs(lse[t, h])
    return out, lse, t_out, t_lse


def compare(c, equal=False, both=True):
    o, l, to, tl = tight(c, equal)
    a = c.device()
    runs = [a] if c.cu is not None or not both else [a, {**a, "cu_q": cuda(list(range(len(c.lengths) + 1)))}]
    for args in runs:
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = hk.attend_pages(scale=c.scale, status=word, **args)
        assert word.item() == 0
        po.check("lse", lse.double().cpu().numpy(), l, tl)
        po.check("out", out.double().cpu().numpy(), o, to)


# (more items than multiprocessors of several tiles each, or few that they share; pieces of prompts)
BATCHES = {"tokens": (Case, [(x, 1) for x in range(300, 460)], True),
           "token": (Case, [(9000, 1)], True),
           "pieces": (AnyCase, [(300, 40), (128, 128), (700, 3), (200, 1)], False)}


def make(batch, d, **kw):
    kind, seqs, single = BATCHES[batch]
    return kind(seqs, Hq=4, Hkv=2, d=d, single=single, seed=d, **kw)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("first,rest", [(-60, 60), (60, -60), (-115, 0), (0, -120), (-126, 118)])
def test_scales_of_v_that_change_after_a_tile(batch, first, rest, d):
    c = make(batch, d, P=128)
    c.v = (c.v & 0x80) | (c.v & 0x7F) % 0x39                # up to 1
    c.vs[:] = 2.0 ** rest
    c.vs[c.table[:, 0]] = np.float32(2.0 ** first * 1.5)
    compare(c)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("q_size,far", [(1.0, 60), (1.0, 120), (64.0, 60), (64.0, 120), (512.0, 120)])
def test_scales_of_v_in_no_order(batch, q_size, far, d):
    """Scores of large queries outweigh scales: rows of tiny values alone, and of huge ones."""
    c = make(batch, d, P=16, q_size=q_size)
    c.v = (c.v & 0x80) | (c.v & 0x7F) % 0x39
    c.vs = (2.0 ** np.random.default_rng(1).uniform(-far, far, c.vs.shape)).astype(np.float32)
    compare(c)


def test_rows_that_see_tiny_values_alone():
    """The first page of a prompt, beside pages of another size in the same tile."""
    for d in (64, 128):
        c = AnyCase([(200, 200), (40, 40)], Hq=4, Hkv=2, d=d, P=16, seed=5)
        c.v = (c.v & 0x80) | (c.v & 0x7F) % 0x39
        c.vs[:] = 1.0
        c.vs[c.table[:, 0]] = 2.0 ** -115
        compare(c)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("log2", [21, 25, 31, 60, -22, -40])
def test_scores_far_from_0_keep_the_scales_of_v(batch, log2, d):
    """All keys alike, so that every weight is the same, whatever the score is."""
    c = make(batch, d, P=64)
    c.k[:] = 0x38
    c.v = c.v & 0x7F
    c.v[c.v == 0x7F] = 0x38
    c.ks[:] = 2.0 ** -6
    c.q = (torch.sign(torch.tensor(float(log2))) * 2.0 ** (abs(log2) - np.log2(d) + 6) *
           torch.ones(c.q.shape)).bfloat16()
    c.scale = 0.7
    compare(c, equal=True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("page", [0, 3, 5, 11])
def test_scores_that_jump(batch, page, d):
    """Two neighbouring pages whose scores lie 2^24 above all others, or below for other heads."""
    c = make(batch, d, P=16)
    c.k[:] = 0x38
    c.v = c.v & 0x7F
    c.v[c.v == 0x7F] = 0x38
    c.ks[:] = 2.0 ** -20
    c.ks[c.table[:, page:page + 2]] = 2.0 ** 18
    c.q[:] = 1.0
    c.q[:, ::2] = -1.0
    compare(c, equal=True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rise", [20, 32])
def test_weights_of_a_tile_whose_reference_rises(rise, d):
    """Keys 2^6.5 times an earlier tile's, then some 2^rise times as heavy in the same tile: what the
    former add to a column that the latter lack. So many items that shares hold whole ones."""
    B, P = 120, 64
    c = AnyCase([(512, 5)] * B, Hq=32, Hkv=1, d=d, P=P, seed=d)
    c.k[:] = 0x38
    c.v[:] = 0
    c.v[..., 1] = 0x38
    c.ks[:] = 2.0 ** -10
    c.vs[:] = 1.0
    c.q[:] = 1.0
    c.scale = float(np.log(2)) / d                 # scores in powers of two: the page's scale of k
    c.ks[c.table[:, 4]], c.ks[c.table[:, 5]] = 6.5, rise
    c.v[c.table[:, 4], :, :, 0] = 0x38
    compare(c)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("log2", [10, 12, 15, 18.3, 19.7, -18.5, -13])
def test_scores_of_middling_size_keep_the_scales_of_v(batch, log2, d):
    """As above: contexts of two pages, the second of whose scales, as a power of two, lies almost half
    a step from any fp32 number of the scores' size."""
    kind, seqs, single = BATCHES[batch]
    seqs = [(128, min(m, 128)) for _, m in seqs]
    c = kind(seqs, Hq=4, Hkv=2, d=d, P=64, seed=d, single=single)
    c.k[:] = 0x38
    c.v[:] = 0x38
    c.ks[:] = 1.0
    c.vs[:] = 1.0
    step = 2.0 ** (np.floor(abs(log2)) - 23)       # of fp32 there
    c.vs[c.table[:, 1]] = np.float32(2.0 ** (-8 + 0.47 * step))
    c.v[c.table[:, 0]] = 0
    c.q[:] = 1.0 if log2 > 0 else -1.0
    c.scale = float(2.0 ** abs(log2) * np.log(2) / d)
    compare(c, equal=True)


@pytest.mark.parametrize("batch", BATCHES)
def test_queries_that_are_not_finite(batch):
    """NaN for their heads, and nothing else for the others of the group."""
    for value in (float("nan"), float("inf"), -float("inf")):
        c = make(batch, 64, P=32)
        o, l, to, tl = tight(c)
        c.q[:, 1, 5] = value
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = hk.attend_pages(scale=c.scale, status=word, **c.device())
        assert word.item() == 0
        # (a score of +inf or NaN makes the row NaN; the first rows of a prompt may only have -inf)
        hurt = torch.isnan(lse[:, 1])
        assert hurt[-1] and hurt.float().mean() > 0.8 and torch.isnan(out[:, 1][hurt]).all()
        assert (out[:, 1][~hurt] == 0).all() and (lse[:, 1][~hurt] == -float("inf")).all()
        for h in (0, 2, 3):
            po.check("lse", lse[:, h].double().cpu().numpy(), l[:, h], tl[:, h])
            po.check("out", out[:, h].double().cpu().numpy(), o[:, h], to[:, h])
