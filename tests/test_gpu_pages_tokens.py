"""Attention over a cache in pages, one new row for each sequence and no cu_q (GPU): against the
formula in 64 bits with the bounds of tests/pages_oracle.py, and what a cu_q of one row each
gives."""
import numpy as np
import pytest
import torch

import exact_top_token_gb300 as hk
from test_gpu_pages_attend import Case as AnyCase
from test_gpu_pages_attend import cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    hk.build()


class Case(AnyCase):
    """With a table so wide that contexts may be long: calls of no more rows than sequences have a
    kernel of their own then (of at most 16 heads on a cache head)."""

    def __init__(self, seqs, Hkv=2, P=16, columns=None, **kw):
        held = max([-(-s[0] // P) for s in seqs] + [1]) + 1
        wide = 2600 * 128 // (len(seqs) * Hkv * P) + 1
        super().__init__(seqs, Hkv=Hkv, P=P, columns=max(columns or 0, held, wide), **kw)


def tokens(lengths, both=True, status=0, **kw):
    """The case run with no cu_q, and with one row a sequence told by a cu_q"""
    c = Case([(x, 1) for x in lengths], single=True, **kw)
    return c, check(c, both, status)


def check(c, both=True, status=0):
    got = c.run(status=status)
    if both:
        c.run(status=status, cu_q=cuda(list(range(len(c.lengths) + 1))))
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (16, 1), (17, 1), (33, 1), (128, 2), (65, 1)])
def test_heads_of_a_group(Hq, Hkv, d):
    tokens([300, 1, 129, 256], Hq=Hq, Hkv=Hkv, d=d, P=32, seed=Hq + d)


@pytest.mark.parametrize("d,P,G", [(64, 16, 4), (64, 128, 40), (128, 64, 8), (128, 256, 64), (128, 16, 1)])
def test_ragged_batches(d, P, G):
    g = np.random.default_rng(d + P)
    lengths = [int(2 ** g.uniform(0, 11)) for _ in range(70)]
    tokens(lengths, Hq=2 * G, Hkv=2, d=d, P=P, seed=G)


@pytest.mark.parametrize("length,G", [(40000, 8), (30000, 16), (25000, 64)])
def test_a_context_that_all_share(length, G):
    tokens([length], Hq=G, Hkv=1, d=128, P=64, seed=G)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cu", [False, True])
def test_runs_of_idle_sequences(cu, d):
    """Many sequences without a context between long ones: a share holds dozens of them."""
    lengths = [9000] + [0] * 300 + [6000, 5] + [0] * 41 + [8000] + [0] * 9
    c = Case([(x, 1) for x in lengths], Hq=16, Hkv=8, d=d, P=64, seed=d, single=True)
    kw = dict(cu_q=cuda(list(range(len(lengths) + 1)))) if cu else {}
    out, lse = c.run(**kw)
    idle = torch.tensor([x == 0 for x in lengths], device="cuda")
    assert (out[idle] == 0).all() and (lse[idle] == -float("inf")).all()


def test_runs_of_rows_before_their_contexts():
    """Prompts' pieces whose rows lie before their contexts, whole blocks of them."""
    seqs = [(700, 3)] + [(0, 200)] * 60 + [(300, 1)] + [(3, 150)] * 20
    Case(seqs, Hq=4, Hkv=2, d=64, P=16, seed=3).run()


def test_one_tile_each():
    """Segments of a single tile, one after another in every share."""
    tokens([int(x) for x in np.random.default_rng(1).integers(1, 129, 1000)], Hq=8, Hkv=4, d=64,
           P=16, seed=2)


@pytest.mark.parametrize("G", [13, 24])
def test_weights_that_grow(G):
    """Scores that rise through a context, so that references are raised in later tiles, by rows
    of their own, and fall in others."""
    for d in (64, 128):
        c = Case([(1500, 1), (900, 1)], Hq=G, Hkv=1, d=d, P=16, seed=4, single=True)
        c.k = (c.k & 0x87) | 0x38                              # 1 .. 1.875, of either sign
        c.q[:, 0] = torch.sign(c.q[:, 0].float()).bfloat16()
        for b in range(2):
            for j in range((c.lengths[b] + 15) // 16):
                c.ks[c.table[b, j]] = 0.02 * (j + 1)
        c.k[..., 0] = 0x38 + 4                                  # one column for the trend
        c.q[..., 0] = torch.linspace(-30, 30, G).bfloat16()
        check(c)


@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -30, 16.0, 2.0 ** 22, 2.0 ** 100])
def test_sizes_of_queries(size):
    tokens([300, 90, 500], Hq=4, Hkv=2, d=128, P=32, seed=4, q_size=size)


@pytest.mark.parametrize("scale", [0.0, -0.125, 2.0, -3.0])
def test_scale_of_either_sign(scale):
    c = Case([(300, 1), (90, 1)], Hq=15, Hkv=1, seed=3, single=True)
    c.scale = scale
    check(c)


def test_scales_far_apart():
    c = Case([(700, 1), (300, 1)], Hq=8, Hkv=2, d=128, P=16, seed=1, spread=18.0, single=True)
    c.ks = (c.ks * 0 + 2.0 ** -6).astype(np.float32)
    check(c)
    c = Case([(700, 1), (300, 1)], Hq=8, Hkv=2, d=64, P=16, seed=2, spread=3.0, single=True)
    c.vs[::2] *= np.float32(2.0 ** 60)
    c.vs[1::2] *= np.float32(2.0 ** -60)
    check(c)


def test_scores_of_minus_infinity_weigh_nothing():
    c = Case([(260, 1), (140, 1)], Hq=2, Hkv=2, d=64, P=16, seed=7, single=True)
    c.k &= 0x7F                                    # codes >= 0
    c.k[c.k == 0x7F] = 1
    c.k[:, :, :, 0] = 0x38
    c.q[:] = -(2.0 ** 126)
    c.ks[:] = 2.0 ** -120
    big = c.table[0, [0, 3, 9]].tolist() + c.table[1, :9].tolist()
    c.ks[big] = 2.0 ** 60                          # all of sequence 1's rows score -inf
    out, lse = check(c)
    assert torch.isinf(lse[1]).all() and (out[1] == 0).all()


def test_codes_of_nan():
    """In a visible key: NaN for the heads that read it; in a visible row of v: in its column."""
    c = Case([(200, 1), (137, 1), (400, 1)], Hq=6, Hkv=2, d=64, P=32, seed=8, single=True)
    c.v[c.table[0, 3], 7, 1, 5] = 0xFF
    c.k[c.table[1, 136 // 32], 136 % 32, 0, 1] = 0x7F
    out, lse = check(c)
    assert torch.isnan(out[0, 3:, 5]).all() and torch.isnan(out[1, :3]).all()
    assert torch.isnan(out).sum() == 3 + 3 * 64 and torch.isnan(lse).sum() == 3


def test_entries_and_scales_that_are_none():
    c = Case([(300, 1), (290, 1), (100, 1), (500, 1)], Hq=4, Hkv=2, d=128, P=16, seed=11, single=True)
    c.table[0, [0, 5, 18]] = -1
    c.table[1, :] = -1
    check(c)
    c.table[2, [1, 6]] = [10 ** 6, -7]
    check(c, status=hk.DEV_BAD_INDEX)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = c.device()
    a["k_scale"][c.table[3, 20], 0] = float("nan")
    a["v_scale"][c.table[3, 2], 1] = -1.0
    a["table"][2, [1, 6]] = -1
    out, lse = hk.attend_pages(scale=c.scale, status=word, **a)
    assert word.item() == hk.DEV_BAD_SCALE
    assert torch.isnan(out[3]).all() and not torch.isnan(out[:3]).any()


def test_lengths_out_of_range():
    c = Case([(40, 1), (64, 1)], Hq=4, Hkv=2, d=64, P=16, seed=14, single=True)
    c.lengths[1] = c.table.shape[1] * 16                   # (most of its entries are -1)
    a = c.device()
    for given, rows in (([40, 10 ** 9], slice(None)), ([-3, c.lengths[1]], slice(1, None))):
        a["lengths"] = cuda(given)
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = hk.attend_pages(scale=c.scale, status=word, **a)
        assert word.item() == hk.DEV_BAD_POSITION
        c.compare(out, lse, rows)
    assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()


def test_strided_queries_given_results_and_same_bits():
    c = Case([(5000, 1), (90, 1), (0, 1)], Hq=8, Hkv=2, d=64, P=32, seed=15, single=True)
    wide = torch.randn(3, 3, 8, 64, device="cuda").bfloat16()
    wide[:, 1] = c.q.cuda()
    a = c.device()
    a["q"] = wide[:, 1]
    out = torch.full((3, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, 8), 7.0, device="cuda")
    got = hk.attend_pages(scale=c.scale, out=out, lse=lse, **a)
    assert got[0] is out and got[1] is lse
    c.compare(out, lse)
    for _ in range(5):
        again = hk.attend_pages(scale=c.scale, **a)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_two_streams_and_graphs():
    """Calls at once on two streams, and two captured ones, replayed with other lengths."""
    c = Case([(5000, 1), (700, 1), (64, 1)], Hq=8, Hkv=2, d=128, P=64, seed=19, single=True)
    e = Case([(900, 1), (3000, 1)], Hq=16, Hkv=1, d=64, P=32, seed=20, single=True)
    a, b = c.device(), e.device()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        got.append((hk.attend_pages(stream=s1, **a), hk.attend_pages(stream=s2, **b)))
    torch.cuda.synchronize()
    for x, y in got:
        c.compare(*x)
        e.compare(*y)
    graphs = []
    for args in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            result = hk.attend_pages(**args)
        graphs.append((graph, result))
    a["lengths"].copy_(cuda([4999, 0, 1]))
    c.lengths = [4999, 0, 1]
    for _ in range(2):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    c.compare(*graphs[0][1])
    e.compare(*graphs[1][1])


@pytest.mark.parametrize("new", [[3, 0, 1, 0, 0, 1], [0, 0, 0, 0, 0, 6], [1, 1, 1, 1, 2, 0], [1] * 6,
                                 [0, 1, 0, 1, 0, 0], [0] * 6])
@pytest.mark.parametrize("d", [64, 128])
def test_no_more_rows_than_sequences(d, new):
    """A cu_q of one row a sequence, or of several of some and none of others; rows of no sequence
    behind them are left."""
    lengths = [3000, 40, 700, 129, 1, 2600]
    c = Case([(x, m) for x, m in zip(lengths, new)], Hq=12, Hkv=4, d=d, P=32, seed=d)
    n = sum(new)
    c.q = torch.cat([c.q, torch.full((6 - n, 12, d), float("nan")).bfloat16()])
    out = torch.full((6, 12, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((6, 12), 7.0, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    hk.attend_pages(scale=c.scale, out=out, lse=lse, status=word, **c.device())
    assert word.item() == 0
    if n:
        c.compare(out, lse, slice(0, n))
    assert (out[n:] == 7.0).all() and (lse[n:] == 7.0).all()


def test_a_graph_whose_rows_change():
    """One captured call whose cu_q tells single rows, then several, then single ones again."""
    c = Case([(900, 1), (3000, 1), (64, 1), (200, 1)], Hq=8, Hkv=2, d=128, P=64, seed=23, single=True)
    a = c.device()
    a["cu_q"] = cuda([0, 1, 2, 3, 4])
    graph = torch.cuda.CUDAGraph()
    hk.attend_pages(scale=c.scale, **a)
    with torch.cuda.graph(graph):
        out, lse = hk.attend_pages(scale=c.scale, **a)
    for cu in ([0, 1, 2, 3, 4], [0, 0, 3, 3, 4], [0, 1, 2, 3, 4], [0, 1, 1, 1, 4]):
        a["cu_q"].copy_(cuda(cu))
        c.cu = cu
        graph.replay()
        torch.cuda.synchronize()
        c.compare(out, lse)
