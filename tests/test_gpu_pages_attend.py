"""Attention over a cache in pages (GPU) against the formula in 64 bits, with bounds derived from
the arithmetic (tests/pages_oracle.py)."""
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
    """Sequences (context length, new rows) with pages in random places of a pool; codes of pages
    that nobody holds, and of rows past the contexts, are NaN."""

    def __init__(self, seqs, Hq=4, Hkv=2, d=64, P=16, seed=0, single=False, q_size=1.0, spread=1.0,
                 columns=None):
        g = np.random.default_rng(seed)
        self.Hq, self.Hkv, self.d, self.P = Hq, Hkv, d, P
        self.lengths = [s[0] for s in seqs]
        self.cu = None if single else np.concatenate([[0], np.cumsum([s[1] for s in seqs])]).tolist()
        n = len(seqs) if single else self.cu[-1]
        held = [po.pages_of(x, P) for x in self.lengths]
        N = sum(held) + 3
        order = g.permutation(N)
        columns = columns or max(held + [1]) + 1
        self.table = np.full((len(seqs), columns), -1, dtype=np.int64)
        self.k = np.full((N, P, Hkv, d), 0x7F, dtype=np.uint8)
        self.v = self.k.copy()
        at = 0
        for b, k in enumerate(held):
            self.table[b, :k] = order[at:at + k]
            for j in range(k):
                rows = min(P, self.lengths[b] - j * P)
                for t in (self.k, self.v):
                    c = g.integers(0, 0x70, (rows, Hkv, d)) | (g.integers(0, 2, (rows, Hkv, d)) << 7)
                    t[order[at + j], :rows] = c
            at += k
        self.ks = (2.0 ** g.uniform(-spread, spread, (N, Hkv)) / 64).astype(np.float32)
        self.vs = (2.0 ** g.uniform(-spread, spread, (N, Hkv)) / 64).astype(np.float32)
        self.q = (torch.from_numpy(g.standard_normal((n, Hq, d))) * q_size / 8).bfloat16()
        self.scale = d ** -0.5

    def device(self):
        return dict(q=self.q.cuda(), k_pages=cuda(self.k, torch.uint8).view(E4M3),
                    v_pages=cuda(self.v, torch.uint8).view(E4M3),
                    k_scale=cuda(self.ks, torch.float32), v_scale=cuda(self.vs, torch.float32),
                    table=cuda(self.table), lengths=cuda(self.lengths),
                    cu_q=None if self.cu is None else cuda(self.cu))

    def reference(self):
        return po.attend(self.q.double().numpy(), self.k, self.ks.astype(np.float64), self.v,
                         self.vs.astype(np.float64), self.table.tolist(), self.lengths, self.cu,
                         self.scale)

    def compare(self, out, lse, rows=slice(None)):
        o, l, to, tl = self.reference()
        po.check("lse", lse.double().cpu().numpy()[rows], l[rows], tl[rows])
        po.check("out", out.double().cpu().numpy()[rows], o[rows], to[rows])

    def run(self, status=0, **kw):
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        a = self.device()
        a.update(kw)
        out, lse = hk.attend_pages(scale=self.scale, status=word, **a)
        torch.cuda.synchronize()
        assert word.item() == status
        self.compare(out, lse)
        return out, lse


@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens_at_page_and_tile_ends(d, P):
    lengths = [1, 2, P - 1, P, P + 1, 127, 128, 129, 255, 256, 257, 383, 0, 500]
    Case([(x, 1) for x in lengths], Hq=4, Hkv=2, d=d, P=P, seed=P + d, single=True).run()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (7, 1), (14, 2), (16, 1), (40, 1), (64, 1),
                                    (100, 1), (128, 1), (130, 2)])
def test_heads_of_a_group(Hq, Hkv):
    Case([(300, 1), (0, 0), (129, 3), (40, 40)], Hq=Hq, Hkv=Hkv, d=128, P=32, seed=Hq).run()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seqs", [
    [(1, 1)], [(0, 0)], [(0, 0), (0, 0), (5, 5)], [(200, 200)], [(130, 17), (700, 129), (64, 64)],
    [(1000, 65), (33, 1), (0, 0), (520, 260), (1, 1), (17, 16)], [(900, 900)], [(128, 128), (256, 128)]])
def test_pieces_of_prompts(seqs, d):
    Case(seqs, Hq=8, Hkv=2, d=d, P=64, seed=len(seqs) + d).run()


@pytest.mark.parametrize("G,m", [(1, 300), (5, 60), (8, 33), (64, 5), (128, 3), (2, 257)])
def test_query_tiles_of_any_group(G, m):
    Case([(m + 150, m), (m, m)], Hq=G, Hkv=1, d=64, P=16, seed=G).run()


@pytest.mark.parametrize("B,length,G", [(1, 20000, 4), (2, 9000, 1), (1, 33000, 16)])
def test_long_contexts_in_parts(B, length, G):
    """A context that many multiprocessors share, joined."""
    Case([(length - 77 * b, 1) for b in range(B)], Hq=G, Hkv=1, d=128, P=64, seed=length,
         single=True).run()


def test_many_sequences():
    g = np.random.default_rng(5)
    seqs = [(int(x), int(min(x, g.integers(0, 4)))) for x in g.integers(0, 400, 333)]
    Case(seqs, Hq=4, Hkv=2, d=64, P=32, seed=9).run()


def test_scales_far_apart():
    c = Case([(700, 1), (300, 20)], Hq=8, Hkv=2, d=128, P=16, seed=1, spread=18.0)
    c.ks = (c.ks * 0 + 2.0 ** -6).astype(np.float32)
    c.run()
    c = Case([(700, 1), (300, 20)], Hq=8, Hkv=2, d=64, P=16, seed=2, spread=3.0)
    c.vs[::2] *= np.float32(2.0 ** 60)
    c.vs[1::2] *= np.float32(2.0 ** -60)
    c.run()


@pytest.mark.parametrize("scale", [0.0, -0.125, 2.0, -3.0])
def test_scale_of_either_sign(scale):
    c = Case([(300, 2), (90, 90)], Hq=4, Hkv=2, seed=3)
    c.scale = scale
    c.run()


@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -30, 16.0, 2.0 ** 22, 2.0 ** 100])
def test_sizes_of_queries(size):
    """Queries far from 1: scores of next to nothing, and ones where a single row is left."""
    c = Case([(300, 2), (90, 90)], Hq=4, Hkv=2, d=128, P=32, seed=4, q_size=size)
    c.run()


def test_uneven_queries():
    """Columns of one query 2^30 apart."""
    c = Case([(300, 3)], Hq=4, Hkv=2, d=64, seed=6)
    c.q[:, :, ::3] *= 2.0 ** 14
    c.q[:, :, 1::3] *= 2.0 ** -16
    c.run()


def test_scores_of_minus_infinity_weigh_nothing():
    c = Case([(260, 2), (140, 1)], Hq=2, Hkv=2, d=64, P=16, seed=7)
    c.k &= 0x7F                                    # codes >= 0
    c.k[c.k == 0x7F] = 1
    c.k[:, :, :, 0] = 0x38
    c.q[:] = -(2.0 ** 126)
    c.ks[:] = 2.0 ** -120
    big = c.table[0, [0, 3, 9]].tolist() + c.table[1, :9].tolist()
    c.ks[big] = 2.0 ** 60                          # all of sequence 1's rows score -inf
    out, lse = c.run()
    assert torch.isinf(lse[2]).all() and (out[2] == 0).all()


def test_codes_of_nan_behind_a_row_do_not_reach_it():
    """Later rows of the same page and tile, NaN in single columns of v and in k."""
    c = Case([(200, 150), (137, 12), (400, 1)], Hq=6, Hkv=2, d=64, P=32, seed=8)
    for b, j, column in ((0, 120, 5), (0, 121, 5), (0, 180, 63), (1, 130, 0), (2, 7, 33)):
        c.v[c.table[b, j // 32], j % 32, :, column] = 0x7F if j % 2 else 0xFF
    c.k[c.table[0, 170 // 32], 170 % 32, 0, 1] = 0x7F     # rows from 170 on: NaN
    c.k[c.table[1, 136 // 32], 136 % 32, :, 1] = 0xFF     # the last row's own key
    out, _ = c.run()
    assert torch.isnan(out).any() and not torch.isnan(out).all()


def test_page_scales_that_are_no_scales():
    """NaN for the rows that see the page, and for no others."""
    for value, which in ((np.nan, "ks"), (0.0, "vs"), (-1.0, "ks"), (np.inf, "vs"), (np.nan, "vs"),
                         (np.inf, "ks")):
        c = Case([(150, 100), (140, 1)], Hq=4, Hkv=2, d=64, P=16, seed=10)
        o, l, to, tl = c.reference()
        page = c.table[0, 6]                              # rows 96 .. 111
        getattr(c, which)[page, 1] = value
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = hk.attend_pages(scale=c.scale, status=word, **c.device())
        assert word.item() == hk.DEV_BAD_SCALE
        seen = np.array([50 + t >= 96 for t in range(100)] + [False])
        got = out.double().cpu().numpy()
        assert np.isnan(got[seen][:, 2:]).all()
        rest = np.ones(got.shape, dtype=bool)
        rest[np.ix_(seen, [2, 3])] = False
        assert not np.isnan(got[rest]).any()
        assert (np.abs(got - o)[rest] <= to[rest] + 1e-30).all()


def test_table_entries_that_are_no_pages():
    c = Case([(300, 30), (290, 1), (100, 1)], Hq=4, Hkv=2, d=128, P=16, seed=11)
    c.table[0, [0, 5, 17]] = -1
    c.table[1, :] = -1
    c.run()
    c.table[2, [1, 6]] = [10 ** 6, -7]
    c.run(status=hk.DEV_BAD_INDEX)


def test_pages_that_sequences_share():
    c = Case([(200, 1), (200, 1), (90, 90)], Hq=8, Hkv=2, d=64, P=32, seed=12)
    c.table[1] = c.table[0]
    out, lse = c.run()
    c.q[1] = c.q[0]
    out, lse = c.run()
    assert torch.equal(out[0], out[1]) and torch.equal(lse[0], lse[1])


def test_rows_past_the_last_sequence_are_left():
    c = Case([(200, 70), (90, 1)], Hq=8, Hkv=2, d=64, P=32, seed=13)
    c.q = torch.cat([c.q, torch.full((9, 8, 64), float("nan")).bfloat16()])
    out = torch.full((80, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((80, 8), 7.0, device="cuda")
    got = hk.attend_pages(scale=c.scale, out=out, lse=lse, **c.device())
    assert got[0] is out and got[1] is lse
    c.compare(out, lse, slice(0, 71))
    assert (out[71:] == 7.0).all() and (lse[71:] == 7.0).all()


def test_lengths_and_offsets_out_of_range():
    """Brought back into the range and reported; rows before the context see nothing."""
    c = Case([(40, 1), (64, 3)], Hq=4, Hkv=2, d=64, P=16, seed=14, columns=4)
    a = c.device()
    a["lengths"] = cuda([40, 10 ** 9])                    # past the table: 64
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = hk.attend_pages(scale=c.scale, status=word, **a)
    assert word.item() == hk.DEV_BAD_POSITION
    c.compare(out, lse)
    a["lengths"] = cuda([-3, 64])
    word.zero_()
    out, lse = hk.attend_pages(scale=c.scale, status=word, **a)
    assert word.item() == hk.DEV_BAD_POSITION
    assert (out[0] == 0).all() and torch.isinf(lse[0]).all()
    c.compare(out, lse, slice(1, None))
    for cu in ([0, 1, 9], [-5, 1, 4], [0, 3, 2]):
        word.zero_()
        a = c.device()
        a["cu_q"] = cuda(cu)
        hk.attend_pages(scale=c.scale, status=word, **a)
        assert word.item() == hk.DEV_BAD_POSITION
    a = c.device()
    a["lengths"] = cuda([40, 2])                          # 3 rows, 2 of context
    c.lengths = [40, 2]
    c.run(lengths=a["lengths"])


def test_strided_queries_and_no_status():
    c = Case([(200, 70), (90, 1)], Hq=8, Hkv=2, d=64, P=32, seed=15)
    wide = torch.randn(71, 3, 8, 64, device="cuda").bfloat16()
    wide[:, 1] = c.q.cuda()
    a = c.device()
    a["q"] = wide[:, 1]
    c.compare(*hk.attend_pages(scale=c.scale, **a))


def test_default_scale():
    c = Case([(60, 1)], Hq=4, Hkv=2, d=64, seed=16)
    c.compare(*hk.attend_pages(**c.device()))


def test_nothing_to_do():
    c = Case([(60, 1)], Hq=4, Hkv=2, d=64, seed=17)
    a = c.device()
    out, lse = hk.attend_pages(**{**a, "q": a["q"][:0], "table": a["table"][:0],
                                  "lengths": a["lengths"][:0], "cu_q": None})
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_same_bits_again():
    c = Case([(5000, 1), (700, 300), (64, 1)], Hq=8, Hkv=2, d=128, P=64, seed=18)
    a = c.device()
    first = hk.attend_pages(**a)
    for _ in range(5):
        again = hk.attend_pages(**a)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_two_streams_and_a_graph():
    """Calls at once on two streams, and captured ones whose lengths change between replays."""
    c = Case([(5000, 1), (700, 30), (64, 1)], Hq=8, Hkv=2, d=128, P=64, seed=19)
    e = Case([(900, 200), (3000, 1)], Hq=4, Hkv=1, d=64, P=32, seed=20)
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
    a["lengths"].copy_(cuda([4999, 650, 1]))
    c.lengths = [4999, 650, 1]
    for _ in range(2):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    c.compare(*graphs[0][1])
    e.compare(*graphs[1][1])


def test_places_past_two_gigabytes():
    """Pages whose bytes lie past 2^31 and 2^32."""
    N, P, H, d = 270000, 128, 1, 128
    k = torch.zeros(N, P, H, d, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    c = Case([(300, 2)], Hq=4, Hkv=1, d=d, P=P, seed=21)
    far = [N - 1, 131072 + 7, 262144 + 9]
    for j, p in enumerate(far):
        k[p] = cuda(c.k[c.table[0, j]], torch.uint8)
        v[p] = cuda(c.v[c.table[0, j]], torch.uint8)
    ks, vs = torch.ones(N, 1, device="cuda"), torch.ones(N, 1, device="cuda")
    a = c.device()
    for j, p in enumerate(far):
        ks[p], vs[p] = a["k_scale"][c.table[0, j]], a["v_scale"][c.table[0, j]]
    a.update(k_pages=k.view(E4M3), v_pages=v.view(E4M3), k_scale=ks, v_scale=vs,
             table=cuda([far]))
    c.compare(*hk.attend_pages(**a))
