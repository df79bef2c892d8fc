"""The pool of a cache in pages (GPU): forks, frees, growth, compaction and copies, number for
number what the definition gives sequence by sequence (tests/pages_oracle.py)."""
import random

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


class Both:
    """The state on the device and in the oracle."""

    def __init__(self, B, columns, N, P, lengths, seed=0):
        g = np.random.default_rng(seed)
        order = g.permutation(N)
        table = np.full((B, columns), -1)
        refs = np.zeros(N, dtype=np.int64)
        at = 0
        for b, x in enumerate(lengths):
            k = po.pages_of(x, P)
            table[b, :k] = order[at:at + k]
            refs[order[at:at + k]] = 1
            at += k
        self.P, self.N = P, N
        self.o = po.Pool(table, lengths, refs, P)
        self.table, self.lengths, self.refs = cuda(table).view(B, columns), cuda(lengths), cuda(refs)
        self.word = torch.zeros(1, dtype=torch.int32, device="cuda")

    def state(self):
        return self.table, self.lengths, self.refs

    def same(self):
        torch.cuda.synchronize()
        assert self.table.tolist() == self.o.table
        assert self.lengths.tolist() == self.o.lengths
        assert self.refs.tolist() == self.o.refs
        assert self.word.item() == (hk.DEV_BAD_INDEX if self.o.bad else 0) | \
            (hk.DEV_NO_PAGE if self.o.short else 0)

    def fork(self, src, dst):
        assert hk.page_fork(*self.state(), cuda(src), cuda(dst), page=self.P, status=self.word) is self.table
        self.o.fork(src, dst)
        self.same()

    def free(self, rows):
        assert hk.page_free(*self.state(), cuda(rows), page=self.P, status=self.word) is self.table
        self.o.free(rows)
        self.same()

    def grow(self, add):
        src, dst = hk.page_grow(*self.state(), cuda(add), page=self.P, status=self.word)
        s, d = self.o.grow(add)
        self.same()
        assert src.tolist() == s and dst.tolist() == d
        return src, dst

    def compact(self):
        src, dst = hk.page_compact(*self.state(), page=self.P, status=self.word)
        s, d = self.o.compact()
        self.same()
        assert src.tolist() == s and dst.tolist() == d
        return src, dst


@pytest.mark.parametrize("seed", range(8))
def test_random_steps(seed):
    """Steps of every kind in a row."""
    r = random.Random(seed)
    P = r.choice([16, 32, 64, 128, 256])
    B, N = r.choice([1, 3, 17, 200]), r.choice([40, 300, 5000, 9001])
    t = Both(B, 12, N, P, [0] * B, seed)
    for _ in range(14):
        kind = r.choice(["grow", "grow", "fork", "free", "compact"])
        if kind == "grow":
            t.grow([r.choice([0, 1, 1, P, r.randrange(3 * P)]) for _ in range(B)])
        elif kind == "fork":
            empty = [b for b in range(B) if t.o.lengths[b] == 0]
            full = [b for b in range(B) if t.o.lengths[b] > 0] or [-1]
            r.shuffle(empty)
            empty = empty[:r.randrange(1, B + 1)]
            t.fork([r.choice(full) for _ in empty], empty)
        elif kind == "free":
            t.free([r.randrange(B) for _ in range(r.randrange(1, B + 1))])
        else:
            t.compact()


def test_grow_at_page_ends():
    P = 16
    t = Both(9, 8, 64, P, [0, 1, 15, 16, 17, 32, 0, 127, 128])
    t.grow([1, 1, 1, 1, 1, 0, 0, 1, 0])
    t.grow([16, 16, 16, 16, 16, 33, 128, 0, 0])


def test_grow_into_shared_pages():
    """The last holder keeps the page if all of them grow; otherwise each that grows copies."""
    t = Both(8, 4, 32, 16, [20, 0, 0, 40, 0, 7, 0, 0])
    t.fork([0, 0, 3, 5], [1, 2, 4, 6])
    src, dst = t.grow([1, 1, 1, 0, 1, 1, 17, 0])
    assert (src >= 0).sum() == 4
    t.grow([1] * 8)


def test_grow_past_the_pool_and_the_table():
    t = Both(5, 4, 10, 16, [16, 30, 64, 16, 16])
    t.grow([1, 10, 1, 33, 1])          # sequence 2 would pass the table, 3 the pool
    assert t.word.item() == hk.DEV_NO_PAGE
    t = Both(3, 4, 6, 16, [16, 16, 16])
    t.grow([1, 40, 0])
    # a page is kept only if the other holders grow too
    t = Both(4, 4, 5, 16, [20, 0, 20, 0])
    t.fork([0, 2], [1, 3])
    t.grow([1, 1, 1, 1])


def test_grow_by_nothing_and_by_less():
    t = Both(4, 4, 10, 16, [16, 30, 0, 5])
    t.grow([0, 0, 0, 0])
    t.grow([1, -1, 0, 1])
    assert t.word.item() == hk.DEV_BAD_INDEX


def test_large_pool():
    g = np.random.default_rng(3)
    B, P = 700, 16
    t = Both(B, 70, 50000, P, g.integers(0, 60 * P, B).tolist(), 4)
    t.grow(g.integers(0, 3 * P, B).tolist())
    t.free(g.permutation(B)[:300].tolist())
    empty = [b for b in range(B) if t.o.lengths[b] == 0][:250]
    full = [b for b in range(B) if t.o.lengths[b] > 0]
    t.fork([full[i % len(full)] for i in range(len(empty))], empty)
    t.grow([1] * B)
    t.compact()
    t.compact()
    t.grow([1] * B)


def test_forks_that_are_refused():
    t = Both(8, 4, 32, 16, [20, 30, 0, 0, 0, 5, 0, 0])
    t.fork([0, 0, 0], [2, 2, -1])                # twice into one place: the first counts
    t.o.bad or pytest.fail("not reported")
    t = Both(8, 4, 32, 16, [20, 30, 0, 0, 0, 5, 0, 0])
    t.fork([0, 3, 9, -2, 1, 0, -1], [3, 4, 6, 7, 5, 8, 2])
    t = Both(4, 4, 32, 16, [20, 0, 0, 0])
    t.fork([0, 1], [1, 2])                       # from a place that is forked into


def test_states_out_of_range():
    """Bad pages and lengths: left out and reported, nothing outside the arrays is touched."""
    for op in ("fork", "free", "grow", "compact"):
        t = Both(5, 4, 32, 16, [20, 30, 0, 64, 9])
        t.table[0, 0], t.table[3, 1] = 1000, -5
        t.o.table[0][0], t.o.table[3][1] = 1000, -5
        if op == "fork":
            t.fork([0], [2])
        elif op == "free":
            t.free([0, 3, 77, -1, 3])
        elif op == "compact":
            t.compact()
        else:
            t.table[1, 1] = t.o.table[1][1] = 31 * 64
            t.grow([1, 1, 1, 0, 1])
        t = Both(5, 4, 32, 16, [20, 30, 0, 64, 9])
        t.lengths[1], t.lengths[4] = 10 ** 6, -4
        t.o.lengths[1], t.o.lengths[4] = 10 ** 6, -4
        if op == "fork":
            t.fork([1, 4], [2, -1])
        elif op == "free":
            t.free([1, 4])
        elif op == "compact":
            t.compact()
        else:
            t.grow([1, 1, 1, 0, 1])


def test_free_twice_and_counts_that_end():
    t = Both(3, 4, 32, 16, [20, 30, 0])
    t.free([0, 0, -1, 0])
    t.refs[t.table[1, 0]] = 0
    t.o.refs[t.o.table[1][0]] = 0
    t.free([1])
    assert t.word.item() == hk.DEV_BAD_INDEX


@pytest.mark.parametrize("N", [1, 2, 3, 4095, 4096, 4097, 8192, 20000])
def test_compact_sizes(N):
    g = np.random.default_rng(N)
    used = min(N, max(1, N // 3))
    t = Both(2, max(1, used), N, 16, [(used + 1) // 2 * 16, used // 2 * 16], N)
    t.compact()
    t = Both(1, 1, N, 16, [0], N)
    t.compact()
    assert g is not None


@pytest.mark.parametrize("N,columns", [(4095, 1500), (4096, 2048), (4096, 2049), (4097, 1500),
                                       (3000, 9000), (16385, 4000), (70001, 20000)])
def test_compact_around_one_block(N, columns):
    """Pools of 4096 pages and tables of 4096 entries are the most that one block takes."""
    t = Both(2, columns, N, 16, [1500 * 8, 1000 * 16 - 5], N)
    t.compact()
    t.free([0])
    t.compact()


def test_compact_refs_at_any_address():
    """refs that start 4 bytes behind a 16-byte boundary."""
    t = Both(2, 60, 300, 16, [900, 700], 4)
    shifted = torch.zeros(301, dtype=torch.int32, device="cuda")[1:]
    shifted.copy_(t.refs)
    t.refs = shifted
    t.compact()
    t.grow([20, 300])


def test_compact_full_and_front():
    t = Both(2, 8, 16, 16, [128, 128])
    t.compact()
    assert (t.compact()[0] == -1).all()


@pytest.mark.parametrize("P,H,d,both", [(16, 1, 64, True), (64, 8, 128, True), (16, 3, 16, False),
                                        (256, 5, 128, True)])
def test_copies(P, H, d, both):
    g = np.random.default_rng(P)
    N, m = 300, 120
    pools = [cuda(g.integers(0, 256, (N, P, H, d)), torch.uint8) for _ in range(2)]
    scales = [torch.rand(N, H, device="cuda") for _ in range(2)]
    order = g.permutation(N)
    src, dst = order[:m].copy(), order[m:2 * m].copy()
    src[5], dst[9], src[11], dst[11] = -1, -1, -1, -1
    src[20] = dst[20] = order[-1]
    src[30] = src[31]                            # one page to two places
    want = [p.clone() for p in pools], [s.clone() for s in scales]
    for a, b in zip(src, dst):
        if a >= 0 and b >= 0:
            for i in range(2 if both else 1):
                want[0][i][b], want[1][i][b] = pools[i][a], scales[i][a]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    v = (pools[1].view(E4M3), scales[1]) if both else (None, None)
    hk.page_copy(pools[0].view(E4M3), v[0], scales[0], v[1], cuda(src), cuda(dst), status=word)
    torch.cuda.synchronize()
    assert word.item() == 0
    for i in range(2):
        assert torch.equal(pools[i], want[0][i]) and torch.equal(scales[i], want[1][i])
    src[0], dst[1] = N, -3
    hk.page_copy(pools[0].view(E4M3), v[0], scales[0], v[1], cuda(src), cuda(dst), status=word)
    torch.cuda.synchronize()
    assert word.item() == hk.DEV_BAD_INDEX
    assert all(torch.equal(p, w) for p, w in zip(pools, want[0]))


def test_long_lists_of_copies():
    """Mostly -1, as a compaction leaves them."""
    N = 6000
    pages = torch.arange(N, device="cuda").to(torch.uint8)[:, None, None, None].expand(N, 16, 1, 64).contiguous()
    scale = torch.arange(N, device="cuda").float()[:, None].contiguous()
    src, dst = torch.full((N,), -1, dtype=torch.int32), torch.full((N,), -1, dtype=torch.int32)
    for i, at in enumerate(range(3, N, 37)):
        src[at], dst[at] = 3000 + i, i
    want = scale.clone()
    k = int((src >= 0).sum())
    want[:k] = scale[3000:3000 + k]
    hk.page_copy(pages.view(E4M3), None, scale, None, src.cuda(), dst.cuda())
    assert torch.equal(scale, want)
    assert torch.equal(pages[:, 3, 0, 5].int(), want[:, 0].int() % 256)


def test_places_past_four_gigabytes():
    N, P, H, d = 5000, 256, 8, 512
    pages = torch.zeros(N, P, H, d, dtype=torch.uint8, device="cuda")
    scale = torch.rand(N, H, device="cuda")
    pages[4990] = 7
    hk.page_copy(pages.view(E4M3), None, scale, None, cuda([4990, 3]), cuda([4999, 4100]))
    assert (pages[4999] == 7).all() and (pages[4998] == 0).all()
    assert torch.equal(scale[4999], scale[4990])


def test_a_run_of_them_captured():
    """A search step by step, as one graph replayed: pages freed, forked, grown, copied, rows written
    and attended; against contexts kept as plain rows."""
    P, H, d, B, columns, N = 16, 2, 64, 8, 6, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.zeros(N, P, H, d, dtype=torch.uint8, device="cuda").view(E4M3)
    v = torch.zeros_like(k)
    ks, vs = torch.zeros(N, H, device="cuda"), torch.zeros(N, H, device="cuda")
    table = torch.full((B, columns), -1, dtype=torch.int32, device="cuda")
    lengths, refs = cuda([0] * B), cuda([0] * N)
    add, drop, src, dst = cuda([0] * B), cuda([-1] * 4), cuda([-1] * 4), cuda([-1] * 4)
    x = torch.zeros(B, H, d, device="cuda")
    y, q = torch.zeros_like(x), torch.zeros(B, 2 * H, d, dtype=torch.bfloat16, device="cuda")
    cu = cuda(list(range(B + 1)))
    word = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        hk.page_free(table, lengths, refs, drop, page=P, status=word)
        hk.page_fork(table, lengths, refs, src, dst, page=P, status=word)
        a, b = hk.page_grow(table, lengths, refs, add, page=P, status=word)
        hk.page_copy(k, v, ks, vs, a, b, status=word)
        hk.page_write(x, k, ks, table, lengths, cu, status=word)
        hk.page_write(y, v, vs, table, lengths, cu, status=word)
        return hk.attend_pages(q, k, v, ks, vs, table, lengths, cu, status=word)

    step()                                       # (nothing grows)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    for t in (k, v):
        t.view(torch.uint8).zero_()
    lengths.zero_(), refs.zero_(), table.fill_(-1), ks.zero_(), vs.zero_(), word.zero_()
    rows = [[] for _ in range(B)]                # of each sequence: (key row, value row)
    add.fill_(1)
    r = random.Random(2)
    for s in range(40):
        drops = r.sample(range(B), 3) if s % 5 == 4 else []
        left = [b for b in range(B) if b not in drops]
        sources = [r.choice(left) for _ in drops]
        drop.copy_(cuda(drops + [-1] * (4 - len(drops))))
        dst.copy_(cuda(drops + [-1] * (4 - len(drops))))
        src.copy_(cuda(sources + [-1] * (4 - len(drops))))
        for a, b in zip(sources, drops):
            rows[b] = list(rows[a])
        x.copy_(torch.randn(B, H, d, device="cuda", generator=g))
        y.copy_(torch.randn(B, H, d, device="cuda", generator=g))
        q.copy_(torch.randn(B, 2 * H, d, device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        assert word.item() == 0
        for b in range(B):
            rows[b].append((x[b].clone(), y[b].clone()))
        assert lengths.tolist() == [len(z) for z in rows]
        held = table.flatten()
        held = held[held >= 0].long()
        assert torch.equal(torch.bincount(held, minlength=N).int(), refs)
        for b in range(B):
            K, V = (torch.stack([z[i] for z in rows[b]]).double() for i in range(2))
            w = torch.softmax(torch.einsum("hgd,jhd->hgj", q[b].double().view(H, 2, d), K) / 8, -1)
            want = torch.einsum("hgj,jhd->hgd", w, V).view(2 * H, d)
            # codes are off by half a step of 2^-4 at most, a few times over as scales grow
            assert ((out[b].double() - want).norm() / want.norm()) < 4 * 2.0 ** -4
    src2, dst2 = hk.page_compact(table, lengths, refs, page=P, status=word)
    hk.page_copy(k, v, ks, vs, src2, dst2, status=word)
    again = hk.attend_pages(q, k, v, ks, vs, table, lengths, cu, status=word)
    torch.cuda.synchronize()
    assert word.item() == 0 and torch.equal(again[0], out) and torch.equal(again[1], lse)
    live = int((refs > 0).sum())
    assert (refs[:live] > 0).all() and (refs[live:] == 0).all()
