"""A cache in pages, in plain numpy and 64 bits (test infrastructure): attention over whole
contexts with first-order bounds of its error, rows written with their page scales, and the
pool's bookkeeping sequence by sequence."""
import numpy as np

U32 = 2.0 ** -23


def e4m3_values():
    """value of each of the 256 codes"""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    v = np.where(c & 128, -v, v)
    v[[0x7F, 0xFF]] = np.nan
    return v


VALUES = e4m3_values()


def pages_of(length, P):
    return -(-length // P)


def context(codes, scale, table_row, length, fill=np.nan):
    """values [length, H, d], scales of each row [length, H] and which rows are there"""
    N, P, H, d = codes.shape
    x, s = np.zeros((length, H, d)), np.ones((length, H))
    there = np.zeros(length, dtype=bool)
    for j in range(length):
        p = table_row[j // P]
        if 0 <= p < N:
            x[j], s[j], there[j] = VALUES[codes[p, j % P]], scale[p], True
    return x, s, there


def attend(q, k, ks, v, vs, table, lengths, cu, scale):
    """q [n, Hq, d] float64 values; k, v [N, P, Hkv, d] codes. Returns out, lse and bounds; rows of
    no sequence are NaN in all four."""
    n, Hq, d = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    out, lse = np.full((n, Hq, d), np.nan), np.full((n, Hq), np.nan)
    t_out, t_lse = np.full((n, Hq, d), np.nan), np.full((n, Hq), np.nan)
    steps = (d / 16 + 16) * U32
    for b, length in enumerate(lengths):
        lo, hi = (b, b + 1) if cu is None else (cu[b], cu[b + 1])
        K, sk, there = context(k, ks, table[b], length)
        V, sv, _ = context(v, vs, table[b], length)
        for t in range(lo, hi):
            p = length - (hi - lo) + t - lo
            rows = np.nonzero(there[:max(p + 1, 0)])[0]
            for h in range(Hq):
                hk = h // G
                out[t, h], lse[t, h], t_out[t, h], t_lse[t, h] = 0.0, -np.inf, 0.0, 0.0
                if not rows.size:
                    continue
                with np.errstate(all="ignore"):
                    s = (K[rows, hk] @ q[t, h]) * sk[rows, hk] * scale
                    # (scores are fp32: past its range they are infinite)
                    s = np.where(np.abs(s) > 3.4028235e38, np.copysign(np.inf, s), s)
                    top = s.max()
                    if top == -np.inf:
                        continue
                    e = np.exp(s - top)
                    z = e.sum()
                    w = e / z
                    val = V[rows, hk] * sv[rows, hk][:, None]
                    o = w @ val
                    out[t, h], lse[t, h] = o, top + np.log(z)
                    # fp32 scores (the tensor core's additions may truncate), queries to 2^-39 of
                    # the row's largest, the exponential, its argument and the normalisation
                    size = np.abs(K[rows, hk]) @ (np.abs(q[t, h]) + 2.0 ** -16 * np.abs(q[t, h]).max())
                    size *= abs(scale) * sk[rows, hk]
                    delta = steps * size[np.isfinite(s)].max(initial=0.0) + 2.0 ** -20 + \
                        2.0 ** -21 * np.abs(s[np.isfinite(s)]).max(initial=0.0)
                    weight = w @ np.abs(val)
                    # weights rounded to f16: half a step, or 2^-28 of the largest where subnormal
                    t_out[t, h] = (2 * delta + 2.0 ** -11 + (rows.size / 16 + 16) * U32) * weight + \
                        2.0 ** -28 * np.abs(val).sum(0) + 2.0 ** -8 * np.abs(o)
                    t_lse[t, h] = 2 * delta + 2.0 ** -22 * abs(lse[t, h])
    return out, lse, t_out, t_lse


def check(name, got, ref, tol):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, name
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), f"{name}: NaN in {np.isnan(got).sum()} places, {nan.sum()} expected"
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]) and not np.isinf(got[~inf]).any(), name
    fine = ~nan & ~inf
    over = np.abs(got[fine] - ref[fine]) - (tol[fine] + 1e-30)
    assert over.size == 0 or over.max() <= 0, \
        f"{name}: {int((over > 0).sum())} of {over.size} past the bound, by {over.max():.3g} " \
        f"(bound there {tol[fine][over.argmax()]:.3g})"


# ---- the pool -----------------------------------------------------------------------

class Pool:
    """table, lengths, refs as lists; `bad` and `short` are the conditions that are reported"""

    def __init__(self, table, lengths, refs, P):
        self.table = [list(map(int, r)) for r in table]
        self.lengths, self.refs = list(map(int, lengths)), list(map(int, refs))
        self.P, self.bad, self.short = P, False, False
        self.columns = len(self.table[0]) if self.table else 0

    def held(self, b):
        return pages_of(self.lengths[b], self.P)

    def fits(self, length):
        return 0 <= length <= self.columns * self.P

    def fork(self, src, dst):
        before = list(self.lengths)
        for i, (s, d) in enumerate(zip(src, dst)):
            if s == -1 or d == -1:
                continue
            B = len(self.lengths)
            if not (0 <= s < B and 0 <= d < B) or d in dst[:i] or s in dst or before[d] != 0 or \
                    not self.fits(before[s]):
                self.bad = True
                continue
            for j in range(self.held(s)):
                p = self.table[s][j]
                if 0 <= p < len(self.refs):
                    self.refs[p] += 1
                else:
                    self.bad |= p != -1
                    p = -1
                self.table[d][j] = p
            self.lengths[d] = self.lengths[s]

    def free(self, rows):
        for i, b in enumerate(rows):
            if b == -1 or b in rows[:i]:
                continue
            if not 0 <= b < len(self.lengths):
                self.bad = True
                continue
            if not self.fits(self.lengths[b]):
                self.bad = True
                self.lengths[b] = min(max(self.lengths[b], 0), self.columns * self.P)
            for j in range(self.held(b)):
                p, self.table[b][j] = self.table[b][j], -1
                if p == -1:
                    continue
                if 0 <= p < len(self.refs) and self.refs[p] > 0:
                    self.refs[p] -= 1
                else:
                    self.bad = True
            self.lengths[b] = 0

    def grow(self, add):
        B, N, P = len(self.lengths), len(self.refs), self.P
        before = list(self.refs)
        free = [p for p in range(N) if before[p] == 0]
        fine = [self.fits(self.lengths[b]) and add[b] >= 0 and self.fits(self.lengths[b] + add[b])
                for b in range(B)]
        last = [-1] * B
        for b in range(B):
            if fine[b] and add[b] > 0 and self.lengths[b] % P:
                p = self.table[b][self.held(b) - 1]
                last[b] = p if 0 <= p < N else -1
        src, dst, at, ended = [-1] * B, [-1] * B, 0, False
        for b in range(B):
            if not fine[b]:
                if self.fits(self.lengths[b]) and add[b] >= 0:
                    self.short = True
                else:
                    self.bad = True
                continue
            same = [o for o in range(B) if last[b] >= 0 and last[o] == last[b]]
            away = last[b] >= 0 and before[last[b]] > 1 and \
                not (len(same) == before[last[b]] and same[-1] == b)
            had, have = self.held(b), pages_of(self.lengths[b] + add[b], P)
            need = have - had + away
            if ended or at + need > len(free):
                ended = self.short = True
                continue
            fresh, at = free[at:at + need], at + need
            if away:
                src[b], dst[b] = last[b], fresh[0]
                self.refs[last[b]] -= 1
            for j, p in enumerate(fresh):
                self.table[b][had - away + j] = p
                self.refs[p] = 1
            self.lengths[b] += add[b]
        return src, dst

    def compact(self):
        N = len(self.refs)
        live = [r > 0 for r in self.refs]
        K = sum(live)
        src = [p for p in range(K, N) if live[p]]
        dst = [p for p in range(K) if not live[p]]
        to = dict(zip(src, dst))
        for b, row in enumerate(self.table):
            length = self.lengths[b]
            self.bad |= not self.fits(length)
            for j in range(pages_of(min(max(length, 0), self.columns * self.P), self.P)):
                p = row[j]
                if p == -1:
                    continue
                if not 0 <= p < N:
                    self.bad = True
                elif p >= K:
                    if live[p]:
                        row[j] = to[p]
                    else:
                        self.bad = True
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        rest = [-1] * (max(1, N // 2) - len(src))
        return src + rest, dst + rest
