"""Operators of a cache in pages, as cases that can be timed and compared:

* ``attend``   attention of each sequence's queries over its whole context, held as e4m3
  codes with one scale per (page, head),
* ``write``    rows, rotated, to the end of each context: codes and page scales,
* ``turn``     a step of page management: sequences freed, others forked into their
  places, every context grown, shared last pages copied,
* ``compact``  the pages in use moved to the front of the pool.

``run`` computes them in elementary 32-bit torch operations, or, where ``own`` is true,
through the package's entry points. ``exact`` computes them from their definitions, in
64 bits.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ------------------------------------------------------------------------------
# Lengths spread over [lo, hi] by sequence; `new`: of them, the tokens of this call.

def listed():
    return [
        # one decoded token, a short context, small pages: latency
        dict(name="attend_one", op="attend", B=1, lo=500, hi=500, new=1, Hq=32, Hkv=8, d=64,
             page=16, pad=0),
        # a decoding batch of ragged contexts, one slot in ten idle
        dict(name="attend_batch", op="attend", B=64, lo=0, hi=16384, new=1, Hq=32, Hkv=8, d=128,
             page=64, pad=0),
        # one token over a million rows, all heads on one cache head
        dict(name="attend_long", op="attend", B=1, lo=1 << 20, hi=1 << 20, new=1, Hq=64, Hkv=1,
             d=128, page=64, pad=0),
        # pieces of prompts and single tokens in one batch, seven heads a group, padded
        dict(name="attend_mixed", op="attend", B=37, lo=1, hi=4099, new=256, Hq=14, Hkv=2, d=64,
             page=32, pad=5),
        # a whole prompt
        dict(name="attend_prompt", op="attend", B=1, lo=8192, hi=8192, new=8192, Hq=32, Hkv=4,
             d=128, page=64, pad=0),
        # the keys of a decoding batch
        dict(name="write_tokens", op="write", B=64, lo=1, hi=16384, new=1, H=8, d=128, page=64,
             rot=64, first=0, inter=False, type="bf16"),
        # the keys of five long prompts
        dict(name="write_prompt", op="write", B=5, lo=13000, hi=13200, new=13200, H=8, d=128,
             page=64, rot=128, first=0, inter=True, type="bf16"),
        # fp32 keys of pieces of prompts, few heads, small pages
        dict(name="write_pieces", op="write", B=37, lo=1, hi=4099, new=500, H=3, d=64, page=16,
             rot=64, first=0, inter=False, type="f32"),
        # a step of a search with 16 branches
        dict(name="turn_few", op="turn", B=16, hi=1000, N=2048, H=8, d=64, page=16),
        # a step of 512 branches: their last pages are copied
        dict(name="turn_many", op="turn", B=512, hi=1500, N=16384, H=4, d=128, page=64),
        # a small pool
        dict(name="compact_few", op="compact", B=16, hi=200, N=512, H=8, d=64, page=16),
        # a large pool, half of it in use
        dict(name="compact_many", op="compact", B=128, hi=4000, N=8192, H=4, d=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "write", "write", "turn", "compact"])
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if op == "attend":
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 4, 5, 8, 16, 64 // Hkv])
        B = _log(rng, 1, 100)
        kind = rng.choice(["token", "token", "pieces", "prompt"])
        if kind == "token":
            hi = _log(rng, 1, min(1 << 18, (1 << 25) // (B * Hkv * d // 8)))
            new = rng.choice([1, 1, 2, 4])
        else:
            hi = _log(rng, 2, 6000 if kind == "prompt" else 4000)
            new = hi if kind == "prompt" else _log(rng, 1, min(hi, 500))
            # (query, key) pairs of all heads and sequences: under the listed prompt's
            B = max(1, min(B, (1 << 31) // (Hq * hi * new)))
            Hq = Hq if Hq * hi * new < 1 << 31 else Hkv
        return dict(op=op, B=B, lo=rng.choice([0, 1, max(1, hi // 2), hi]), hi=hi, new=new, Hq=Hq,
                    Hkv=Hkv, d=d, page=page, pad=rng.choice([0, 0, 3]))
    if op == "write":
        H, B = rng.choice([1, 2, 3, 8, 16]), _log(rng, 1, 100)
        hi = _log(rng, 1, max(2, min(20000, 65000 * 8 // (B * H))))
        rot = rng.choice([d, d // 2])
        return dict(op=op, B=B, lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi,
                    new=rng.choice([1, max(1, hi // 3), hi]), H=H, d=d, page=page, rot=rot,
                    first=rng.choice([0, d - rot]), inter=rng.random() < 0.5,
                    type=rng.choice(["bf16", "bf16", "f32"]))
    H = rng.choice([1, 2, 4, 8])
    if op == "turn":
        B, hi = 2 * _log(rng, 1, 200), _log(rng, 2, 1500)
    else:
        B, hi = _log(rng, 1, 128), _log(rng, 2, 4000)
    need = B * (hi // page + 2)
    N = min(need * rng.choice([2, 3]), (1 << 28) // (page * H * d))
    return dict(op=op, B=max(2, B if need * 2 <= N else B * N // (2 * need) // 2 * 2),
                hi=hi, N=max(N, 4 * (hi // page + 2)), H=H, d=d, page=page)


def _spread(B, lo, hi):
    """B lengths over [lo, hi] in no order, the first of them hi."""
    return [lo + int((hi - lo + 0.999) * (1.0 - (b * 0.6180339887498949) % 1.0)) for b in range(B)]


def _lengths(c):
    """Context lengths (one in ten idle where lo is 0) and new tokens of each sequence."""
    full = _spread(c["B"], max(1, c["lo"]), c["hi"])
    if c["lo"] == 0:
        full = [0 if b % 10 == 7 else x for b, x in enumerate(full)]
    most = _spread(c["B"], min(1, c["new"]), c["new"])
    return full, [min(x, y) for x, y in zip(full, most)]


def _pages_of(length, page):
    return -(-length // page)


# ---- inputs -----------------------------------------------------------------------------

def _frequencies(rot, base=10000.0):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (base ** (-2.0 * i / rot)).float().cuda()


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _quantised_pages(x):
    """codes and [N, H] scales of 32-bit pages [N, P, H, d]"""
    scale = x.abs().amax((1, 3)) / E4M3_MAX
    return (x / scale[:, None, :, None]).to(E4M3), scale


def _tables(lengths, page, N, columns, order):
    """[B, columns] page ids, -1 past each context, ids in the order given"""
    held = [_pages_of(x, page) for x in lengths]
    table = torch.full((len(lengths), columns), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(held):
        table[b, :k] = order[at:at + k]
        at += k
    return table


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 23)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def pages(N, H):
        # rows of about the same size, pages that differ
        x = normal(N, c["page"], H, c["d"]) * (0.5 + torch.rand(N, 1, H, 1, device="cuda", generator=g))
        return _quantised_pages(x)

    if c["op"] in ("attend", "write"):
        full, new = _lengths(c)
        held = sum(_pages_of(x, c["page"]) for x in full)
        N = held + held // 8 + 1
        order = torch.randperm(N, device="cuda", generator=g).int()
        c["table"] = _tables(full, c["page"], N, max(1, _pages_of(c["hi"], c["page"])), order)
        c["lengths"] = _int(full)
        c["cu_q"] = _int([0] + new).cumsum(0).int()
        c["total"], c["longest"], c["most"] = sum(new), max(full), max(new)
    if c["op"] == "attend":
        c["k"], c["k_scale"] = pages(N, c["Hkv"])
        c["v"], c["v_scale"] = pages(N, c["Hkv"])
        n = c["total"] + c["pad"]
        c["q"] = (1.5 * normal(n, c["Hq"], c["d"])).bfloat16()
        c["out"] = torch.zeros(n, c["Hq"], c["d"], device="cuda", dtype=torch.bfloat16)
        c["lse"] = torch.zeros(n, c["Hq"], device="cuda")
    elif c["op"] == "write":
        c["pages"], c["page_scale"] = pages(N, c["H"])
        # activations with a few strong columns, as projections have them
        strong = 1 + 6 * (torch.rand(c["d"], device="cuda", generator=g) > 0.95)
        c["x"] = (normal(c["total"], c["H"], c["d"]) * strong).to(TYPES[c["type"]])
        c["inv_freq"] = _frequencies(c["rot"])
    else:
        full = _spread(c["B"], max(1, c["hi"] // 4), c["hi"])
        order = torch.randperm(c["N"], device="cuda", generator=g).int()
        if c["op"] == "compact":
            order = order[:max(sum(_pages_of(x, c["page"]) for x in full), 1)]
        c["table"] = _tables(full, c["page"], c["N"], _pages_of(c["hi"], c["page"]) + 1, order)
        c["lengths"] = _int(full)
        held = c["table"][c["table"] >= 0].long()
        c["refs"] = torch.zeros(c["N"], dtype=torch.int32, device="cuda")
        c["refs"][held] = 1
        c["k"], c["k_scale"] = pages(c["N"], c["H"])
        c["v"], c["v_scale"] = pages(c["N"], c["H"])
        if c["op"] == "turn":
            src, dst, add = _branches(c)
            c["src"], c["dst"], c["add"] = _int(src), _int(dst), _int(add)
    return c


def _branches(c):
    """Of B sequences every second one ends; others, some of them twice, are forked into the
    places; all but one in nine grow by a token."""
    dst = list(range(1, c["B"], 2))
    src = [2 * (i * 7 % max(1, len(dst) // 2)) for i in range(len(dst))]
    return src, dst, [0 if b % 9 == 8 else 1 for b in range(c["B"])]


# ---- the plain forms, 32 bits -----------------------------------------------------------

def _turns(pos, f):
    """exp(i pos f), [n, r/2]: the angle in 64 bits, of far positions 32 lose the turn"""
    angle = torch.remainder(pos.double()[:, None] * f.double()[None, :], 2 * math.pi).float()
    return torch.polar(torch.ones_like(angle), angle)


def _rotate(x, turns, c):
    lo, r = c["first"], c["rot"]
    if c["inter"]:
        a, b = slice(lo, lo + r, 2), slice(lo + 1, lo + r, 2)
    else:
        a, b = slice(lo, lo + r // 2), slice(lo + r // 2, lo + r)
    cos, sin = turns.real[:, None, :], turns.imag[:, None, :]
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def _where(c):
    """of every new row: its sequence, its number there, its position"""
    rows = torch.arange(c["total"], device="cuda")
    new = (c["cu_q"][1:] - c["cu_q"][:-1]).long()
    seq = torch.searchsorted(c["cu_q"][1:].long(), rows, right=True)
    i = rows - c["cu_q"].long()[seq]
    return seq, i, c["lengths"].long()[seq] - new[seq] + i


def _attend(c):
    B, P, Hkv, d, G = c["B"], c["page"], c["Hkv"], c["d"], c["Hq"] // c["Hkv"]
    L, m = max(1, c["longest"]), max(1, c["most"])
    at = torch.arange(L, device="cuda")
    page = c["table"].long()[:, at // P].clamp(min=0)                     # [B, L]

    def rows(t, scale):                                                   # [B, Hkv, L, d]
        x = t.view(torch.uint8)[page, at % P].view(E4M3).float() * scale[page][..., None]
        return x.transpose(1, 2)

    seq, i, pos = _where(c)
    q = torch.zeros(B, m, Hkv, G, d, device="cuda")
    q[seq, i] = c["q"][:c["total"]].float().view(-1, Hkv, G, d)
    p = torch.full((B, m), -1, device="cuda")
    p[seq, i] = pos
    s = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * m, d),
                     rows(c["k"], c["k_scale"]).transpose(2, 3)).view(B, Hkv, G, m, L)
    s *= 1.0 / math.sqrt(d)
    s.masked_fill_((at > p[:, :, None])[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    s -= top
    s.exp_()
    z = s.sum(-1, keepdim=True)
    lse = (top + torch.log(z))[..., 0]                                    # [B, Hkv, G, m]
    o = torch.matmul(s.view(B, Hkv, G * m, L), rows(c["v"], c["v_scale"])).view(B, Hkv, G, m, d)
    o = o / torch.where(z == 0, 1.0, z)
    out, l = o.permute(0, 3, 1, 2, 4)[seq, i], lse.permute(0, 3, 1, 2)[seq, i]
    c["out"][:c["total"]] = out.reshape(-1, c["Hq"], d).bfloat16()
    c["lse"][:c["total"]] = l.reshape(-1, c["Hq"])
    return c["out"], c["lse"]


def _write(c):
    P, N, H, d = c["page"], c["pages"].shape[0], c["H"], c["d"]
    seq, _, pos = _where(c)
    y = _rotate(c["x"].float(), _turns(pos, c["inv_freq"]), c)
    page, row = c["table"].long()[seq, pos // P], pos % P
    # pages that hold rows of this call, and those that held rows before it
    touched = torch.zeros(N, dtype=torch.bool, device="cuda")
    touched[page] = True
    start = c["lengths"].long() - (c["cu_q"][1:] - c["cu_q"][:-1]).long()
    column = (start // P).clamp(max=c["table"].shape[1] - 1)
    first = c["table"].long().gather(1, column[:, None])[:, 0]
    keeps = (start % P > 0) & (first >= 0)
    kept = torch.zeros(N, dtype=torch.int64, device="cuda")               # rows kept
    kept[first[keeps]] = (start % P)[keeps]
    amax = torch.zeros(N, H, device="cuda")
    amax.scatter_reduce_(0, page[:, None].expand(-1, H), y.abs().amax(-1), "amax")
    fresh = torch.where(amax > 0, (amax / E4M3_MAX).clamp(min=2.0 ** -126), 0.0)
    old = torch.where((kept > 0)[:, None], c["page_scale"], 0.0)
    scale = torch.maximum(old, fresh)
    scale = torch.where(scale > 0, scale, 1.0)
    # codes kept, under the new scale
    grew = touched & (kept > 0)
    at = grew.nonzero()[:, 0]
    codes = c["pages"][at].float() * (old[at] / scale[at])[:, None, :, None]
    keep = torch.arange(P, device="cuda")[None, :] < kept[at][:, None]
    bits = c["pages"].view(torch.uint8)
    bits[at] = torch.where(keep[:, :, None, None], codes.to(E4M3).view(torch.uint8), bits[at])
    bits[page, row] = (y / scale[page][..., None]).to(E4M3).view(torch.uint8)
    c["page_scale"].copy_(torch.where(touched[:, None], scale, c["page_scale"]))
    return c["pages"], c["page_scale"]


def _copy_pages(c, src, dst):
    """pages src to dst, both lists without -1"""
    for t in ("k", "v"):
        c[t].view(torch.uint8)[dst] = c[t].view(torch.uint8)[src]
        c[t + "_scale"][dst] = c[t + "_scale"][src]


def _turn(c):
    table, lengths, refs = c["table"].clone(), c["lengths"].clone(), c["refs"].clone()
    P, N, columns = c["page"], c["N"], torch.arange(c["table"].shape[1], device="cuda")

    def count(t, by):
        held = t.reshape(-1)
        refs.add_(torch.bincount(held[held >= 0].long(), minlength=N).int(), alpha=by)

    dst = c["dst"].long()
    count(table[dst], -1)                                # free
    table[dst], lengths[dst] = -1, 0
    src = c["src"].long()
    table[dst], lengths[dst] = table[src], lengths[src]  # fork
    count(table[dst], 1)
    # grow: fresh pages, the lowest numbered first, to rows in order; a row whose last page is
    # shared takes another for it, but for the last of its holders if all of them grow
    grown = lengths + c["add"]
    had, have = (lengths + P - 1) // P, (grown + P - 1) // P
    last = table.gather(1, (had - 1).clamp(min=0)[:, None].long())[:, 0]
    open_ = (lengths % P > 0) & (c["add"] > 0)
    same = (last[:, None] == last[None, :]) & open_[:, None] & open_[None, :]
    later = same.triu(1).any(1)
    away = open_ & (refs[last.clamp(min=0).long()] > 1) & (
        later | (same.sum(1) != refs[last.clamp(min=0).long()]))
    need = (have - had) + away.int()
    offset = need.cumsum(0) - need
    free = (refs == 0).nonzero()[:, 0].int()
    # columns that take a fresh page, in order
    j = columns[None, :]
    takes = ((j >= had[:, None]) & (j < have[:, None])) | (away[:, None] & (j == had[:, None] - 1))
    rank = offset[:, None] + takes.int().cumsum(1) - 1
    given = free[rank.clamp(min=0).long()]
    from_, to = torch.where(away, last, -1), torch.where(away, free[offset.long()], -1)
    refs.add_(torch.bincount(last[away].long(), minlength=N).int(), alpha=-1)
    refs[given[takes].long()] = 1
    table = torch.where(takes, given, table)
    _copy_pages(c, last[away].long(), to[away].long())
    return table, grown.int(), refs, from_, to, c["k"], c["v"], c["k_scale"], c["v_scale"]


def _compact(c):
    table, refs = c["table"].clone(), c["refs"].clone()
    live = refs > 0
    K = live.sum()
    number = torch.arange(c["N"], device="cuda")
    src = (live & (number >= K)).nonzero()[:, 0]
    dst = (~live & (number < K)).nonzero()[:, 0]
    to = number.clone()
    to[src] = dst
    held = table >= 0
    table = torch.where(held, to[table.clamp(min=0).long()].int(), table)
    refs[dst], refs[src] = refs[src], 0
    lists = torch.full((2, max(1, c["N"] // 2)), -1, dtype=torch.int32, device="cuda")
    lists[0, :src.numel()], lists[1, :src.numel()] = src.int(), dst.int()
    _copy_pages(c, src, dst)
    return table, refs, lists[0], lists[1], c["k"], c["v"], c["k_scale"], c["v_scale"]


# ---- the package's calls ----------------------------------------------------------------

def _package(c):
    import exact_top_token_gb300 as hk

    if c["op"] == "attend":
        return hk.attend_pages(c["q"], c["k"], c["v"], c["k_scale"], c["v_scale"], c["table"],
                               c["lengths"], c["cu_q"], out=c["out"], lse=c["lse"])
    if c["op"] == "write":
        hk.page_write(c["x"], c["pages"], c["page_scale"], c["table"], c["lengths"], c["cu_q"],
                      inv_freq=c["inv_freq"], first=c["first"], interleaved=c["inter"])
        return c["pages"], c["page_scale"]
    table, lengths, refs, page = c["table"].clone(), c["lengths"].clone(), c["refs"].clone(), c["page"]
    if c["op"] == "turn":
        hk.page_free(table, lengths, refs, c["dst"], page=page)
        hk.page_fork(table, lengths, refs, c["src"], c["dst"], page=page)
        src, dst = hk.page_grow(table, lengths, refs, c["add"], page=page)
        hk.page_copy(c["k"], c["v"], c["k_scale"], c["v_scale"], src, dst)
        return table, lengths, refs, src, dst, c["k"], c["v"], c["k_scale"], c["v_scale"]
    src, dst = hk.page_compact(table, lengths, refs, page=page)
    hk.page_copy(c["k"], c["v"], c["k_scale"], c["v_scale"], src, dst)
    return table, refs, src, dst, c["k"], c["v"], c["k_scale"], c["v_scale"]


def run(state):
    if own:
        return _package(state)
    return {"attend": _attend, "write": _write, "turn": _turn, "compact": _compact}[state["op"]](state)


# ---- the definitions in 64 bits ---------------------------------------------------------

def _context(pages, scale, ids, length, page):
    """[length, H, d] of one sequence in 64 bits"""
    x = pages[ids.long()].float().double() * scale[ids.long()].double()[:, None, :, None]
    return x.flatten(0, 1)[:length]


def _attend64(c):
    full, new = _lengths(c)
    out = torch.zeros(c["out"].shape, device="cuda", dtype=torch.float64)
    lse = torch.zeros(c["lse"].shape, device="cuda", dtype=torch.float64)
    G, first = c["Hq"] // c["Hkv"], 0
    for b, (length, m) in enumerate(zip(full, new)):
        if m:
            ids = c["table"][b, :_pages_of(length, c["page"])]
            k = _context(c["k"], c["k_scale"], ids, length, c["page"])
            v = _context(c["v"], c["v_scale"], ids, length, c["page"])
            step = max(1, (1 << 26) // (length * G))
            for h in range(c["Hkv"]):
                for t in range(0, m, step):
                    e = min(m, t + step)
                    see = length - m + e                 # rows that the last of them sees
                    rows = slice(first + t, first + e)
                    q = c["q"][rows, h * G:(h + 1) * G].double()
                    s = torch.einsum("thd,jd->thj", q, k[:see, h]) / math.sqrt(c["d"])
                    pos = torch.arange(length - m + t, see, device="cuda")
                    hidden = torch.arange(see, device="cuda")[None, :] > pos[:, None]
                    s = s.masked_fill(hidden[:, None, :], -math.inf)
                    z = torch.logsumexp(s, -1)
                    out[rows, h * G:(h + 1) * G] = torch.einsum(
                        "thj,jd->thd", torch.exp(s - z[..., None]), v[:see, h])
                    lse[rows, h * G:(h + 1) * G] = z
        first += m
    return out, lse


def _write64(c):
    full, new = _lengths(c)
    P, lo, r = c["page"], c["first"], c["rot"]
    values, scales = c["pages"].float().double(), c["page_scale"].double()
    first = 0
    for b, (length, m) in enumerate(zip(full, new)):
        pos = torch.arange(length - m, length, device="cuda")
        theta = pos.double()[:, None] * c["inv_freq"].double()[None, :]
        x = c["x"][first:first + m].double()
        part = x[..., lo:lo + r]
        turn = torch.polar(torch.ones_like(theta), theta)[:, None]
        if c["inter"]:
            z = torch.view_as_complex(part.reshape(*part.shape[:-1], r // 2, 2).contiguous())
            part = torch.view_as_real(z * turn).flatten(-2)
        else:
            z = torch.complex(part[..., :r // 2].contiguous(), part[..., r // 2:].contiguous()) * turn
            part = torch.cat([z.real, z.imag], -1)
        y = torch.cat([x[..., :lo], part, x[..., lo + r:]], -1)
        for column in range((length - m) // P, _pages_of(length, P)):
            rows = (pos // P) == column
            kept = max(0, min(P, length - m - column * P))
            page = int(c["table"][b, column])
            scale = y[rows].abs().amax((0, 2)) / E4M3_MAX
            if kept:
                scale = torch.maximum(scale, scales[page])
                values[page, :kept] *= (scales[page] / scale)[None, :, None]
            values[page, kept:kept + int(rows.sum())] = y[rows] / scale[None, :, None]
            scales[page] = scale                         # codes unrounded
        first += m
    return values, scales


def _moved64(c, src, dst):
    """the pools after copies, as values in 64 bits"""
    got = []
    for t in ("k", "v", "k_scale", "v_scale"):
        x = c[t].float()
        x[_int(dst).long()] = x[_int(src).long()]
        got.append(x.double())
    return got


def _turn64(c):
    P = c["page"]
    table, lengths, refs = c["table"].tolist(), c["lengths"].tolist(), c["refs"].tolist()
    src, dst, add = _branches(c)
    for b in dst:
        for j in range(_pages_of(lengths[b], P)):
            refs[table[b][j]] -= 1
            table[b][j] = -1
        lengths[b] = 0
    for a, b in zip(src, dst):
        for j in range(_pages_of(lengths[a], P)):
            refs[table[a][j]] += 1
            table[b][j] = table[a][j]
        lengths[b] = lengths[a]
    free = [p for p, n in enumerate(refs) if n == 0][::-1]
    before = list(refs)
    open_ = [lengths[b] % P > 0 and add[b] > 0 for b in range(c["B"])]
    last = [table[b][_pages_of(lengths[b], P) - 1] for b in range(c["B"])]
    source, target = [-1] * c["B"], [-1] * c["B"]
    holders = {}
    for b in range(c["B"]):
        if open_[b]:
            holders.setdefault(last[b], []).append(b)
    for b in range(c["B"]):
        keeps = open_[b] and len(holders[last[b]]) == before[last[b]] and holders[last[b]][-1] == b
        if open_[b] and before[last[b]] > 1 and not keeps:
            source[b], target[b] = last[b], free.pop()
            refs[last[b]] -= 1
            refs[target[b]] = 1
            table[b][_pages_of(lengths[b], P) - 1] = target[b]
        for j in range(_pages_of(lengths[b], P), _pages_of(lengths[b] + add[b], P)):
            table[b][j] = free.pop()
            refs[table[b][j]] = 1
        lengths[b] += add[b]
    pairs = [(a, b) for a, b in zip(source, target) if a >= 0]
    return (_int(table), _int(lengths), _int(refs), _int(source), _int(target),
            *_moved64(c, [a for a, _ in pairs], [b for _, b in pairs]))


def _compact64(c):
    refs = c["refs"].tolist()
    K = sum(n > 0 for n in refs)
    src = [p for p in range(K, c["N"]) if refs[p] > 0]
    dst = [p for p in range(K) if refs[p] == 0]
    to = dict(zip(src, dst))
    table = [[to.get(p, p) for p in row] for row in c["table"].tolist()]
    for a, b in to.items():
        refs[b], refs[a] = refs[a], 0
    rest = [-1] * (max(1, c["N"] // 2) - len(src))
    return (_int(table), _int(refs), _int(src + rest), _int(dst + rest), *_moved64(c, src, dst))


def exact(case, seed):
    c = prepare(case, seed)
    return {"attend": _attend64, "write": _write64, "turn": _turn64, "compact": _compact64}[c["op"]](c)


# ---- what a pass cannot do without ------------------------------------------------------

def work(case):
    c = case
    page_bytes = c["page"] * c.get("H", 1) * c["d"] + 4 * c.get("H", 1)
    if c["op"] == "turn":
        # copies: of the holders of a partly filled last page, where all grow, all but one
        full = _spread(c["B"], max(1, c["hi"] // 4), c["hi"])
        src, dst, add = _branches(c)
        held = {b: [b] for b in range(c["B"]) if b not in set(dst)}
        for a, b in zip(src, dst):
            held[a].append(b)
        copies = sum(max(0, sum(add[b] for b in rows) - (len(rows) == sum(add[b] for b in rows)))
                     for a, rows in held.items() if full[a] % c["page"])
        entries = sum(_pages_of(full[b], c["page"]) for b in dst) + \
            sum(_pages_of(full[a], c["page"]) for a in src)
        return {"bytes": 4 * copies * page_bytes + 4 * c["N"] + 16 * entries + 28 * c["B"], "flops": 0}
    if c["op"] == "compact":
        full = _spread(c["B"], max(1, c["hi"] // 4), c["hi"])
        live = min(c["N"], sum(_pages_of(x, c["page"]) for x in full))
        moves = live * (c["N"] - live) // c["N"]
        return {"bytes": 4 * moves * page_bytes + 8 * c["N"] + 8 * live, "flops": 0}
    full, new = _lengths(c)
    if c["op"] == "write":
        elems = sum(new) * c["H"] * c["d"]
        touched = sum(_pages_of(x, c["page"]) - (x - m) // c["page"] for x, m in zip(full, new) if m)
        return {"bytes": (3 if c["type"] == "bf16" else 5) * elems + touched * (4 + 4 * c["H"]),
                "flops": 6 * elems}
    pairs = sum(m * (x - m) + m * (m + 1) // 2 for x, m in zip(full, new))
    seen = sum(x for x, m in zip(full, new) if m)
    blocks = sum(_pages_of(x, c["page"]) for x, m in zip(full, new) if m)
    return {"bytes": 2 * c["Hkv"] * (seen * c["d"] + 4 * blocks) + 4 * blocks +
            sum(new) * c["Hq"] * (4 * c["d"] + 4) + 8 * c["B"],
            "flops": 4.0 * pairs * c["Hq"] * c["d"]}
