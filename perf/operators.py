"""The serving-side operators of the library, as cases that can be timed and compared.

Four groups, which a serving loop runs one after the other and of which the first is also part of training:

  rotary   rotary positions on q and k (and their gradients), half and interleaved pairs, part of the head, scaled frequencies
  append   new keys and values (rotated on the way) into the pages of a key/value cache, prompts and single tokens
  decode   attention of the last positions of each sequence over its pages, split over the cache's length and joined
  pages    extending, forking, freeing and compacting sequences' pages, with the copies that follow

``own`` false: elementary torch operations in 32 bits (64 for angles).  ``own`` true: the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

BF16 = torch.bfloat16


def listed():
    return [
        # one new token of one sequence, as a latency-bound generation step rotates it
        dict(name="rotary one token", op="rotary", B=1, H=16, H_kv=16, N=1, d=64, r=64, interleaved=False, dtype="bf16",
             scaling="none", start=1000, token_major=True, backward=False),
        # the benchmark's grouped-head prefill shape, forward and gradients of a training step
        dict(name="rotary training 8192", op="rotary", B=2, H=32, H_kv=8, N=8192, d=128, r=128, interleaved=False,
             dtype="bf16", scaling="none", start=0, token_major=True, backward=True),
        # a long-context tail in fp32: odd length, wide head of which a part turns, neighbouring pairs, far positions
        dict(name="rotary far ragged fp32", op="rotary", B=3, H=10, H_kv=5, N=1531, d=256, r=96, interleaved=True,
             dtype="f32", scaling="yarn", start=1000000, token_major=False, backward=True),
        # one token each of a full serving batch
        dict(name="append tokens", op="append", B=64, H=32, H_kv=8, d=128, r=128, interleaved=False, page=16, N=1,
             length=4096, ragged=True, packed=False, heads_first=False),
        # prompts of mixed lengths, packed, into fresh pages
        dict(name="append prompts", op="append", B=12, H=32, H_kv=8, d=128, r=128, interleaved=False, page=64, N=8192,
             length=8192, ragged=True, packed=True, heads_first=True),
        # one short sequence: latency
        dict(name="decode one short", op="decode", B=1, H=16, H_kv=16, Lq=1, length=301, ragged=False, d=64, page=16,
             heads_first=False),
        # the benchmark's decode shape on pages
        dict(name="decode 16 x 8192", op="decode", B=16, H=32, H_kv=8, Lq=1, length=8192, ragged=False, d=128, page=64,
             heads_first=True),
        # continuous batching: lengths from a few tokens to 16384, small pages, token-major pages
        dict(name="decode ragged batch", op="decode", B=64, H=32, H_kv=8, Lq=1, length=16384, ragged=True, d=128, page=16,
             heads_first=False),
        # four guessed tokens at once, the widest head, pages that end inside a tile
        dict(name="decode four tokens wide", op="decode", B=4, H=16, H_kv=4, Lq=4, length=9001, ragged=True, d=256, page=48,
             heads_first=True),
        # the longest caches of the benchmark's range
        dict(name="decode 16 x 65536", op="decode", B=16, H=32, H_kv=8, Lq=1, length=65536, ragged=False, d=128, page=128,
             heads_first=False),
        # branches of running sequences, one step later
        dict(name="fork and extend", op="fork", S=128, n=48, length=4000, page=32, H_kv=8, d=128, pages=20000,
             heads_first=False),
        # half of the sequences end, the pages of the others move together
        dict(name="free and compact", op="compact", S=64, length=4096, page=64, H_kv=8, d=128, moved=0.9, heads_first=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "decode", "decode", "fork", "compact"])
    d = rng.choice([64, 128, 256])
    H_kv = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([8, 16, 32, 48, 64, 128, 256])
    heads_first = rng.random() < 0.5
    if op == "rotary":
        B = rng.choice([1, 2, 3, 4])
        N = _log(rng, 1, 40_000_000 // (B * H_kv * (group + 1) * d))
        r = rng.choice([d, d, d // 2, 32, d // 4 + 8 if d > 64 else 10])
        return dict(op=op, B=B, H=H_kv * group, H_kv=H_kv, N=min(N, 40000), d=d, r=r, interleaved=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), scaling=rng.choice(["none", "linear", "yarn"]),
                    start=_log(rng, 1, 1_000_000) - 1, token_major=rng.random() < 0.5, backward=rng.random() < 0.6)
    if op == "append":
        packed = rng.random() < 0.5
        B = _log(rng, 1, 128)
        N = _log(rng, 1, max(2, 60_000_000 // (B * H_kv * (group + 2) * d))) if packed else rng.choice([1, 1, 2, 5])
        N = min(N, 20000)
        length = max(N, _log(rng, 1, 3000) + N if not packed else N)
        return dict(op=op, B=B, H=H_kv * group, H_kv=H_kv, d=d, r=rng.choice([d, d // 2]), interleaved=rng.random() < 0.5,
                    page=page, N=N, length=length, ragged=rng.random() < 0.7, packed=packed, heads_first=heads_first)
    if op == "decode":
        B = _log(rng, 1, 200)
        length = _log(rng, 1, min(100_000, 500_000_000 // (B * H_kv * d)))
        return dict(op=op, B=B, H=H_kv * group, H_kv=H_kv, Lq=rng.choice([1, 1, 1, 2, 3, 5, 9]), length=length,
                    ragged=rng.random() < 0.6, d=d, page=page, heads_first=heads_first)
    length = _log(rng, 1, 8000)
    S = _log(rng, 4, max(5, min(256, 400_000_000 // (H_kv * d * (length + page)))))
    if op == "fork":
        n = max(1, S // 2 - rng.randrange(S // 2))
        total = sum(-(-x // page) for x in _lengths(S // 2, length, True))
        return dict(op=op, S=S, n=n, length=length, page=page, H_kv=H_kv, d=d, pages=total + 2 * n + rng.randrange(50),
                    heads_first=heads_first)
    return dict(op=op, S=S, length=length, page=page, H_kv=H_kv, d=d, moved=round(rng.random(), 2), heads_first=heads_first)


# ------------------------------------------------------------------------------------------------- shapes of a case
def _lengths(n, most, ragged, least=1):
    """n sequence lengths up to `most`, spread over the logarithm, the first one the longest; the same for every seed."""
    if not ragged:
        return [most] * n
    rng = random.Random(n * 1000003 + most)
    return [most] + [max(least, int(math.exp(rng.uniform(0.0, math.log(most + 0.99))))) for _ in range(n - 1)]


def _append_lengths(c):
    """(lengths after the call, new tokens) of each sequence."""
    if c["packed"]:
        new = _lengths(c["B"], c["N"], c["ragged"])
        return list(new), new
    return _lengths(c["B"], c["length"], c["ragged"], least=c["N"]), [c["N"]] * c["B"]


def _compact_plan(c):
    """Lengths of the sequences; pages that survive the freeing, pages in all, pages that have to move.
    Sequences 0, 2, 4, ... stay; sequence 4 i + 2 shares the first half of its pages with sequence 4 i."""
    lens = _lengths(c["S"], c["length"], True)
    need = [-(-x // c["page"]) for x in lens]
    shared = [min(need[i - 2], need[i]) // 2 if i % 4 == 2 else 0 for i in range(c["S"])]
    live = sum(need[i] - shared[i] for i in range(0, c["S"], 2))
    total = live + sum(need[i] for i in range(1, c["S"], 2)) + 3
    return lens, need, shared, live, total, int(c["moved"] * min(live, total - live))


def _rotary_tables(c, device):
    """Frequencies (radians per position, float64) and the factor on cos and sin."""
    r, base = c["r"], 10000.0
    f = base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    magnitude = 1.0
    if c.get("scaling") == "linear":
        f = f / 4.0
    elif c.get("scaling") == "yarn":
        s, original = 16.0, 8192
        turn = lambda n: r * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(turn(32)), 0), min(math.ceil(turn(1)), r - 1)
        ramp = ((torch.arange(r // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / s * ramp + f * (1 - ramp)
        magnitude = 0.1 * math.log(s) + 1.0
    return f.to(device), magnitude


# ------------------------------------------------------------------------------------------------- inputs
def _randn(g, shape, dtype=BF16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype) if math.prod(shape) < (1 << 26) else \
        torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _heads(g, B, H, N, d, token_major, dtype=BF16):
    return _randn(g, (B, N, H, d), dtype).transpose(1, 2) if token_major else _randn(g, (B, H, N, d), dtype)


def _pages(g, P, H_kv, page, d, heads_first):
    """[pages, heads, rows, d], as it lies in memory or as a view of [pages, rows, heads, d]."""
    return _randn(g, (P, H_kv, page, d)) if heads_first else _randn(g, (P, page, H_kv, d)).transpose(1, 2)


def _table(seed, lens, page, P, M):
    """A page table whose sequences hold pages in no particular order; -1 behind their ends."""
    order = torch.from_numpy(np.random.RandomState(seed % (1 << 31)).permutation(P).astype(np.int32))
    t = torch.full((len(lens), M), -1, dtype=torch.int32)
    at = 0
    for b, x in enumerate(lens):
        n = -(-x // page)
        t[b, :n] = order[at:at + n]
        at += n
    return t


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "rotary":
        dt = BF16 if c["dtype"] == "bf16" else torch.float32
        s["q"] = _heads(g, c["B"], c["H"], c["N"], c["d"], c["token_major"], dt)
        s["k"] = _heads(g, c["B"], c["H_kv"], c["N"], c["d"], c["token_major"], dt)
        if c["backward"]:
            s["dq"] = _heads(g, c["B"], c["H"], c["N"], c["d"], c["token_major"], dt)
            s["dk"] = _heads(g, c["B"], c["H_kv"], c["N"], c["d"], c["token_major"], dt)
        first = c["start"] + seed % 7
        s["positions"] = torch.arange(first, first + c["N"], dtype=torch.int32, device="cuda")
        s["freqs"], s["magnitude"] = _rotary_tables(c, "cuda")
    elif c["op"] == "append":
        lens, new = _append_lengths(c)
        B, M = c["B"], -(-max(lens) // c["page"])
        P = sum(-(-x // c["page"]) for x in lens) + 5
        s["k_pages"], s["v_pages"] = (_pages(g, P, c["H_kv"], c["page"], c["d"], c["heads_first"]) for _ in range(2))
        s["page_table"] = _table(seed, lens, c["page"], P, M).cuda()
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if c["packed"]:
            s["q"], s["k"], s["v"] = (_randn(g, (sum(new), h, c["d"])) for h in (c["H"], c["H_kv"], c["H_kv"]))
            s["cu_seqlens"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
        else:
            s["q"], s["k"], s["v"] = (_heads(g, B, h, c["N"], c["d"], True) for h in (c["H"], c["H_kv"], c["H_kv"]))
            s["cu_seqlens"] = None
        s["freqs"], s["magnitude"] = _rotary_tables(c, "cuda")
    elif c["op"] == "decode":
        lens = _lengths(c["B"], c["length"], c["ragged"])
        M = -(-max(lens) // c["page"])
        P = sum(-(-x // c["page"]) for x in lens) + 3
        s["k_pages"], s["v_pages"] = (_pages(g, P, c["H_kv"], c["page"], c["d"], c["heads_first"]) for _ in range(2))
        s["page_table"] = _table(seed, lens, c["page"], P, M).cuda()
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = _heads(g, c["B"], c["H"], c["Lq"], c["d"], True)
        s["scale"] = 1.0 / math.sqrt(c["d"])
    else:
        page, S = c["page"], c["S"]
        if c["op"] == "fork":
            lens, P = _lengths(S // 2, c["length"], True) + [0] * (S - S // 2), c["pages"]
            M = -(-(c["length"] + 1) // page)
            table = _table(seed, lens, page, P, M)
            refs = torch.zeros(P, dtype=torch.int32)
            refs[table[table >= 0].long()] = 1
            rng = np.random.RandomState(seed % (1 << 31))
            s["src"] = torch.from_numpy(rng.randint(0, S // 2, c["n"]).astype(np.int32)).cuda()
            s["dst"] = torch.from_numpy((S // 2 + rng.permutation(S - S // 2)[:c["n"]]).astype(np.int32)).cuda()
            s["ones"] = torch.ones(c["n"], dtype=torch.int32, device="cuda")
        else:
            lens, need, shared, live, P, moved = _compact_plan(c)
            M = max(need)
            rng = np.random.RandomState(seed % (1 << 31))
            low, high = rng.permutation(live), live + rng.permutation(P - live)
            keep = rng.permutation(np.concatenate([low[moved:], high[:moved]]))
            rest = np.concatenate([low[:moved], high[moved:]])
            table, refs = torch.full((S, M), -1, dtype=torch.int32), torch.zeros(P, dtype=torch.int32)
            for i in range(S):
                take, n = need[i] - shared[i], shared[i]
                if n:
                    table[i, :n] = table[i - 2, :n]
                own_pages, left = (keep, rest) if i % 2 == 0 else (rest, keep)
                table[i, n:n + take] = torch.from_numpy(own_pages[:take].astype(np.int32))
                keep, rest = (own_pages[take:], left) if i % 2 == 0 else (left, own_pages[take:])
                refs.index_add_(0, table[i, :need[i]].long(), torch.ones(need[i], dtype=torch.int32))
            s["ended"] = torch.arange(1, S, 2, dtype=torch.int32, device="cuda")
        s["k_pages"], s["v_pages"] = (_pages(g, P, c["H_kv"], page, c["d"], c["heads_first"]) for _ in range(2))
        # the cache's bookkeeping in one buffer, so that a pass can start again from the same state
        s["meta"] = torch.cat([refs, torch.tensor(lens, dtype=torch.int32), table.reshape(-1)]).cuda()
        s["now"] = s["meta"].clone()
        s["refcounts"], s["seq_lens"] = s["now"][:P], s["now"][P:P + S]
        s["page_table"] = s["now"][P + S:].view(S, M)
    return s


# ------------------------------------------------------------------------------------------------- the plain forms
def _turned(x, cos, sin, r, interleaved, inverse=False):
    """x [..., d] in 32 bits with its first r columns turned by the angles of cos, sin (which broadcast over [..., r / 2])."""
    sin = -sin if inverse else sin
    x = x.float()
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., r:]], dim=-1)


def _cos_sin(positions, freqs, magnitude):
    angle = positions.double()[..., None] * freqs
    return (angle.cos() * magnitude).float(), (angle.sin() * magnitude).float()


def _plain_rotary(s):
    c = s["case"]
    cos, sin = _cos_sin(s["positions"], s["freqs"], s["magnitude"])
    turn = lambda x, back: _turned(x, cos, sin, c["r"], c["interleaved"], back).to(x.dtype)  # noqa: E731
    out = [turn(s["q"], False), turn(s["k"], False)]
    return out + [turn(s["dq"], True), turn(s["dk"], True)] if c["backward"] else out


def _plain_append(s):
    c, page = s["case"], s["case"]["page"]
    if s["cu_seqlens"] is not None:
        cu = s["cu_seqlens"].long()
        rows = torch.arange(s["k"].shape[0], device="cuda")
        b = torch.searchsorted(cu, rows, right=True) - 1
        pos = s["seq_lens"].long()[b] - (cu[b + 1] - rows)
        q, k, v = s["q"], s["k"], s["v"]
    else:
        B, N = c["B"], c["N"]
        b = torch.arange(B, device="cuda").repeat_interleave(N)
        pos = (s["seq_lens"].long()[:, None] - N + torch.arange(N, device="cuda")).reshape(-1)
        q, k, v = (s[n].transpose(1, 2).reshape(B * N, -1, c["d"]) for n in ("q", "k", "v"))
    cos, sin = _cos_sin(pos, s["freqs"], s["magnitude"])
    cos, sin = cos[:, None], sin[:, None]
    q = _turned(q, cos, sin, c["r"], c["interleaved"]).to(BF16)
    k = _turned(k, cos, sin, c["r"], c["interleaved"]).to(BF16)
    at = s["page_table"].long()[b, pos // page]
    s["k_pages"].transpose(1, 2)[at, pos % page] = k
    s["v_pages"].transpose(1, 2)[at, pos % page] = v
    if s["cu_seqlens"] is None:
        q = q.view(c["B"], c["N"], c["H"], c["d"]).transpose(1, 2)
    return [q, s["k_pages"], s["v_pages"]]


def _plain_decode(s):
    c, page = s["case"], s["case"]["page"]
    B, H, H_kv, Lq, d = c["B"], c["H"], c["H_kv"], c["Lq"], c["d"]
    M = s["page_table"].shape[1]
    idx = s["page_table"].long().clamp(min=0)

    def cached(p):      # [B, H_kv, M * page, d]
        return p[idx].transpose(1, 2).reshape(B, H_kv, M * page, d).float()

    n = s["seq_lens"].long()[:, None]
    j = torch.arange(M * page, device="cuda")
    last = n - Lq + torch.arange(Lq, device="cuda")                       # the last key each query sees
    seen = (j < n)[:, None, :] & (j <= last[:, :, None])                  # [B, Lq, keys]
    q = s["q"].float().reshape(B, H_kv, H // H_kv, Lq, d)
    x = torch.einsum("bhgqd,bhkd->bhgqk", q, cached(s["k_pages"])) * s["scale"]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = (x - m).exp()
    l = p.sum(-1, keepdim=True)
    v = cached(s["v_pages"]).masked_fill(~(j < n)[:, None, :, None], 0.0)
    o = torch.einsum("bhgqk,bhkd->bhgqd", p, v) / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + l.log()).squeeze(-1)
    return [o.reshape(B, H, Lq, d).to(BF16), lse.reshape(B, H, Lq)]


def _free_pages(refs):
    """Page numbers with the free ones first, lowest first."""
    return torch.sort((refs > 0).int(), stable=True).indices


def _plain_copy(s, copies):
    page = s["case"]["page"]
    copies = copies[copies[:, 0] >= 0].long()
    src, dst, rows = copies[:, 0], copies[:, 1], copies[:, 2]
    keep = (torch.arange(page, device="cuda") < rows[:, None])[:, None, :, None]
    for p in (s["k_pages"], s["v_pages"]):
        p[dst] = torch.where(keep, p[src], p[dst])


def _plain_fork(s):
    page, src, dst = s["case"]["page"], s["src"].long(), s["dst"].long()
    refs, lens, table = s["refcounts"], s["seq_lens"], s["page_table"]
    n, M, free = src.numel(), table.shape[1], (refs == 0).sum()
    # fork: whole pages are shared, the page that is still being filled is copied into a new one
    full, rest = lens[src] // page, lens[src] % page
    want = (rest > 0).int()
    ok = (want == 0) | (want.cumsum(0) <= free)
    status = torch.where(ok, 0, 4).int()
    new = _free_pages(refs)[(want.cumsum(0) - 1).clamp(min=0)].int()
    taken = ok & (want > 0)
    col = torch.arange(M, device="cuda")
    row = torch.where(col < full[:, None], table[src], table[dst])
    old = table[src].gather(1, full[:, None].long().clamp(max=M - 1)).squeeze(1)
    row = torch.where((col == full[:, None]) & taken[:, None], new[:, None], row)
    table[dst] = torch.where(ok[:, None], row, table[dst])
    use = ((col < full[:, None]) & ok[:, None]).int()
    refs.index_add_(0, table[src].clamp(min=0).reshape(-1).long(), use.reshape(-1))
    refs.index_add_(0, new.long(), taken.int())
    lens[dst] = torch.where(ok, lens[src], lens[dst])
    copies = torch.full((n, 3), -1, dtype=torch.int32, device="cuda")
    listed_ = torch.stack([old, new, rest], 1)[taken].int()
    copies[:listed_.shape[0]] = listed_
    _plain_copy(s, copies)
    # extend the new sequences by a token each
    status2 = _plain_extend(s, dst, s["ones"])
    return [status, copies, status2]


def _plain_extend(s, seqs, tokens):
    page = s["case"]["page"]
    refs, lens, table = s["refcounts"], s["seq_lens"], s["page_table"]
    M, free = table.shape[1], (refs == 0).sum()
    have, after = -(-lens[seqs] // page), -(-(lens[seqs] + tokens) // page)
    want = after - have
    upto = want.cumsum(0)
    ok = (want == 0) | (upto <= free)
    col = torch.arange(M, device="cuda")
    fill = (col >= have[:, None]) & (col < after[:, None]) & ok[:, None]
    rank = (upto - want)[:, None] + col - have[:, None]
    pages = _free_pages(refs)[rank.clamp(0, refs.numel() - 1)].int()
    table[seqs] = torch.where(fill, pages, table[seqs])
    refs.index_add_(0, pages.reshape(-1).long(), fill.int().reshape(-1))
    lens[seqs] = torch.where(ok, lens[seqs] + tokens, lens[seqs])
    return torch.where(ok, 0, 4).int()


def _plain_compact(s):
    page, ended = s["case"]["page"], s["ended"].long()
    refs, lens, table = s["refcounts"], s["seq_lens"], s["page_table"]
    P, col = refs.numel(), torch.arange(table.shape[1], device="cuda")
    # free
    used = col < (-(-lens[ended] // page))[:, None]
    refs.index_add_(0, table[ended].clamp(min=0).reshape(-1).long(), -used.int().reshape(-1))
    table[ended] = torch.where(used, -1, table[ended])
    lens[ended] = 0
    # compact: the j-th page in use behind the first `live` ones moves to the j-th free page among them
    idx = torch.arange(P, device="cuda")
    live = (refs > 0).sum()
    mover, hole = (refs > 0) & (idx >= live), (refs == 0) & (idx < live)
    src, dst = idx[mover], idx[hole]
    copies = torch.full((P // 2, 3), -1, dtype=torch.int32, device="cuda")
    copies[:src.numel()] = torch.stack([src, dst, torch.full_like(src, page)], 1).int()
    place = idx.clone()
    place[src] = dst
    used = col < (-(-lens // page))[:, None]
    table.copy_(torch.where(used, place[table.clamp(min=0).long()].int(), table))
    refs[dst] = refs[src]
    refs[src] = 0
    _plain_copy(s, copies)
    return [copies]


# ------------------------------------------------------------------------------------------------- one pass
def run(state):
    s, c = state, state["case"]
    if own:
        import exact_io_aware_100_b200 as fa
    if c["op"] == "rotary":
        if not own:
            return _plain_rotary(s)
        out = fa.rotary(s["q"], s["k"], s["freqs"], s["positions"], c["interleaved"], s["magnitude"])
        if c["backward"]:
            out += fa.rotary_backward(s["dq"], s["dk"], s["freqs"], s["positions"], c["interleaved"], s["magnitude"])
        return out
    if c["op"] == "append":
        if not own:
            return _plain_append(s)
        q = fa.paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"], q=s["q"],
                            freqs=s["freqs"], interleaved=c["interleaved"], magnitude=s["magnitude"],
                            cu_seqlens=s["cu_seqlens"])
        return [q, s["k_pages"], s["v_pages"]]
    if c["op"] == "decode":
        if not own:
            return _plain_decode(s)
        return fa.paged_decode(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"], True, s["scale"])
    s["now"].copy_(s["meta"])
    book = (s["page_table"], s["seq_lens"], s["refcounts"])
    if not own:
        told = _plain_fork(s) if c["op"] == "fork" else _plain_compact(s)
    elif c["op"] == "fork":
        copies, status = fa.pages_fork(*book, c["page"], s["src"], s["dst"])
        fa.pages_copy(s["k_pages"], s["v_pages"], copies)
        told = [status, copies, fa.pages_extend(*book, c["page"], s["dst"], s["ones"])]
    else:
        fa.pages_free(*book, c["page"], s["ended"])
        copies = fa.pages_compact(*book, c["page"])
        fa.pages_copy(s["k_pages"], s["v_pages"], copies)
        told = [copies]
    return told + [s["page_table"], s["seq_lens"], s["refcounts"], s["k_pages"], s["v_pages"]]


def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["B"] * (c["H"] + c["H_kv"]) * c["N"] * c["d"]
        passes = 2 if c["backward"] else 1
        return {"bytes": passes * (2 * n * (2 if c["dtype"] == "bf16" else 4) + 4 * c["N"]),
                "flops": passes * 3 * n * c["r"] // c["d"]}
    if c["op"] == "append":
        _, new = _append_lengths(c)
        t = sum(new)
        return {"bytes": t * (c["H"] + 2 * c["H_kv"]) * c["d"] * 2 * 2, "flops": 3 * t * (c["H"] + c["H_kv"]) * c["r"]}
    if c["op"] == "decode":
        lens = _lengths(c["B"], c["length"], c["ragged"])
        keys, rows = sum(lens), c["B"] * c["H"] * c["Lq"]
        return {"bytes": keys * c["H_kv"] * c["d"] * 4 + rows * (c["d"] * 4 + 4) + 4 * sum(-(-x // c["page"]) for x in lens),
                "flops": 4 * keys * c["H"] * c["Lq"] * c["d"]}
    row = c["H_kv"] * c["d"] * 2 * 2 * 2          # a row of K and of V, read and written
    if c["op"] == "fork":
        lens = _lengths(c["S"] // 2, c["length"], True)
        mean = sum(x % c["page"] for x in lens) / len(lens)
        pages = sum(-(-x // c["page"]) for x in lens) / len(lens)
        return {"bytes": c["n"] * (mean * row + 4 * 4 * pages) + 2 * 4 * c["pages"], "flops": 0}
    lens, need, shared, live, total, moved = _compact_plan(c)
    return {"bytes": moved * c["page"] * row + 4 * 4 * sum(need) + 2 * 4 * total, "flops": 0}


# ------------------------------------------------------------------------------------------------- the definitions in 64 bits
def _exact_turn(x, positions, freqs, magnitude, interleaved, inverse=False):
    """x [rows, heads, d] in float64: each pair of columns is a complex number, multiplied by magnitude * e^(+-i position f)."""
    r = 2 * freqs.numel()
    x = x.double()
    pairs = x[..., :r].unflatten(-1, (r // 2, 2) if interleaved else (2, r // 2))
    pairs = pairs if interleaved else pairs.transpose(-1, -2)
    z = torch.view_as_complex(pairs.contiguous())
    angle = positions.double()[:, None] * freqs[None, :]
    w = torch.polar(torch.full_like(angle, magnitude), -angle if inverse else angle)
    y = torch.view_as_real(z * w[:, None])
    y = y if interleaved else y.transpose(-1, -2)
    return torch.cat([y.reshape(*x.shape[:-1], r), x[..., r:]], -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rotary":
        def turned(x, back):
            y = [_exact_turn(x[b].transpose(0, 1), s["positions"], s["freqs"], s["magnitude"], c["interleaved"], back)
                 for b in range(c["B"])]
            return torch.stack(y).transpose(1, 2)
        out = [turned(s["q"], False), turned(s["k"], False)]
        return out + [turned(s["dq"], True), turned(s["dk"], True)] if c["backward"] else out
    if c["op"] == "append":
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        lens, new = _append_lengths(c)
        start, qs = 0, []
        for b, (n, t) in enumerate(zip(lens, new)):
            if c["packed"]:
                q, k, v = (s[x][start:start + t] for x in ("q", "k", "v"))
            else:
                q, k, v = (s[x][b].transpose(0, 1) for x in ("q", "k", "v"))
            start += t
            pos = torch.arange(n - t, n, device="cuda")
            qs.append(_exact_turn(q, pos, s["freqs"], s["magnitude"], c["interleaved"]))
            where = s["page_table"][b, (pos // c["page"])].long()
            kp[where, :, pos % c["page"]] = _exact_turn(k, pos, s["freqs"], s["magnitude"], c["interleaved"])
            vp[where, :, pos % c["page"]] = v.double()
        q = torch.cat(qs) if c["packed"] else torch.stack(qs).transpose(1, 2)
        return [q, kp, vp]
    if c["op"] == "decode":
        lens = _lengths(c["B"], c["length"], c["ragged"])
        os_, ls = [], []
        for b, n in enumerate(lens):
            rows = s["page_table"][b, :-(-n // c["page"])].long()
            k, v = (p[rows].double().transpose(0, 1).flatten(1, 2)[:, :n].repeat_interleave(c["H"] // c["H_kv"], 0)
                    if n * c["H"] * c["d"] < (1 << 28) else None for p in (s["k_pages"], s["v_pages"]))
            heads = []
            for h in range(c["H"]):
                if k is None:
                    kh, vh = (p[rows, h // (c["H"] // c["H_kv"])].double().flatten(0, 1)[:n] for p in (s["k_pages"], s["v_pages"]))
                else:
                    kh, vh = k[h], v[h]
                x = s["q"][b, h].double() @ kh.T * s["scale"]
                hidden = torch.ones_like(x).triu(n - c["Lq"] + 1).bool()
                x[hidden] = -math.inf
                l = torch.logsumexp(x, -1)
                p = torch.where(hidden, torch.zeros_like(x), (x - torch.where(l == -math.inf, 0.0, l)[:, None]).exp())
                heads.append((p @ vh, l))
            os_.append(torch.stack([h[0] for h in heads]))
            ls.append(torch.stack([h[1] for h in heads]))
        return [torch.stack(os_), torch.stack(ls)]
    # page bookkeeping, one request after the other on the host; only the cache's contents are values
    page, refs = c["page"], s["refcounts"].tolist()
    lens, table = s["seq_lens"].tolist(), s["page_table"].tolist()
    moves, kp, vp = [], s["k_pages"].double(), s["v_pages"].double()
    if c["op"] == "fork":
        free = [i for i, n in enumerate(refs) if n == 0]
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            if lens[a] % page and free:
                moves.append((table[a][lens[a] // page], free.pop(0), lens[a] % page))
        hold = 3
    else:
        for b in s["ended"].tolist():
            for p in table[b][:-(-lens[b] // page)]:
                refs[p] -= 1
        live = sum(n > 0 for n in refs)
        holes = iter([i for i in range(live) if refs[i] == 0])
        moves = [(i, next(holes), page) for i in range(live, len(refs)) if refs[i] > 0]
        hold = 1
    for src, dst, rows in moves:
        kp[dst, :, :rows], vp[dst, :, :rows] = kp[src, :, :rows].clone(), vp[src, :, :rows].clone()
    return [None] * (hold + 3) + [kp, vp]
