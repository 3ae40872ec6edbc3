"""The paged cache on the GPU against the float64 oracle: append, and attention over pages.

O and lse: the bounds of the dense decode (helpers).  Appended values are copies (bit for bit) or, when turned, what
``rotary`` gives for the same tokens (bit for bit), which has its own parity tests.
"""
import numpy as np
import pytest

from helpers import assert_close, to_f64
from oracle import serving as ref

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _cache(P, H_kv, page, d, heads_first, fill=NAN):
    """k, v pages full of NaN: what nobody wrote must not matter."""
    import torch
    shape = (P, H_kv, page, d) if heads_first else (P, page, H_kv, d)
    return [t if heads_first else t.transpose(1, 2)
            for t in (torch.full(shape, fill, device="cuda", dtype=torch.bfloat16) for _ in range(2))]


def _table(lens, page, P, M=None, seed=0):
    import torch
    order = np.random.default_rng(seed).permutation(P)
    M = M or max(1, -(-max(lens) // page))
    t, at = np.full((len(lens), M), -1, np.int32), 0
    for b, n in enumerate(lens):
        k = -(-n // page)
        t[b, :k] = order[at:at + k]
        at += k
    return torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def _fill(kp, vp, table, lens, page, k_scale=1.0, seed=0):
    """Random keys and values at the positions in use."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    for b, n in enumerate(lens):
        for e in range(-(-n // page)):
            rows = min(page, n - e * page)
            for p, s in ((kp, k_scale), (vp, 1.0)):
                x = torch.randn(p.shape[1], rows, p.shape[3], device="cuda", generator=g) * s
                p[int(table[b, e]), :, :rows] = x.bfloat16()


def _host(p):
    return np.nan_to_num(to_f64(p))


def _check_decode(q, kp, vp, table, lens, causal=True, scale=None, lse_tol=1e-5):
    import torch
    import exact_io_aware_100_b200 as fa
    o, lse = fa.paged_decode(q, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), causal, scale)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    ro, rl = ref.paged_decode(to_f64(q), _host(kp), _host(vp), table.cpu().numpy(), lens,
                              1 / np.sqrt(q.shape[-1]) if scale is None else scale, causal)
    assert_close("O", to_f64(o), ro, scale_max_abs=True)
    got, empty = to_f64(lse), np.isneginf(rl)
    assert np.array_equal(np.isneginf(got), empty) and not np.isnan(got).any()
    # lse: fp32 scores of up to |s| and an fp32 sum, a few steps of each
    assert (np.abs(got - rl)[~empty] <= lse_tol * np.maximum(1, np.abs(rl[~empty]))).all()
    assert not np.any(to_f64(o)[empty]) if empty.any() else True
    return o, lse


@pytest.mark.parametrize("B,H,H_kv,N,lens,d,page,heads_first,causal", [
    (1, 1, 1, 1, [1], 64, 16, True, True),                       # one key
    (2, 8, 2, 1, [1000, 0], 128, 16, False, True),               # and an empty sequence
    (3, 4, 4, 1, [15, 16, 17], 64, 16, True, True),              # around a page's end
    (4, 8, 1, 1, [63, 64, 65, 129], 128, 64, False, True),       # around a tile's end
    (2, 16, 1, 1, [700, 333], 128, 8, True, True),               # the smallest pages, 16 rows per head
    (2, 6, 2, 3, [2, 500], 128, 48, True, True),                 # pages that end inside a tile; more queries than keys
    (2, 6, 2, 3, [2, 500], 128, 48, True, False),
    (1, 4, 2, 16, [300], 64, 32, False, True),                   # 32 rows per head: several row tiles
    (1, 24, 1, 5, [1030], 128, 128, True, True),                 # 120 rows
    (2, 8, 4, 2, [3001, 77], 256, 16, False, True),
    (1, 16, 1, 1, [5000], 256, 256, True, False),
    (1, 3, 1, 1, [40000], 128, 64, True, True),                  # one long sequence: split over the GPU
    (70, 2, 1, 1, list(range(0, 700, 10)), 64, 24, False, True), # many sequences of every length
    (1, 7, 7, 1, [129], 128, 40, True, True),
])
def test_decode_matches_oracle(B, H, H_kv, N, lens, d, page, heads_first, causal):
    import torch
    P = sum(-(-n // page) for n in lens) + 2
    kp, vp = _cache(P, H_kv, page, d, heads_first)
    table, _ = _table(lens, page, P, seed=B + N)
    _fill(kp, vp, table, lens, page)
    q = torch.randn(B, H, N, d, device="cuda").bfloat16()
    _check_decode(q, kp, vp, table, lens, causal)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_sharp_scores_and_negative_ones(d):
    """Keys times 4: rows that a single key decides; a scale of its own."""
    import torch
    lens, page = [900, 40], 32
    kp, vp = _cache(40, 2, page, d, True)
    table, _ = _table(lens, page, 40, seed=3)
    _fill(kp, vp, table, lens, page, k_scale=4.0)
    q = torch.randn(2, 8, 2, d, device="cuda").bfloat16()
    _check_decode(q, kp, vp, table, lens, scale=0.3)
    kp.copy_(-kp.abs())
    _check_decode(q.abs(), kp, vp, table, lens, scale=1.0)       # every score far below zero


def test_decode_query_and_table_views():
    """q of token-major and of wider memory, a table with spare columns and garbage behind the ends, shared pages."""
    import torch
    import exact_io_aware_100_b200 as fa
    lens, page = [100, 37, 100], 16
    kp, vp = _cache(30, 2, page, 128, False)
    small, sl = _table(lens[:2], page, 30, seed=4)
    _fill(kp, vp, small, lens[:2], page)
    table = torch.randint(-2**31, 2**31 - 1, (3, 60), device="cuda").int()[:, 10:40]    # strided rows
    for b, src in ((0, 0), (1, 1), (2, 0)):                                             # sequence 2 holds 0's pages
        n = -(-lens[b] // page)
        table[b, :n] = small[src, :n]
    wide = torch.randn(3, 2, 8, 256, device="cuda").bfloat16()
    q = wide.transpose(1, 2)[..., 64:192]
    o, lse = _check_decode(q, kp, vp, table, lens)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o2, lse2 = fa.paged_decode(q.contiguous(), kp, vp, table, sl)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o3, _ = fa.paged_decode(q.contiguous(), kp.contiguous(), vp.contiguous(), table, sl)  # the other page layout
    assert torch.equal(o, o3)


def test_decode_matches_the_dense_decode():
    import torch
    import exact_io_aware_100_b200 as fa
    B, H, H_kv, n, d, page = 2, 8, 2, 513, 128, 32
    k, v = (torch.randn(B, H_kv, n, d, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(B, H, 1, d, device="cuda").bfloat16()
    kp, vp = _cache(40, H_kv, page, d, True)
    table, lens = _table([n] * B, page, 40)
    fa.paged_append(k, v, kp, vp, table, lens)
    o, lse = fa.paged_decode(q, kp, vp, table, lens)
    ro, rl = fa.decode(q, k, v, True)
    # two roundings of one value: a step of bf16 apart at most
    assert ((o.float() - ro.float()).abs() <= 2.0 ** -7 * ro.float().abs() + 1e-3).all()
    assert (lse - rl).abs().max() < 1e-4


def test_decode_repeats_bit_for_bit():
    import torch
    import exact_io_aware_100_b200 as fa
    lens, page = [5000, 3, 900, 12000], 16
    P = sum(-(-n // page) for n in lens)
    kp, vp = _cache(P, 2, page, 128, True)
    table, sl = _table(lens, page, P)
    _fill(kp, vp, table, lens, page)
    q = torch.randn(4, 8, 1, 128, device="cuda").bfloat16()
    o, lse = fa.paged_decode(q, kp, vp, table, sl)
    for _ in range(3):
        o2, lse2 = fa.paged_decode(q, kp, vp, table, sl)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_decode_cache_beyond_32_bit_offsets():
    """Pages more than 2^31 elements into the cache."""
    import torch
    import exact_io_aware_100_b200 as fa
    page, d = 64, 128
    P = (1 << 31) // (page * d) + 8
    kp, vp = (torch.empty(P, 1, page, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    lens = [200]
    table = torch.tensor([[P - 1, 0, P - 3, P // 2]], dtype=torch.int32, device="cuda")
    small = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    _fill(kp, vp, table, lens, page)
    k4, v4 = (p[table[0].long()].contiguous() for p in (kp, vp))
    q = torch.randn(1, 4, 1, d, device="cuda").bfloat16()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = fa.paged_decode(q, kp, vp, table, sl)
    o4, lse4 = _check_decode(q, k4, v4, small, lens)
    assert torch.equal(o, o4) and torch.equal(lse, lse4)
    n = torch.randn(1, 1, 2, d, device="cuda").bfloat16()
    fa.paged_append(n, n, kp, vp, table, sl)
    assert torch.equal(kp[P // 2, :, 6:8], n[0]) and torch.equal(vp[P // 2, :, 6:8], n[0])


def test_decode_bad_pages_and_lengths_are_reported():
    """No fault: the numbers are checked before they are used; other sequences keep their results."""
    import torch
    import exact_io_aware_100_b200 as fa
    lens, page = [100, 100, 100], 16
    kp, vp = _cache(30, 2, page, 128, True)
    table, sl = _table(lens, page, 30)
    _fill(kp, vp, table, lens, page)
    q = torch.randn(3, 4, 1, 128, device="cuda").bfloat16()
    good, _ = fa.paged_decode(q, kp, vp, table, sl)
    assert fa.fa_get_device_status() == fa.FA_OK
    for bad_page, bad_len in ((30, 100), (-1, 100), (2**31 - 1, 100), (5, -3), (5, 113), (5, 2**31 - 1)):
        t, n = table.clone(), sl.clone()
        t[1, 2], n[1] = bad_page, bad_len
        o, _ = fa.paged_decode(q, kp, vp, t, n)
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
        assert fa.fa_get_device_status() == fa.FA_ERR_INVALID
        before = kp.clone(), vp.clone()
        fa.paged_append(q[:, :2], q[:, :2], kp, vp, t, n)
        assert fa.fa_get_device_status() == (fa.FA_OK if bad_len == 100 else fa.FA_ERR_INVALID)
        kp.copy_(before[0])
        vp.copy_(before[1])


@pytest.mark.parametrize("B,H,H_kv,N,lens,d,page,heads_first,r,interleaved", [
    (1, 2, 1, 1, [1], 64, 16, True, 64, False),
    (3, 4, 2, 1, [16, 17, 1], 128, 16, False, 128, False),
    (2, 4, 2, 5, [3, 70], 128, 8, True, 64, True),          # padding: the first sequence is shorter than N
    (2, 3, 3, 1, [0, 9], 256, 48, False, 256, True),        # an idle slot
    (1, 1, 1, 300, [300], 64, 32, True, 40, False),
    (2, 8, 2, 33, [100, 40], 128, 64, False, 0, False),     # not turned
])
def test_append_writes_the_right_rows(B, H, H_kv, N, lens, d, page, heads_first, r, interleaved):
    import torch
    import exact_io_aware_100_b200 as fa
    P = sum(-(-max(n, 1) // page) for n in lens) + 2
    kp, vp = _cache(P, H_kv, page, d, heads_first, fill=3.0)
    table, sl = _table(lens, page, P, seed=N)
    q, k, v = (torch.randn(B, h, N, d, device="cuda").bfloat16() for h in (H, H_kv, H_kv))
    freqs = fa.rotary_frequencies(r)[0] if r else None
    pos = sl[:, None] - N + torch.arange(N, dtype=torch.int32, device="cuda")
    tq, tk = fa.rotary(q, k, freqs, pos, interleaved, 1.1) if r else (q, k)
    hk, hv = ref.paged_append(to_f64(kp), to_f64(vp), table.cpu().numpy(), lens,
                              [(to_f64(tk[b]), to_f64(v[b])) for b in range(B)])
    got = fa.paged_append(k, v, kp, vp, table, sl, q=q, freqs=freqs, interleaved=interleaved, magnitude=1.1)
    assert fa.fa_get_device_status() == fa.FA_OK
    assert np.array_equal(to_f64(kp), hk) and np.array_equal(to_f64(vp), hv)
    want = tq.masked_fill((pos < 0)[:, None, :, None], 0.0)
    assert torch.equal(got, want)
    kp.fill_(3.0)
    assert fa.paged_append(k, v, kp, vp, table, sl, freqs=freqs, interleaved=interleaved, magnitude=1.1) is None
    assert np.array_equal(to_f64(kp), hk)
    fa.paged_append(k, v, kp, vp, table, sl, q=q, freqs=freqs, interleaved=interleaved, magnitude=1.1, out=q)
    assert torch.equal(q, want)


@pytest.mark.parametrize("cu,lens", [
    ([0, 5, 5, 40, 41], [5, 20, 60, 1]),            # a prompt, an idle sequence, a later piece of one, a token
    ([2, 9], [7]),                                  # rows before the first sequence
    ([0, 30], [12]),                                # 18 rows of padding
])
def test_append_packed(cu, lens):
    """Rows outside every sequence and padding rows touch nothing and come back as zeros, or unchanged in place."""
    import torch
    import exact_io_aware_100_b200 as fa
    H, H_kv, d, page, total = 4, 2, 128, 16, 45
    P = sum(-(-n // page) for n in lens) + 1
    kp, vp = _cache(P, H_kv, page, d, True, fill=3.0)
    table, sl = _table(lens, page, P)
    q, k, v = (torch.randn(total, h, d, device="cuda").bfloat16() for h in (H, H_kv, H_kv))
    freqs, _ = fa.rotary_frequencies(d)
    pos = torch.full((total,), -1, dtype=torch.int32)
    outside = torch.ones(total, dtype=torch.bool)
    for b, n in enumerate(lens):
        t = cu[b + 1] - cu[b]
        pos[cu[b]:cu[b + 1]] = torch.arange(n - t, n, dtype=torch.int32)
        outside[cu[b]:cu[b + 1]] = False
    pos, outside = pos.cuda(), outside.cuda()
    tq, tk = fa.rotary(q, k, freqs, pos)
    hk, hv = ref.paged_append(to_f64(kp), to_f64(vp), table.cpu().numpy(), lens, [
        (to_f64(tk[cu[b]:cu[b + 1]].transpose(0, 1)), to_f64(v[cu[b]:cu[b + 1]].transpose(0, 1))) for b in range(len(lens))])
    dcu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    got = fa.paged_append(k, v, kp, vp, table, sl, q=q, freqs=freqs, cu_seqlens=dcu)
    assert fa.fa_get_device_status() == fa.FA_OK
    assert np.array_equal(to_f64(kp), hk) and np.array_equal(to_f64(vp), hv)
    zero = tq.masked_fill((pos < 0)[:, None, None], 0.0)
    assert torch.equal(got, zero)
    fa.paged_append(k, v, kp, vp, table, sl, q=q.clone(), freqs=freqs, cu_seqlens=dcu, out=(mine := q.clone()))
    assert torch.equal(mine, zero)
    fa.paged_append(k, v, kp, vp, table, sl, q=mine.copy_(q), freqs=freqs, cu_seqlens=dcu, out=mine)
    assert torch.equal(mine, torch.where(outside[:, None, None], q, zero))


def test_append_bad_offsets_are_reported():
    import torch
    import exact_io_aware_100_b200 as fa
    kp, vp = _cache(8, 1, 16, 64, True, fill=3.0)
    table, sl = _table([20, 20], 16, 8)
    k = torch.randn(10, 1, 64, device="cuda").bfloat16()
    before = kp.clone()
    for cu in ([0, 4, 11], [-5, 4, 4]):
        fa.paged_append(k, k, kp, vp, table, sl, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert fa.fa_get_device_status() == fa.FA_ERR_INVALID
    kp.copy_(before)
    fa.paged_append(k, k, kp, vp, table, sl, cu_seqlens=torch.tensor([0, 7, 3], dtype=torch.int32, device="cuda"))
    fa.fa_get_device_status()


def test_decode_two_streams_and_a_graph():
    """Calls that overlap, each with a workspace of its own; a captured call follows lengths and tables that change."""
    import torch
    import exact_io_aware_100_b200 as fa
    page, lens = 16, [3000, 50]
    P = 300
    kp, vp = _cache(P, 2, page, 128, True, fill=0.0)
    kp.copy_(torch.randn(kp.shape, device="cuda"))
    vp.copy_(torch.randn(vp.shape, device="cuda"))
    table, sl = _table([4000, 400], page, P)
    sl.copy_(torch.tensor(lens, dtype=torch.int32))
    q = torch.randn(2, 8, 1, 128, device="cuda").bfloat16()
    want = fa.paged_decode(q, kp, vp, table, sl)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [fa.paged_decode(q, kp, vp, table, sl, stream=s) for s in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(g[0], want[0]) and torch.equal(g[1], want[1]) for g in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.paged_decode(q, kp, vp, table, sl)
    for lens in ([3000, 50], [1, 0], [4000, 399]):
        sl.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ro, rl = fa.paged_decode(q, kp, vp, table, sl)
        assert torch.equal(o, ro) and torch.equal(lse, rl)
    assert fa.fa_get_device_status() == fa.FA_OK


def _reference(q, kp, vp, table, lens, causal, scale):
    """Float64 attention of the gathered cache, one sequence at a time, on the device."""
    import torch
    B, H, N, d = q.shape
    H_kv, page = kp.shape[1:3]
    o, lse = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.full((B, H, N), -float("inf"), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        rows = table[b, :-(-n // page)].long()
        k, v = (p[rows].transpose(0, 1).reshape(H_kv, -1, d)[:, :n].double().repeat_interleave(H // H_kv, 0) for p in (kp, vp))
        x = q[b].double() @ k.transpose(1, 2) * scale
        if causal:
            hidden = torch.arange(n, device="cuda")[None, :] > (n - N + torch.arange(N, device="cuda"))[:, None]
            x.masked_fill_(hidden, -float("inf"))
        lse[b] = torch.logsumexp(x, -1)
        top = lse[b].masked_fill(lse[b] == -float("inf"), 0.0)
        o[b] = (x - top[..., None]).exp() @ v
    return o, lse


def _random_decode(seed, rng, d, page, H_kv, group, N, B, most, idle):
    """One call on random lengths up to `most`, NaN wherever no key is, against float64."""
    import torch
    import exact_io_aware_100_b200 as fa
    pick = lambda *x: x[int(rng.integers(len(x)))]  # noqa: E731
    lens = [most] + [int(np.exp(rng.uniform(0, np.log(most + 0.99)))) - pick(0, 0, idle) for _ in range(B - 1)]
    P = sum(-(-n // page) for n in lens) + 3
    kp, vp = _cache(P, H_kv, page, d, pick(True, False), fill=NAN)
    table, sl = _table(lens, page, P, M=-(-most // page) + pick(0, 0, 7), seed=seed)
    for p in (kp, vp):                               # values at the positions in use, NaN everywhere else
        for b, n in enumerate(lens):
            if n:
                rows = table[b, :-(-n // page)].long()
                x = torch.full((len(rows) * page, H_kv, d), NAN, device="cuda")
                x[:n] = torch.randn(n, H_kv, d, device="cuda")
                p[rows] = x.view(len(rows), page, H_kv, d).transpose(1, 2).bfloat16()
    q = torch.randn(B, N, H_kv * group, d, device="cuda").bfloat16().transpose(1, 2)
    causal, scale = pick(True, False), pick(None, 0.2)
    o, lse = fa.paged_decode(q, kp, vp, table, sl, causal, scale)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    ro, rl = _reference(q, kp, vp, table, lens, causal, 1 / np.sqrt(d) if scale is None else scale)
    assert_close("O", to_f64(o), ro.cpu().numpy(), scale_max_abs=True)
    rl, got = rl.cpu().numpy(), to_f64(lse)
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(got), empty) and not np.isnan(got).any()
    assert (np.abs(got[~empty] - rl[~empty]) <= 1e-5 * np.maximum(1, np.abs(rl[~empty]))).all()
    assert not to_f64(o)[empty].any()


@pytest.mark.parametrize("seed", range(40))
def test_decode_anywhere_in_the_range(seed):
    """Sizes, lengths and layouts at random: cut and uncut pairs, every row tile, every box, idle and tiny sequences."""
    rng = np.random.default_rng(9000 + seed)
    pick = lambda *x: x[int(rng.integers(len(x)))]  # noqa: E731
    d, page, H_kv, group, N = pick(64, 128, 256), pick(8, 16, 24, 32, 48, 64, 128), pick(1, 2, 5, 8), pick(1, 2, 3, 4, 8), pick(1, 1, 2, 4, 9)
    B = int(np.exp(rng.uniform(0, np.log(160))))
    most = int(np.exp(rng.uniform(0, np.log(min(20000, 6_000_000 // (B * H_kv * d) * 8 + 2)))))
    _random_decode(seed, rng, d, page, H_kv, group, N, B, most, 1)


@pytest.mark.parametrize("seed", range(36))
def test_decode_short_tables(seed):
    """Tables of 1 to 70 tiles and 1 to 1300 pairs: pairs of a warp, of a block, and cut ones, one query row to 40."""
    rng = np.random.default_rng(400 + seed)
    pick = lambda *x: x[int(rng.integers(len(x)))]  # noqa: E731
    d = (64, 128, 256)[seed % 3]
    H_kv = pick(1, 2, 4, 8)
    B = max(1, int(np.exp(rng.uniform(0, np.log(1300 / H_kv)))))
    tiles = int(np.exp(rng.uniform(0, np.log(70))))
    most = max(1, tiles * (32 if d == 64 else 16) - pick(0, 1, 5, 15))
    _random_decode(seed, rng, d, pick(8, 16, 40, 64), H_kv, pick(1, 2, 4, 8), pick(1, 1, 1, 2, 5), B, most, 1)


def test_calls_from_several_threads():
    import threading

    import torch
    import exact_io_aware_100_b200 as fa
    page, lens = 16, [3000, 50]
    P = 200
    kp, vp = _cache(P, 2, page, 128, True, fill=0.0)
    kp.copy_(torch.randn(kp.shape, device="cuda"))
    vp.copy_(torch.randn(vp.shape, device="cuda"))
    table, sl = _table(lens, page, P)
    q = torch.randn(2, 8, 1, 128, device="cuda").bfloat16()
    freqs, _ = fa.rotary_frequencies(128)
    want, turned = fa.paged_decode(q, kp, vp, table, sl), fa.rotary(q, None, freqs)[0]
    torch.cuda.synchronize()
    bad = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(50):
                o, lse = fa.paged_decode(q, kp, vp, table, sl)
                y, _ = fa.rotary(q, None, freqs)
                stream.synchronize()
                if not (torch.equal(o, want[0]) and torch.equal(lse, want[1]) and torch.equal(y, turned)):
                    bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and fa.fa_get_device_status() == fa.FA_OK


@pytest.mark.parametrize("d,page,H_kv,group,N,B,most", [
    (64, 8, 1, 4, 1, 3000, 700),       # more sequences than planning threads, most of them short, some empty
    (128, 16, 2, 2, 300, 1, 1000),     # a piece of a prompt: 600 rows per key/value head
    (64, 32, 1, 2, 70, 3, 40),         # more queries than keys
    (256, 64, 2, 3, 40, 2, 5000),
    (128, 24, 1, 1, 1, 1, 30000),      # one pair over the whole GPU
])
def test_decode_large_in_one_way(d, page, H_kv, group, N, B, most):
    _random_decode(77, np.random.default_rng(d + N), d, page, H_kv, group, N, B, most, 1)


def test_decode_bad_pages_in_a_long_table_are_reported():
    """As above, where pairs are cut: other sequences keep their results."""
    import torch
    import exact_io_aware_100_b200 as fa
    lens, page = [2000, 2000, 2000], 16
    P = 400
    kp, vp = _cache(P, 2, page, 64, True)
    table, sl = _table(lens, page, P, M=300)
    _fill(kp, vp, table, lens, page)
    q = torch.randn(3, 4, 1, 64, device="cuda").bfloat16()
    good, glse = fa.paged_decode(q, kp, vp, table, sl)
    assert fa.fa_get_device_status() == fa.FA_OK
    for bad_page, bad_len in ((P, 2000), (-1, 2000), (2**31 - 1, 2000), (5, -3), (5, 4801), (5, 2**31 - 1)):
        t, n = table.clone(), sl.clone()
        t[1, 100], n[1] = bad_page, bad_len
        o, lse = fa.paged_decode(q, kp, vp, t, n)
        assert fa.fa_get_device_status() == fa.FA_ERR_INVALID
        if bad_len == 2000:                          # the line is cut at the same places: the same bits
            assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
        # else: other partial sums, each of them 32-bit, and one rounding of o
        assert ((o[[0, 2]].float() - good[[0, 2]].float()).abs() <= 2.0 ** -7 * good[[0, 2]].float().abs() + 1e-6).all()
        assert (lse[[0, 2]] - glse[[0, 2]]).abs().max() < 1e-5


def test_keys_and_values_that_are_not_finite():
    """A NaN or an infinity among the keys a row sees comes out as NaN, in the rows that see it only."""
    import torch
    import exact_io_aware_100_b200 as fa
    for n, M in ((60, 4), (3000, 188)):
        kp, vp = _cache(400, 2, 16, 64, True)
        table, sl = _table([n, n], 16, 400, M=M)
        q = torch.randn(2, 4, 1, 64, device="cuda").bfloat16()
        for pages, value in ((kp, NAN), (vp, NAN), (vp, float("inf"))):
            _fill(kp, vp, table, [n, n], 16)
            want = fa.paged_decode(q, kp, vp, table, sl)
            pages[int(table[0, 1]), 1, 3] = value    # head 1 of sequence 0
            o, lse = fa.paged_decode(q, kp, vp, table, sl)
            assert torch.equal(o[1], want[0][1]) and torch.equal(o[0, :2], want[0][0, :2])
            assert not torch.isfinite(o[0, 2:].float()).any()
            assert torch.isnan(lse[0, 2:]).all() if pages is kp else torch.equal(lse, want[1])
