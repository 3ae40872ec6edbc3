"""Page bookkeeping and copies on the GPU against the oracle's one-request-at-a-time bookkeeping (equal, not near), and
a serving loop of all the operators together."""
import numpy as np
import pytest

from helpers import assert_close, to_f64
from oracle import serving as ref

pytestmark = pytest.mark.gpu


def _state(S, P, M, page, lens, seed=0, stride=None):
    """Device (table, lens, refs) and the oracle's state, sequences on pages in no order."""
    import torch
    order = np.random.default_rng(seed).permutation(P)
    t, refs, at = np.full((S, M), -1, np.int32), np.zeros(P, np.int32), 0
    for b, n in enumerate(lens):
        k = -(-n // page)
        t[b, :k] = order[at:at + k]
        refs[order[at:at + k]] = 1
        at += k
    full = np.zeros(S, np.int32)
    full[:len(lens)] = lens
    wide = torch.full((S, stride or M), 77, dtype=torch.int32, device="cuda")
    table = wide[:, :M]
    table.copy_(torch.from_numpy(t))
    return (table, torch.from_numpy(full).cuda(), torch.from_numpy(refs).cuda()), ref.Pages(t, full, refs, page), wide


def _i(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _same(dev, want):
    for name, d, w in zip(("table", "lens", "refs"), dev, (want.table, want.lens, want.refs)):
        assert np.array_equal(d.cpu().numpy(), w), name


def _ok(code=0):
    import exact_io_aware_100_b200 as fa
    assert fa.fa_get_device_status() == code


@pytest.mark.parametrize("S,P,M,page,lens,seqs,tokens", [
    (1, 1, 1, 8, [0], [0], [8]),                                      # the only page
    (4, 20, 5, 16, [10, 16, 0, 80], [0, 1, 2, 3], [6, 1, 33, 0]),     # up to a page's end, over it, from nothing, nothing
    (4, 9, 5, 16, [10, 16, 0, 0], [3, 0, 2, 1], [80, 30, 70, 17]),    # pages run out on the way
    (3, 20, 3, 4, [5, 0, 12], [0, 0, 2, -1, 3, 1, 1], [1, 1, 1, 1, 1, -2, 9]),   # repeated, full, out of range, negative
    (300, 20000, 70, 16, [], list(range(299, -1, -1)), [(i * 37) % 1100 for i in range(300)]),
    (1500, 40000, 3, 8, [], list(range(1500)), [i % 25 for i in range(1500)]),   # more requests than threads
    (3000, 5000, 3, 8, [], list(range(2999, -1, -1)), [i % 25 for i in range(3000)]),   # lists beyond shared memory; pages run out
])
def test_extend(S, P, M, page, lens, seqs, tokens):
    import exact_io_aware_100_b200 as fa
    dev, want, wide = _state(S, P, M, page, lens, stride=M + 3)
    status = fa.pages_extend(*dev, page, _i(seqs), _i(tokens))
    assert status.tolist() == want.extend(seqs, tokens)
    _same(dev, want)
    assert (wide[:, M:] == 77).all()
    _ok()


@pytest.mark.parametrize("S,P,M,page,lens,src,dst", [
    (2, 4, 2, 8, [5], [0], [1]),
    (2, 4, 2, 8, [8], [0], [1]),                                      # nothing but whole pages
    (6, 30, 4, 16, [50, 16, 7], [0, 0, 1], [3, 4, 5]),                # one source twice
    (6, 6, 4, 16, [50, 16], [0, 0, 0, 1], [2, 3, 4, 5]),              # one page left for three copies; the last wants none
    (6, 30, 4, 16, [50, 16], [0, 2, 3, 0, 9, 0, -1, 4], [2, 3, 3, 1, 4, 6, 5, 4]),   # empty source, taken, range, itself
    (400, 9000, 40, 16, [(i * 53) % 640 for i in range(200)], [i // 2 for i in range(200)], list(range(200, 400))),
    (5000, 9000, 2, 16, [(i * 7) % 32 for i in range(2500)], list(range(2500)), list(range(2500, 5000))),
])
def test_fork(S, P, M, page, lens, src, dst):
    import exact_io_aware_100_b200 as fa
    dev, want, _ = _state(S, P, M, page, lens)
    copies, status = fa.pages_fork(*dev, page, _i(src), _i(dst))
    wc, ws = want.fork(src, dst)
    assert status.tolist() == ws and copies.tolist() == np.asarray(wc).tolist()
    _same(dev, want)
    _ok()


@pytest.mark.parametrize("S,P,M,page,lens,ended", [
    (1, 1, 1, 8, [8], [0]),
    (4, 30, 4, 16, [50, 16, 7], [1]),
    (4, 30, 4, 16, [50, 16, 7], [0, 1, 2, 3, 0, 2]),                  # twice, and an empty one
    (64, 2500, 64, 8, [(i * 71) % 512 for i in range(64)], list(range(0, 64, 3))),
    (200, 70000, 600, 8, [(i * 997) % 4800 for i in range(100)], list(range(1, 100, 2))),
])
def test_free_and_compact(S, P, M, page, lens, ended):
    import exact_io_aware_100_b200 as fa
    dev, want, _ = _state(S, P, M, page, lens, seed=S)
    if S > 100:                                                       # shared pages among those that move
        src, dst = list(range(0, 90)), list(range(100, 190))
        fa.pages_fork(*dev, page, _i(src), _i(dst))
        want.fork(src, dst)
    fa.pages_free(*dev, page, _i(ended))
    want.free(sorted(set(ended)))
    _same(dev, want)
    copies = fa.pages_compact(*dev, page)
    assert copies.tolist() == np.asarray(want.compact()).reshape(-1, 3).tolist()
    _same(dev, want)
    again = fa.pages_compact(*dev, page)                              # nothing is left to move
    assert (again == -1).all()
    _same(dev, want)
    _ok()


def test_no_requests_and_bad_ones():
    import exact_io_aware_100_b200 as fa
    dev, want, _ = _state(3, 10, 4, 16, [20, 5])
    none = _i([])
    assert fa.pages_extend(*dev, 16, none, none).numel() == 0
    assert fa.pages_fork(*dev, 16, none, none)[0].shape == (0, 3)
    fa.pages_free(*dev, 16, none)
    _same(dev, want)
    _ok()
    fa.pages_free(*dev, 16, _i([7, -1]))
    _same(dev, want)
    _ok(fa.FA_ERR_INVALID)
    dev[0][0, 0] = 99                                                 # a table that names no page
    fa.pages_compact(*dev, 16)
    _ok(fa.FA_ERR_INVALID)
    fa.pages_free(*dev, 16, _i([0]))
    _ok(fa.FA_ERR_INVALID)
    assert dev[1].tolist() == [0, 5, 0] and int(dev[2].min()) >= 0


@pytest.mark.parametrize("H_kv,page,d,heads_first", [(1, 8, 64, True), (3, 48, 128, False), (8, 64, 128, True), (2, 16, 256, False)])
def test_copies(H_kv, page, d, heads_first):
    import torch
    import exact_io_aware_100_b200 as fa
    P = 40
    pages = [torch.randn(P, H_kv, page, d, device="cuda").bfloat16() for _ in range(2)]
    if not heads_first:
        pages = [p.transpose(1, 2).contiguous().transpose(1, 2) for p in pages]
    rng = np.random.default_rng(page)
    order = rng.permutation(P)
    for n in (0, 1, 15):
        moves = [[order[i], order[20 + i], [page, 0, 1, page - 1][i % 4]] for i in range(n)] + [[-1, -1, -1], [5, 6, page]]
        want = [ref.copy_pages(to_f64(p), moves) for p in pages]
        fa.pages_copy(*pages, _i(moves))
        # page 6, written here from 5, is itself a source in some of these lists (and 5 a destination): the call says
        # nothing about pages written from a page that the same call writes
        written = {int(m[1]) for m in moves if m[0] >= 0}
        told = [p for p in range(P) if not any(m[1] == p and int(m[0]) in written for m in moves)]
        assert len(told) >= P - 2
        assert all(np.array_equal(to_f64(p)[told], w[told]) for p, w in zip(pages, want))
    _ok()
    before = [p.clone() for p in pages]
    fa.pages_copy(*pages, _i([[P, 0, page], [0, P, page], [0, 1, page + 1], [0, -1, 1], [0, 1, -1]]))
    assert all(torch.equal(p, b) for p, b in zip(pages, before))
    _ok(fa.FA_ERR_INVALID)


@pytest.mark.parametrize("H_kv,page,d,heads_first", [(1, 8, 64, True), (5, 48, 128, False), (8, 64, 128, True), (2, 16, 256, False)])
def test_copies_of_disjoint_pages(H_kv, page, d, heads_first):
    """Sources of 0 .. 39, destinations of 40 .. 79, one source several times; everything else is left as it was."""
    import torch
    import exact_io_aware_100_b200 as fa
    shape = (80, H_kv, page, d) if heads_first else (80, page, H_kv, d)
    pages = [torch.randn(shape, device="cuda").bfloat16() for _ in range(2)]
    pages = pages if heads_first else [p.transpose(1, 2) for p in pages]
    rng = np.random.default_rng(page)
    for n in (0, 1, 40):
        to = 40 + rng.permutation(40)[:n]
        moves = [[-1, -1, -1]] + [[int(rng.integers(40)), int(t), [page, 0, 1, page - 1][i % 4]] for i, t in enumerate(to)]
        want = [ref.copy_pages(to_f64(p), moves) for p in pages]
        fa.pages_copy(*pages, _i(moves))
        assert all(np.array_equal(to_f64(p), w) for p, w in zip(pages, want))
    _ok()


@pytest.mark.parametrize("graph", [False, True])
def test_a_serving_loop(graph):
    """Prompts, steps, a fork, an end and a compaction, against float64 attention on what each sequence was given."""
    import torch
    import exact_io_aware_100_b200 as fa
    S, P, M, page, H, H_kv, d = 6, 60, 8, 16, 8, 2, 128
    freqs, m = fa.rotary_frequencies(d, scaling="linear", factor=2.0)
    hf = freqs.cpu().numpy()
    table = torch.full((S, M), -1, dtype=torch.int32, device="cuda")
    lens, refs = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (S, P))
    book = (table, lens, refs, page)
    kp, vp = (torch.full((P, page, H_kv, d), float("nan"), device="cuda", dtype=torch.bfloat16).transpose(1, 2) for _ in range(2))
    said = {s: [] for s in range(S)}                                  # the keys and values each sequence was given
    rng = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *shape: torch.randn(*shape, device="cuda", generator=rng).bfloat16()  # noqa: E731

    prompts, active = [40, 16, 7], [0, 1, 2]
    assert fa.pages_extend(*book, _i(active), _i(prompts)).tolist() == [0] * 3
    k, v = new(sum(prompts), H_kv, d), new(sum(prompts), H_kv, d)
    cu = _i([0, 40, 56, 63, 63, 63, 63])
    fa.paged_append(k, v, kp, vp, table, lens, freqs=freqs, magnitude=m, cu_seqlens=cu)
    for s, (a, b) in enumerate([(0, 40), (40, 56), (56, 63)]):
        said[s] += [(to_f64(k[i]), to_f64(v[i])) for i in range(a, b)]

    seqs, ones = _i(list(range(S))), _i([0] * S)
    q, k, v = new(S, H, 1, d), new(S, H_kv, 1, d), new(S, H_kv, 1, d)

    def step():
        status = fa.pages_extend(*book, seqs, ones)
        out = fa.paged_append(k, v, kp, vp, table, lens, q=q, freqs=freqs, magnitude=m)
        return (status,) + fa.paged_decode(out, kp, vp, table, lens)

    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            result = step()

    def run(active):
        ones.copy_(_i([int(s in active) for s in range(S)]))
        for t in (q, k, v):
            t.copy_(new(*t.shape))
        if graph:
            captured.replay()
            status, o, lse = result
        else:
            status, o, lse = step()
        assert status.tolist() == [0] * S
        for s in range(S):
            if s in active:
                said[s].append((to_f64(k[s, :, 0]), to_f64(v[s, :, 0])))
            elif said[s]:
                # an idle sequence's token went where its last one is
                said[s][-1] = (to_f64(k[s, :, 0]), to_f64(v[s, :, 0]))
            n = len(said[s])
            assert int(lens[s]) == n
            if n == 0:
                assert not o[s].any() and (lse[s] == -float("inf")).all()
                continue
            hk = np.stack([x for x, _ in said[s]], 1)[None]
            hv = np.stack([x for _, x in said[s]], 1)[None]
            hk = ref.rotary(hk, np.arange(n), hf, m)
            hq = ref.rotary(to_f64(q[s:s + 1]), [n - 1], hf, m)
            want, wl = ref.attention_fwd_general(hq, hk, hv, 1 / np.sqrt(d), True)
            # keys and queries are rounded to bf16 after the turn: the scores move by about 2^-8 of their size
            assert_close("O", to_f64(o[s:s + 1]), want, max_abs=4e-2, rel_l2=1.5e-2)
            assert np.abs(to_f64(lse[s:s + 1]) - wl).max() < 2e-2

    for _ in range(3):
        run([0, 1, 2])
    copies, status = fa.pages_fork(*book, _i([0, 2]), _i([3, 5]))
    fa.pages_copy(kp, vp, copies)
    assert status.tolist() == [0, 0]
    said[3], said[5] = list(said[0]), list(said[2])
    for _ in range(9):
        run([0, 1, 2, 3, 5])
    fa.pages_free(*book, _i([0, 1]))
    said[0], said[1] = [], []
    run([2, 3, 5])
    fa.pages_copy(kp, vp, fa.pages_compact(*book))
    used = refs.nonzero().flatten().tolist()
    assert used == list(range(len(used)))
    for _ in range(2):
        run([2, 3, 5])
    _ok()


def test_low_level_names_give_the_same():
    """The mirrors of the C ABI, with layouts and workspaces of the caller's, against the calls that make their own."""
    import torch
    import exact_io_aware_100_b200 as fa
    S, P, M, page, H, H_kv, d = 3, 12, 4, 16, 4, 2, 64
    freqs, _ = fa.rotary_frequencies(d)
    q, k, v = (torch.randn(S, h, 5, d, device="cuda").bfloat16() for h in (H, H_kv, H_kv))
    strides = lambda *ts: [s for t in ts for s in (t.stride()[:3] if t is not None else (0, 0, 0))]  # noqa: E731
    yq, yk = torch.empty_like(q), torch.empty_like(k)
    fa.fa_rotary(q, k, yq, yk, None, freqs, fa.FaRotaryLayout(S, H, H_kv, 5, d, d, 0, 0, *strides(q, k, yq, yk)), 1.0, False,
                 fa.FA_BF16)
    want = fa.rotary(q, k, freqs)
    assert torch.equal(yq, want[0]) and torch.equal(yk, want[1])

    def run(low):
        table = torch.full((S, M), -1, dtype=torch.int32, device="cuda")
        lens, refs = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (S, P))
        kp, vp = (torch.zeros(P, H_kv, page, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        seqs, tokens, src, dst = _i([0, 1]), _i([21, 7]), _i([0]), _i([2])
        if not low:
            status = fa.pages_extend(table, lens, refs, page, seqs, tokens)
            copies, forked = fa.pages_fork(table, lens, refs, page, src, dst)
            fa.pages_copy(kp, vp, copies)
            turned = fa.paged_append(k, v, kp, vp, table, lens, q=q, freqs=freqs)
            o, lse = fa.paged_decode(turned, kp, vp, table, lens)
            fa.pages_free(table, lens, refs, page, seqs)
            moves = fa.pages_compact(table, lens, refs, page)
        else:
            G = fa.FaPagesLayout(S, P, page, M, M)
            ws = torch.empty(fa.fa_pages_workspace_size(G, 2), dtype=torch.uint8, device="cuda")
            status, forked, copies = torch.empty_like(seqs), torch.empty_like(src), torch.empty(1, 3, dtype=torch.int32, device="cuda")
            fa.fa_pages_extend(table, lens, refs, G, seqs, tokens, status, ws)
            fa.fa_pages_fork(table, lens, refs, G, src, dst, copies, forked, ws)
            turned, o = torch.empty_like(q), torch.empty_like(q)
            lse = torch.empty(S, H, 5, device="cuda")
            L = fa.FaPagedLayout(S, H, H_kv, d, 5, P, page, M, M, *strides(q, o, k, v, kp, vp), None, 0, d, 0)
            fa.fa_pages_copy(kp, vp, copies, L)
            fa.fa_paged_append(q, k, v, turned, kp, vp, table, lens, freqs, L)
            big = torch.empty(fa.fa_paged_decode_workspace_size(L), dtype=torch.uint8, device="cuda")
            fa.fa_paged_decode(turned, kp, vp, table, lens, o, lse, L, True, big)
            fa.fa_pages_free(table, lens, refs, G, seqs)
            moves = torch.empty(P // 2, 3, dtype=torch.int32, device="cuda")
            fa.fa_pages_compact(table, lens, refs, G, moves, ws)
        return table, lens, refs, kp, vp, status, copies, forked, turned, o, lse, moves

    assert all(torch.equal(x, y) for x, y in zip(run(False), run(True)))
    _ok()


def test_steps_in_a_row_give_what_single_steps_give():
    """Every call may come up while the one before it ends: 60 steps with forks, ends and moves between them, queued
    without a wait, against the same with a wait behind every call."""
    import torch
    import exact_io_aware_100_b200 as fa
    S, P, M, page, H, H_kv, d = 40, 700, 24, 8, 8, 2, 64
    freqs, _ = fa.rotary_frequencies(d)

    def run(wait):
        g = torch.Generator(device="cuda").manual_seed(5)
        table = torch.full((S, M), -1, dtype=torch.int32, device="cuda")
        lens, refs = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (S, P))
        kp, vp = (torch.zeros(P, page, H_kv, d, device="cuda", dtype=torch.bfloat16).transpose(1, 2) for _ in range(2))
        book, everyone = (table, lens, refs, page), _i(list(range(S)))
        done = torch.cuda.synchronize if wait else (lambda: None)
        outs = []
        fa.pages_extend(*book, _i(list(range(20))), _i([3 * i + 1 for i in range(20)]))
        grow = [_i([int(s < 20 + n) for s in range(S)]) for n in range(20)]
        torch.cuda.synchronize()
        for t in range(60):
            q, k, v = (torch.randn(S, h, 1, d, device="cuda", generator=g).bfloat16() for h in (H, H_kv, H_kv))
            done()
            outs.append(fa.pages_extend(*book, everyone, grow[min(19, t // 2)]))
            done()
            q = fa.paged_append(k, v, kp, vp, table, lens, q=q, freqs=freqs)
            done()
            outs += fa.paged_decode(q, kp, vp, table, lens)
            done()
            if t % 2 == 0 and t // 2 < 18:
                copies, status = fa.pages_fork(*book, _i([t // 2]), _i([20 + t // 2]))
                done()
                fa.pages_copy(kp, vp, copies)
                outs += [copies, status]
                done()
            if t in (21, 45):
                fa.pages_free(*book, _i([1, 30 + t % 7]))
                done()
                moves = fa.pages_compact(*book)
                done()
                fa.pages_copy(kp, vp, moves)
                outs.append(moves)
                done()
        torch.cuda.synchronize()
        return outs + [table, lens, refs, kp, vp]

    want = run(True)
    for _ in range(3):
        got = run(False)
        assert len(got) == len(want) and all(torch.equal(x, y) for x, y in zip(got, want))
    _ok()
