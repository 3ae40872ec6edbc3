"""A generation step whose sequences do not all go on: idle ones, and ones that were refused a page.

What the cache holds is compared bit for bit: keys are not turned unless the test says so, so a row is what was given.
"""
import numpy as np
import pytest

from helpers import assert_close, to_f64
from oracle import serving as ref

pytestmark = pytest.mark.gpu


def _i(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(P, H_kv, page, d):
    import torch
    return [torch.randn(P, H_kv, page, d, device="cuda").bfloat16() for _ in range(2)]


@pytest.mark.parametrize("graph", [False, True])
def test_a_refused_step_leaves_shared_pages_alone(graph):
    """Two full pages, forked twice; one page is left for three branches that want one, and one sequence is idle."""
    import torch
    import exact_io_aware_100_b200 as fa
    S, P, M, page, H, H_kv, d = 5, 4, 4, 8, 4, 2, 64
    table = torch.full((S, M), -1, dtype=torch.int32, device="cuda")
    lens, refs = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (S, P))
    book = (table, lens, refs, page)
    kp, vp = _cache(P, H_kv, page, d)
    assert fa.pages_extend(*book, _i([0, 3]), _i([16, 5])).tolist() == [0, 0]
    _, status = fa.pages_fork(*book, _i([0, 0]), _i([1, 2]))
    assert status.tolist() == [0, 0] and int((refs == 0).sum()) == 1
    freqs, m = fa.rotary_frequencies(d)
    tokens, seqs = _i([1, 1, 1, 0, 0]), _i(list(range(S)))
    q, k, v = (torch.randn(S, h, 1, d, device="cuda").bfloat16() for h in (H, H_kv, H_kv))

    def step():
        status = fa.pages_extend(*book, seqs, tokens)
        out = fa.paged_append(k, v, kp, vp, table, lens, q=q, freqs=freqs, magnitude=m, tokens=tokens, status=status)
        return (status, out) + fa.paged_decode(out, kp, vp, table, lens)

    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            result = step()

    def run(want_status, grown):
        """One step: new positions of the sequences `grown`, and nothing else, change."""
        before, n = [kp.clone(), vp.clone()], lens.tolist()
        if graph:
            captured.replay()
            status, out, o, lse = result
        else:
            status, out, o, lse = step()
        assert status.tolist() == want_status
        assert lens.tolist() == [x + (s in grown) for s, x in enumerate(n)]
        pos = _i(n)[:, None]
        tq, tk = fa.rotary(q, k, freqs, pos, False, m)
        for s in grown:
            p, row = int(table[s, n[s] // page]), n[s] % page
            before[0][p, :, row], before[1][p, :, row] = tk[s, :, 0], v[s, :, 0]
        assert torch.equal(kp, before[0]) and torch.equal(vp, before[1])
        on = torch.tensor([s in grown for s in range(S)], device="cuda")[:, None, None, None]
        assert torch.equal(out, torch.where(on, tq, torch.zeros_like(tq)))
        wo, wl = ref.paged_decode(to_f64(out), to_f64(kp), to_f64(vp), table.cpu().numpy(), lens.tolist(), 1 / np.sqrt(d))
        assert_close("O", to_f64(o), wo, scale_max_abs=True)

    run([0, 4, 4, 0, 0], [0])
    tokens.copy_(_i([0, 1, 1, 0, 0]))
    run([0, 4, 4, 0, 0], [])
    fa.pages_free(*book, _i([3]))                    # room for one of the two
    run([0, 0, 4, 0, 0], [1])
    tokens.copy_(_i([1, 0, 0, 1, 0]))
    run([0, 0, 0, 4, 0], [0])
    assert fa.fa_get_device_status() == fa.FA_OK


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("r", [0, 64, 20])           # copied; turned in vectors; turned column by column
def test_counts_name_the_last_rows(packed, r):
    """tokens[b] of n rows, on the right; the others are padding: zero in q (in place too), and nothing in the cache."""
    import torch
    import exact_io_aware_100_b200 as fa
    B, H, H_kv, N, d, page = 6, 3, 2, 5, 64, 8
    counts, lens = [0, 1, 3, 5, 5, 2], [30, 30, 3, 40, 4, 9]      # sequence 4: a token more than it is long
    refused = [0, 0, 0, 0, 0, 4]
    P, M = 24, 6
    table = torch.full((B, M), -1, dtype=torch.int32)
    order, at = np.random.default_rng(3).permutation(P), 0
    for b, n in enumerate(lens):
        table[b, :-(-n // page)] = torch.from_numpy(order[at:at + -(-n // page)].astype(np.int32))
        at += -(-n // page)
    kp, vp = _cache(P, H_kv, page, d)
    q, k, v = (torch.randn(B, h, N, d, device="cuda").bfloat16() for h in (H, H_kv, H_kv))
    freqs = fa.rotary_frequencies(r)[0] if r else None
    pos = _i(lens)[:, None] - N + torch.arange(N, dtype=torch.int32, device="cuda")
    tq, tk = fa.rotary(q, k, freqs, pos) if r else (q, k)
    n = [0 if refused[b] else counts[b] for b in range(B)]
    hk, hv = ref.paged_append(to_f64(kp), to_f64(vp), table.numpy(), lens,
                              [(to_f64(tk[b, :, N - n[b]:]), to_f64(v[b, :, N - n[b]:])) for b in range(B)])
    row = torch.arange(N, device="cuda")
    real = (pos >= 0) & (row >= N - _i(n)[:, None])
    want = tq.masked_fill(~real[:, None, :, None], 0.0)
    pack = (lambda x: x.transpose(1, 2).reshape(B * N, -1, d).contiguous()) if packed else (lambda x: x.clone())
    cu = _i([N * b for b in range(B + 1)]) if packed else None
    args = (kp, vp, table.cuda(), _i(lens))
    got = fa.paged_append(pack(k), pack(v), *args, q=pack(q), freqs=freqs, cu_seqlens=cu, tokens=_i(counts), status=_i(refused))
    assert fa.fa_get_device_status() == fa.FA_OK
    assert np.array_equal(to_f64(kp), hk) and np.array_equal(to_f64(vp), hv)
    assert torch.equal(got, pack(want))
    there = pack(q)
    fa.paged_append(pack(k), pack(v), *args, q=there, freqs=freqs, cu_seqlens=cu, out=there, tokens=_i(counts),
                    status=_i(refused), stream=torch.cuda.current_stream())
    assert torch.equal(there, pack(want))
    assert np.array_equal(to_f64(kp), hk)


def test_counts_that_make_no_sense_are_reported():
    import torch
    import exact_io_aware_100_b200 as fa
    kp, vp = _cache(12, 1, 8, 64)
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    k = torch.randn(3, 1, 2, 64, device="cuda").bfloat16()
    for bad in (-1, 3, 2**31 - 1, -2**31):
        before = kp.clone()
        fa.paged_append(k, k, kp, vp, table, _i([9, 20, 30]), tokens=_i([2, bad, 1]))
        assert fa.fa_get_device_status() == fa.FA_ERR_INVALID
        before[0, 0, 7], before[1, 0, 0] = k[0, 0, 0], k[0, 0, 1]          # sequence 0: positions 7 and 8
        before[11, 0, 5] = k[2, 0, 1]                                      # sequence 2: position 29
        assert torch.equal(kp, before)
        fa.paged_append(k, k, kp, vp, table, _i([9, 20, 30]), tokens=_i([2, bad, 1]), status=_i([0, 1, 0]))
        assert fa.fa_get_device_status() == fa.FA_OK                       # a refused sequence's count is not looked at
        assert torch.equal(kp, before)


@pytest.mark.parametrize("r", [0, 64, 20])
@pytest.mark.parametrize("cu,kept", [
    ([0, 7, 3], []),                    # sequence 1 ends before it begins
    ([0, 10, 4, 12], []),               # rows 4 to 9 belong to two sequences
    ([0, 3, 9, 6, 12, 12], [0]),        # sequence 0 is not beside the place
    ([0, 4, 4, 13], [0, 1]),            # more rows than there are
    ([-1, 4, 12], [1]),
    ([0, 12, 12, 5], [0]),              # no row looks at sequence 2
    ([0, 12, 14, 14], [0]),             # sequences behind the last row
    ([0, 5, 5, 12], [0, 1, 2]),         # in order: nothing to report
])
def test_packed_offsets_out_of_order_are_reported(cu, kept, r):
    import torch
    import exact_io_aware_100_b200 as fa
    H, H_kv, d, page, total, B = 3, 2, 64, 8, 12, len(cu) - 1
    lens = [20] * B
    kp, vp = _cache(3 * B, H_kv, page, d)
    table = torch.arange(3 * B, dtype=torch.int32, device="cuda").view(B, 3)
    q, k, v = (torch.randn(total, h, d, device="cuda").bfloat16() for h in (H, H_kv, H_kv))
    freqs = fa.rotary_frequencies(r)[0] if r else None
    pos = torch.zeros(total, dtype=torch.int32, device="cuda")
    real = torch.zeros(total, dtype=torch.bool, device="cuda")
    for b in kept:
        pos[cu[b]:cu[b + 1]] = torch.arange(20 - (cu[b + 1] - cu[b]), 20, dtype=torch.int32, device="cuda")
        real[cu[b]:cu[b + 1]] = True
    tq, tk = fa.rotary(q, k, freqs, pos) if r else (q, k)
    rows = [(cu[b], cu[b + 1]) if b in kept else (0, 0) for b in range(B)]
    hk, hv = ref.paged_append(to_f64(kp), to_f64(vp), table.cpu().numpy(), lens,
                              [(to_f64(tk[x:y].transpose(0, 1)), to_f64(v[x:y].transpose(0, 1))) for x, y in rows])
    got = fa.paged_append(k, v, kp, vp, table, _i(lens), q=q, freqs=freqs, cu_seqlens=_i(cu))
    assert fa.fa_get_device_status() == (fa.FA_OK if len(kept) == B else fa.FA_ERR_INVALID)
    assert np.array_equal(to_f64(kp), hk) and np.array_equal(to_f64(vp), hv)
    assert torch.equal(got, tq.masked_fill(~real[:, None, None], 0.0))


def test_packed_offsets_of_more_sequences_than_threads():
    """One wrong offset among many sequences of one row or none."""
    import torch
    import exact_io_aware_100_b200 as fa
    B = 5000
    kp, vp = _cache(B, 1, 8, 64)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
    k = torch.randn(20, 1, 64, device="cuda").bfloat16()
    cu = torch.arange(B + 1, device="cuda").clamp(max=20).int()
    fa.paged_append(k, k, kp, vp, table, torch.ones(B, dtype=torch.int32, device="cuda"), cu_seqlens=cu)
    assert fa.fa_get_device_status() == fa.FA_OK
    assert torch.equal(kp[:20, :, 0], k)
    cu[4321] = 19
    fa.paged_append(k, k, kp, vp, table, torch.ones(B, dtype=torch.int32, device="cuda"), cu_seqlens=cu)
    assert fa.fa_get_device_status() == fa.FA_ERR_INVALID


def test_no_sequences_and_no_rows():
    """A batch that has run empty goes through the same calls."""
    import torch
    import exact_io_aware_100_b200 as fa
    kp, vp = _cache(6, 2, 8, 64)
    before = kp.clone()
    new = lambda *shape: torch.zeros(*shape, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    freqs, _ = fa.rotary_frequencies(64)
    none, refs = _i([]), _i([0, 1, 0, 0, 0, 0])
    table = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    book = (table, none, refs, 8)
    for n in (1, 0, 5):
        q, k = new(0, 4, n, 64), new(0, 2, n, 64)
        got = fa.rotary(q, k, freqs)
        assert got[0].shape == q.shape and got[1].shape == k.shape
        got = fa.paged_append(k, k, kp, vp, table, none, q=q, freqs=freqs, tokens=none, status=none)
        assert got.shape == q.shape
        o, lse = fa.paged_decode(q, kp, vp, table, none)
        assert o.shape == q.shape and lse.shape == (0, 4, n) and lse.dtype == torch.float32
    got = fa.paged_append(new(0, 2, 64), new(0, 2, 64), kp, vp, table, none, q=new(0, 4, 64), cu_seqlens=_i([0]))
    assert got.shape == (0, 4, 64)
    assert fa.pages_extend(*book, none, none).shape == (0,)
    copies, status = fa.pages_fork(*book, none, none)
    assert copies.shape == (0, 3) and status.shape == (0,)
    fa.pages_free(*book, none)
    assert fa.pages_compact(*book).tolist() == [[-1] * 3] * 3 and refs.tolist() == [0, 1, 0, 0, 0, 0]
    fa.pages_copy(kp, vp, torch.empty(0, 3, dtype=torch.int32, device="cuda"))
    # one sequence, no rows
    one, lens = torch.zeros(1, 3, dtype=torch.int32, device="cuda"), _i([4])
    o, lse = fa.paged_decode(new(1, 4, 0, 64), kp, vp, one, lens)
    assert o.shape == (1, 4, 0, 64) and lse.shape == (1, 4, 0)
    assert fa.paged_append(new(1, 2, 0, 64), new(1, 2, 0, 64), kp, vp, one, lens, q=new(1, 4, 0, 64)).shape == (1, 4, 0, 64)
    torch.cuda.synchronize()
    assert torch.equal(kp, before) and fa.fa_get_device_status() == fa.FA_OK
    # what makes no sense is refused as before: rows or requests of no sequence
    with pytest.raises(fa.FaError):
        fa.paged_append(new(3, 2, 64), new(3, 2, 64), kp, vp, table, none, cu_seqlens=_i([0]))
    with pytest.raises(fa.FaError):
        fa.pages_extend(*book, _i([0]), _i([1]))
