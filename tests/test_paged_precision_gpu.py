"""How exactly the probabilities enter the second product of paged decode, whatever the rows, the lengths and the table.

Values come in pairs a, -a under nearly equal keys, so O is a difference of large sums and shows what rounding P costs.  With
A = sum p |v| / sum p, every element is within

    2^-8 |O|          the output's rounding to bf16
    2^-16 A           P as a bf16 and the bf16 of what that left: 2^-8 of 2^-8 of each p
    2^-17 A           the 32-bit arithmetic before and after: a score's sum of d products, sum |q k| scale 2^-22 < 11 * 2^-22
                      here, the exponent's rounding (|x| < 16: 2^-21) and ex2 (2^-22): under 2^-18 of each p; as much for sums
of the float64 result.  P rounded to bf16 alone would be 2^-8 of each p.
"""
import numpy as np
import pytest


pytestmark = pytest.mark.gpu


def _call(d, H_kv, group, N, lens, page, wide, seed):
    """(q, k_pages, v_pages, table, lens) with paired values."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, n = len(lens), max(lens)
    M = -(-n // page)
    base = torch.randn(B, H_kv, (n + 1) // 2, d, device="cuda", generator=g)
    near = base + 0.05 * torch.randn(base.shape, device="cuda", generator=g)
    a = torch.randn(base.shape, device="cuda", generator=g)
    k = torch.stack([base, near], 3).flatten(2, 3)[:, :, :n].bfloat16()
    v = torch.stack([a, -a], 3).flatten(2, 3)[:, :, :n].bfloat16()
    kp, vp = (torch.full((B * M, H_kv, page, d), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table = torch.full((B, wide // page if wide else M), -1, dtype=torch.int32, device="cuda")
    table[:, :M] = torch.randperm(B * M, device="cuda", generator=g).int().view(B, M)
    for b, m in enumerate(lens):
        for e in range(-(-m // page)):
            rows = min(page, m - e * page)
            kp[int(table[b, e]), :, :rows], vp[int(table[b, e]), :, :rows] = (x[b, :, e * page:e * page + rows] for x in (k, v))
    q = torch.randn(B, H_kv * group, N, d, device="cuda", generator=g).bfloat16()
    return q, k, v, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("wide", [0, 1 << 17])          # a table as wide as the sequences, and one for 131072 positions
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group,N", [(1, 1), (8, 1), (4, 4), (12, 1), (8, 3), (16, 2), (20, 2)])
def test_probabilities_keep_16_bits(d, group, N, wide):
    import torch
    import exact_io_aware_100_b200 as fa
    lens, H_kv = [70, 400, 1, 33, 1000], 2
    q, k, v, kp, vp, table, sl = _call(d, H_kv, group, N, lens, 16, wide, seed=d + group)
    o, _ = fa.paged_decode(q, kp, vp, table, sl)
    assert fa.fa_get_device_status() == fa.FA_OK
    for b, n in enumerate(lens):
        kb, vb = (x[b, :, :n].double().repeat_interleave(group, 0) for x in (k, v))
        s = q[b].double() @ kb.transpose(1, 2) / np.sqrt(d)
        hidden = torch.arange(n, device="cuda")[None, :] > (n - N + torch.arange(N, device="cuda"))[:, None]
        s.masked_fill_(hidden, -float("inf"))
        p = torch.softmax(s, -1).nan_to_num(0.0)                 # a query before the sequence's start sees nothing
        want, size = p @ vb, p @ vb.abs()
        bound = 2.0 ** -8 * want.abs() + (2.0 ** -16 + 2.0 ** -17) * size
        worst = ((o[b].double() - want).abs() - bound).max()
        assert worst <= 0, (b, n, float(worst), float(((o[b].double() - want).abs() / size.clamp(min=1e-9)).max()))


def test_probabilities_keep_16_bits_in_many_and_long_calls():
    """Where the row tiles are 16 and 32 rows high: many pairs, and long ones."""
    import torch
    import exact_io_aware_100_b200 as fa
    for d, H_kv, group, lens in ((128, 8, 16, [300] * 40), (64, 8, 32, [600] * 60), (128, 4, 32, [30000, 20000]), (256, 4, 16, [20000])):
        q, k, v, kp, vp, table, sl = _call(d, H_kv, group, 1, lens, 64, 0, seed=d)
        o, _ = fa.paged_decode(q, kp, vp, table, sl)
        for b, n in list(enumerate(lens))[:3]:
            kb, vb = (x[b, :, :n].double().repeat_interleave(group, 0) for x in (k, v))
            p = torch.softmax(q[b].double() @ kb.transpose(1, 2) / np.sqrt(d), -1)
            want, size = p @ vb, p @ vb.abs()
            assert ((o[b].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -16 + 2.0 ** -17) * size).all()
    assert fa.fa_get_device_status() == fa.FA_OK
