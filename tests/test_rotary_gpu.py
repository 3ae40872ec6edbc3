"""Rotary positions on the GPU against the float64 oracle.

Bound per element: half a step of the output type, |ref| 2^-8 (bf16) or |ref| 2^-24 (fp32), and what 32-bit arithmetic
before that rounding can add: the angle is rounded to 2^-24 of half a turn (pi 2^-24 = 1.9e-7), sin and cos to two
steps (2.4e-7), two products and a sum to half a step each (1.8e-7), all of them times m (|x_a| + |x_b|): under 1e-6 of
that.  The frequency itself, a double divided by 2 pi, is good to 2^-52 relative, so position p adds |p f| 2^-52 2 pi.
"""
import numpy as np
import pytest

from exact_io_aware_100_b200 import inputs
from helpers import to_device, to_f64
from oracle import serving as ref

pytestmark = pytest.mark.gpu


def _data(seed, shape, dtype, name="q"):
    host = inputs.make_tensor(seed, name, shape, dtype=dtype)
    return to_device(host, dtype), inputs.to_f64(host, dtype)


def _check(got, x, pos, freqs, m, interleaved, inverse, dtype):
    want = ref.rotary(x, pos, freqs, m, interleaved, inverse)
    r = 2 * len(freqs)
    size = np.zeros_like(want)
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    both = m * (np.abs(a) + np.abs(b))
    far = np.abs(np.broadcast_to(np.asarray(pos, float), (x.shape[0], x.shape[2])))[:, None, :, None] * np.asarray(freqs)
    add = both * (1e-6 + 2 * np.pi * 2.0 ** -52 * far)
    if interleaved:
        size[..., 0:r:2] = size[..., 1:r:2] = add
    else:
        size[..., :r // 2] = size[..., r // 2:r] = add
    bound = size + np.abs(want) * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24)
    g = to_f64(got)
    assert np.isfinite(g).all()
    assert (np.abs(g - want) <= bound).all(), float((np.abs(g - want) - bound).max())
    assert np.array_equal(g[..., r:], x[..., r:])               # what is not turned is copied


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,H_kv,N,d,r,interleaved,first", [
    (1, 1, 1, 1, 64, 64, False, 0),           # one row, position 0
    (2, 4, 2, 37, 64, 64, True, 5),
    (2, 8, 2, 130, 128, 128, False, 1000),
    (1, 3, 1, 17, 128, 40, True, 7),          # a part of the head: whole vectors
    (1, 3, 3, 17, 128, 40, False, 7),         # half pairs of 20 columns: no whole vectors
    (1, 2, 1, 9, 96, 32, False, 3),
    (2, 2, 1, 5, 30, 10, True, 3),            # d not a multiple of 8
    (2, 2, 1, 5, 31, 10, False, 3),           # odd d: rows start at odd elements
    (1, 5, 1, 3, 256, 0, False, 0),           # nothing to turn: a copy
    (1, 2, 2, 3, 256, 256, False, 2**31 - 4), # the furthest positions
    (1, 2, 2, 3, 64, 64, True, -3),           # positions before the start
    (3, 1, 0, 8, 1024, 512, True, 10**6),     # no k, the widest head
    (1, 40, 8, 300, 128, 128, False, 0),
])
def test_rotary_matches_oracle(B, H, H_kv, N, d, r, interleaved, first, dtype):
    import torch
    import exact_io_aware_100_b200 as fa
    q, fq = _data(700 + N, (B, H, N, d), dtype)
    k, fk = _data(700 + N, (B, H_kv, N, d), dtype, "k") if H_kv else (None, None)
    freqs, _ = fa.rotary_frequencies(r)
    pos = torch.arange(first, first + N, dtype=torch.int64).to(torch.int32).cuda()
    hf, hp = freqs.cpu().numpy(), pos.cpu().numpy()
    yq, yk = fa.rotary(q, k, freqs, pos, interleaved, 1.25)
    gq, gk = fa.rotary_backward(q, k, freqs, pos, interleaved, 1.25)
    assert (yk is None) == (k is None)
    _check(yq, fq, hp, hf, 1.25, interleaved, False, dtype)
    _check(gq, fq, hp, hf, 1.25, interleaved, True, dtype)
    if H_kv:
        _check(yk, fk, hp, hf, 1.25, interleaved, False, dtype)
        _check(gk, fk, hp, hf, 1.25, interleaved, True, dtype)
    assert fa.fa_get_device_status() == fa.FA_OK


def test_rotary_positions_per_batch_entry_and_default():
    import torch
    import exact_io_aware_100_b200 as fa
    q, fq = _data(801, (3, 2, 11, 64), "bf16")
    freqs, m = fa.rotary_frequencies(32, 500.0, "yarn", 8.0, 64)
    pos = torch.randint(-50, 5000, (3, 22), dtype=torch.int32, device="cuda")[:, ::1][:, 4:15]     # a strided view
    y, _ = fa.rotary(q, None, freqs, pos, magnitude=m)
    _check(y, fq, pos.cpu().numpy(), freqs.cpu().numpy(), m, False, False, "bf16")
    y, _ = fa.rotary(q, None, freqs)
    _check(y, fq, np.arange(11), freqs.cpu().numpy(), 1.0, False, False, "bf16")


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_layouts_give_the_same_bits(interleaved):
    """Token-major, sliced, misaligned, expanded and packed inputs, other output strides, and in place."""
    import torch
    import exact_io_aware_100_b200 as fa
    freqs, _ = fa.rotary_frequencies(64)
    base = torch.randn(2, 21, 6, 64, device="cuda").bfloat16()
    x = base.transpose(1, 2)                                            # [B, H, N, d] of token-major memory
    want, want_k = fa.rotary(x.contiguous(), x[:, :2].contiguous(), freqs, interleaved=interleaved)
    got, got_k = fa.rotary(x, x[:, :2], freqs, interleaved=interleaved)
    assert got.stride() == x.stride() and torch.equal(got, want) and torch.equal(got_k, want_k)
    odd = torch.empty(2 * 6 * 21 * 67 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(2, 6, 21, 67)[..., 2:66]
    odd.copy_(x)                                                        # rows of 67 elements, not even 4-byte aligned
    out = torch.full_like(odd, 7.0)
    fa.rotary(odd, None, freqs, interleaved=interleaved, out=(out, None))
    assert torch.equal(out, want)
    one = x[:1, :1].expand(2, 6, 21, 64)                                 # broadcast over batch and heads: strides 0
    got, _ = fa.rotary(one, None, freqs, interleaved=interleaved)
    assert torch.equal(got, want[:1, :1].expand_as(got))
    packed = base.reshape(42, 6, 64)
    pos = torch.arange(21, dtype=torch.int32, device="cuda").repeat(2)
    got, _ = fa.rotary(packed, None, freqs, pos, interleaved)
    assert torch.equal(got.view(2, 21, 6, 64).transpose(1, 2), want)
    there = x.clone()
    res, _ = fa.rotary(there, None, freqs, interleaved=interleaved, out=(there, None))
    assert res is there and torch.equal(there, want)


def test_rotary_empty_and_large_batches():
    import torch
    import exact_io_aware_100_b200 as fa
    freqs, _ = fa.rotary_frequencies(64)
    y, _ = fa.rotary(torch.empty(2, 3, 0, 64, device="cuda", dtype=torch.bfloat16), None, freqs)
    assert y.shape == (2, 3, 0, 64)
    x = torch.randn(1, 1, 70001, 64, device="cuda").bfloat16()
    y, _ = fa.rotary(x, None, freqs)
    f = freqs.cpu().numpy()
    for i in (0, 4095, 65536, 70000):
        _check(y[:, :, i:i + 1], to_f64(x[:, :, i:i + 1]), [i], f, 1.0, False, False, "bf16")


def test_rotary_offsets_beyond_32_bits():
    """Rows more than 2^31 elements apart."""
    import torch
    import exact_io_aware_100_b200 as fa
    freqs, _ = fa.rotary_frequencies(64)
    store = torch.empty((1 << 31) + 4096, device="cuda", dtype=torch.bfloat16)
    x = torch.as_strided(store, (2, 2, 3, 64), ((1 << 31) + 512, 256, 64, 1))
    x.copy_(torch.randn(2, 2, 3, 64, device="cuda"))
    want, _ = fa.rotary(x.contiguous(), None, freqs)
    fa.rotary(x, None, freqs, out=(x, None))
    assert torch.equal(x, want)


def test_rotary_stream_and_graph():
    import torch
    import exact_io_aware_100_b200 as fa
    freqs, _ = fa.rotary_frequencies(128)
    q, k = torch.randn(2, 4, 33, 128, device="cuda").bfloat16(), torch.randn(2, 2, 33, 128, device="cuda").bfloat16()
    want = fa.rotary(q, k, freqs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.rotary(q, k, freqs, stream=side)
    raw = fa.rotary(q, k, freqs, stream=side.cuda_stream)
    side.synchronize()
    for g in (got, raw):
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fa.rotary(q, k, freqs)
        back = fa.rotary_backward(*out, freqs)
    q.copy_(torch.randn_like(q))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], fa.rotary(q, None, freqs)[0])
    assert (back[0].float() - q.float()).abs().max() < 0.06       # a turn there and back: two roundings of |x| < 6


@pytest.mark.parametrize("H,H_kv,N,d,r", [(40000, 20000, 2, 16, 16), (1, 0, 300000, 16, 8), (65535, 0, 1, 8, 8)])
def test_rotary_many_heads_or_rows(H, H_kv, N, d, r):
    import torch
    import exact_io_aware_100_b200 as fa
    freqs, _ = fa.rotary_frequencies(r)
    q = torch.randn(1, H, N, d, device="cuda").bfloat16()
    k = torch.randn(1, H_kv, N, d, device="cuda").bfloat16() if H_kv else None
    y, yk = fa.rotary(q, k, freqs)
    at = [0, H // 2, H - 1]
    rows = [0, N // 2, N - 1]
    _check(y[:, at][:, :, rows], to_f64(q[:, at][:, :, rows]), np.asarray(rows), freqs.cpu().numpy(), 1.0, False, False, "bf16")
    if H_kv:
        _check(yk[:, -2:], to_f64(k[:, -2:]), np.arange(N), freqs.cpu().numpy(), 1.0, False, False, "bf16")


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_gradient_is_the_transpose(interleaved):
    """<dy, f(x)> = <f^T(dy), x> in float32, and differences: f is linear, so f(x + h e) - f(x) = h f(e)."""
    import torch
    import exact_io_aware_100_b200 as fa
    freqs, _ = fa.rotary_frequencies(48)
    x, dy = (torch.randn(2, 3, 17, 64, device="cuda") for _ in range(2))
    pos = torch.randint(0, 5000, (2, 17), dtype=torch.int32, device="cuda")
    y, _ = fa.rotary(x, None, freqs, pos, interleaved, 1.3)
    dx, _ = fa.rotary_backward(dy, None, freqs, pos, interleaved, 1.3)
    a, b = (dy.double() * y.double()).sum(), (dx.double() * x.double()).sum()
    # 6528 products of size about 1.3, each good to 1e-6 (the bound above) of 1.3 (|x_a| + |x_b|) |dy|
    assert abs(float(a - b)) <= 6528 * 1e-6 * 1.3 * 8
    h = 0.5
    for col in (0, 1, 24, 47, 50):
        e = torch.zeros_like(x)
        e[..., col] = h
        # two outputs of up to 8, each good to 1e-6 of |x_a| + |x_b| < 10, in two columns, times |dy| < 5, over h
        step = fa.rotary(x + e, None, freqs, pos, interleaved, 1.3)[0].double() - y.double()
        assert (((step * dy.double()).sum(-1) / h - dx[..., col].double()).abs() <= 4e-4).all()


@pytest.mark.parametrize("size,stride", [
    ((1, 1, 4, 64), (1, 1, 1, 1)),            # rows one element apart: windows over one line
    ((2, 3, 5, 64), (7, 1, 100, 1)),          # heads one element apart
    ((2, 3, 5, 64), (1, 64, 200, 1)),         # batch entries
    ((2, 3, 5, 64), (0, 0, 3, 1)),
    ((5, 3, 64), (1, 70, 1)),                 # packed rows
])
def test_rotary_of_overlapping_inputs(size, stride):
    """Inputs may have any strides; the outputs made for them are tensors of their own, d contiguous."""
    import torch
    import exact_io_aware_100_b200 as fa
    freqs, _ = fa.rotary_frequencies(64)
    x = torch.randn(4096, device="cuda").bfloat16().as_strided(size, stride)
    want = fa.rotary(x.contiguous(), x.contiguous(), freqs)
    for f, want in ((fa.rotary, want), (fa.rotary_backward, fa.rotary_backward(x.contiguous(), x.contiguous(), freqs))):
        got = f(x, x, freqs)
        for g, w in zip(got, want):
            assert g.stride(-1) == 1 and torch.equal(g, w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rotary_by_negative_frequencies_is_the_inverse_turn(dtype):
    """The same angle with the other sign: the same bits."""
    import torch
    import exact_io_aware_100_b200 as fa
    q, _ = _data(911, (2, 3, 40, 64), dtype)
    pos = torch.arange(2**31 - 40, 2**31, dtype=torch.int64).int().cuda()
    for f in (fa.rotary_frequencies(64)[0], torch.logspace(-18, -6, 32, dtype=torch.float64, device="cuda")):
        for interleaved in (False, True):
            for p in (pos, -pos):
                a, _ = fa.rotary(q, None, -f, p, interleaved, 1.5)
                b, _ = fa.rotary_backward(q, None, f, p, interleaved, 1.5)
                assert torch.equal(a, b)


@pytest.mark.parametrize("sign", [1, -1])
def test_rotary_small_angles_of_far_positions(sign):
    """x_a = 0, x_b = 1: y_a = -sin t, for t from 2e-9 to 2e3.  The fraction of a turn is cut to 2^-32, after a product with a
    step that is cut to 2^-64 and taken up to 2^31 times (2^-33): 2 pi (2^-32 + 2^-33) = 2.2e-9 rad.  It is rounded to 2^-24 of
    itself; the sine has two steps, freqs / 2 pi 2^-52 of t."""
    import torch
    import exact_io_aware_100_b200 as fa
    f = sign * 10.0 ** np.linspace(-18, -6, 32)
    x = torch.zeros(1, 1, 64, 64, device="cuda")
    x[..., 32:] = 1.0
    pos = np.arange(2**31 - 64, 2**31)
    y, _ = fa.rotary(x, None, torch.tensor(f, device="cuda"), torch.from_numpy(pos).int().cuda())
    t = pos[:, None].astype(np.longdouble) * f.astype(np.longdouble)
    want = -np.sin(t)
    small = np.minimum(np.abs(t), np.pi)             # the reduced angle is no further out
    bound = 2 * np.pi * (2.0 ** -32 + 2.0 ** -33) + small * 2.0 ** -24 + np.abs(want) * 2.0 ** -22 + np.abs(t) * 2.0 ** -52
    assert (np.abs(to_f64(y)[0, 0, :, :32] - want) <= bound).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_float32_angles(interleaved):
    """x_a = 1, x_b = 0: y = (cos t, sin t) all around the turn.  The reduced angle, an eighth of a turn at most once the
    nearest quarter is off, is rounded to 2^-24 of itself (half of pi / 4's step: pi 2^-27) and cut to 2^-32 of a turn;
    freqs / 2 pi adds 2^-52 of t, and the sine or cosine two steps.  An angle rounded as half a turn would be off by pi 2^-25."""
    import torch
    import exact_io_aware_100_b200 as fa
    f = np.array([0.001, 0.37, 1.0, 1.5707963, 2.9])
    x = torch.zeros(1, 1, 40000, 10, device="cuda")
    x[..., 0::2 if interleaved else 1] = 1.0
    if not interleaved:
        x[..., 5:] = 0.0
    y, _ = fa.rotary(x, None, torch.tensor(f, device="cuda"), interleaved=interleaved)
    t = np.arange(40000)[:, None].astype(np.longdouble) * f.astype(np.longdouble)
    y = to_f64(y)[0, 0]
    for got, want in ((y[:, 0::2] if interleaved else y[:, :5], np.cos(t)), (y[:, 1::2] if interleaved else y[:, 5:], np.sin(t))):
        bound = np.pi * 2.0 ** -27 + 2 * np.pi * 2.0 ** -32 + 2.0 ** -52 * np.abs(t) + np.abs(want) * 2.0 ** -22
        assert (np.abs(got - want) <= bound).all()
        # the sine's own two steps apart, the angle's error shows near its zeros
        near = np.abs(want) < 2.0 ** -6
        assert near.sum() > 1000 and (np.abs(got - want)[near] <= (bound - np.abs(want) * 2.0 ** -22 + 2.0 ** -28)[near]).all()
