"""The float64 oracle of the serving operators against hand-made values, identities, differences and each other."""
import math

import numpy as np
import pytest

from oracle import attention_fwd_general
from oracle import serving as ref


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_is_a_scaled_rotation_and_its_inverse_the_transpose(interleaved):
    rng = np.random.default_rng(1)
    x, y = rng.standard_normal((2, 2, 3, 5, 12))
    f, pos, m = 10.0 ** -np.arange(4), np.array([[0, 1, 7, 100, 2**31 - 1]] * 2), 1.25
    a = ref.rotary(x, pos, f, m, interleaved)
    assert np.allclose((a[..., :8] ** 2).sum(-1), m * m * (x[..., :8] ** 2).sum(-1))
    assert np.array_equal(a[..., 8:], x[..., 8:])
    # <R x, y> = <x, R^T y>
    b = ref.rotary(y, pos, f, m, interleaved, inverse=True)
    assert np.allclose((a * y).sum(), (x * b).sum())
    assert np.allclose(ref.rotary(a, pos, f, 1 / m, interleaved, inverse=True)[..., :8], x[..., :8])
    assert np.allclose(a[:, :, 0], np.concatenate([m * x[:, :, 0, :8], x[:, :, 0, 8:]], -1))     # position 0


def test_rotary_hand_values():
    x = np.arange(1.0, 5.0).reshape(1, 1, 1, 4)
    f = [math.pi / 2, math.pi / 6]
    half = ref.rotary(x, [1], f)[0, 0, 0]            # pairs (1, 3) by 90 degrees, (2, 4) by 30
    c, s = math.cos(math.pi / 6), 0.5
    assert np.allclose(half, [-3, 2 * c - 4 * s, 1, 4 * c + 2 * s])
    near = ref.rotary(x, [1], f, interleaved=True)[0, 0, 0]    # pairs (1, 2), (3, 4)
    assert np.allclose(near, [-2, 1, 3 * c - 4 * s, 4 * c + 3 * s])


def test_rotary_scores_depend_on_the_distance_alone():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 1, 8))
    f = 100.0 ** -(np.arange(4) / 4)
    score = lambda i, j: (ref.rotary(q, [i], f) * ref.rotary(k, [j], f)).sum()  # noqa: E731
    assert np.isclose(score(5, 2), score(1005, 1002)) and not np.isclose(score(5, 2), score(5, 3))


def test_rotary_gradient_by_differences():
    rng = np.random.default_rng(3)
    x, g = rng.standard_normal((2, 1, 2, 3, 6))
    f, pos = [0.7, 0.1], [3, 4, 9]
    grad = ref.rotary(g, pos, f, 1.1, inverse=True)
    for at in [(0, 0, 0, 0), (0, 1, 2, 3), (0, 1, 1, 5)]:
        d = np.zeros_like(x)
        d[at] = 1e-6
        slope = ((ref.rotary(x + d, pos, f, 1.1) - ref.rotary(x - d, pos, f, 1.1)) * g).sum() / 2e-6
        assert abs(slope - grad[at]) < 1e-6


def test_paged_attention_is_the_dense_one_on_gathered_keys():
    rng = np.random.default_rng(4)
    kp, vp = rng.standard_normal((2, 9, 2, 4, 8))
    table, lens = [[7, 2, 5], [1, 8, 0], [3, -1, -1]], [11, 4, 0]
    q = rng.standard_normal((3, 4, 2, 8))
    o, lse = ref.paged_decode(q, kp, vp, table, lens, 0.3)
    k = np.concatenate([kp[7], kp[2], kp[5]], axis=1)[None, :, :11]
    v = np.concatenate([vp[7], vp[2], vp[5]], axis=1)[None, :, :11]
    ro, rl = attention_fwd_general(q[:1], k, v, 0.3, True)
    assert np.allclose(o[:1], ro) and np.allclose(lse[:1], rl)
    assert np.all(o[2] == 0) and np.all(np.isneginf(lse[2]))


def test_bookkeeping_by_hand():
    # pages of 4; sequence 0 holds 6 positions on pages 5, 1; sequence 1 4 positions on page 3
    refs = np.zeros(8, int)
    refs[[5, 1, 3]] = 1
    st = ref.Pages([[5, 1, -1], [3, -1, -1], [-1, -1, -1], [-1, -1, -1]], [6, 4, 0, 0], refs, 4)
    copies, status = st.fork([0, 1, 0], [2, 3, 2])
    assert status == [0, 0, 1]
    assert copies == [[1, 0, 2], [-1, -1, -1], [-1, -1, -1]]
    assert st.table.tolist() == [[5, 1, -1], [3, -1, -1], [5, 0, -1], [3, -1, -1]]
    assert st.refs.tolist() == [1, 1, 0, 2, 0, 2, 0, 0] and st.lens.tolist() == [6, 4, 6, 4]
    assert st.extend([3, 0, 1, 1], [1, 2, 9, 1]) == [0, 0, 1, 0]
    assert st.table[3].tolist() == [3, 2, -1] and st.table[1].tolist() == [3, 4, -1] and st.lens.tolist() == [8, 5, 6, 5]
    st.free([0])
    assert st.refs.tolist() == [1, 0, 1, 2, 1, 1, 0, 0] and st.table[0].tolist() == [-1, -1, -1]
    assert st.compact()[:2] == [[5, 1, 4], [-1, -1, -1]]
    assert st.refs.tolist() == [1, 1, 1, 2, 1, 0, 0, 0] and st.table[2].tolist() == [1, 0, -1]


def test_pages_run_out_in_the_order_of_the_requests():
    st = ref.Pages(np.full((4, 3), -1), [0, 0, 0, 0], np.zeros(3, int), 2)
    assert st.extend([0, 1, 2, 3], [3, 4, 1, 0]) == [0, 4, 4, 0]
    assert st.table[0].tolist() == [0, 1, -1] and st.lens.tolist() == [3, 0, 0, 0]


def test_planted_mistake_turning_by_the_wrong_sign_is_seen():
    """The transpose check above fails for a backward pass that forgets to turn the other way."""
    rng = np.random.default_rng(5)
    x, y = rng.standard_normal((2, 1, 1, 4, 4))
    f, pos = [0.5, 0.2], [1, 2, 3, 4]
    wrong = ref.rotary(y, pos, f)
    assert not np.allclose((ref.rotary(x, pos, f) * y).sum(), (x * wrong).sum())
