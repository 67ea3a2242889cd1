"""Pins of the float64 oracles of the decayed linear attention and the rotary embedding."""
import numpy as np
import pytest

import oracle
from oracle import decay as od


def test_hand_worked_example():
    # d = 1, g = 1/2, scale 3, S_0 = 8:  S_1 = 4 + 2*5 = 14, S_2 = 7 + 1*1 = 8
    q, k, v = ([[[[x] for x in xs]]] for xs in ([1.0, 2.0], [2.0, 1.0], [5.0, 1.0]))
    o, S = od.decay_attention(q, k, v, [np.log(0.5)], 3.0, np.full((1, 1, 1, 1), 8.0))
    assert o.ravel().tolist() == [42.0, 48.0]
    assert S.item() == 8.0


def test_equals_the_masked_pair_sum():
    """o_i = scale sum_{j <= i} g^{i-j} (q_i . k_j) v_j, by a dense matrix."""
    rng = np.random.default_rng(0)
    B, H, N, d = 2, 3, 37, 5
    q, k, v = rng.standard_normal((3, B, H, N, d))
    lg = -rng.exponential(0.2, H)
    o, S = od.decay_attention(q, k, v, lg, 0.7)
    i, j = np.indices((N, N))
    D = np.where(i >= j, np.exp(lg.reshape(H, 1, 1) * np.maximum(i - j, 0)), 0.0)
    np.testing.assert_allclose(o, 0.7 * (np.einsum("bhid,bhjd->bhij", q, k) * D) @ v, rtol=1e-12, atol=1e-12)
    w = np.exp(lg[:, None] * (N - 1 - np.arange(N)))
    np.testing.assert_allclose(S, np.einsum("hn,bhni,bhnj->bhij", w, k, v), rtol=1e-12, atol=1e-12)


def test_splits_and_lengths():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 2, 2, 20, 4))
    lg = [-0.1, -np.inf]
    full, S = od.decay_attention(q, k, v, lg)
    a, Sa = od.decay_attention(q[:, :, :7], k[:, :, :7], v[:, :, :7], lg)
    b, Sb = od.decay_attention(q[:, :, 7:], k[:, :, 7:], v[:, :, 7:], lg, S=Sa)
    np.testing.assert_array_equal(np.concatenate([a, b], axis=2), full)
    np.testing.assert_array_equal(Sb, S)
    # a head that forgets at once attends to its own token alone
    own = np.einsum("bnd,bnd->bn", q[:, 1], k[:, 1])[..., None] * v[:, 1]
    np.testing.assert_allclose(full[:, 1], own, rtol=1e-13)
    r, Sr = od.decay_attention(q, k, v, lg, lengths=[7, 0])
    np.testing.assert_array_equal(r[0, :, :7], a[0])
    assert not r[0, :, 7:].any() and not r[1].any() and not Sr[1].any()
    np.testing.assert_array_equal(Sr[0], Sa[0])


def test_without_decay_it_is_the_attention_oracle_with_one_token_blocks():
    """g = 1, positive features and positions 0: the numerator of the block-causal oracle with
    one-token blocks (its denominator is multiplied back)."""
    rng = np.random.default_rng(2)
    H, N, d = 2, 9, 32
    q, k = np.abs(rng.standard_normal((2, 1, H, N, d)))
    v = rng.standard_normal((1, H, N, d))
    o, S, z = oracle.recurrence(q, k, v, np.zeros((N, 3), np.int32), np.arange(N, dtype=np.int32), (8, 12, 12), 1e4, 1.0)
    den = np.einsum("bhnd,bhnd->bhn", q, np.cumsum(k, axis=2)) + 1.0
    mine, Sm = od.decay_attention(q, k, v, np.zeros(H))
    np.testing.assert_allclose(mine, o * den[..., None], rtol=1e-5, atol=1e-4)  # the C oracle takes float32 inputs
    np.testing.assert_allclose(Sm[0], S, rtol=1e-5, atol=1e-5)


def test_rope_is_the_attention_oracles_rotation():
    pos = od.rope_positions(3, 4, 5, t0=2)
    ref_pos, _ = oracle.grid(3, 4, 5, 1, 2)
    np.testing.assert_array_equal(pos, ref_pos)
    # one pair of one axis, a quarter turn's worth of positions by hand
    x = np.zeros((1, 1, 1, 4))
    x[..., 0] = 1.0
    y = od.rope(x, [[0, 3, 0]], (0, 2, 2))
    np.testing.assert_allclose(y.ravel(), [np.cos(3.0), np.sin(3.0), 0, 0], atol=1e-15)


def test_rope_inverse_is_transpose_and_gradient():
    rng = np.random.default_rng(3)
    split, N, d = (4, 6, 2), 6, 16
    pos = rng.integers(-50, 5000, (2, N, 3))
    x, g = rng.standard_normal((2, 2, 1, N, d))
    y = od.rope(x, pos, split)
    np.testing.assert_allclose(od.rope(y, pos, split, inverse=True), x, atol=1e-12)
    np.testing.assert_array_equal(y[..., 12:], x[..., 12:])
    np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-13)
    # <g, rope(x)> has the gradient rope^-1(g): against central differences
    grad = od.rope(g, pos, split, inverse=True)
    for idx in [(0, 0, 1, 0), (1, 0, 5, 7), (1, 0, 2, 11), (0, 0, 0, 15)]:
        e = np.zeros_like(x)
        e[idx] = 1e-3
        diff = (np.vdot(g, od.rope(x + e, pos, split)) - np.vdot(g, od.rope(x - e, pos, split))) / 2e-3
        assert diff == pytest.approx(grad[idx], abs=1e-9)
