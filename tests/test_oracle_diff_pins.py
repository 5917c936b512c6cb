"""Pins of the oracle's norm-and-rotation and differential attention: closed forms,
invariants and a complex-number restatement."""

import numpy as np
import pytest

import oracle


def _rows(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    x = _rows(0, 64)
    ang = _rows(1, 12)
    got = oracle.norm_rotate_row(x, None, np.cos(ang), np.sin(ang), 0.0, interleaved)
    a, b = (x[0:24:2], x[1:24:2]) if interleaved else (x[:12], x[12:24])
    z = (a + 1j * b) * np.exp(1j * ang)
    want = x.copy()
    if interleaved:
        want[0:24:2], want[1:24:2] = z.real, z.imag
    else:
        want[:12], want[12:24] = z.real, z.imag
    assert np.allclose(got, want, rtol=0, atol=1e-14)
    wrong = oracle.norm_rotate_row(x, None, np.cos(ang), -np.sin(ang), 0.0, interleaved)
    assert not np.allclose(wrong, want, atol=1e-3)                  # turned the other way
    other = oracle.norm_rotate_row(x, None, np.cos(ang), np.sin(ang), 0.0, not interleaved)
    assert not np.allclose(other, want, atol=1e-3)                  # the other pairing


def test_rotation_keeps_scores_of_equal_distances():
    """Rotated q and k have a dot product that depends on the distance alone."""
    q, k = _rows(2, 32), _rows(3, 32)
    f = 10.0 ** -np.linspace(0, 3, 16)

    def turned(x, pos):
        return oracle.norm_rotate_row(x, None, np.cos(pos * f), np.sin(pos * f), 0.0)
    dots = [turned(q, 7 + d) @ turned(k, 3 + d) for d in (0, 1, 50, 1000)]
    assert np.ptp(dots) < 1e-10
    assert abs(turned(q, 8) @ turned(k, 3) - dots[0]) > 1e-3


def test_norm_closed_forms():
    x = np.full(64, -3.0)
    assert np.allclose(oracle.norm_rotate_row(x, np.ones(64), [], [], 0.0), -1.0)
    assert np.allclose(oracle.norm_rotate_row(x, np.arange(64.0), [], [], 0.0), -np.arange(64.0))
    assert np.allclose(oracle.norm_rotate_row(x, np.ones(64), [], [], 16.0), -3.0 / 5.0)
    assert np.all(oracle.norm_rotate_row(np.zeros(64), np.ones(64), [], [], 1e-6) == 0)
    y = oracle.norm_rotate_row(_rows(4, 64), np.ones(64), [], [], 0.0)
    assert abs(np.mean(y * y) - 1) < 1e-12


def _case(seed, L, hq=8, hkv=4, d=16):
    return _rows(seed, hq, d), list(_rows(seed + 1, hkv, L, d)), list(_rows(seed + 2, hkv, L, d))


def test_diff_lambda_zero_is_plain_attention_on_even_heads():
    q, k, v = _case(5, 9)
    out, maps = oracle.decode_attention_diff(q, k, v, np.zeros(4), 0.3)
    for j in range(4):
        p = j // 2
        for half in range(2):
            want, w = oracle.attend_one_head(q[2 * j], k[2 * p], v[2 * p + half], 0.3)
            assert np.allclose(out[j, half * 16:(half + 1) * 16], want, atol=1e-13)
            assert np.allclose(maps[j, 0], w)


def test_diff_closed_forms():
    q, k, v = _case(6, 1)                                   # one token: (1 - lambda) V'
    lam = np.array([0.25, 0.5, 1.0, 3.0])
    out, _ = oracle.decode_attention_diff(q, k, v, lam, 1.0)
    for j in range(4):
        p = j // 2
        assert np.allclose(out[j], (1 - lam[j]) * np.concatenate([v[2 * p][0], v[2 * p + 1][0]]))
    q, k, v = _case(7, 6)
    out, maps = oracle.decode_attention_diff(q, k, v, np.ones(4), 0.0)   # equal maps cancel
    assert np.abs(out).max() < 1e-14 and np.allclose(maps, 1 / 6)
    same = oracle.decode_attention_diff(np.repeat(q[::2], 2, 0), [k[0], k[0], k[2], k[2]], v,
                                        np.ones(4), 0.7)[0]
    assert np.abs(same).max() < 1e-14
    empty, _ = oracle.decode_attention_diff(*_case(8, 0), np.ones(4), 1.0)
    assert np.all(empty == 0)


def test_diff_norm_and_scale():
    q, k, v = _case(9, 11)
    lam = np.full(4, 0.4)
    raw, _ = oracle.decode_attention_diff(q, k, v, lam, 0.5)
    out, _ = oracle.decode_attention_diff(q, k, v, lam, 0.5, np.ones(32), 0.0, 0.2)
    assert np.allclose(np.sqrt(np.mean(out ** 2, 1)), 0.2)
    assert np.allclose(out / out[:, :1], raw / raw[:, :1])


def test_planted_mistakes_show():
    """A map over the other head's keys, halves of V' exchanged, an interleaved pairing and a
    dropped lambda each change the result."""
    q, k, v = _case(10, 8)
    lam = np.array([0.3, 0.6, 0.2, 0.8])
    out, _ = oracle.decode_attention_diff(q, k, v, lam, 0.5)
    swapped_k = oracle.decode_attention_diff(q, [k[1], k[0], k[3], k[2]], v, lam, 0.5)[0]
    swapped_v = oracle.decode_attention_diff(q, k, [v[1], v[0], v[3], v[2]], lam, 0.5)[0]
    halves = oracle.decode_attention_diff(q[[0, 4, 1, 5, 2, 6, 3, 7]], k, v, lam, 0.5)[0]
    ones = oracle.decode_attention_diff(q, k, v, np.ones(4), 0.5)[0]
    for wrong in (swapped_k, swapped_v, halves, ones):
        assert np.abs(wrong - out).max() > 1e-2
