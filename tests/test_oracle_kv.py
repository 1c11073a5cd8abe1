"""Pins of the rotated key/value cache oracle: hand-worked cases and identities that need no kernel."""
import numpy as np
import pytest

from oracle import kvcache as kc


def test_places_and_slots():
    # sequence 0: two tokens of five positions; 1: none; 2: three tokens of two positions (one lies before the start)
    assert kc.places([1, 3, 3, 6], [5, 4, 2], 8) == [(None, None), (0, 3), (0, 4), (2, -1), (2, 0), (2, 1), (None, None),
                                                     (None, None)]
    table = np.array([[7, 2], [9, -1]])
    assert kc.slot(table, 8, 4, 0, 0) == (7, 0)
    assert kc.slot(table, 8, 4, 0, 6) == (2, 2)
    assert kc.slot(table, 8, 4, 0, 8) is None and kc.slot(table, 8, 4, 0, -1) is None
    assert kc.slot(table, 8, 4, 1, 0) is None and kc.slot(table, 8, 4, 1, 5) is None


def test_rope_by_hand():
    x = np.array([1.0, 2.0, 3.0, 4.0, 5.0])
    a = np.array([np.pi / 2, np.pi])
    np.testing.assert_allclose(kc.rope(x, a, False), [-3.0, -2.0, 1.0, -4.0, 5.0], atol=1e-15)
    np.testing.assert_allclose(kc.rope(x, a, True), [-2.0, 1.0, -3.0, -4.0, 5.0], atol=1e-15)
    # relative: the score of two turned vectors goes by the difference of their positions
    r = np.random.RandomState(0)
    f, q, k = r.rand(8), r.randn(16), r.randn(16)
    for il in (False, True):
        s = [kc.rope(q, kc.angles(f, p + 5, 0), il) @ kc.rope(k, kc.angles(f, p, 0), il) for p in (0, 3, 900)]
        np.testing.assert_allclose(s, s[0], rtol=1e-11)


def test_angles_of_several_axes():
    pos = np.array([[10, 20], [3, 4]])
    np.testing.assert_allclose(kc.angles([1.0, 0.5, 0.25], 99, 1, pos, [0, 1, 2]), [20.0, 2.0, 0.0])
    np.testing.assert_allclose(kc.angles([1.0, 0.5], 99, 0), [99.0, 49.5])


@pytest.mark.parametrize("d", [64, 128])
def test_rotation_keeps_scores_and_inverts(d):
    r = np.random.RandomState(d)
    s = r.choice([-1, 1], d)
    x, y = r.randn(3, d), r.randn(3, d)
    np.testing.assert_allclose((kc.rotate(x, s) * kc.rotate(y, s)).sum(-1), (x * y).sum(-1), rtol=1e-10)
    np.testing.assert_allclose(kc.unrotate(kc.rotate(x, s), s), x, atol=1e-13)
    e = np.zeros(d)
    e[3] = 2.0  # column 3 of H is + - pattern of popcount(3 & i)
    ref = [2.0 * s[3] * (-1) ** bin(3 & i).count("1") / np.sqrt(d) for i in range(d)]
    np.testing.assert_allclose(kc.rotate(e, s), ref, atol=1e-15)


def test_quantize_by_hand():
    q, s, t = kc.quantize(np.array([[7.0, -3.5, 0.5, 2.49], [0.0, 0.0, 0.0, 0.0], [1.0, np.nan, 0.0, 0.0]]), 4)
    assert q[0].tolist() == [7, -4, 0, 2] and s[0] == 1.0  # -3.5 and 0.5 tie to even
    assert q[1].tolist() == [0] * 4 and s[1] == 0.0
    assert q[2].tolist() == [0] * 4 and np.isnan(s[2])
    assert kc.pack(np.array([-8, 7, 0, 1]) + 0, 4).tolist() == [0xF0, 0x98]
    assert kc.unpack(np.array([0xF0, 0x98], dtype=np.uint8), 4).tolist() == [-8, 7, 0, 1]
    assert kc.pack(np.array([-127, 127]), 8).tolist() == [1, 255]


def test_attention_of_one_key_is_its_value():
    r = np.random.RandomState(1)
    codes = r.randint(1, 16, (2, 1, 4, 64)).astype(np.uint8)
    codes = (codes[..., ::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
    scales = r.rand(2, 1, 4)
    vs = r.choice([-1, 1], 64)
    q = r.randn(2, 3, 64)
    out, _ = kc.attention(q, (codes, scales), (codes, scales), np.array([[1]]), [0, 2], [1], 4, None, vs, 0.125)
    assert (out[0] == 0.0).all()  # position -1 sees nothing
    value = kc.unrotate(kc.unpack(codes[1, 0, 0], 4) * scales[1, 0, 0], vs)
    np.testing.assert_allclose(out[1], np.tile(value, (3, 1)), atol=1e-13)


def test_visible():
    assert list(kc.visible(5, 9, True, 0)) == [0, 1, 2, 3, 4, 5]
    assert list(kc.visible(5, 9, True, 2)) == [4, 5]
    assert list(kc.visible(5, 4, False, 0)) == [0, 1, 2, 3]
    assert list(kc.visible(-1, 4, True, 0)) == []
