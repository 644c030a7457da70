"""Pins of the rotation's, the 4-bit cache's and the norm's oracles."""
import numpy as np
import pytest

from oracle import kv4, norm


def test_rotation_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(5, 3, 32))
    table = kv4.rotary_table(50, 16).astype(np.float64)
    for inter in (False, True):
        y = kv4.rotate(x, table[[0, 1, 7, 49, 20]], inter, exact=True)
        assert np.array_equal(y[0], x[0])                     # position 0: no angle
        assert np.array_equal(y[..., 16:], x[..., 16:])       # past rotary_dim
        pair = (lambda a: a[..., :16].reshape(5, 3, 8, 2)) if inter else \
            (lambda a: a[..., :16].reshape(5, 3, 2, 8).swapaxes(2, 3))
        assert np.allclose((pair(y) ** 2).sum(-1), (pair(x) ** 2).sum(-1), rtol=1e-6)
        z = pair(x)[..., 0] + 1j * pair(x)[..., 1]
        turned = z * np.exp(1j * np.array([0, 1, 7, 49, 20])[:, None, None] *
                            10000.0 ** (-np.arange(8) / 8))
        assert np.allclose(pair(y)[..., 0], turned.real, atol=1e-6)
        assert np.allclose(pair(y)[..., 1], turned.imag, atol=1e-6)


def test_scores_of_rotated_pairs_depend_on_the_distance():
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(2, 1, 1, 64))
    table = kv4.rotary_table(400, 64).astype(np.float64)
    dot = lambda a, b: (kv4.rotate(q, table[[a]], exact=True) *
                        kv4.rotate(k, table[[b]], exact=True)).sum()
    assert abs(dot(300, 290) - dot(10, 0)) < 1e-4


def test_values_that_can_be_held_come_back():
    code = np.arange(16, dtype=np.uint8)
    for sb in (1, 7, 8, 56, 100, 126):
        x = kv4.decode(code, np.array([sb]))
        c, s = kv4.encode(x)
        assert s[0] == sb and np.array_equal(kv4.decode(c, s), x)


def test_ties_and_ends():
    half = lambda a, b: (a + b) / 2
    x = np.array([half(0, .5), half(.5, 1), half(1, 1.5), half(1.5, 2), half(2, 3), half(3, 4),
                  half(4, 6), 6] + [0.0] * 8)
    c, s = kv4.encode(x)
    assert s[0] == 56  # scale 1
    assert kv4.CODES[c[:8]].tolist() == [0, 1, 1, 2, 2, 4, 4, 6]
    c, s = kv4.encode(np.full(16, 1e30))
    assert s[0] == 126 and (c == 7).all()               # 448 * 6 at most
    c, s = kv4.encode(np.full(16, 6 * 2.0 ** -11))      # nothing that small
    assert s[0] == 0 and (kv4.decode(c, s) == 0).all()
    c, s = kv4.encode(np.array([np.nan, -np.inf] + [1.0] * 14))
    assert s[0] == 126 and c[0] == 0 and c[1] == 15


def test_error_of_a_block():
    """A code is within a sixth of the largest value's share (codes 4 and 6 are furthest apart), and
    the scale within half a step of three bits of mantissa."""
    rng = np.random.default_rng(2)
    x = rng.normal(size=(200, 64))
    c, s = kv4.encode(x, 0.5)
    back = kv4.decode(c, s, 0.5)
    top = np.abs(x).reshape(200, 4, 16).max(-1).repeat(16, -1)
    assert (np.abs(back - x) <= top * (1 / 6 + 1 / 16)).all()


def test_pack_and_unpack():
    rng = np.random.default_rng(3)
    code = rng.integers(0, 16, (3, 16, 2, 64)).astype(np.uint8)
    sb = rng.integers(0, 127, (3, 16, 2, 4)).astype(np.uint8)
    for values in (False, True):
        b = kv4.pack(code, sb, values)
        assert b.shape == (3, 2, 576)
        c, s = kv4.unpack(b, 64, values)
        assert np.array_equal(c, code) and np.array_equal(s, sb)
    # the second token's third byte holds its values 4 and 5; block 1's scale of token 2
    k, v = kv4.pack(code, sb, False), kv4.pack(code, sb, True)
    assert k[1, 0, 32 + 2] == code[1, 1, 0, 4] | code[1, 1, 0, 5] << 4
    assert k[1, 0, 512 + 2 * 4 + 1] == sb[1, 2, 0, 1] == v[1, 0, 512 + 16 + 2]


@pytest.mark.parametrize("group", [0, 4])
def test_norm(group):
    y = norm.rms_norm(np.array([[3.0, 4.0, 0, 0], [0, 0, 0, 0]]), [1, 2, 1, 1], 0.0 + 1e-30)
    assert np.allclose(y, [[1.2, 3.2, 0, 0], [0, 0, 0, 0]])
    assert np.allclose(norm.scales_of(y, group), [[3.2 / 448], [0]])
