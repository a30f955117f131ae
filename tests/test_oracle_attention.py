"""The oracle of the calls around an 8-bit cache against closed forms and
hand-worked values (CPU)."""
import numpy as np
import pytest

from oracle import attention as oa


def test_norm_by_hand():
    x = np.array([[[3.0, 4.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0]]])      # mean of squares 25 / 8
    y, _ = oa.norm_rope(x, np.full(8, 2.0), 0.0, None, [0], 0, 0)
    assert np.allclose(y[0, 0, :2], np.array([6.0, 8.0]) / np.sqrt(25 / 8))
    y, _ = oa.norm_rope(x, None, 0.0, None, [0], 0, 0)
    assert np.array_equal(y, x)


@pytest.mark.parametrize("interleaved", [0, 1])
def test_quarter_turns_and_padding(interleaved):
    x = np.arange(1.0, 17.0).reshape(1, 1, 16).repeat(3, 0)
    table = np.array([[1.0] * 4 + [0.0] * 4, [0.0] * 4 + [1.0] * 4])          # no turn, a quarter turn
    y, size = oa.norm_rope(x, None, 0.0, table, [0, 1, 2], 8, interleaved)
    assert np.array_equal(y[0], x[0]) and np.isnan(y[2]).all()
    want = [-2, 1, -4, 3, -6, 5, -8, 7] if interleaved else [-5, -6, -7, -8, 1, 2, 3, 4]
    assert y[1, 0, :8].tolist() == want and np.array_equal(y[1, 0, 8:], x[1, 0, 8:])
    assert np.array_equal(size[1], np.abs(y[1]))


def test_rotated_products_depend_on_the_distance():
    rng = np.random.default_rng(0)
    angle = np.arange(20)[:, None] * 0.7 ** np.arange(8)
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    a, b = rng.normal(size=(1, 1, 16)), rng.normal(size=(1, 1, 16))
    for inter in (0, 1):
        turn = lambda x, at: oa.norm_rope(x, None, 0.0, table, [at], 16, inter)[0][0, 0]  # noqa: E731
        assert np.isclose(turn(a, 3) @ turn(b, 9), turn(a, 11) @ turn(b, 17))


@pytest.mark.parametrize("page,D", [(16, 64), (32, 128), (64, 192), (128, 256)])
def test_every_byte_has_one_token_and_channel(page, D):
    for values in (False, True):
        assert np.array_equal(np.sort(oa.byte_index(page, D, values).ravel()), np.arange(page * D))


def test_bytes_by_hand():
    assert oa.key_byte(17, 70, 128) == 2048 + 1024 + 0 + 16 + 6
    assert oa.value_byte(17, 70, 128) == 2048 + 1024 + 0 + 16 * 6 + 0 + 1
    assert oa.value_byte(6, 35, 64) == 256 + 16 * 3 + 4 * 2 + 2


def test_a_scale_grows_and_a_page_starts_anew():
    c = oa.Cache(oa.INT8, 1, 64, 16, 2)
    table = np.array([[1]])
    one = np.zeros((1, 1, 64), np.float32)
    one[0, 0, 0] = 127.0
    c.append([0, 1], [1], table, one, one)
    assert c.scales[0][1, 0] == 1 and c.token(0, table, 0, 0)[0, 0] == 127
    c.append([0, 1], [2], table, 3 * one, one / 2)
    assert c.scales[0][1, 0] == 3 and c.scales[1][1, 0] == 1
    assert c.token(0, table, 0, 0)[0, 0] == 126                      # 127 / 3 = 42.33 -> 42
    assert c.token(1, table, 0, 1)[0, 0] == 64                       # 63.5 -> 64 (even)
    assert np.isnan(c.scales[0][0, 0]) and (c.codes[0][0] == 0x7F).all()
    c.append([0, 1], [1], table, one, one)
    assert c.scales[0][1, 0] == 1 and c.token(0, table, 0, 0)[0, 0] == 127


def test_absent_tokens_are_not_stored():
    c = oa.Cache(oa.FP8, 1, 64, 16, 2)
    x = np.ones((20, 1, 64), np.float32)
    c.append([0, 20], [18], np.array([[0, 2]]), x, x)                # positions -2 .. 17; page 2 does not exist
    index = c.index[0]
    assert (c.codes[0][0, 0][index] == 0x7E).all() and (c.codes[0][1] == 0x7F).all()
    assert c.token(0, np.array([[0, 2]]), 0, 16) is None and c.token(0, np.array([[0, 2]]), 0, 32) is None


def filled(rng, fmt=oa.FP8, n=40, heads=2, D=64, page=16):
    c = oa.Cache(fmt, heads, D, page, 5)
    table = np.array([[4, 0, 2]])
    k, v = rng.normal(size=(2, n, heads, D)).astype(np.float32)
    c.append([0, n], [n], table, k, v)
    return c, table


def test_attention_of_equal_scores_is_the_mean_and_of_one_token_is_it():
    c, table = filled(np.random.default_rng(1))
    v = c.exact(1, table, 0, range(40))
    y, W, E, F = oa.attention(c, [0, 2], [40], table, np.zeros((2, 4, 64)), 0.3)
    assert np.allclose(y[1], v.mean(0).repeat(2, 0)) and np.allclose(y[0], v[:39].mean(0).repeat(2, 0))
    assert np.allclose(W[1], np.abs(v).mean(0).repeat(2, 0)) and (E == 0).all()
    assert np.allclose(F, W)                                         # all p are 1
    q = np.random.default_rng(2).normal(size=(2, 4, 64))
    y, *_ = oa.attention(c, [0, 2], [40], table, q, 0.3, window=1)
    assert np.allclose(y, v[38:40].repeat(2, 1))
    y, *_ = oa.attention(c, [0, 2], [40], table, q, 0.3, causal=False)
    for t in range(2):
        for h in range(4):
            s = np.exp(c.exact(0, table, 0, range(40))[:, h // 2] @ q[t, h] * 0.3)
            assert np.allclose(y[t, h], s @ v[:, h // 2] / s.sum())


def test_tokens_that_see_nothing():
    c, table = filled(np.random.default_rng(3))
    q = np.ones((3, 2, 64))
    y, *_ = oa.attention(c, [0, 3], [2], table, q, 1.0)              # positions -1, 0, 1
    assert (y[0] == 0).all() and np.allclose(y[1], c.exact(1, table, 0, [0])[0])
    y, *_ = oa.attention(c, [0, 3], [40], np.full((1, 3), -1), q, 1.0)
    assert (y == 0).all()
    y, *_ = oa.attention(c, [0, 0, 2], [5, 40], np.repeat(table, 2, 0), q, 1.0)
    assert np.isnan(y[2]).all() and not np.isnan(y[:2]).any()
