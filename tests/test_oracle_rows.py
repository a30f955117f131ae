"""The per-row oracle (routing, combine, adapters) against hand-worked values
and brute force (CPU)."""
import numpy as np
import pytest

from oracle import rows

INF, NAN = np.inf, np.nan


def test_softmax_route_by_hand():
    # exp: 1, 2, 4, 1 -> sum 8
    l = np.log(np.array([[1.0, 2.0, 4.0, 1.0], [4.0, 1.0, 1.0, 2.0]]))
    ids, w, off, r, s = rows.route(l, 2, renormalize=0)
    assert ids.tolist() == [[2, 1], [0, 3]]
    assert np.allclose(w, [[0.5, 0.25], [0.5, 0.25]], rtol=1e-14)
    assert off.tolist() == [0, 1, 2, 3, 4] and r.tolist() == [1, 0, 0, 1] and s.tolist() == [[2, 1], [0, 3]]
    _, w, *_ = rows.route(l, 2, scale=3.0)
    assert np.allclose(w, [[2.0, 1.0], [2.0, 1.0]], rtol=1e-14)


def test_sigmoid_bias_only_steers():
    l = np.array([[0.0, -np.log(3.0), np.log(3.0)]])        # 1/2, 1/4, 3/4
    ids, w, *_ = rows.route(l, 2, rows.SIGMOID, bias=[0.0, 0.6, 0.0], renormalize=0)
    assert ids.tolist() == [[1, 2]] and np.allclose(w, [[0.25, 0.75]])
    ids, w, *_ = rows.route(l, 3, rows.SIGMOID, bias=[-INF, NAN, 0.0])
    assert ids.tolist() == [[2, -1, -1]] and np.allclose(w, [[1.0, 0.0, 0.0]])


def test_ties_masks_and_extremes():
    ids, w, off, r, s = rows.route([[1.0, 1.0, 1.0], [-INF, -INF, -INF], [NAN, 2.0, -INF], [INF, 0.0, 0.0]], 2)
    assert ids.tolist() == [[0, 1], [-1, -1], [1, -1], [0, 1]]
    assert np.allclose(w, [[0.5, 0.5], [0, 0], [1, 0], [1, 0]])
    assert off.tolist() == [0, 2, 5, 5] and r.tolist() == [0, 3, 0, 2, 3, -1, -1, -1]
    assert s.tolist() == [[0, 2], [-1, -1], [3, -1], [1, 4]]
    ids, w, *_ = rows.route(np.full((1, 4), -rows.FLT_MAX), 2)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, 0.5)
    ids, w, *_ = rows.route(np.full((1, 4), -rows.FLT_MAX), 2, rows.SIGMOID)
    assert ids.tolist() == [[0, 1]] and (w == 0).all()


def test_groups_by_hand():
    l = np.log(np.array([[8.0, 1.0, 5.0, 5.0, 7.0, 1.0]]))     # three groups of two
    assert rows.route(l, 2, groups=3, topk_groups=1)[0].tolist() == [[0, 1]]
    assert rows.route(l, 2, groups=3, topk_groups=1, group_score=rows.TOP2)[0].tolist() == [[2, 3]]
    assert rows.route(l, 2, groups=3, topk_groups=2)[0].tolist() == [[0, 4]]
    # a group with one open expert is worth that expert
    l2 = l.copy()
    l2[0, 1] = -INF
    assert rows.route(l2, 2, groups=3, topk_groups=1, group_score=rows.TOP2)[0].tolist() == [[2, 3]]
    assert rows.route(l2, 2, groups=3, topk_groups=1)[0].tolist() == [[0, -1]]


def test_rows_invert_slots():
    rng = np.random.default_rng(5)
    l = rng.normal(size=(23, 11))
    l[rng.random((23, 11)) < 0.4] = -INF
    ids, _, off, r, s = rows.route(l, 5)
    seen = set()
    for t in range(23):
        for j in range(5):
            if ids[t, j] < 0:
                assert s[t, j] == -1
                continue
            i = s[t, j]
            assert off[ids[t, j]] <= i < off[ids[t, j] + 1] and r[i] == t
            seen.add(i)
    assert seen == set(range(off[-1])) and (r[off[-1]:] == -1).all()


def test_combine_and_lora_by_hand():
    h = np.array([[1.0, 2.0], [3.0, 5.0]])
    y, size = rows.combine(h, np.array([[1, 0], [-1, 0], [7, -1]]), np.array([[2.0, -1.0], [NAN, 4.0], [1.0, 1.0]]),
                           np.array([[1.0, 1.0], [0.0, 0.0], [6.0, 7.0]]))
    assert y.tolist() == [[6.0, 9.0], [4.0, 8.0], [6.0, 7.0]] and size.tolist() == [[8.0, 13.0], [4.0, 8.0], [6.0, 7.0]]
    A = np.array([[[1.0, 1.0], [NAN, NAN]], [[2.0, 0.0], [0.0, 1.0]]])
    B = np.array([[[1.0, NAN], [3.0, NAN]], [[1.0, 1.0], [0.0, 1.0]]])
    x = np.array([[1.0, 2.0]] * 4)
    y, *_ = rows.lora(x, [0, 1, -1, 2], A, B, [1, 2], [1.0, 0.5], np.ones((4, 2)))
    assert y.tolist() == [[4.0, 10.0], [3.0, 2.0], [1.0, 1.0], [1.0, 1.0]]


@pytest.mark.parametrize("seed", range(3))
def test_lora_equals_one_product_per_adapter(seed):
    rng = np.random.default_rng(seed)
    x, A, B = rng.normal(size=(9, 16)), rng.normal(size=(3, 4, 16)), rng.normal(size=(3, 8, 4))
    ids = rng.integers(-1, 4, 9)
    y, of_v, of_terms = rows.lora(x, ids, A, B)
    want = np.zeros((9, 8))
    for a in range(3):
        want[ids == a] = x[ids == a] @ A[a].T @ B[a].T
    assert np.allclose(y, want, rtol=1e-12, atol=1e-12)
    assert (np.abs(y) <= of_v + 1e-12).all() and (of_v <= of_terms + 1e-12).all()
