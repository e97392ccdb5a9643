"""Pins of oracle/rules.py: worked examples, the neutral rules, the pinned top-k
and draw of oracle/select.py, and the words of a mask."""
import numpy as np

from oracle import rules, select

INF = float("inf")


def test_worked_example():
    y = [2.0, -1.0, 0.0, 4.0, 1.0]
    got = rules.adjust(y, history=[0, 1, 3, 3, 9, -1, 3, 1], prompt=3, repetition=2.0, frequency=0.25, presence=0.5,
                       bias=[(4, 3.0), (0, 7.0), (4, -0.5), (2, -INF), (5, 1.0)])
    # 0: prompt only, halved, +7; 1: doubled, once generated; 3: halved, twice generated; 4: the last bias; 2 banned
    assert np.array_equal(got, np.array([8.0, -2.75, -INF, 2.0 - 0.5 - 0.5, 0.5], dtype=np.float32))
    masked = rules.adjust(y, mask=[1, 0, 0, 1, 0])
    assert np.array_equal(masked, np.array([2.0, -INF, -INF, 4.0, -INF], dtype=np.float32))


def test_neutral_rules_change_nothing():
    y = np.array([0.1, -0.0, -INF, INF, 3e38, 1e-40], dtype=np.float32)
    assert np.array_equal(rules.adjust(y, history=[0, 1, 2, 3, 4, 5]), y)


def test_top_and_draw_are_those_of_the_head():
    rng = np.random.default_rng(0)
    for _ in range(50):
        y = np.round(rng.normal(0, 1, 40), 1).astype(np.float32)  # many ties
        v, i = rules.top(y, 7)
        want_v, want_i = select.top_k(y[None], 7)
        assert np.array_equal(i, want_i[0]) and np.array_equal(v, want_v[0])
        u, tau = rng.random(), rng.uniform(0.2, 2.0)
        assert rules.draw(v, i, u, tau) == select.sample_top_k(want_v, want_i, tau, np.array([u]))[0]


def test_rows_with_nothing_left_and_ends_of_the_draw():
    assert rules.draw([-INF, -INF], [0, 1], 0.3, 1.0) == -1
    assert rules.draw([np.nan, 1.0], [4, 1], 0.3, 1.0) == -1
    assert rules.draw([INF, INF, 1.0], [3, 5, 1], 0.9, 1.0) == 3
    assert rules.draw([2.0, 1.0], [7, 1], 0.99, 0.0) == 7
    assert rules.draw([2.0, -INF], [7, 1], 1.0 - 2.0 ** -24, 1.0) == 7
    v, i = rules.top(np.array([1.0, np.nan, -0.0, 0.0, np.nan], dtype=np.float32), 5)
    assert list(i) == [1, 4, 0, 2, 3]


def test_words_of_a_mask():
    m = np.zeros((2, 40), dtype=bool)
    m[0, [0, 31, 32]] = True
    m[1, 39] = True
    assert rules.bits(m).tolist() == [[1 - 2 ** 31, 1], [0, 128]]
