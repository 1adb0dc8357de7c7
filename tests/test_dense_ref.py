"""The tests' plain forms against worked examples (CPU)."""
import numpy as np

import dense_ref as ref


def test_route_worked_example():
    logits = np.array([[0.0, 2.0, 1.0, 2.0]])
    ids, w = ref.route(logits, 3)
    e = np.exp([2.0, 2.0, 1.0])
    assert ids.tolist() == [[1, 3, 2]]                      # the tie goes to the lower index
    assert np.allclose(w[0], e / e.sum(), rtol=1e-15)
    ids, w = ref.route(logits, 2, renorm=False, scale=2.0)
    assert np.allclose(w[0], 2 * np.exp([2.0, 2.0]) / np.exp(logits[0]).sum(), rtol=1e-15)


def test_route_bias_decides_but_does_not_weigh():
    ids, w = ref.route(np.zeros((1, 4)), 2, score="sigmoid", bias=[0.0, 0.0, 0.5, 0.25], renorm=False)
    assert ids.tolist() == [[2, 3]] and w.tolist() == [[0.5, 0.5]]


def test_route_groups():
    # groups {0,1}, {2,3}, {4,5}: best single expert in the first, best pair in the last
    logits = np.array([[4.0, -4.0, 1.0, 1.0, 3.0, 2.5]])
    assert ref.route(logits, 2, groups=3, topk_groups=1)[0].tolist() == [[0, 1]]
    assert ref.route(logits, 2, score="sigmoid", groups=3, topk_groups=1, group_score="top2")[0].tolist() == [[4, 5]]


def test_route_masked():
    nan, inf = np.nan, np.inf
    ids, w = ref.route(np.array([[nan, -inf, 1.0, -inf], [-inf] * 4, [inf, 0, inf, 0]]), 3)
    assert ids.tolist() == [[2, 0, 1], [0, 1, 2], [0, 2, 1]]
    assert w.tolist() == [[1, 0, 0], [0, 0, 0], [0.5, 0.5, 0]]


def test_route_nan_or_infinite_bias_decides_but_does_not_weigh():
    """The bias puts an expert last; its score stays, in its own weight and in the sum."""
    for b in (np.nan, -np.inf):
        ids, w = ref.route(np.zeros((1, 3)), 3, score="sigmoid", bias=[b, 0.0, 0.0])
        assert ids.tolist() == [[1, 2, 0]] and np.allclose(w, 1 / 3, rtol=1e-15)


def test_quant_worked_example():
    q, s = ref.quant(np.array([[0.0, 0.0, 0.0], [127.0, 0.5, -1.5], [254.0, 1.0, 3.0], [np.inf, 1.0, 0.0]]))
    assert q.tolist() == [[0, 0, 0], [127, 0, -2], [127, 0, 2], [0, 0, 0]]   # halves go to even
    assert s[:3].tolist() == [0.0, 1.0, 2.0] and np.isnan(s[3])


def test_linear_worked_example():
    a, w = np.array([[1, 2]], np.int8), np.array([[3, 4], [5, -6]], np.int8)
    y, _ = ref.linear(a, np.array([0.5]), w, np.array([1.0, 2.0]), bias=np.array([1.0, 0.0]))
    assert y.tolist() == [[6.5, -7.0]]
    y, _ = ref.linear(a, np.array([0.5]), w, np.array([1.0, 2.0]), act="swiglu", add=np.array([[1.0]]))
    assert np.allclose(y, 5.5 / (1 + np.exp(-5.5)) * -7.0 + 1.0)
