"""The fp64 routing oracle: closed forms, invariants, and its gradient against central
differences of its own forward definitions."""
import numpy as np
import pytest

from oracle import routing_oracle as R


def _logits(t, e, seed):
    return np.random.default_rng(seed).normal(size=(t, e)) * 1.5


def test_plain_softmax_topk_by_hand():
    idx, w = R.route(np.array([[1.0, 3.0, 2.0, 3.0]]), 2)
    assert idx.tolist() == [[1, 3]]                      # equal logits: the lower index first
    assert np.allclose(w, 0.5)
    idx, w = R.route(np.array([[1.0, 3.0, 2.0, 0.0]]), 2, renormalize=False, scale=2.0)
    p = np.exp([1.0, 3.0, 2.0, 0.0]) / np.exp([1.0, 3.0, 2.0, 0.0]).sum()
    assert idx.tolist() == [[1, 2]] and np.allclose(w, 2 * p[[1, 2]])


def test_bias_moves_the_choice_and_not_the_weight():
    l = np.array([[2.0, 1.0, 0.0, -1.0]])
    idx, w = R.route(l, 1, "sigmoid", bias=[0, 0, 0, 5.0], renormalize=False)
    assert idx.tolist() == [[3]] and np.allclose(w, 1 / (1 + np.e))


def test_groups_close_the_other_experts():
    l = np.array([[9.0, -9.0, 5.0, 5.0, 0.0, 0.0]])
    assert R.route(l, 2, num_groups=3, topk_groups=1)[0].tolist() == [[0, 1]]
    # by the two best of a group, the even pair beats the single peak under sigmoid scores
    assert R.route(l, 2, "sigmoid", 3, 1, 2)[0].tolist() == [[2, 3]]


def test_dead_rows_and_special_logits():
    l = np.full((1, 4), -np.inf)
    idx, w = R.route(l, 2)
    assert idx.tolist() == [[0, 1]] and np.all(w == 0)
    idx, w = R.route(np.array([[np.nan, 1.0, np.inf, -np.inf]]), 3)
    assert idx.tolist() == [[2, 1, 0]] and w.tolist() == [[1.0, 0.0, 0.0]]
    los, counts, p = R.losses(l, np.array([[0, 1]]))
    assert los.tolist() == [0, 0] and counts.tolist() == [1, 1, 0, 0, 1] and np.all(p == 0)


def test_uniform_routing_has_balance_k():
    l = np.zeros((8, 4))
    idx = np.array([[i % 4, (i + 1) % 4] for i in range(8)])
    los, counts, p = R.losses(l, idx)
    assert np.allclose(los, [2.0, np.log(4) ** 2]) and counts.tolist() == [4, 4, 4, 4, 8]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(scoring, renorm):
    rng = np.random.default_rng(3)
    l = _logits(5, 7, 1)
    idx, _ = R.route(l, 3, scoring)
    d_w, d_losses = rng.normal(size=(5, 3)), rng.normal(size=2)
    mask = np.array([1, 0, 1, 1, 1])
    _, counts, _ = R.losses(l, idx, scoring, mask)

    def total(x):
        return ((R.weights(x, idx, scoring, renorm, 1.7) * d_w).sum()
                + R.losses(x, idx, scoring, mask, counts)[0] @ d_losses)

    grad, size = R.route_backward(l, idx, scoring, renorm, 1.7, d_w, counts, d_losses, mask)
    h = 1e-5
    for t in range(5):
        for e in range(7):
            up, down = l.copy(), l.copy()
            up[t, e] += h
            down[t, e] -= h
            # second-order differences: error h^2 |f'''| / 6 + 2^-52 |f| / h, both below 1e-9
            assert abs((total(up) - total(down)) / (2 * h) - grad[t, e]) < 1e-8
    assert np.all(size >= np.abs(grad) - 1e-15)
