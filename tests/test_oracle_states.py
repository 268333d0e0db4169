"""What ties the oracle of the operators over rows of hidden states to the
mathematics: cases by hand, invariances, and gradients against differences."""
import numpy as np
import pytest

from oracle import states as os_


def test_embed_by_hand():
    table = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    got = os_.embed(table, [2, -1, 0, 3, -2], 2.0)
    np.testing.assert_array_equal(got[:3], [[10, 12], [0, 0], [2, 4]])
    assert np.isnan(got[3:]).all()


def test_embed_grad_by_hand():
    grad = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0], [7.0, 8.0], [9.0, 1.0]])
    got = os_.embed_grad(grad, [1, -1, 1, 0, 5], 3, 0.5)
    np.testing.assert_array_equal(got, [[3.5, 4], [3, 4], [0, 0]])
    np.testing.assert_array_equal(os_.embed_grad(grad, [1, -1, 1, 0, 5], 3, 0.5, np.ones((3, 2))),
                                  got + 1)


def test_embed_grad_is_the_lookups_transpose():
    """<embed(T), G> is linear in T with the gradient as its matrix."""
    rng = np.random.default_rng(0)
    table, grad = rng.normal(size=(7, 5)), rng.normal(size=(20, 5))
    ids = rng.integers(-1, 7, 20)
    left = (os_.embed(table, ids, 1.7) * grad).sum()
    assert abs(left - (table * os_.embed_grad(grad, ids, 7, 1.7)).sum()) < 1e-12


def test_layernorm_by_hand():
    y = os_.layernorm(np.array([[1.0, 3.0]]), np.array([2.0, 5.0]), np.array([0.5, -0.5]), 0.0)
    np.testing.assert_allclose(y, [[-1.5, 4.5]])
    np.testing.assert_allclose(os_.layernorm(np.full((1, 4), 7.0), None, None, 1e-5), 0.0)


def test_layernorm_knows_no_shift_and_no_scale():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(3, 50))
    y = os_.layernorm(x, None, None, 0.0)
    np.testing.assert_allclose(os_.layernorm(4.0 * x - 9.0, None, None, 0.0), y, atol=1e-12)
    np.testing.assert_allclose(y.mean(1), 0.0, atol=1e-14)
    np.testing.assert_allclose((y * y).mean(1), 1.0)


@pytest.mark.parametrize("weighted", [False, True])
def test_layernorm_gradients_against_differences(weighted):
    rng = np.random.default_rng(2)
    x, grad = rng.normal(size=(4, 9)), rng.normal(size=(4, 9))
    weight = rng.normal(size=9) if weighted else None
    bias = rng.normal(size=9)
    eps, h = 1e-3, 1e-5

    def loss(x, weight, bias):
        return (os_.layernorm(x, weight, bias, eps) * grad).sum()

    mean, inverse = os_.norm_stats(x, eps)
    gx, gw, gb = os_.layernorm_grad(x, mean, inverse, weight, grad)
    for at in np.ndindex(x.shape):
        step = np.zeros_like(x)
        step[at] = h
        d = (loss(x + step, weight, bias) - loss(x - step, weight, bias)) / (2 * h)
        assert abs(d - gx[at]) < 1e-8
    w = np.ones(9) if weight is None else weight
    for c in range(9):
        step = np.zeros(9)
        step[c] = h
        d = (loss(x, w + step, bias) - loss(x, w - step, bias)) / (2 * h)
        assert abs(d - gw[c]) < 1e-8
        d = (loss(x, w, bias + step) - loss(x, w, bias - step)) / (2 * h)
        assert abs(d - gb[c]) < 1e-8
