"""The oracle of the operators over rows of logits, pinned to hand-computed
values and to central differences of its own losses (CPU only)."""
import math

import numpy as np
import pytest

from oracle import logits as ol


def test_two_token_row_by_hand():
    z = np.array([math.log(3.0), 0.0])
    lp = ol.log_softmax(z, 1.0)
    np.testing.assert_allclose(np.exp(lp), [0.75, 0.25], rtol=1e-15)
    h = -(0.75 * math.log(0.75) + 0.25 * math.log(0.25))
    assert abs(ol.entropy(lp) - h) < 1e-15
    lp2 = ol.log_softmax(z, 0.5)                     # x = 2 log 3: 9 to 1
    np.testing.assert_allclose(np.exp(lp2), [0.9, 0.1], rtol=1e-14)


def test_shift_and_uniform_rows():
    z = np.random.default_rng(0).normal(size=50)
    np.testing.assert_allclose(ol.log_softmax(z + 7.0, 1.3), ol.log_softmax(z, 1.3), atol=1e-13)
    u = ol.log_softmax(np.full(8, -3.3e38), 1.0)
    np.testing.assert_allclose(u, -math.log(8.0), rtol=1e-15)
    assert abs(ol.entropy(u) - math.log(8.0)) < 1e-14


def test_rows_without_a_distribution():
    lp = ol.log_softmax(np.full(4, -np.inf), 1.0)
    assert np.isneginf(lp).all() and ol.entropy(lp) == 0.0
    assert (ol.logprobs_grad(np.full(4, -np.inf), 1.0, 2, 1.0) == 0).all()
    for bad in (np.nan, np.inf):
        assert np.isnan(ol.log_softmax(np.array([0.0, bad]), 1.0)).all()
    assert ol.token_logprob(np.log([0.5, 0.5]), -1) == 0.0
    assert np.isnan(ol.token_logprob(np.log([0.5, 0.5]), 2))
    assert np.isnan(ol.logprobs_grad(np.zeros(3), 1.0, 3, 1.0)).all()


def test_best_orders_by_value_then_index():
    z = np.array([1.0, -0.0, 0.0, np.nan, 1.0, -np.inf])
    assert ol.best(z, 6).tolist() == [0, 4, 1, 2, 3, 5]


def test_masked_tokens_drop_out():
    z = np.array([0.3, -np.inf, 1.1, -np.inf])
    lp = ol.log_softmax(z, 1.0)
    np.testing.assert_allclose(lp[[0, 2]], ol.log_softmax(z[[0, 2]], 1.0), rtol=1e-15)
    g = ol.logprobs_grad(z, 1.0, 0, 1.0, 0.7)
    assert g[1] == 0 and g[3] == 0


def _differences(f, z, h=1e-6):
    g = np.zeros(len(z))
    for j in range(len(z)):
        a, b = z.copy(), z.copy()
        a[j] += h
        b[j] -= h
        g[j] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("tau", [1.0, 0.6, 2.5])
def test_logprobs_gradient_is_the_difference_quotient(tau):
    rng = np.random.default_rng(1)
    z = rng.normal(size=23) * 2
    ids, gi = [4, 9, 4, -1], [0.3, -0.8, 0.2, 5.0]

    def f(x):
        lp = ol.log_softmax(x, tau)
        return 0.9 * lp[7] - 0.4 * ol.entropy(lp) + sum(g * lp[i] for i, g in zip(ids, gi)
                                                        if i >= 0)

    got = ol.logprobs_grad(z, tau, 7, 0.9, -0.4, ids, gi)
    # Central differences: truncation h^2 f''' / 6 plus 2^-53 |f| / h.
    np.testing.assert_allclose(got, _differences(f, z), atol=2e-8)


@pytest.mark.parametrize("mode", [ol.RENORM, ol.TAIL])
@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_distill_gradient_is_the_difference_quotient(mode, tau):
    rng = np.random.default_rng(2)
    z = rng.normal(size=30) * 2
    t = ol.log_softmax(rng.normal(size=30) * 2, 1.0)
    ids = np.array([3, 11, 29, -1, 0, 11])
    scores = np.where(ids >= 0, t[ids], 0.0)
    loss, grad, _ = ol.distill(z, tau, scores, ids, mode, 1.7)
    want = _differences(lambda x: 1.7 * ol.distill(x, tau, scores, ids, mode)[0], z)
    np.testing.assert_allclose(grad, want, atol=2e-8)
    assert abs(grad.sum()) < 1e-12                    # shifting a row changes nothing


def test_distill_is_zero_at_the_teacher_and_positive_elsewhere():
    rng = np.random.default_rng(3)
    z = rng.normal(size=40)
    lp = ol.log_softmax(z, 1.0)
    ids = ol.best(z, 6)
    loss, grad, _ = ol.distill(z, 1.0, lp[ids], ids, ol.TAIL)
    assert abs(loss) < 1e-14 and np.abs(grad).max() < 1e-15
    # Renormalised over every token it is the full divergence, 0 as well.
    allids = np.arange(40)
    loss, grad, _ = ol.distill(z, 1.0, z + 5.0, allids, ol.RENORM)
    assert abs(loss) < 1e-14 and np.abs(grad).max() < 1e-15
    assert ol.distill(z[::-1].copy(), 1.0, lp[ids], ids, ol.TAIL)[0] > 0


def test_distill_tail_by_hand():
    # Teacher 0.5 / 0.25 listed, 0.25 left; student uniform over 4 tokens.
    z = np.zeros(4)
    loss, grad, tail = ol.distill(z, 1.0, np.log([0.5, 0.25]), [0, 3], ol.TAIL)
    want = 0.5 * math.log(2.0) + 0.25 * math.log(1.0) + 0.25 * math.log(0.5)
    assert abs(loss - want) < 1e-15 and abs(tail - math.log(0.5)) < 1e-15
    np.testing.assert_allclose(grad, [-0.25, 0.125, 0.125, 0.0], atol=1e-16)


def test_distill_edges():
    z = np.array([0.0, 1.0, 2.0])
    for mode in (ol.RENORM, ol.TAIL):
        loss, grad, _ = ol.distill(z, 1.0, [0.0, 0.0], [-1, -1], mode)
        assert abs(loss) < 1e-15 and np.abs(grad).max() < 1e-15
        assert np.isnan(ol.distill(z, 1.0, [0.0], [3], mode)[0])
        loss, grad, _ = ol.distill(np.full(3, -np.inf), 1.0, [-0.7], [1], mode)
        assert loss == np.inf and (grad == 0).all()
    # Every token listed: no tail, whatever the sum's rounding leaves.
    lp = np.log([0.3, 0.3, 0.3])
    assert np.isfinite(ol.distill(z, 1.0, lp, [0, 1, 2], ol.TAIL)[0])
    # The student rules out what the teacher wants.
    loss, grad, _ = ol.distill(np.array([-np.inf, 0.0]), 1.0, [-0.5, -1.0], [0, 1], ol.RENORM)
    assert loss == np.inf and np.isfinite(grad).all() and grad[0] < 0


def test_distill_rounding_of_a_list_that_holds_all_of_the_mass():
    """Rows constrained to fewer tokens than are listed: FP32 scores leave 1 -
    sum q of either sign, which no loss may turn into an infinity."""
    rng = np.random.default_rng(4)
    for mask in (-np.inf, -3.4028234663852886e38, -65504.0):
        for _ in range(50):
            allowed = rng.choice(300, 12, replace=False)
            t, z = np.full(300, mask), np.full(300, mask)
            t[allowed] = rng.normal(size=12) * 3
            z[allowed] = rng.normal(size=12) * 3
            ids = ol.best(t, 20)
            scores = ol.log_softmax(t, 1.0)[ids].astype(np.float32).astype(np.float64)
            loss, grad, _ = ol.distill(z, 1.0, scores, ids, ol.TAIL)
            lt, lz = ol.log_softmax(t[allowed], 1.0), ol.log_softmax(z[allowed], 1.0)
            # Each score is off by at most 2^-24 of itself.
            assert abs(loss - (np.exp(lt) * (lt - lz)).sum()) < 1e-5
            np.testing.assert_allclose(grad[allowed], np.exp(lz) - np.exp(lt), atol=1e-6)
            assert np.abs(np.delete(grad, allowed)).max() == 0
    # What rounding cannot explain stays: the student rules out a real tail.
    assert ol.distill(np.array([0.0, -np.inf]), 1.0, [-1e-3], [0], ol.TAIL)[0] == np.inf


def test_distill_token_listed_twice_by_hand():
    """Two terms of the loss, one token of p_t and of the gradient: teacher 0.25
    and 0.25 on one token of a uniform student's four, 0.5 left."""
    loss, grad, tail = ol.distill(np.zeros(4), 1.0, np.log([0.25, 0.25]), [2, 2], ol.TAIL)
    want = 2 * 0.25 * math.log(0.25 / 0.25) + 0.5 * math.log(0.5 / 0.75)
    assert abs(loss - want) < 1e-15 and abs(tail - math.log(0.75)) < 1e-15
    np.testing.assert_allclose(grad, [0.25 / 3, 0.25 / 3, -0.25, 0.25 / 3], atol=1e-16)
