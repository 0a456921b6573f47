"""The fp64 definitions of the losses, the clipping and the bounded update, pinned by
central differences, closed forms and invariants."""
import math

import numpy as np
import pytest

from oracle import loss_oracle as lo


def _rows(seed, rows, vocab):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((rows, vocab)) * 2
    token = rng.integers(0, vocab, rows)
    return rng, z, token


def _differences(f, z, h=1e-5):
    """Central differences of f in every element: f(z +- h), error O(h^2) f''' and rounding eps f / h."""
    g = np.zeros_like(z)
    for i in np.ndindex(z.shape):
        keep = z[i]
        z[i] = keep + h
        up = f()
        z[i] = keep - h
        down = f()
        z[i] = keep
        g[i] = (up - down) / (2 * h)
    return g


def test_row_logp_is_a_distribution():
    _, z, token = _rows(0, 5, 9)
    for t in range(5):
        l, p = lo.row_logp(z[t], token[t])
        assert abs(p.sum() - 1) < 1e-14 and abs(math.exp(l) - p[token[t]]) < 1e-14
    l, p = lo.row_logp(np.array([0.0, -np.inf, 0.0]), 0)
    assert l == pytest.approx(-math.log(2)) and p[1] == 0


@pytest.mark.parametrize("begin,by_sequence", [(None, False), ([0, 3, 3, 6], True), ([1, 4, 5], False)])
@pytest.mark.parametrize("kl", [0.0, 0.3])
def test_policy_gradient_is_the_differences(begin, by_sequence, kl):
    rng, z, token = _rows(1, 7, 5)
    old = np.array([lo.row_logp(z[t], token[t])[0] for t in range(7)]) + 0.3 * rng.standard_normal(7)
    ref = old + 0.2 * rng.standard_normal(7)
    adv = rng.standard_normal(7)
    mask = np.array([1, 1, 0, 1, 1, 1, 1])
    kw = dict(ref=ref, mask=mask, begin=begin, by_sequence=by_sequence, low=0.1, high=0.15, kl_coef=kl)
    stats, logp, grad = lo.policy_loss(z, token, old, adv, scale=2.0, **kw)
    ratio = np.exp(np.array([lo.row_logp(z[t], token[t])[0] for t in range(7)]) - old)
    assert np.abs(ratio - 0.9).min() > 1e-3 and np.abs(ratio - 1.15).min() > 1e-3   # no kink within the steps
    assert (ratio > 1.15).any() or (ratio < 0.9).any()
    num = _differences(lambda: lo.policy_loss(z, token, old, adv, **kw)[0][0], z)
    got = np.where(np.isnan(grad), 0.0, grad) / 2.0
    assert np.abs(got - num).max() < 1e-8
    assert stats[0] == pytest.approx(stats[1] + kl * stats[2])


def test_policy_at_the_old_policy_is_the_policy_gradient():
    rng, z, token = _rows(2, 4, 6)
    logp = np.array([lo.row_logp(z[t], token[t])[0] for t in range(4)])
    adv = rng.standard_normal(4)
    stats, got, grad = lo.policy_loss(z, token, logp, adv, ref=logp, kl_coef=1.0)
    assert stats[0] == pytest.approx(-adv.mean()) and abs(stats[2]) < 1e-15 and stats[3] == 0
    for t in range(4):
        one = np.eye(6)[token[t]]
        assert np.allclose(grad[t], -adv[t] / 4 * (one - lo.row_logp(z[t], token[t])[1]), atol=1e-15)
    assert np.allclose(got, logp)


def test_policy_without_rows_that_count():
    _, z, token = _rows(3, 3, 4)
    stats, logp, grad = lo.policy_loss(z, token, np.zeros(3), np.ones(3), mask=np.zeros(3))
    assert not stats.any() and not logp.any() and not grad.any()
    stats, _, grad = lo.policy_loss(z, np.array([-100, 4, 1 << 40]), np.zeros(3), np.ones(3))
    assert not stats.any() and not grad.any()


@pytest.mark.parametrize("smooth", [0.0, 0.2, 1.0])
def test_preference_gradient_is_the_differences(smooth):
    rng, z, token = _rows(4, 9, 4)
    begin = [0, 2, 4, 4, 8]
    mask = np.array([1, 1, 1, 0, 1, 1, 1, 1, 1])
    ref = rng.standard_normal(4)
    kw = dict(ref=ref, mask=mask, beta=0.7, smooth=smooth)
    loss, x, sums, grad = lo.preference_loss(z, token, begin, scale=3.0, **kw)
    num = _differences(lambda: lo.preference_loss(z, token, begin, **kw)[0], z)
    assert np.abs(np.where(np.isnan(grad), 0.0, grad) / 3.0 - num).max() < 1e-8
    assert np.isnan(grad[8]).all() and sums[2] == 0 and not grad[3].any()
    assert x[0] == pytest.approx(0.7 * ((sums[0] - ref[0]) - (0 - ref[2])))


def test_preference_closed_forms():
    _, z, token = _rows(5, 4, 3)
    loss, x, _, _ = lo.preference_loss(z, token, [0, 2, 4], ref=None, beta=0.0)
    assert loss == pytest.approx(math.log(2)) and x[0] == 0
    a = lo.preference_loss(z, token, [0, 2, 4], beta=0.5, smooth=0.25)[0]
    b = lo.preference_loss(z, token, [0, 2, 4], beta=-0.5, smooth=0.75)[0]   # both labels turned round
    assert a == pytest.approx(b)
    assert lo.preference_loss(z, token, [0])[0] == 0.0


def test_clip_and_trust_closed_forms():
    assert lo.global_norm([np.array([3.0]), np.zeros(0), np.array([[0.0, 4.0]])]) == 5.0
    assert lo.clip_scale(5.0, 1.0) == 0.2 and lo.clip_scale(0.5, 1.0) == 1.0 and lo.clip_scale(0.0, 1.0) == 1.0
    assert lo.clip_scale(math.inf, 1.0) == 1.0 and lo.clip_scale(math.nan, 1.0) == 1.0
    rng = np.random.default_rng(6)
    F = rng.standard_normal((6, 6))
    F = F @ F.T + np.eye(6)
    g = rng.standard_normal(6)
    P = np.linalg.solve(F, g)
    s, q = lo.trust_step([P], [g], 10.0, 1e-2)
    assert 0.5 * s * s * (P @ F @ P) == pytest.approx(1e-2)      # the bound is reached
    assert lo.trust_step([P], [g], 1e-6, 1e-2)[0] == 1e-6        # or the rate is the bound
    d = np.abs(rng.standard_normal(6))
    assert lo.trust_step([P], [None], 1.0, 1e-2, [d], 0.5) == lo.trust_step([P], [P * (d + 0.5)], 1.0, 1e-2)
    assert lo.trust_step([np.zeros(3)], [np.ones(3)], 0.3, 1e-2) == (0.3, 0.0)


def test_a_token_without_probability():
    """A logit of -inf at the token: the loss of its pair, or its KL, is infinite, and 0 where it has no share."""
    z = np.array([[0.0, -np.inf, 0.0], [1.0, 0.0, 0.0]])
    token = np.array([1, 0])
    for smooth in (0.0, 0.25, 1.0):
        loss, margin, sums, grad = lo.preference_loss(z, token, [0, 1, 2], beta=0.5, smooth=smooth)
        assert margin[0] == -np.inf and sums[0] == -np.inf and loss == (0.0 if smooth == 1 else np.inf)
        assert np.isfinite(grad).all() and grad[0, 1] == pytest.approx((smooth - 1) * 0.5)
        loss, margin, _, grad = lo.preference_loss(z[::-1], token[::-1], [0, 1, 2], beta=0.5, smooth=smooth)
        assert margin[0] == np.inf and loss == (0.0 if smooth == 0 else np.inf)
        assert grad[1, 1] == pytest.approx(-smooth * 0.5)
    stats, logp, grad = lo.policy_loss(z, token, np.array([-1.0, -1.0]), np.array([1.0, 1.0]),
                                       ref=np.array([-1.0, -1.0]))
    assert logp[0] == -np.inf and stats[2] == np.inf and np.isfinite(stats[:2]).all() and not grad[0].any()
