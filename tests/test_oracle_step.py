"""Pins of the float64 reference of the fine-tuning step: gradients against
central differences, closed forms, and the orthogonalised update's spectrum."""

import numpy as np
import pytest

from oracle import step_oracle as S


def _rng(*key):
    return np.random.Generator(np.random.PCG64(list(key)))


def _central(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_label_logprobs_are_normalised_and_uniform_rows_give_minus_ln_v():
    z = _rng(1).normal(size=(3, 11)) * 4
    every = np.stack([S.label_logprobs(z, [y] * 3) for y in range(11)], 1)
    assert np.allclose(np.exp(every).sum(1), 1, rtol=0, atol=1e-14)
    assert np.allclose(S.label_logprobs(np.full((2, 7), -3.0e38), [0, 6], 2.0), -np.log(7))
    assert np.array_equal(S.label_logprobs(z, [-100, 11, -1]), np.zeros(3))


@pytest.mark.parametrize("tau", [1.0, 0.5])
def test_label_logprobs_gradient(tau):
    r = _rng(2)
    z, g, y = r.normal(size=(4, 6)) * 2, r.normal(size=4), [0, 5, -100, 2]
    num = _central(lambda v: float((S.label_logprobs(v, y, tau) * g).sum()), z)
    assert np.allclose(S.label_logprobs_grad(z, y, g, tau), num, atol=1e-8)


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
@pytest.mark.parametrize("average", [False, True])
def test_preference_gradient(kind, average):
    r = _rng(3)
    T, cu = 14, [0, 3, 3, 8, 14]     # an empty sequence
    y = [1] * T
    y[4] = -100
    logp, ref, w = -r.random(T), -r.random(T), np.array([0.5, 2.0])
    kw = dict(ref=ref, kind=kind, average=average, smoothing=0.1 if kind == "sigmoid" else 0.0, margin=0.2, weight=w)
    f = lambda v: float((S.preference(v, y, 5, cu, 0.7, **kw)[0] * w).sum())  # noqa: E731
    assert np.allclose(S.preference(logp, y, 5, cu, 0.7, **kw)[2], _central(f, logp), atol=1e-7)


def test_preference_of_a_policy_at_its_reference_is_ln_2():
    logp = -_rng(4).random(9)
    loss, reward, d = S.preference(logp, [0] * 9, 1, [0, 4, 9], 0.1, ref=logp)
    assert np.allclose(loss, np.log(2)) and np.array_equal(reward, np.zeros(2))
    assert np.allclose(d, [-0.05] * 4 + [0.05] * 5)


def test_policy_gradient_and_clip():
    r = _rng(5)
    T = 12
    logp, adv = -r.random(T) * 3, r.normal(size=T)
    old, ref, w = logp - 0.3 * r.normal(size=T), logp + 0.2 * r.normal(size=T), r.random(T)
    y = [0] * T
    y[3] = -100
    f = lambda v: float((S.policy(v, y, 4, adv, old, ref, w, kl_coef=0.3)[0] * w).sum())  # noqa: E731
    assert np.allclose(S.policy(logp, y, 4, adv, old, ref, w, kl_coef=0.3)[2], _central(f, logp), atol=1e-7)
    # a ratio past the clip on its advantage's side has no gradient; on the other side it keeps it
    up = S.policy(np.array([0.0, 0.0]), [0, 0], 1, np.array([1.0, -1.0]), old=np.array([-1.0, -1.0]))[2]
    assert up[0] == 0.0 and np.isclose(up[1], np.e)


@pytest.mark.parametrize("shape", [(8, 40), (40, 8), (16, 16)])
def test_orthogonalised_is_a_function_of_the_singular_values(shape):
    u = _rng(6).normal(size=shape)
    x = S.orthogonalised(u, (S.USUAL,) * 5)
    U, s, Vt = np.linalg.svd(u, full_matrices=False)
    f = s / (np.sqrt((s * s).sum()) + 1e-7)
    for a, b, c in (S.USUAL,) * 5:
        f = a * f + b * f ** 3 + c * f ** 5
    assert np.allclose(x, (U * f) @ Vt, atol=1e-12)
    if shape != (16, 16):  # well away from singular: every value near one
        assert np.all((0.6 < f) & (f < 1.3))
    # the cubic steps (1.5, -0.5, 0) converge to the orthogonal factor
    x = S.orthogonalised(u, ((1.5, -0.5, 0.0),) * 60)
    assert np.allclose(x, U @ Vt, atol=1e-9)


def test_muon_momentum_and_decay():
    r = _rng(7)
    W, g = r.normal(size=(4, 9)), r.normal(size=(4, 9))
    W1, m1 = S.muon(W, g, np.zeros((4, 9)), 0.1, momentum=0.9, nesterov=False, wd=0.5, scale=2.0)
    assert np.array_equal(m1, g)
    assert np.allclose(W1, 0.95 * W - 0.2 * S.orthogonalised(g, (S.USUAL,) * 5))
    # a zero gradient leaves only the decay
    W2, _ = S.muon(W, 0 * g, 0 * g, 0.1, wd=0.5)
    assert np.allclose(W2, 0.95 * W)
