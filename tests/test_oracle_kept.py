"""Pins of the plain references of the 8-bit checkpoint and of the scores:
hand-made blocks, error bounds, differences, and torch's own functions."""

import numpy as np
import pytest
import torch

import oracle as O
import workloads as WL
from oracle import checkpoint_oracle as K
from oracle import scores_oracle as S


def _bits(v):
    return O.bf16_rne_bits_from_f64(np.asarray(v, np.float64))


def test_blocks_by_hand():
    x = np.zeros((3, 128))
    x[0, :4] = [127, -127, 1, 0.5]       # a = 127: codes are the values, a tie goes to the even code
    x[0, 4:6] = [1.5, -2.5]
    x[1, 64:67] = [1.0, 0.5, -0.25]      # a = 1: 63.5 -> 64, -31.75 -> -32
    codes, a = K.encode(_bits(x))
    assert codes[0, :6].tolist() == [127, -127, 1, 0, 2, -2] and not codes[0, 64:].any()
    assert codes[1, 64:67].tolist() == [127, 64, -32] and not codes[2].any()
    assert a.tolist() == [[127, 0], [0, 1], [0, 0]]
    back = O.bf16_bits_to_f64(K.decode(codes, a))
    assert back[0, :3].tolist() == [127, -127, 1] and back[1, 64] == 1 and not back[2].any()


def test_checkpoint_error_and_extremes():
    b = WL.normal_bf16((64, 256), 3.0, (5, 1))
    x, y = O.bf16_bits_to_f64(b), O.bf16_bits_to_f64(K.restored(b))
    a = np.abs(x).reshape(64, 4, 64).max(axis=2).repeat(64, axis=1)
    # half a code's step, and half of a bf16's of the restored value
    assert np.all(np.abs(y - x) <= a * (0.5 / 127) * (1 + 1e-6) + np.abs(y) * 2.0 ** -8)
    at = np.abs(x) == a
    assert np.array_equal(x[at], y[at])  # a block's largest come back exactly
    for size in (2.0 ** -133, 2.0 ** -120, 2.0 ** -100, 2.0 ** 127):  # the type's smallest and largest
        codes, _ = K.encode(_bits(np.full((1, 64), size) * np.where(np.arange(64) % 2, 1, -1)))
        assert np.array_equal(np.abs(codes), np.full((1, 64), 127))
    z = np.ones((1, 128))
    z[0, 70] = np.inf
    back = O.bf16_bits_to_f64(K.restored(_bits(z)))
    assert np.all(back[0, :64] == 1) and np.isnan(back[0, 64:]).all()


def test_scores_against_torch():
    g = torch.Generator().manual_seed(3)
    z = torch.randn(7, 50, generator=g, dtype=torch.float64) * 3
    y = torch.randint(0, 50, (7, 4), generator=g)
    y[2, 1], y[3] = -100, -1
    logp, ent, ids, top = S.scores(z.numpy(), y.numpy(), 5, 0.7)
    lp = torch.log_softmax(0.7 * z, 1)
    H = torch.distributions.Categorical(logits=0.7 * z).entropy()
    for i in range(7):
        if i == 3:
            assert not logp[i].any() and ent[i] == 0 and (ids[i] == -1).all() and np.isneginf(top[i]).all()
            continue
        for j in range(4):
            want = float(lp[i, y[i, j]]) if y[i, j] >= 0 else 0.0
            assert abs(logp[i, j] - want) < 1e-12
        assert abs(ent[i] - float(H[i])) < 1e-12
        t = lp[i].topk(5)
        assert ids[i].tolist() == t.indices.tolist() and np.allclose(top[i], t.values.numpy(), atol=1e-12)


def test_scores_of_ties_masks_and_rows_without_a_distribution():
    z = np.array([[1.0, 2.0, 2.0, 0.0, 2.0], [-np.inf, 1.0, -np.inf, 1.0, -np.inf], [np.nan, 1, 1, 1, 1],
                  [np.inf, 1, 1, 1, 1], [-np.inf] * 5, [0.0, -0.0, 0.0, -0.0, -1.0]])
    _, ent, ids, top = S.scores(z, None, 3)
    assert ids[0].tolist() == [1, 2, 4] and ids[1].tolist() == [1, 3, -1] and np.isneginf(top[1, 2])
    assert abs(ent[1] - np.log(2)) < 1e-12
    assert np.isnan(ent[2:5]).all() and (ids[2:5] == -1).all() and np.isnan(top[2:5]).all()
    assert ids[5].tolist() == [0, 1, 2]


@pytest.mark.parametrize("tau", [1.0, 0.6])
def test_scores_gradient_against_differences(tau):
    r = np.random.default_rng(4)
    z = r.normal(size=(4, 12)) * 2
    z[1, 5] = -np.inf
    y = np.array([[3, 3, 7], [0, -1, 2], [12, -5, 99], [1, 2, 1]])
    g, gh = r.normal(size=(4, 3)), r.normal(size=4)
    d = S.scores_grad(z, y, g, gh, tau)
    assert not d[2].any()

    def total(z):
        logp, ent, _, _ = S.scores(z, y, 1, tau)
        return (np.where((y >= 0) & (y < 12), g, 0) * logp).sum() + (gh * ent).sum()

    for i in range(4):
        for v in range(12):
            if np.isinf(z[i, v]):
                assert d[i, v] == 0
                continue
            a, b = z.copy(), z.copy()
            a[i, v] += 1e-6
            b[i, v] -= 1e-6
            assert abs((total(a) - total(b)) / 2e-6 - d[i, v]) < 1e-7
