"""The policy loss where a factor of 0 meets what fp32 cannot hold."""

import numpy as np
import pytest
import torch

from gpu_util import DEV
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _rows(dtype, V, at):
    """Three tokens of equal logits but the label's, `at` above the others."""
    z = torch.zeros(3, V, device=DEV).to(dtype)
    y = torch.tensor([0, V // 2, V - 1], dtype=torch.int32, device=DEV)
    z[torch.arange(3, device=DEV), y.long()] = at
    return z, y


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [50, 5000, 140000])
def test_kl_that_only_is_watched_takes_no_part(lib, V, dtype):
    # kl_coef = 0: whatever kl is, loss and gradient are those without a reference
    print("case: kl watched", V, dtype, flush=True)
    adv = torch.tensor([1.0, -2.0, 0.5], device=DEV)
    for at in (-100.0, -float("inf")):
        z, y = _rows(dtype, V, at)
        lp = lib.token_logprobs(z, y)
        old = torch.where(torch.isfinite(lp), lp, -3.0) - 0.1
        ref = torch.full((3,), 0.0, device=DEV)
        want = lib.policy_loss(z, y, adv, old_logp=old)
        loss, kl, logp, dz = lib.policy_loss(z, y, adv, old_logp=old, ref_logp=ref, kl_coef=0.0)
        assert torch.isfinite(loss).all() and torch.isfinite(dz).all()
        assert torch.equal(loss, want[0]) and torch.equal(logp, want[2]) and torch.equal(dz, want[3])
        assert (kl == float("inf")).all()          # exp(100) is past fp32
    # an ordinary kl is written all the same
    z, y = _rows(dtype, V, 1.0)
    lp = lib.token_logprobs(z, y)
    kl = lib.policy_loss(z, y, adv, ref_logp=lp + 0.25, kl_coef=0.0)[1].double().cpu().numpy()
    d = (lp + 0.25).double().cpu().numpy() - S.label_logprobs(z.double().cpu().numpy(), y.cpu().numpy())
    # d is off by lp's error, at most 64 half steps of ln V for these rows; the series by 12 half steps of its own
    assert np.all(np.abs(kl - (np.exp(d) - d - 1)) <= (64 * np.log(V) * U) * np.expm1(0.26) + 12 * U * kl)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [50, 5000, 140000])
def test_an_advantage_of_zero_adds_nothing(lib, V, dtype):
    # however far the ratio has gone: exp(100) is past fp32
    print("case: advantage 0", V, dtype, flush=True)
    z, y = _rows(dtype, V, 1.0)
    adv = torch.tensor([0.0, -0.0, 0.5], device=DEV)
    lp = lib.token_logprobs(z, y)
    old = lp - torch.tensor([100.0, 100.0, 0.1], device=DEV)
    loss, kl, logp, dz = lib.policy_loss(z, y, adv, old_logp=old)
    assert torch.all(loss[:2] == 0) and torch.all(dz[:2] == 0) and torch.isfinite(dz).all() and torch.all(kl == 0)
    # what the KL term adds stays
    ref = lp + 0.25
    both = lib.policy_loss(z, y, adv, old_logp=old, ref_logp=ref, kl_coef=0.5)
    alone = lib.policy_loss(z, y, adv, old_logp=lp, ref_logp=ref, kl_coef=0.5)
    for a, b in zip(both, alone):
        assert torch.equal(a[:2], b[:2]) and torch.isfinite(a).all()
    # a row without a distribution is NaN all the same
    z[0] = float("nan")
    loss, _, logp, _ = lib.policy_loss(z, y, adv, old_logp=old)
    assert torch.isnan(loss[0]) and torch.isnan(logp[0]) and loss[1] == 0
