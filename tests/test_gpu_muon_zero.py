"""The orthogonalised update of a zero gradient with a small eps."""

import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(2, 8, 256), (2, 16, 1024), (2, 1024, 16), (2, 64, 512), (2, 512, 40)])
def test_no_update_of_a_zero_gradient(lib, shape):
    # X = 0 / (0 + eps) = 0, however large what multiplies it is (3.4445^16 / 1e-30 is past fp32): weights decay alone
    print("case: muon zero", shape, flush=True)
    g = torch.Generator(device=DEV).manual_seed(1)
    W = torch.randn(*shape, device=DEV, generator=g)
    G, m = torch.zeros(*shape, device=DEV, dtype=torch.bfloat16), torch.zeros(*shape, device=DEV)
    G[1] = 1.0                                       # the other matrix of the stack has one
    P, W0 = W.bfloat16(), W.clone()
    lib.muon_step(P, W, G, m, lr=0.0078125, weight_decay=0.5, ns_steps=16, eps=1e-30)
    assert torch.equal(W[0], W0[0] * (1 - 0.0078125 * 0.5)) and torch.equal(P[0], W[0].bfloat16())
    assert torch.isfinite(W[1]).all() and not torch.equal(W[1], W0[1] * (1 - 0.0078125 * 0.5))


@pytest.mark.parametrize("shape", [(1, 8, 256), (1, 1024, 16), (1, 64, 512)])
def test_a_tiny_gradient_has_a_whole_update(lib, shape):
    # |u| far above eps, both at the lower end of what is taken: the update is the one of the gradient times 2^80
    print("case: muon tiny", shape, flush=True)
    g = torch.Generator(device=DEV).manual_seed(2)
    W = torch.randn(*shape, device=DEV, generator=g)
    G = torch.randn(*shape, device=DEV, generator=g).bfloat16() * 2.0 ** -85
    got = []
    for scale in (1.0, 2.0 ** 80):
        P, w, m = W.bfloat16(), W.clone(), torch.zeros(*shape, device=DEV)
        lib.muon_step(P, w, G * scale, m, lr=0.01, eps=1e-30)
        got.append(w)
    # 1.95 |G| of 2048 elements or more is about 2^-78.5, so eps = 2^-99.7 takes 2^-21.2 of X_0, and five steps, whose
    # slopes are at most 3.4445, make at most 485 |X_0| = 485 times that of it: 2^-12.2, where |X_5| is above 1
    change = (got[1] - W).norm()
    assert (got[0] - got[1]).norm() <= 2.0 ** -12 * change and change > 0.001
