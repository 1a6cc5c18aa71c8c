"""Log-probabilities of rows whose mass two words hold, next to each other and
in every place of a 16-byte piece."""

import numpy as np
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("tau", [0.6934478282928467, 0.6936106085777283, 1.0])
@pytest.mark.parametrize("V,dtype", [(140000, BF), (131072, BF), (70001, F32), (32000, BF), (8191, F32), (500, BF)],
                         ids=lambda x: str(x).split(".")[-1])
def test_two_words_hold_the_mass(lib, V, dtype, tau):
    # temperatures whose scale tau log2 e rounds by most, either way.  With x the runner-up's exponent and p its
    # probability, ln S is off by p (2 |x| + 3) half steps (x's two roundings and a step of the hardware's exp2) and
    # 5 of the sum, of the factor that its parts are joined with and of the product with it; the result by half a step
    print("case: peaked", V, dtype, tau, flush=True)
    T, a = 256, 1.84375
    z = torch.full((T, V), -100.0, dtype=dtype, device=DEV)
    rows = torch.arange(T, device=DEV)
    z[rows, rows] = 3.0 - a
    z[rows, rows + 1] = 3.0
    y = rows.int() + 1
    logp = lib.token_logprobs(z, y, tau).double().cpu().numpy()
    t = float(np.float32(tau)) * a
    want = -np.log1p(np.exp(-t))
    p = np.exp(-t + want)
    assert np.abs(logp - want).max() <= U * (p * (2 * t / np.log(2) + 3) + 5 - want)


@pytest.mark.parametrize("tau", [1e-45, 1e-40, 1e-33, 1e-20, 1e20, 3.3e38])
@pytest.mark.parametrize("V,dtype", [(140000, BF), (20011, F32), (500, BF)], ids=lambda x: str(x).split(".")[-1])
def test_masked_words_at_every_scale(lib, V, dtype, tau):
    # a masked word's exponent is -inf whatever bits the scale has left: two words of equal logits are left of the row
    print("case: masked", V, dtype, tau, flush=True)
    z = torch.full((2, V), -float("inf"), dtype=dtype, device=DEV)
    z[0, 5] = z[0, V - 1] = 2.0
    z[1, 5] = z[1, V - 1] = 0.0
    y = torch.tensor([5, V - 1], dtype=torch.int32, device=DEV)
    logp, stats = lib.token_logprobs(z, y, tau, save_stats=True)
    half = float(np.float32(np.log(0.5)))
    assert logp.tolist() == [half, half]               # S = 2, rounded once
    g = torch.tensor([1.0, -1.0], device=DEV)
    dz = lib.token_logprobs_backward(g, z, y, stats, tau).double()
    t = float(torch.tensor(tau).float()) / 2
    want = torch.zeros(2, V, dtype=torch.float64, device=DEV)
    want[0, 5], want[0, V - 1], want[1, V - 1], want[1, 5] = t, -t, -t, t
    # four half steps, one to the output's type, and at the lower end of its range a step of that
    assert ((dz - want).abs() <= (4 * U + torch.finfo(dtype).eps / 2) * want.abs() + 2.0 ** -126).all()


@pytest.mark.parametrize("tau", [1.0, 0.6934478282928467])
@pytest.mark.parametrize("V,T,dtype", [(32000, 4096, BF), (140000, 500, BF), (32000, 40, BF), (32003, 1100, F32),
                                       (8191, 5, F32)], ids=lambda x: str(x).split(".")[-1])
def test_logits_around_any_level(lib, V, T, dtype, tau):
    # a level that all logits share changes no probability: both ways of forming exponents (the largest logit's is 2^9
    # at 355 or 512), gradients above and below what is written past the cache.  The bounds are those of
    # test_gpu_logprobs.py, from the logits as the type holds them
    print("case: level", V, T, dtype, tau, flush=True)
    g = torch.Generator(device=DEV).manual_seed(V)
    z, adv = torch.empty(T, V, dtype=dtype, device=DEV), torch.randn(T, device=DEV, generator=g)
    y = torch.randint(0, V, (T,), device=DEV, generator=g, dtype=torch.int32)
    for level in (-600.0, -120.0, 80.0, 340.0, 500.0, 5000.0):
        for part in z.split(256):
            part.copy_(2 * torch.randn(len(part), V, device=DEV, generator=g) + level)
        logp, stats = lib.token_logprobs(z, y, tau, save_stats=True)
        dz = lib.token_logprobs_backward(adv, z, y, stats, tau)
        pdz = lib.policy_loss(z, y, -adv, inv_temperature=tau)[3]
        t32 = float(np.float32(tau))
        for i in (0, 1, T // 2, T - 1):
            t = t32 * (z[i].double() - z[i].double().max())
            p, label = t.softmax(0), int(y[i])
            want = float(t[label] - t.logsumexp(0))
            b = U * (12 * (np.log(V) + 1) + V / 256 + 32 + 3 * abs(float(t[label])) + abs(want))
            assert abs(float(logp[i]) - want) <= b, (level, i)
            d = -p
            d[label] += 1
            a = float(adv[i]) * t32
            d *= a
            bound = abs(a) * (3 * U + p * b) + (4 * U + torch.finfo(dtype).eps / 2) * d.abs() + 1e-37
            assert ((dz[i].double() - d).abs() <= bound).all(), (level, i)
            assert ((pdz[i].double() - d).abs() <= bound).all(), (level, i)
