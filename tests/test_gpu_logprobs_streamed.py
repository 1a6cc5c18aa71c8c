"""Gradients larger than half the last-level cache (128 MiB), which are written
past it: the same rows in calls below that size give the same bits, and some of
them are checked in float64 (the bounds are those of test_gpu_logprobs.py)."""

import numpy as np
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32

# (T, V, row stride, first element): ordinary batches, odd strides, rows in registers and in pieces
CASES = [(4096, 32000, 32000, 0, BF), (2200, 32003, 32003, 0, BF), (4100, 20011, 20011, 3, BF),
         (600, 131071, 131071, 0, BF), (520, 140000, 140001, 1, BF), (1000, 70001, 70008, 5, BF),
         (1100, 32003, 32003, 0, F32), (1100, 32000, 32064, 0, F32), (600, 70001, 70001, 1, F32),
         (530, 66001, 66001, 0, F32), (40000, 1001, 1001, 0, F32)]


@pytest.mark.parametrize("T,V,ld,offset,dtype", CASES, ids=lambda x: str(x).split(".")[-1])
def test_streamed_gradients(lib, T, V, ld, offset, dtype):
    print("case: streamed", T, V, ld, offset, dtype, flush=True)
    tau, n = 0.8, 300
    assert T * ld * dtype.itemsize > 128 << 20 and n * ld * dtype.itemsize < 128 << 20
    g = torch.Generator(device=DEV).manual_seed(V)
    buf = torch.empty(T * ld + offset + 64, dtype=dtype, device=DEV)
    for part in buf.split(1 << 26):
        part.copy_(2 * torch.randn(len(part), device=DEV, generator=g))
    z = buf[offset:offset + T * ld].view(T, ld)[:, :V]
    y = torch.randint(0, V, (T,), device=DEV, generator=g, dtype=torch.int32)
    y[::9], y[1], y[2] = -1, 0, V - 1
    adv = torch.randn(T, device=DEV, generator=g)
    adv[5] = 0
    logp, stats = lib.token_logprobs(z, y, tau, save_stats=True)
    own = torch.full_like(buf, 7.0)
    out = own[offset:offset + T * ld].view(T, ld)
    ends = (own[:offset], own[offset + T * ld:])

    def grad(s, dst):
        return lib.token_logprobs_backward(adv[s], z[s], y[s], stats[s], tau, out=dst)

    def policy(s, dst):
        return lib.policy_loss(z[s], y[s], -adv[s], inv_temperature=tau, out=dst)[3]

    whole = slice(0, T)
    first = buf.clone()
    for f in (grad, policy):
        out.fill_(7.0)
        f(whole, out[:, :V])
        assert torch.all(out[:, V:] == 0) and all(torch.all(e == 7) for e in ends)
        assert not out[y < 0].any() and not out[5].any()
        for s in (slice(0, n), slice(T - n, T)):
            assert torch.equal(f(s, None), out[s, :V])
        for i in (1, 2, 4, T // 2 + 1, T - 1):
            t = tau * (z[i].double() - z[i].double().max())
            p, label = t.softmax(0), int(y[i])
            want = torch.zeros(V, dtype=torch.float64, device=DEV)
            bound = torch.full_like(want, 1e-37)
            if label >= 0:
                want = -p
                want[label] += 1
                a = float(adv[i]) * float(np.float32(tau))
                want *= a
                b = U * (12 * (np.log(V) + 1) + V / 256 + 32 + 3 * float(t[label].abs()) + float(logp[i].abs()))
                bound += abs(a) * (3 * U + p * b) + (4 * U + torch.finfo(dtype).eps / 2) * want.abs()
            assert ((out[i, :V].double() - want).abs() <= bound).all()
        f(whole, z)                                     # in place
        assert torch.equal(z, out[:, :V])
        buf.copy_(first)
