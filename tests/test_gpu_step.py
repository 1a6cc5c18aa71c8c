"""One preference step and one policy step of an adapted NF4 head as they are
used together: reference and policy logits from one frozen weight, label
log-probabilities, loss, its gradient as the dY of the head's backward, and
the optimiser step on both adapter factors.  The gradients are the formulas'
(float64, from the head's own bf16 logits) and follow differences of the loss
in the adapter."""

import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import DEV, Layer, bits_host, rel
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.detach().double().cpu().numpy()


def test_preference_step_of_an_adapted_head(lib):
    # a vocabulary of 1000 in a head padded to 1024 rows
    d, k, r, M, V, beta = 1024, 512, 16, 96, 1000, 0.5
    print("case: preference step", d, k, r, M, V, flush=True)
    H = Layer(lib, d, k, r, M, cfg=81)
    y = torch.randint(0, V, (M,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    y[:9] = -100
    y = y.to(DEV)
    cu_h = [0, 30, 50, 80, 96]
    cu = torch.tensor(cu_h, dtype=torch.int32, device=DEV)

    ref_logp = lib.token_logprobs(lib.forward(H.X, H.w)[:, :V], y)          # the adapter left off
    logits, T = lib.forward(H.X, H.w, H.A, H.B, H.alpha, save_t=True)
    logp, stats = lib.token_logprobs(logits[:, :V], y, save_stats=True)
    loss, reward, dlogp = lib.preference_loss(logp, y, V, cu, beta, ref_logp=ref_logp,
                                              weight=torch.full((2,), 0.5, device=DEV))
    dY = torch.full((M, d), 5.0, dtype=torch.bfloat16, device=DEV)
    lib.token_logprobs_backward(dlogp, logits[:, :V], y, stats, out=dY[:, :V])
    dX, dA, dB = lib.backward(dY, H.X, H.w, H.A, H.B, H.alpha, T_saved=T)

    yh, z = y.cpu().numpy(), _f64(logits[:, :V])
    lp64 = S.label_logprobs(z, yh)
    want = S.preference(lp64, yh, V, cu_h, beta, ref=_f64(ref_logp), weight=[0.5, 0.5])
    assert np.allclose(_f64(loss), want[0], rtol=1e-4) and np.allclose(_f64(dlogp), want[2], rtol=1e-4, atol=1e-7)
    dY64 = np.zeros((M, d))
    dY64[:, :V] = S.label_logprobs_grad(z, yh, want[2])
    assert np.all(np.abs(_f64(dY) - dY64) <= 2.0 ** -8 * np.abs(dY64) * 1.01 + 1e-6)
    assert torch.all(dY[:, V:] == 0) and torch.all(dY[:9] == 0)
    dXr, dAr, dBr = O.backward(bits_host(dY), H.inp["X"], H.Wt, H.inp["A"], H.inp["B"], H.alpha)
    assert rel(bits_host(dX), dXr) <= 1e-2 and rel(bits_host(dA), dAr) <= 2e-2 and rel(bits_host(dB), dBr) <= 2e-2

    # the loss in float64 along the gradients' own direction, against its differences
    A, B = (O.bf16_bits_to_f64(H.inp[n]) for n in "AB")
    X, s = O.bf16_bits_to_f64(H.inp["X"]), H.alpha / r
    base = X @ np.asarray(O.bf16_bits_to_f64(H.Wt) if H.Wt.dtype == np.uint16 else H.Wt, np.float64).T

    def total(a, b):
        lp = S.label_logprobs((base + s * (X @ a.T) @ b.T)[:, :V], yh)
        return 0.5 * S.preference(lp, yh, V, cu_h, beta, ref=_f64(ref_logp))[0].sum()

    gA, gB = _f64(dA), _f64(dB)
    for dirA, dirB in ((gA / np.linalg.norm(gA), 0 * gB), (0 * gA, gB / np.linalg.norm(gB))):
        h = 1e-4
        slope = (total(A + h * dirA, B + h * dirB) - total(A - h * dirA, B - h * dirB)) / (2 * h)
        assert abs(slope - ((gA * dirA).sum() + (gB * dirB).sum())) <= 2e-2 * abs(slope)

    # the optimiser step on both factors: the copies that the next forward reads
    for P, G in ((H.A, dA), (H.B, dB)):
        W, m = P.float(), torch.zeros_like(P, dtype=torch.float32)
        W0 = _f64(W)
        lib.muon_step(P, W, G, m, lr=0.01)
        w64, _ = S.muon(W0, _f64(G), np.zeros(W0.shape), float(np.float32(0.01)))
        assert np.linalg.norm(_f64(W) - w64) <= 1e-4 * np.linalg.norm(w64 - W0) + 1e-6 * np.linalg.norm(W0)
        assert torch.equal(P, W.bfloat16())
    after = lib.forward(H.X, H.w, H.A, H.B, H.alpha)
    assert torch.isfinite(after.float()).all() and not torch.equal(after, logits)


def test_policy_step_of_an_adapted_head_in_place(lib):
    # the logits' own memory takes the gradient; sections give the stacked factors of two heads' worth of rows
    d, k, r, M = 512, 256, 16, 40
    print("case: policy step", d, k, r, M, flush=True)
    H = Layer(lib, d, k, r, M, cfg=82)
    y = torch.randint(0, d, (M,), generator=torch.Generator().manual_seed(2), dtype=torch.int32).to(DEV)
    logits = lib.forward(H.X, H.w, H.A, H.B, H.alpha)
    ref = lib.token_logprobs(lib.forward(H.X, H.w), y)
    old = lib.token_logprobs(logits, y)
    adv = torch.linspace(-1, 1, M).to(DEV)
    w = torch.full((M,), 1.0 / M, device=DEV)
    z, yh = _f64(logits), y.cpu().numpy()
    loss, kl, logp, dY = lib.policy_loss(logits, y, adv, old, ref, w, kl_coef=0.1, out=logits)
    assert dY is logits and torch.equal(logp, old)
    lp = S.label_logprobs(z, yh)
    wl, wk, wg = S.policy(lp, yh, d, _f64(adv), lp, _f64(ref), np.full(M, 1 / M), kl_coef=0.1)
    assert np.allclose(_f64(loss), wl, rtol=1e-4, atol=1e-5) and np.allclose(_f64(kl), wk, rtol=1e-3, atol=1e-5)
    want = S.label_logprobs_grad(z, yh, wg)
    assert np.all(np.abs(_f64(dY) - want) <= 2.0 ** -8 * 1.01 * np.abs(want) + 1e-6)
    dX, dA, dB = lib.backward(dY, H.X, H.w, H.A, H.B, H.alpha)
    dXr, dAr, dBr = O.backward(bits_host(dY), H.inp["X"], H.Wt, H.inp["A"], H.inp["B"], H.alpha)
    assert rel(bits_host(dX), dXr) <= 1e-2 and rel(bits_host(dA), dAr) <= 2e-2 and rel(bits_host(dB), dBr) <= 2e-2


def test_preference_steps_captured(lib):
    # whole steps replayed from a graph, between eager ones on a second copy of the adapter: the same bits each time
    d, k, r, M, V = 512, 256, 16, 64, 500
    print("case: captured preference steps", d, k, r, M, V, flush=True)
    H = Layer(lib, d, k, r, M, cfg=83)
    y = torch.randint(0, V, (M,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(DEV)
    cu = torch.tensor([0, 20, 31, 50, 64], dtype=torch.int32, device=DEV)

    def state():
        f = [H.A.clone(), H.B.clone()]
        return f + [p.float() for p in f] + [torch.zeros_like(p, dtype=torch.float32) for p in f]

    def step(s):
        A, B, WA, WB, mA, mB = s
        ref = lib.token_logprobs(lib.forward(H.X, H.w)[:, :V], y)
        logits, T = lib.forward(H.X, H.w, A, B, H.alpha, save_t=True)
        logp, stats = lib.token_logprobs(logits[:, :V], y, save_stats=True)
        _, _, dlogp = lib.preference_loss(logp, y, V, cu, 0.5, ref_logp=ref)
        lib.token_logprobs_backward(dlogp, logits[:, :V], y, stats, out=logits[:, :V])
        _, dA, dB = lib.backward(logits, H.X, H.w, A, B, H.alpha, T_saved=T)
        lib.muon_step(A, WA, dA, mA, lr=0.01)
        lib.muon_step(B, WB, dB, mB, lr=0.01)

    eager, replayed, warm = state(), state(), state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(warm)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(replayed)
    for n in range(4):
        step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, eager)), n
    assert not torch.equal(eager[0], H.A) and torch.isfinite(eager[2]).all()
