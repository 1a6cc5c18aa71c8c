"""Fine-tuning steps with the inputs kept at 8 bits, as they are used together: a
projection of two sections and an adapted head over a padded vocabulary, the
frozen model's best words as a teacher, a loss on log-probabilities and entropy
from the head's scores, and both layers' backwards from their checkpoints.
Gradients are the formulas' (float64, on what the checkpoints stand for) and
follow differences of the loss; a whole step is replayed from a graph."""

import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import DEV, Layer, bits_host, rel
from oracle import checkpoint_oracle as K
from oracle import scores_oracle as S

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.detach().double().cpu().numpy()


def _head(lib, H, V, n, coef):
    """Teacher (the frozen head's n best words), the head's scores, the coefficients of the loss
    sum_t (-sum_j q_j logp_j - coef H) / M, and the gradient in the logits of the padded head."""
    M, d = H.M, H.d
    _, _, ids, top = lib.token_scores(lib.forward(H.X, H.w)[:, :V], top=n)
    q = torch.softmax(top, dim=1)
    logits, T, ck = lib.forward_checkpoint(H.X, H.w, H.A, H.B, H.alpha)
    logp, entropy, _, _, stats = lib.token_scores(logits[:, :V], ids, save_stats=True)
    dlogp, dentropy = -q / M, torch.full((M,), -coef / M, device=DEV)
    dY = torch.full((M, d), 5.0, dtype=torch.bfloat16, device=DEV)
    lib.token_scores_backward(dlogp, dentropy, logits[:, :V], ids, stats, out=dY[:, :V])
    return ids, q, logits, T, ck, logp, entropy, dlogp, dentropy, dY


def test_distillation_step_of_an_adapted_head(lib):
    d, k, r, M, V, n, coef = 1024, 512, 16, 96, 1000, 8, 0.05
    print("case: distillation step", d, k, r, M, V, flush=True)
    H = Layer(lib, d, k, r, M, cfg=91)
    ids, q, logits, T, ck, logp, entropy, dlogp, dentropy, dY = _head(lib, H, V, n, coef)
    dX, dA, dB = lib.backward_checkpoint(dY, ck, H.w, H.A, H.B, H.alpha, T)

    # the scores and their gradient, from the head's own bf16 logits
    z, y = _f64(logits[:, :V]), ids.cpu().numpy()
    lp, ent, _, _ = S.scores(z, y, 1)
    assert np.allclose(_f64(logp), lp, rtol=1e-5, atol=1e-6) and np.allclose(_f64(entropy), ent, rtol=1e-5, atol=1e-6)
    want = S.scores_grad(z, y, _f64(dlogp), _f64(dentropy))
    # rounded to bf16 (2^-8 of the value), on fp32 exponents (2^-16 of a word's own share)
    share = np.abs(S.scores_grad(z, y, np.abs(_f64(dlogp)), None)) + np.abs(want)
    assert np.all(np.abs(_f64(dY[:, :V]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -14 * share + 1e-9)
    assert torch.all(dY[:, V:] == 0)

    # the layer's gradients: dX and dB of the input itself, dA of what the checkpoint stands for
    dXr, _, dBr = O.backward(bits_host(dY), H.inp["X"], H.Wt, H.inp["A"], H.inp["B"], H.alpha)
    kept = K.restored(H.inp["X"])
    _, dAr, _ = O.backward(bits_host(dY), kept, H.Wt, H.inp["A"], H.inp["B"], H.alpha)
    assert rel(bits_host(dX), dXr) <= 1e-2 and rel(bits_host(dA), dAr) <= 2e-2 and rel(bits_host(dB), dBr) <= 2e-2
    # the 8 bits against the input itself: half a code's step, uniformly spread, is 0.29 of it; a block's largest of 64
    # normal values is below 5, so 0.29 * 5 / 127 = 1.2 % of the input and, the errors being independent, of dA
    _, dAx, _ = O.backward(bits_host(dY), H.inp["X"], H.Wt, H.inp["A"], H.inp["B"], H.alpha)
    assert np.linalg.norm(dAr - dAx) <= 0.02 * np.linalg.norm(dAx)

    # the loss in float64 along dB, which the 8 bits do not touch, against its differences
    A, B = (O.bf16_bits_to_f64(H.inp[n_]) for n_ in "AB")
    X, s = O.bf16_bits_to_f64(H.inp["X"]), H.alpha / r
    base = X @ (O.bf16_bits_to_f64(H.Wt) if H.Wt.dtype == np.uint16 else np.asarray(H.Wt, np.float64)).T
    qh = _f64(q)

    def total(b):
        lp, ent, _, _ = S.scores((base + s * (X @ A.T) @ b.T)[:, :V], y, 1)
        return -((qh * lp).sum() + coef * ent.sum()) / M

    g = _f64(dB)
    way = g / np.linalg.norm(g)
    slope = (total(B + 1e-4 * way) - total(B - 1e-4 * way)) / 2e-4
    assert abs(slope - (g * way).sum()) <= 2e-2 * abs(slope)


def test_two_layers_captured(lib):
    # sections, then the head on their output; whole steps of both, replayed between eager ones
    k, ds, r, M, V, n = 256, 256, 16, 48, 500, 5
    print("case: captured steps of two layers", k, ds, r, M, V, flush=True)
    g = torch.Generator().manual_seed(7)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(DEV)

    w1 = lib.quantize_sections([normal(ds, k, std=0.06), normal(ds, k, std=0.06)])
    w2 = lib.quantize(normal(512, 2 * ds, std=0.06))
    X = normal(M, k).bfloat16()
    P0 = [normal(2 * r, k, std=k ** -0.5).bfloat16(), normal(2 * ds, r, std=0.05).bfloat16(),
          normal(r, 2 * ds, std=(2 * ds) ** -0.5).bfloat16(), normal(512, r, std=0.05).bfloat16()]
    H0 = lib.forward_sections(X, w1)
    _, _, ids, top = lib.token_scores(lib.forward(H0, w2)[:, :V], top=n)
    dlogp = -torch.softmax(top, dim=1) / M
    dentropy = torch.full((M,), -0.01 / M, device=DEV)

    def state():
        return [[p.clone(), p.float(), torch.zeros_like(p, dtype=torch.float32), torch.zeros_like(p, dtype=torch.float32)]
                for p in P0]

    def step(s, number):
        A1, B1, A2, B2 = (p[0] for p in s)
        Y1, T1, ck1 = lib.forward_checkpoint(X, w1, A1, B1, 16.0)
        logits, T2, ck2 = lib.forward_checkpoint(Y1, w2, A2, B2, 16.0)
        z = logits[:, :V]
        _, _, _, _, stats = lib.token_scores(z, ids, save_stats=True)
        lib.token_scores_backward(dlogp, dentropy, z, ids, stats, out=z)  # in the logits' place, with the padding
        dY1, dA2, dB2 = lib.backward_checkpoint(logits, ck2, w2, A2, B2, 16.0, T2)
        _, dA1, dB1 = lib.backward_checkpoint(dY1, ck1, w1, A1, B1, 16.0, T1, need_dx=False)
        for p, grad in zip(s, (dA1, dB1, dA2, dB2)):
            lib.adam_step(p[0], p[1], grad, p[2], p[3], lr=1e-3, step=number)
        return dA1, dB1, dA2, dB2

    def loss(s):
        Y1 = lib.forward_sections(X, w1, s[0][0], s[1][0], 16.0)
        logp, ent, _, _ = lib.token_scores(lib.forward(Y1, w2, s[2][0], s[3][0], 16.0)[:, :V], ids)
        return float((dlogp * logp).sum() + (dentropy * ent).sum())

    eager, replayed, warm = state(), state(), state()
    # the first step's gradients against the same layers on the restored inputs
    grads = step(warm, 1)
    fresh = state()
    A1, B1, A2, B2 = (p[0] for p in fresh)
    Y1, T1 = lib.forward_sections(X, w1, A1, B1, 16.0, save_t=True)
    logits, T2 = lib.forward(Y1, w2, A2, B2, 16.0, save_t=True)
    _, _, _, _, stats = lib.token_scores(logits[:, :V], ids, save_stats=True)
    dY = torch.zeros_like(logits)
    lib.token_scores_backward(dlogp, dentropy, logits[:, :V], ids, stats, out=dY[:, :V])
    r2 = lib.checkpoint_load(lib.checkpoint_save(Y1))
    dY1, dA2, dB2 = lib.backward(dY, r2, w2, A2, B2, 16.0, T_saved=T2)
    r1 = lib.checkpoint_load(lib.checkpoint_save(X))
    _, dA1, dB1 = lib.backward_sections(dY1, r1, w1, A1, B1, 16.0, T_saved=T1, need_dx=False)
    assert all(torch.equal(a, b) for a, b in zip(grads, (dA1, dB1, dA2, dB2)))
    assert all(torch.isfinite(a.float()).all() for a in grads) and all(a.any() for a in grads)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(replayed, 1)
    for i in range(4):
        got = step(eager, 1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, got)), i
        assert all(torch.equal(a, b) for p, q in zip(replayed, eager) for a, b in zip(p, q)), i
    assert np.isfinite(loss(eager))
