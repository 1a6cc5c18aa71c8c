"""GPU parity of the orthogonalised update step (qlora_muon_step) against the
float64 reference.

Tolerances.  u = 2^-24.  The momentum takes two roundings: |dm| <= 2 u (|mu m| +
|m'|).  X_0 = U / |U| is formed from a U whose entries carry at most 4 u of
their size (|dX_0|_F <= 4 u), and a step maps singular values by a x + b x^3 +
c x^5, whose slope is at most a on [0, 1.3]: n steps enlarge that error by at
most a^n (and by K = max over the matrix's own singular values of X_n / X_0 for
the part along them).  Q is rounded to fp32 and its product with X_0 sums S
terms: (S + 4) u | |Q| |X_0| |_F <= (S + 4) u sqrt(S) K.  So

  |dX_n|_F <= u (4 a^n + (S + 4) sqrt(S) K),   K <= a^n,

the weights |dW|_F <= lr scale |dX_n|_F + 3 u (|W|_F + |lr scale X_n|_F), and P
is W rounded, exactly.
"""

import numpy as np
import pytest
import torch

from gpu_util import DEV
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _case(*args):
    print("case:", *args, flush=True)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _state(n, rows, cols, seed, low_rank=False):
    r = np.random.Generator(np.random.PCG64(seed))
    shape = (n, rows, cols)
    g = r.normal(size=shape)
    if low_rank:
        k = min(2, rows, cols)
        g = 1e-3 * g + r.normal(size=(n, rows, k)) @ r.normal(size=(n, k, cols))
    G = torch.from_numpy(g * 1e-3).float().bfloat16().to(DEV)
    m = torch.from_numpy(r.normal(size=shape) * (0 if low_rank else 2e-3)).float().to(DEV)
    W = torch.from_numpy(r.normal(size=shape) * 0.02).float().to(DEV)
    return G, m, W, torch.full(shape, 9.0, device=DEV).bfloat16()


def _check(G, m0, W0, P, W, m, *, lr, mu=0.95, nesterov=True, wd=0.0, coef=(S.USUAL,) * 5, scale=None):
    f = lambda v: float(np.float32(v))  # noqa: E731
    coef = [tuple(f(v) for v in c) for c in coef]
    grow = np.prod([abs(c[0]) for c in coef])
    assert torch.equal(P, W.bfloat16())
    rows, cols = W.shape[-2:]
    s = max(1.0, rows / cols) ** 0.5 if scale is None else scale
    short = min(rows, cols)
    for i in range(W.shape[0]):
        g, m1, w0 = _f64(G[i]), _f64(m0[i]), _f64(W0[i])
        want, wm = S.muon(w0, g, m1, f(lr), f(mu), nesterov, f(wd), coef, f(s))
        assert np.all(np.abs(_f64(m[i]) - wm) <= 2 * U * (np.abs(mu * m1) + np.abs(wm)) + 1e-45)
        u = g + f(mu) * wm if nesterov else wm
        x = S.orthogonalised(u, coef)
        x0 = S.orthogonalised(u, ())
        sv0, sv = np.linalg.svd(x0, compute_uv=False), np.linalg.svd(x, compute_uv=False)
        # singular values do not keep their order: K bounded by the scalar iteration
        k, v = np.zeros_like(sv0), sv0.copy()
        for a, b, c in coef:
            v = a * v + b * v ** 3 + c * v ** 5
        k = np.max(np.abs(v) / np.maximum(sv0, 1e-300), initial=0, where=sv0 > 1e-12)
        dx = U * (4 * grow + (short + 4) * short ** 0.5 * min(max(k, 1), grow))
        bound = lr * s * dx + 3 * U * (np.linalg.norm(w0) + lr * s * np.linalg.norm(sv))
        assert np.linalg.norm(_f64(W[i]) - want) <= bound, (i, np.linalg.norm(_f64(W[i]) - want), bound)


SHAPES = [(1, 1, 1), (2, 1, 64), (1, 64, 1), (3, 2, 3), (1, 8, 256), (2, 256, 8), (3, 7, 1001), (3, 1001, 7),
          (2, 15, 129), (2, 129, 15), (2, 16, 4096), (2, 4096, 16), (2, 17, 640), (2, 640, 17), (1, 32, 4160),
          (2, 33, 130), (2, 130, 33), (1, 48, 1000), (1, 1000, 48), (1, 63, 65), (1, 65, 63), (2, 64, 64),
          (2, 64, 8192), (1, 11008, 64), (5, 11008, 16), (40, 16, 300), (1, 60, 22016), (300, 4, 64),
          # tall, with a rank that no vector divides
          (3, 5000, 1), (3, 5000, 2), (3, 5000, 3), (3, 5001, 5), (2, 5000, 6), (2, 2003, 13), (2, 700, 19),
          (2, 2001, 31), (2, 700, 35), (2, 1300, 47), (2, 700, 50), (2, 1111, 53), (1, 900, 61), (70, 333, 62),
          # long: many partials; m, g, w and p larger than half the last-level cache, rows on lines or not
          (1, 40, 20000), (1, 16, 70000), (1, 70001, 3), (2, 32, 40000), (3, 52, 65536), (3, 65536, 52), (2, 50, 98305)]


@pytest.mark.parametrize("n,rows,cols", SHAPES)
@pytest.mark.parametrize("nesterov", [True, False])
def test_muon_parity(lib, n, rows, cols, nesterov):
    _case("muon", n, rows, cols, nesterov)
    G, m, W, P = _state(n, rows, cols, rows * 7 + cols)
    m0, W0, G0 = m.clone(), W.clone(), G.clone()
    lib.muon_step(P, W, G, m, lr=0.01, nesterov=nesterov, weight_decay=0.1)
    _check(G, m0, W0, P, W, m, lr=0.01, nesterov=nesterov, wd=0.1)
    assert torch.equal(G, G0)


@pytest.mark.parametrize("n,rows,cols", [(2, 64, 4096), (2, 4096, 64), (2, 16, 1024), (2, 1024, 12)])
def test_muon_low_rank_gradients(lib, n, rows, cols):
    # two strong directions over weak ones, as a first step's gradients are
    _case("muon low rank", n, rows, cols)
    G, m, W, P = _state(n, rows, cols, 5, low_rank=True)
    m0, W0 = m.clone(), W.clone()
    lib.muon_step(P, W, G, m, lr=0.02)
    _check(G, m0, W0, P, W, m, lr=0.02)


def test_muon_coefficients_steps_and_scale(lib):
    _case("muon coefficients")
    G, m, W, P = _state(3, 24, 500, 6)
    for coef, kw in (((S.USUAL,), dict(ns_steps=1)),
                     (((1.5, -0.5, 0.0),) * 16, dict(ns_steps=16, coefficients=(1.5, -0.5, 0.0))),
                     (((4.0, -7.0, 3.5), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0)),
                      dict(ns_steps=3, coefficients=[(4.0, -7.0, 3.5), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0)]))):
        m0, W0 = m.clone(), W.clone()
        lib.muon_step(P, W, G, m, lr=0.05, momentum=0.5, scale=0.2, **kw)
        _check(G, m0, W0, P, W, m, lr=0.05, mu=0.5, coef=coef, scale=0.2)


def test_muon_one_matrix_is_the_stack_of_one(lib):
    G, m, W, P = _state(4, 16, 768, 7)
    single = [t.clone() for t in (P, W, G, m)]
    lib.muon_step(P, W, G, m, lr=0.01)
    for i in range(4):
        p, w, g, b = (t[i] for t in single)
        lib.muon_step(p, w, g, b, lr=0.01)
    # the work is split otherwise; both are within rounding of each other
    assert torch.allclose(W, single[1], rtol=0, atol=1e-6)
    assert torch.equal(m, single[3])


def test_muon_zero_and_tiny_and_nan_gradients(lib):
    _case("muon zero")
    for shape in ((3, 16, 512), (3, 512, 16)):
        G, m, W, P = _state(*shape, 8)
        G.zero_()
        m.zero_()
        W0 = W.clone()
        lib.muon_step(P, W, G, m, lr=0.01, weight_decay=0.5)
        assert torch.equal(W, W0 * torch.tensor(1 - float(np.float32(0.01)) * 0.5, device=DEV).float())
        assert torch.equal(P, W.bfloat16())
        # sizes at which the squares leave fp32's range: the direction is the same
        G, m, W, P = _state(*shape, 9)
        m.zero_()
        G[0] *= 2.0 ** 90
        G[1] = float("nan")
        m0, W0 = m.clone(), W.clone()
        lib.muon_step(P, W, G, m, lr=0.01)
        assert torch.isnan(W[1]).all()
        keep = [0, 2]
        _check(G[keep], m0[keep], W0[keep], P[keep], W[keep], m[keep], lr=0.01)


def test_muon_several_steps_stay_close(lib):
    # five steps in a row: each one starts from what the last one wrote
    _case("muon steps")
    G, m, W, P = _state(2, 1024, 16, 10)
    for step in range(5):
        G = (G.float() * (1 - 0.3 * step) + 1e-4).bfloat16()
        m0, W0 = m.clone(), W.clone()
        lib.muon_step(P, W, G, m, lr=0.01, weight_decay=0.01)
        _check(G, m0, W0, P, W, m, lr=0.01, wd=0.01)


def test_muon_writes_nothing_behind_the_stack(lib):
    for n, rows, cols in ((3, 7, 101), (2, 101, 7), (1, 64, 130), (2, 16, 64)):
        k = n * rows * cols
        bufs = [torch.full((k + 256,), 3.0, device=DEV, dtype=t) for t in (torch.bfloat16, torch.float32,
                                                                          torch.bfloat16, torch.float32)]
        P, W, G, m = (b[:k].view(n, rows, cols) for b in bufs)
        lib.muon_step(P, W, G, m, lr=0.01)
        assert all(torch.all(b[k:] == 3) for b in bufs)
        assert torch.all(G == 3) and torch.isfinite(W).all()


def test_muon_state_in_pinned_host_memory(lib):
    _case("muon pinned")
    G, m, W, P = _state(2, 16, 1024, 11)
    mp, Wp = (torch.empty(t.shape, pin_memory=True).copy_(t) for t in (m, W))
    P2 = P.clone()
    lib.muon_step(P, W, G, m, lr=0.01)
    lib.muon_step(P2, Wp, G, mp, lr=0.01)
    torch.cuda.synchronize()
    assert torch.equal(P, P2) and torch.equal(W.cpu(), Wp) and torch.equal(m.cpu(), mp)


def test_muon_captured_replays_and_streams(lib):
    _case("muon graph")
    a, b = _state(3, 16, 512, 12), _state(2, 4096, 32, 13)

    def step(s):
        G, m, W, P = s
        lib.muon_step(P, W, G, m, lr=0.01)

    eager = [[t.clone() for t in s] for s in (a, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    warm = [[t.clone() for t in s] for s in (a, b)]
    with torch.cuda.stream(side):
        for s in warm:
            step(s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for s in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step(s)
    for rep in range(4):
        for s in eager:
            step(s)
        torch.cuda.synchronize()
        graphs[rep % 2].replay()
        graphs[1 - rep % 2].replay()
        torch.cuda.synchronize()
        for s, e in zip((a, b), eager):
            assert all(torch.equal(x, y) for x, y in zip(s, e)), rep


def test_muon_on_two_streams_at_once(lib):
    _case("muon streams")
    shapes = ((2, 64, 2048), (3, 3000, 16), (40, 8, 256))
    states = [_state(*s, 20 + i) for i, s in enumerate(shapes)]
    eager = [[t.clone() for t in s] for s in states]
    for G, m, W, P in eager:
        for _ in range(3):
            lib.muon_step(P, W, G, m, lr=0.01)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in shapes]
    for _ in range(3):
        for st, (G, m, W, P) in zip(streams, states):
            with torch.cuda.stream(st):
                lib.muon_step(P, W, G, m, lr=0.01)
    torch.cuda.synchronize()
    for s, e in zip(states, eager):
        assert all(torch.equal(a, b) for a, b in zip(s, e))


@pytest.mark.parametrize("rows,cols", [(64, 8388600), (8388480, 63)])
def test_muon_largest_matrix(lib, rows, cols):
    # just below 2^29 elements, offsets of 2 GiB: the ends of the long axis against the formula in float64.  With no
    # decay and no weights before, w = -lr scale X, off by Q's and the products' roundings, S + 8 half steps of
    # sum |Q| |u| / |u|, and two of its own.
    _case("muon largest", rows, cols)
    short, tall, lr, mu = min(rows, cols), rows > cols, 0.01, float(np.float32(0.95))
    gen = torch.Generator(device=DEV).manual_seed(rows)
    G = torch.randn(rows, cols, device=DEV, generator=gen, dtype=torch.bfloat16)
    m, W = (torch.zeros(rows, cols, device=DEV) for _ in range(2))
    P = torch.empty(rows, cols, device=DEV, dtype=torch.bfloat16)
    lib.muon_step(P, W, G, m, lr=lr, scale=1.0)
    update = lambda g: (g.float() + mu * g.float()).double()  # noqa: E731
    axis = 0 if tall else 1
    gram = torch.zeros(short, short, device=DEV, dtype=torch.float64)
    for part in G.split(1 << 19, dim=axis):
        u = update(part)
        gram += u.t() @ u if tall else u @ u.t().contiguous()
    norm = gram.trace().sqrt()
    g, eye = gram / norm ** 2, torch.eye(short, device=DEV, dtype=torch.float64)
    q = eye
    for _ in range(5):
        a, b, c = (float(np.float32(v)) for v in S.USUAL)
        p = a * eye + b * g + c * g @ g
        q, g = p @ q, p @ g @ p
    n = 1000
    for at in (0, max(rows, cols) - n):
        u, w, pp = (update(G.narrow(axis, at, n)), W.narrow(axis, at, n).double(), P.narrow(axis, at, n))
        want = -lr * (u @ q if tall else q @ u) / norm
        size = lr * (u.abs() @ q.abs() if tall else q.abs() @ u.abs()) / norm
        assert ((w - want).abs() <= U * ((short + 8) * size + 2 * want.abs())).all()
        assert torch.equal(pp, w.float().bfloat16())
    assert torch.equal(m, G.float())
