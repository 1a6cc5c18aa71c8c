"""Host-side checks of the fine-tuning step's calls (no GPU needed): argument
validation of qlora_token_logprobs (and its backward), qlora_preference_loss,
qlora_policy_loss and qlora_muon_step, and of their Python forms.  The device
pointers are fake addresses that are never dereferenced."""

import ctypes

import pytest
import torch

OK, E_NULL, E_SHAPE, E_RANK, E_ALIGN, E_WS, E_ALPHA, E_ALIAS, E_HIP, E_TYPE = range(10)
GB = 1 << 30
Z, DZ, LAB, LP, ST, DLP, CU, W_, LOSS, REW, REF, ADV, OLD, KL = (p * GB for p in range(1, 15))
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L(lib):
    return lib.lib()


def test_status_string_of_an_unknown_type(L, lib):
    assert L.qlora_status_string(E_TYPE) != b"unknown status"
    assert lib.STATUS[E_TYPE] == "QLORA_ERR_TYPE"


def test_token_logprobs_validation(L):
    def f(z=Z, dt=0, T=100, V=1000, ld=1000, y=LAB, tau=1.0, lp=LP, st=ST):
        return L.qlora_token_logprobs(z, dt, T, V, ld, y, tau, lp, st, None)

    def b(g=DLP, z=Z, dt=0, T=100, V=1000, ld=1000, y=LAB, tau=1.0, st=ST, dz=DZ, ldd=1000):
        return L.qlora_token_logprobs_backward(g, z, dt, T, V, ld, y, tau, st, dz, ldd, None)

    for call in (f, b):
        assert call(dt=2) == E_TYPE and call(dt=-1) == E_TYPE
        assert call(T=-1) == E_SHAPE and call(T=1 << 31) == E_SHAPE
        assert call(V=0) == E_SHAPE and call(ld=999) == E_SHAPE
        assert call(V=1 << 30, ld=1 << 30) == E_SHAPE
        for tau in (0.0, -1.0, INF, NAN):
            assert call(tau=tau) == E_ALPHA
        assert call(z=None) == E_NULL and call(y=None) == E_NULL
        assert call(z=Z + 1) == E_ALIGN and call(z=Z + 2, dt=1) == E_ALIGN and call(y=LAB + 2) == E_ALIGN
        assert call(T=0) == OK and call(T=0, z=None, y=None) == OK
    assert f(lp=None) == E_NULL
    assert f(lp=LP + 2) == E_ALIGN and f(st=ST + 1) == E_ALIGN
    assert f(lp=Z + 4) == E_ALIAS and f(st=LP + 396) == E_ALIAS and f(lp=LAB) == E_ALIAS
    # the last row ends at its V-th element
    assert f(lp=Z + (99 * 1200 + 1000) * 2 - 4, ld=1200) == E_ALIAS
    assert b(g=None) == E_NULL and b(st=None) == E_NULL and b(dz=None) == E_NULL
    assert b(ldd=999) == E_SHAPE and b(ldd=1 << 30) == E_SHAPE
    assert b(dz=DZ + 1) == E_ALIGN and b(g=DLP + 1) == E_ALIGN
    assert b(dz=Z + 2) == E_ALIAS                                # off by an element: not in place
    assert b(dz=Z, ldd=1008) == E_ALIAS                          # another stride: not in place
    assert b(dz=DLP) == E_ALIAS and b(dz=ST - 100) == E_ALIAS and b(dz=LAB) == E_ALIAS
    # dlogits rows are written to their whole stride
    assert b(dz=ST - (100 * 1004 * 2 - 2), ldd=1004) == E_ALIAS


def test_preference_validation(L):
    def f(lp=LP, ref=REF, y=LAB, T=100, V=1000, cu=CU, P=4, kind=0, beta=0.1, e=0.0, mg=0.0, w=W_, loss=LOSS,
          rew=REW, g=DLP):
        return L.qlora_preference_loss(lp, ref, y, T, V, cu, P, kind, 0, beta, e, mg, w, loss, rew, g, None)

    assert f(kind=3) == E_TYPE and f(kind=-1) == E_TYPE
    assert f(T=-1) == E_SHAPE and f(V=0) == E_SHAPE and f(P=-1) == E_SHAPE and f(P=1 << 20) == E_SHAPE
    for bad in (0.0, -0.1, INF, NAN):
        assert f(beta=bad) == E_ALPHA
    assert f(e=-0.1) == E_ALPHA and f(e=0.51) == E_ALPHA and f(e=NAN) == E_ALPHA and f(mg=INF) == E_ALPHA
    assert f(P=0) == OK and f(P=0, cu=None, loss=None) == OK
    assert f(lp=None) == E_NULL and f(y=None) == E_NULL and f(cu=None) == E_NULL and f(loss=None) == E_NULL
    for name in ("lp", "ref", "y", "cu", "w", "loss", "rew", "g"):
        assert f(**{name: 20 * GB + 2}) == E_ALIGN, name
    assert f(g=LP) == E_ALIAS and f(loss=CU + 32) == E_ALIAS and f(rew=LOSS) == E_ALIAS and f(g=W_) == E_ALIAS


def test_policy_validation(L):
    def f(z=Z, dt=0, T=100, V=1000, ld=1000, y=LAB, tau=1.0, adv=ADV, old=OLD, ref=REF, w=W_, lo=0.2, hi=0.2, kc=0.1,
          loss=LOSS, kl=KL, lp=LP, dz=DZ, ldd=1000):
        return L.qlora_policy_loss(z, dt, T, V, ld, y, tau, adv, old, ref, w, lo, hi, kc, loss, kl, lp, dz, ldd, None)

    assert f(dt=7) == E_TYPE and f(ld=10) == E_SHAPE and f(tau=0.0) == E_ALPHA
    assert f(lo=-0.1) == E_ALPHA and f(lo=1.1) == E_ALPHA and f(hi=-0.1) == E_ALPHA and f(hi=INF) == E_ALPHA
    assert f(kc=-1.0) == E_ALPHA and f(kc=NAN) == E_ALPHA
    assert f(T=0) == OK
    assert f(adv=None) == E_NULL and f(loss=None) == E_NULL and f(lp=None) == E_NULL and f(z=None) == E_NULL
    for name in ("adv", "old", "ref", "w", "loss", "kl", "lp"):
        assert f(**{name: 20 * GB + 2}) == E_ALIGN, name
    assert f(ldd=999) == E_SHAPE and f(dz=DZ + 1) == E_ALIGN
    assert f(dz=Z + 2) == E_ALIAS and f(dz=ADV) == E_ALIAS and f(dz=KL) == E_ALIAS and f(dz=W_ - 64) == E_ALIAS
    assert f(loss=LP) == E_ALIAS and f(kl=OLD) == E_ALIAS and f(lp=Z) == E_ALIAS


def test_muon_validation(L):
    P, W, G, m, ws = (p * GB for p in (21, 22, 23, 24, 25))
    F = ctypes.c_float

    def f(P=P, W=W, G=G, m=m, n=2, rows=16, cols=4096, lr=1e-3, mu=0.95, wd=0.0, scale=1.0, eps=1e-7, steps=5,
          coef=None, ws=ws, wsb=1 << 40):
        return L.qlora_muon_step(P, W, G, m, n, rows, cols, lr, mu, 1, wd, scale, eps, steps, coef, ws, wsb, None)

    assert f(n=-1) == E_SHAPE and f(n=65536) == E_SHAPE and f(rows=0) == E_SHAPE and f(cols=0) == E_SHAPE
    assert f(rows=64, cols=1 << 25) == E_SHAPE and f(n=4, rows=64, cols=1 << 23) == E_SHAPE
    assert f(rows=65, cols=65) == E_RANK
    assert f(steps=0) == E_SHAPE and f(steps=17) == E_SHAPE
    assert f(lr=-1.0) == E_ALPHA and f(lr=INF) == E_ALPHA and f(mu=1.0) == E_ALPHA and f(mu=NAN) == E_ALPHA
    assert f(wd=-1.0) == E_ALPHA and f(scale=NAN) == E_ALPHA and f(eps=0.0) == E_ALPHA and f(eps=INF) == E_ALPHA
    assert f(coef=(F * 15)(*([1.0] * 14 + [INF]))) == E_ALPHA
    assert f(n=0) == OK and f(n=0, P=None) == OK
    assert f(P=None) == E_NULL and f(W=None) == E_NULL and f(G=None) == E_NULL and f(m=None) == E_NULL
    assert f(W=W + 4) == E_ALIGN and f(ws=ws + 8) == E_ALIGN
    assert f(ws=None) == E_WS and f(wsb=64) == E_WS
    assert f(m=W + 16) == E_ALIAS and f(P=G) == E_ALIAS and f(ws=G) == E_ALIAS and f(ws=m - 16) == E_ALIAS
    need = L.qlora_muon_workspace_bytes
    assert need(2, 16, 4096) > 0 and need(2, 4096, 16) > 0
    assert need(2, 16, 256) == 0 and f(cols=256, ws=None, wsb=0, W=W + 4) == E_ALIGN   # small: none needed
    assert need(0, 16, 4096) == 0 and need(2, 65, 65) == 0 and need(1, 0, 5) == 0


# --------------------------------------------------- the Python forms ----
# Every call below is refused before its pointers are used.

def test_python_refusals(lib):
    z, y = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError):
        lib.token_logprobs(z.half(), y)
    with pytest.raises(TypeError):
        lib.token_logprobs(z[0], y)
    with pytest.raises(ValueError):
        lib.token_logprobs(z.t(), torch.zeros(8, dtype=torch.int32))   # rows not contiguous
    with pytest.raises(ValueError):
        lib.token_logprobs(z, y.long())
    with pytest.raises(ValueError):
        lib.token_logprobs(z, y[:3])
    with pytest.raises(ValueError):
        lib.token_logprobs(z, torch.zeros(8, dtype=torch.int32)[::2])
    g, st = torch.zeros(4), torch.zeros(4, 2)
    with pytest.raises(ValueError):
        lib.token_logprobs_backward(g, z, y, torch.zeros(4, 3))
    with pytest.raises(ValueError):
        lib.token_logprobs_backward(g.double(), z, y, st)
    with pytest.raises(ValueError):
        lib.token_logprobs_backward(g, z, y, st, out=torch.zeros(4, 8))              # another type
    wide = torch.zeros(4 * 10 - 1, dtype=torch.bfloat16).as_strided((4, 8), (10, 1))
    with pytest.raises(ValueError):
        lib.token_logprobs_backward(g, z, y, st, out=wide)                           # the last row's stride is missing
    cu = torch.tensor([0, 2, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        lib.preference_loss(g, y, 8, cu, 0.1, kind="other")
    with pytest.raises(ValueError):
        lib.preference_loss(g, y, 8, cu[:2], 0.1)
    with pytest.raises(ValueError):
        lib.preference_loss(g, y, 8, cu, 0.1, weight=torch.zeros(2))
    with pytest.raises(ValueError):
        lib.policy_loss(z, y, g, old_logp=torch.zeros(5))
    W = torch.zeros(2, 8, 32)
    P = W.bfloat16()
    with pytest.raises(ValueError):
        lib.muon_step(P, W, W, W.clone(), lr=0.1)                                    # fp32 gradients
    with pytest.raises(ValueError):
        lib.muon_step(P, W.transpose(1, 2), P.clone(), W.clone(), lr=0.1)
    with pytest.raises(ValueError):
        lib.muon_step(P[0, 0], W[0, 0], P[0, 0], W[0, 0], lr=0.1)
    with pytest.raises(ValueError):
        lib.muon_step(P, W, P.clone(), W.clone(), lr=0.1, coefficients=[(1.0, 2.0, 3.0)] * 4)


def test_python_calls_refuse_host_memory(lib):
    z, y, g = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    W = torch.zeros(8, 32)
    calls = (lambda: lib.token_logprobs(z, y), lambda: lib.token_logprobs_backward(g, z, y, torch.zeros(4, 2)),
             lambda: lib.policy_loss(z, y, g),
             lambda: lib.preference_loss(g, y, 8, torch.tensor([0, 2, 4], dtype=torch.int32), 0.1),
             lambda: lib.muon_step(W.bfloat16(), W, W.bfloat16(), W.clone(), lr=0.1))
    for call in calls:
        with pytest.raises(ValueError, match="GPU"):
            call()
