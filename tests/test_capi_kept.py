"""Host-side checks of the 8-bit checkpoint's and the scores' calls (no GPU
needed): argument validation at the C ABI and of the Python forms.  The device
pointers are fake addresses that are never dereferenced."""

import ctypes

import pytest
import torch

OK, E_NULL, E_SHAPE, E_RANK, E_ALIGN, E_WS, E_ALPHA, E_ALIAS, E_HIP, E_TYPE = range(10)
GB = 1 << 30
X, CODES, AM, Y, T_, A, B, WS, DY, DX, DA, DB, KEEP, W0, W1, W2, W3 = (p * 8 * GB for p in range(1, 18))
Z, DZ, TOK, LP, ENT, IDS, TOP, ST, DLP, DENT = (p * 8 * GB for p in range(20, 30))
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L(lib):
    return lib.lib()


def _desc(lib, d=256, k=512):
    return ctypes.byref(lib._Nf4Desc(d, k, W0, W1, W2, W3))


def test_checkpoint_sizes(L):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()

    def f(M, k):
        s = L.qlora_checkpoint_sizes(M, k, ctypes.byref(a), ctypes.byref(b))
        return s if s else (a.value, b.value)

    assert f(1, 64) == (64, 128) and f(64, 64) == (4096, 128) and f(65, 128) == (8320, 512) and f(0, 64) == (0, 0)
    assert f(4096, 4096) == (1 << 24, 1 << 19)
    for bad in ((-1, 64), (1, 0), (1, 63), (1, 96), (1 << 31, 64), (1 << 25, 64), (1, 1 << 31)):
        assert f(*bad) == E_SHAPE, bad
    assert L.qlora_checkpoint_sizes(5, 64, None, None) == OK


def test_checkpoint_validation(L):
    def save(x=X, M=100, k=512, c=CODES, a=AM):
        return L.qlora_checkpoint_save(x, M, k, c, a, None)

    def load(x=X, M=100, k=512, c=CODES, a=AM):
        return L.qlora_checkpoint_load(c, a, M, k, x, None)

    for f in (save, load):
        assert f(M=-1) == E_SHAPE and f(k=500) == E_SHAPE and f(k=0) == E_SHAPE and f(M=1 << 22) == E_SHAPE
        assert f(M=0) == OK and f(M=0, x=None, c=None, a=None) == OK
        for name in "xca":
            assert f(**{name: None}) == E_NULL
            assert f(**{name: 200 * GB + 8}) == E_ALIGN
        assert f(c=X + 16) == E_ALIAS and f(a=X + 100 * 1024 - 16) == E_ALIAS and f(x=CODES + 51184) == E_ALIAS
    assert save(a=CODES + 51184) == E_ALIAS
    # the constants' rows end behind the last token
    assert save(a=X - 8 * 128 * 2 + 16) == E_ALIAS


def test_forward_checkpoint_validation(L, lib):
    def f(x=X, M=100, w=None, nsec=1, a=A, b=B, r=16, al=1.0, y=Y, t=T_, c=CODES, m=AM, ws=WS, wb=1 << 40):
        return L.qlora_forward_checkpoint(x, M, w or _desc(lib), nsec, a, b, r, al, y, t, c, m, ws, wb, None)

    assert f(c=None) == E_NULL and f(m=None) == E_NULL and f(x=None) == E_NULL and f(y=None) == E_NULL
    assert f(a=None) == E_NULL and f(M=-1) == E_SHAPE and f(r=65) == E_RANK and f(al=NAN) == E_ALPHA
    assert f(M=0) == OK
    assert f(c=CODES + 8) == E_ALIGN and f(m=AM + 2) == E_ALIGN and f(ws=None) == E_WS
    for other in (X, Y, A, B, T_, WS, W0):
        assert f(c=other) == E_ALIAS and f(m=other) == E_ALIAS
    assert f(c=AM + 512) == E_ALIAS


def test_backward_checkpoint_validation(L, lib):
    def f(g=DY, c=CODES, m=AM, M=100, w=None, nsec=1, a=A, b=B, r=16, al=1.0, keep=None, p=0.0, t=T_, dx=DX, da=DA,
          db=DB, ws=WS, wb=1 << 40):
        return L.qlora_backward_checkpoint(g, c, m, M, w or _desc(lib), nsec, a, b, r, al, keep, p, t, dx, da, db, ws,
                                           wb, None)

    for name in ("g", "c", "m", "a", "b", "t", "da", "db"):
        assert f(**{name: None}) == E_NULL, name
    assert f(M=-1) == E_SHAPE and f(r=65) == E_RANK and f(al=INF) == E_ALPHA and f(M=0) == OK
    for name in ("g", "c", "m", "a", "b", "t", "da", "db", "dx"):
        assert f(**{name: 300 * GB + 8}) == E_ALIGN, name
    assert f(ws=None) == E_WS and f(wb=64) == E_WS
    for other in (CODES, AM, DY, A, B, T_, W1):
        for name in ("dx", "da", "db"):
            assert f(**{name: other}) == E_ALIAS, (name, other)
    assert f(ws=CODES) == E_ALIAS and f(ws=AM) == E_ALIAS
    # dropout: a mask for one section, and its probability
    assert f(keep=KEEP, p=1.0) == E_ALPHA and f(keep=KEEP, p=NAN) == E_ALPHA and f(keep=KEEP + 1, p=0.1) == E_ALIGN
    assert f(keep=KEEP, p=0.1, nsec=2, w=_desc(lib, 512)) == E_SHAPE
    assert f(keep=DX, p=0.1) == E_ALIAS


def test_scores_validation(L):
    def f(z=Z, dt=0, T=100, V=1000, ld=1000, y=TOK, m=3, n=5, tau=1.0, lp=LP, e=ENT, i=IDS, t=TOP, st=ST):
        return L.qlora_token_scores(z, dt, T, V, ld, y, m, n, tau, lp, e, i, t, st, None)

    def b(g=DLP, ge=DENT, z=Z, dt=0, T=100, V=1000, ld=1000, y=TOK, m=3, tau=1.0, st=ST, dz=DZ, ldd=1000):
        return L.qlora_token_scores_backward(g, ge, z, dt, T, V, ld, y, m, tau, st, dz, ldd, None)

    for call in (f, b):
        assert call(dt=2) == E_TYPE and call(T=-1) == E_SHAPE and call(T=1 << 31) == E_SHAPE
        assert call(V=0) == E_SHAPE and call(ld=999) == E_SHAPE and call(V=1 << 30, ld=1 << 30) == E_SHAPE
        assert call(m=-1) == E_SHAPE and call(m=65) == E_SHAPE
        for tau in (0.0, -1.0, INF, NAN):
            assert call(tau=tau) == E_ALPHA
        assert call(z=None) == E_NULL and call(y=None) == E_NULL
        assert call(z=Z + 1) == E_ALIGN and call(z=Z + 2, dt=1) == E_ALIGN and call(y=TOK + 2) == E_ALIGN
        assert call(T=0) == OK and call(T=0, z=None, y=None) == OK
    assert f(n=-1) == E_SHAPE and f(n=65) == E_SHAPE and f(V=4, ld=8, n=5) == E_SHAPE
    assert f(lp=None) == E_NULL and f(e=None) == E_NULL and f(i=None) == E_NULL and f(t=None) == E_NULL
    assert f(z=None, y=None, m=0, lp=None) == E_NULL
    for name in ("lp", "e", "i", "t", "st"):
        assert f(**{name: 300 * GB + 2}) == E_ALIGN, name
    assert f(lp=Z + 4) == E_ALIAS and f(e=LP + 1196) == E_ALIAS and f(i=TOP + 1996) == E_ALIAS and f(st=TOK) == E_ALIAS
    assert f(lp=TOK + 1196) == E_ALIAS and f(st=IDS - 1196) == E_ALIAS
    assert b(g=None) == E_NULL and b(st=None) == E_NULL and b(dz=None) == E_NULL
    assert b(g=DLP + 1) == E_ALIGN and b(ge=DENT + 2) == E_ALIGN and b(st=ST + 2) == E_ALIGN and b(dz=DZ + 1) == E_ALIGN
    assert b(ldd=999) == E_SHAPE and b(ldd=1 << 30) == E_SHAPE
    assert b(dz=Z + 2) == E_ALIAS and b(dz=Z, ldd=1008) == E_ALIAS
    assert b(dz=DLP + 1184) == E_ALIAS and b(dz=DENT) == E_ALIAS and b(dz=ST) == E_ALIAS and b(dz=TOK) == E_ALIAS


def test_python_refusals(lib):
    z, y = torch.zeros(4, 80, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    for bad in (y.long(), y[:3], y[:, :1].expand(4, 2), y.view(4, 2, 1), torch.zeros(4, 65, dtype=torch.int32)):
        with pytest.raises(ValueError):
            lib.token_scores(z, bad)
    for top in (-1, 65):
        with pytest.raises(ValueError):
            lib.token_scores(z, y, top=top)
    with pytest.raises(ValueError):
        lib.token_scores(z[:, :8], y, top=9)
    with pytest.raises(TypeError):
        lib.token_scores(z.half(), y)
    with pytest.raises(ValueError):
        lib.token_scores(z.t(), None)
    g, st = torch.zeros(4, 2), torch.zeros(4, 3)
    for args in ((g, None, z, None, st), (None, None, z, y, st), (g[:, 0], None, z, y, st), (g.double(), None, z, y, st),
                 (g, torch.zeros(3), z, y, st), (g, None, z, y, torch.zeros(4, 2)), (g, None, z, y.long(), st)):
        with pytest.raises(ValueError):
            lib.token_scores_backward(*args)
    with pytest.raises(ValueError):
        lib.token_scores_backward(g, None, z, y, st, out=torch.zeros(4, 80))
    for M, k in ((-1, 64), (4, 63), (4, 0)):
        with pytest.raises(ValueError):
            lib.Checkpoint.empty(M, k, "cpu")
    ck = lib.Checkpoint.empty(4, 128, "cpu")
    assert ck.codes.shape == (4, 128) and ck.absmax.shape == (2, 64)
    ck.check(4, 128, torch.device("cpu"))
    for bad in (lib.Checkpoint(4, 128, ck.codes.view(torch.uint8), ck.absmax), lib.Checkpoint(4, 128, ck.codes, ck.absmax.half()),
                lib.Checkpoint(4, 128, ck.codes, ck.absmax[:, :4]), lib.Checkpoint(4, 128, ck.codes[:, ::2], ck.absmax),
                lib.Checkpoint(5, 128, ck.codes, ck.absmax)):
        with pytest.raises(ValueError):
            bad.check(4, 128, torch.device("cpu"))


def test_python_calls_refuse_host_memory(lib):
    z, y = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    ck = lib.Checkpoint.empty(4, 128, "cpu")
    calls = (lambda: lib.token_scores(z, y), lambda: lib.token_scores_backward(torch.zeros(4, 2), None, z, y, torch.zeros(4, 3)),
             lambda: lib.checkpoint_save(z), lambda: lib.checkpoint_load(ck),
             lambda: lib.forward_checkpoint(z, lib.NF4Weight.empty(64, 128, "cpu")),
             lambda: lib.backward_checkpoint(z, ck, lib.NF4Weight.empty(128, 128, "cpu")))
    for call in calls:
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_shapes_are_refused_before_a_call(lib):
    for X_ in (torch.zeros(4, 128), torch.zeros(4, 128, dtype=torch.bfloat16)[:, :64], torch.zeros(128, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            lib.checkpoint_save(X_)
