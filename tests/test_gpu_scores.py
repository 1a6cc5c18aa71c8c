"""GPU parity of the scores of a head's logits and of their gradient against
the float64 reference.

Tolerances.  u = 2^-24.  With t = tau (z - max z), S the sum of exp t over V
words, E the mean under p:

* ln S and a token's logp as for the label log-probabilities: an exponent is
  off by at most 4 u |t| (two fused steps, the constant, the difference), ln S by
  4 u E|t| <= 4 u ln V and by its sum's (V/256 + 24) u, exp2 and the logarithms by
  8 u (1 + ln S), a token's own term by 3 u |t_y| and the last rounding:
  |d logp| <= u (12 (ln V + 1) + V/256 + 32 + 3 |t_y| + |logp|) = B.
* the mean exponent E t = sum e t / sum e: each e is off by (4 |t| + 8) u of it,
  each t by 4 u |t|, both sums by (V/256 + 32) u of sum e |t|, the quotient by 4 u:
  |d E t| <= u ((4 E t^2 + 8 E|t|) + (4 E|t| + 8) E|t| + (2 V/256 + 72) E|t|) = C,
  and |d H| <= B0 + C + u H, B0 being B without a token's own terms.
* gradient: with f = G + gH (t - E t), p f is off by p (6 u |ln p| + B0) |f| + p
  |gH| (8 u (|t| + E|t|) + C) + 4 u p |f|, G by m u sum |g|, a token's sum by m u of
  its own, bf16's one-part exponent (2^-16 of p f) and the rounding to the type.
  The hardware's exp2 gives 0 below 2^-126: a word of p s < 2^-126, s >= 1/2, has no
  gradient of its own instead of p f < 2^-125 f.
"""

import numpy as np
import pytest
import torch

from gpu_util import DEV
from oracle import scores_oracle as S

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def _case(*args):
    print("case:", *args, flush=True)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _logits(T, V, dtype, seed, ld=None, offset=0, std=3.0):
    ld = V if ld is None else ld
    g = torch.Generator().manual_seed(seed)
    buf = (torch.randn(T * ld + offset, generator=g) * std).to(dtype).to(DEV)
    return buf[offset:].view(T, ld)[:, :V]


def _tokens(T, V, m, seed):
    """Given tokens: some out of range, some twice in a row, a row without one that counts."""
    g = torch.Generator().manual_seed(seed + 1)
    y = torch.randint(0, V, (T, m), generator=g, dtype=torch.int32)
    if m > 1:
        y[:, -1] = y[:, 0]
        y[::3, m // 2] = -100
    if T > 3:
        y[1::5] = V
        y[2, 0] = V - 1
    return y.to(DEV)


def _bounds(z, tau, H):
    """(B0 [T], C [T], E|t| [T]) of rows with a distribution; zeros elsewhere."""
    V = z.shape[1]
    with np.errstate(all="ignore"):
        t = tau * (z - z.max(axis=1, keepdims=True))
        p = np.exp(t)
        p /= p.sum(axis=1, keepdims=True)
        t = np.where(p > 0, t, 0.0)
        e1, e2 = (p * np.abs(t)).sum(axis=1), (p * t * t).sum(axis=1)
    B0 = U * (12 * (np.log(V) + 1) + V / 256 + 32) * np.ones(len(z))
    C = U * (4 * e2 + 8 * e1 + (4 * e1 + 8) * e1 + (2 * V / 256 + 72) * e1)
    return B0, np.nan_to_num(C), np.nan_to_num(e1)


def _token_bound(z, ids, logp, tau, B0):
    with np.errstate(all="ignore"):
        t = tau * np.abs(z - z.max(axis=1, keepdims=True))
    ty = np.take_along_axis(t, np.clip(ids, 0, z.shape[1] - 1), axis=1)
    ty, lp = (np.where(np.isfinite(v), np.abs(v), 0.0) for v in (ty, logp))
    return B0[:, None] + U * (3 * ty + lp)


def _near(got, want, bound):
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        return bool(np.all(same | (np.abs(got - want) <= bound)))


def _check(lib, z, y, n, tau):
    T, V = z.shape
    out = lib.token_scores(z, y, top=n, inv_temperature=tau, save_stats=True)
    zh, yh = _f64(z), None if y is None else y.cpu().numpy().reshape(T, -1)
    logp, H, ids, top = S.scores(zh, yh, n, tau)
    B0, C, _ = _bounds(zh, tau, H)
    if y is None:
        assert out[0] is None
    else:
        assert out[0].shape == y.shape and _near(_f64(out[0]).reshape(T, -1), logp, _token_bound(zh, yh, logp, tau, B0))
    assert _near(_f64(out[1]), H, B0 + C + U * np.abs(np.nan_to_num(H)))
    assert out[2].dtype == torch.int32 and np.array_equal(out[2].cpu().numpy(), ids)
    assert _near(_f64(out[3]), top, _token_bound(zh, ids, top, tau, B0))
    return out


def _check_grad(lib, z, y, g, gh, stats, tau, dtype, out=None, zh=None):
    T, V = z.shape
    zh = _f64(z) if zh is None else zh
    yh = None if y is None else y.cpu().numpy().reshape(T, -1)
    got = lib.token_scores_backward(g, gh, z, y, stats, inv_temperature=tau, out=out)
    gg = np.zeros((T, 0)) if g is None else _f64(g).reshape(T, -1)
    hh = np.zeros(T) if gh is None else _f64(gh)
    want = S.scores_grad(zh, yh, gg, hh, tau)
    B0, C, e1 = _bounds(zh, tau, None)
    m = gg.shape[1]
    with np.errstate(all="ignore"):
        t = tau * (zh - zh.max(axis=1, keepdims=True))
        p = np.exp(t)
        p /= p.sum(axis=1, keepdims=True)
        t = np.where(p > 0, t, 0.0)
        lnp = np.where(p > 0, np.abs(np.log(np.where(p > 0, p, 1.0))), 0.0)
    mean = (p * t).sum(axis=1, keepdims=True)
    use = np.zeros((T, m), bool) if yh is None else (yh >= 0) & (yh < V)
    live = np.ones(T) if yh is None else use.any(axis=1).astype(float)
    G, Gabs = np.where(use, gg, 0).sum(axis=1), np.abs(np.where(use, gg, 0)).sum(axis=1)
    f = np.abs(G[:, None] + (live * hh)[:, None] * (t - mean))
    ah = np.abs(live * hh)[:, None]
    off = p * f * (6 * U * lnp + B0[:, None] + 8 * U + (2.0 ** -16 if dtype == BF else 0))
    off += p * ah * (8 * U * (np.abs(t) + e1[:, None]) + C[:, None]) + ((m + 4) * U * Gabs)[:, None] * p
    if m:
        own = np.zeros((T, V))
        for i in range(T):
            for j in range(m):
                if use[i, j]:
                    own[i, yh[i, j]] += abs(gg[i, j])
        off += (m + 4) * U * own
    off += 2.0 ** -125 * f
    off = tau * off + (4 * U + torch.finfo(dtype).eps / 2) * np.abs(want) + 1e-37
    assert got.dtype == dtype and got.shape == z.shape
    assert _near(_f64(got), want, off)
    return got


# (T, V, m, n): every kernel by row length, in registers and in pieces; few rows and many
SIZES = [(1, 1, 1, 1), (2, 2, 3, 2), (3, 7, 2, 7), (5, 8, 1, 5), (9, 64, 4, 64), (33, 200, 1, 20), (4, 255, 5, 64),
         (7, 513, 2, 64), (9, 2048, 64, 64), (7, 2049, 2, 33), (6, 4099, 1, 20), (5, 8191, 9, 5), (4, 16385, 3, 20),
         (3, 32000, 33, 20), (3, 32769, 1, 64), (2, 50021, 2, 1), (2, 65537, 1, 20), (2, 131072, 1, 20),
         (2, 131077, 4, 64), (1, 262147, 1, 20), (2, 600011, 2, 64), (300, 9001, 1, 20), (300, 33000, 2, 8), (270, 70001, 1, 5)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,V,m,n", SIZES)
def test_scores_and_gradient_parity(lib, T, V, m, n, dtype):
    _case("scores", T, V, m, n, dtype)
    tau = 1.0 if V % 2 else 0.75
    z, y = _logits(T, V, dtype, 11 + V), _tokens(T, V, m, V)
    out = _check(lib, z, y, n, tau)
    gen = torch.Generator().manual_seed(V)
    g, gh = torch.randn(T, m, generator=gen).to(DEV), torch.randn(T, generator=gen).to(DEV)
    if T > 2:
        gh[0] = 0
    _check_grad(lib, z, y, g, gh, out[4], tau, dtype)
    _check_grad(lib, z, y, g, None, out[4], tau, dtype)
    # fewer outputs do not change those that are left
    again = lib.token_scores(z, y, inv_temperature=tau)
    assert torch.equal(again[0], out[0]) and torch.equal(again[1], out[1])
    assert again[2] is None and again[3] is None
    flat = lib.token_scores(z, y[:, 0].contiguous(), top=n, inv_temperature=tau)
    rows = ((y[:, 0] >= 0) & (y[:, 0] < V))
    assert flat[0].shape == (T,) and torch.equal(flat[0], out[0][:, 0])
    assert torch.equal(flat[2][rows], out[2][rows]) and not flat[1][~rows].any()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [100, 3000, 40000, 140000])
def test_without_tokens(lib, V, dtype):
    _case("no tokens", V, dtype)
    z = _logits(4, V, dtype, V)
    out = _check(lib, z, None, 20, 1.0)
    gh = torch.tensor([1.0, -2.0, 0.0, 0.5], device=DEV)
    d = _check_grad(lib, z, None, None, gh, out[4], 1.0, dtype)
    assert not d[2].any()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("ld,offset", [(1000, 1), (1001, 0), (1003, 5), (1008, 0), (1024, 3), (4000, 7)])
def test_strides_and_starts(lib, ld, offset, dtype):
    # rows that start anywhere; the gradient's rows are written whole, nothing before or behind them
    _case("strides", ld, offset, dtype)
    T, V, m = 21, 1000, 3
    z, y = _logits(T, V, dtype, 5, ld, offset), _tokens(T, V, m, 5)
    out = _check(lib, z, y, 20, 1.0)
    g, gh = torch.linspace(-1, 1, T * m).view(T, m).to(DEV), torch.linspace(1, -1, T).to(DEV)
    want = _check_grad(lib, z, y, g, gh, out[4], 1.0, dtype)
    buf = torch.full((T * ld + offset + 64,), 7.0, dtype=dtype, device=DEV)
    dst = buf[offset:offset + T * ld].view(T, ld)
    got = lib.token_scores_backward(g, gh, z, y, out[4], out=dst[:, :V])
    assert torch.equal(got, want) and torch.all(dst[:, V:] == 0)
    assert torch.all(buf[:offset] == 7) and torch.all(buf[offset + T * ld:] == 7)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [1000, 32000, 70001, 300000])
def test_in_place(lib, V, dtype):
    _case("in place", V, dtype)
    T, m = 9, 5
    z, y = _logits(T, V, dtype, 6), _tokens(T, V, m, 6)
    stats = lib.token_scores(z, y, save_stats=True)[4]
    g, gh = torch.linspace(-2, 2, T * m).view(T, m).to(DEV), torch.linspace(1, -1, T).to(DEV)
    want = lib.token_scores_backward(g, gh, z, y, stats)
    a = z.clone()
    assert lib.token_scores_backward(g, gh, a, y, stats, out=a) is a and torch.equal(a, want)


def _crowded(T, V, dtype):
    """Rows of 64 tokens: one word throughout, neighbours (of them the row's first and last words), words a list's
    number of pieces apart, both ends and every border between the columns of two work-groups."""
    per = 16 // torch.finfo(dtype).bits * 8
    j = torch.arange(64)
    rows = [torch.full((64,), V // 2), j % V, V - 1 - (j % V), (j // 2 * 1024 * per + 3) % V,
            torch.where(j % 2 == 0, j // 2 * 1024 * per, j // 2 * 1024 * per - 1) % V,
            torch.where(j % 3 == 0, V - 1, j % 3 - 1)]
    return torch.stack([rows[i % len(rows)] for i in range(T)]).to(torch.int32).to(DEV)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V,offset", [(1, 0), (5, 1), (200, 3), (1023, 0), (9001, 1), (40000, 0), (70001, 5)])
def test_tokens_close_together(lib, V, offset, dtype):
    _case("crowded", V, offset, dtype)
    T = 6
    z, y = _logits(T, V, dtype, 31, offset=offset), _crowded(T, V, dtype)
    stats = lib.token_scores(z, y, save_stats=True)[4]
    g, gh = torch.linspace(-1, 2, T * 64).view(T, 64).to(DEV), torch.linspace(1, -1, T).to(DEV)
    d = _check_grad(lib, z, y, g, gh, stats, 1.0, dtype)
    a = z.clone()
    assert torch.equal(lib.token_scores_backward(g, gh, a, y, stats, out=a), d)


@pytest.mark.parametrize("V,T", [(33001, 2100), (70001, 1000)])
def test_tokens_close_together_streamed(lib, V, T):
    _case("crowded, streamed", V, T)
    z8, y8 = _logits(6, V, BF, 32), _crowded(6, V, BF)
    n = -(-T // 6)
    z, y = z8.repeat(n, 1)[:T].contiguous(), y8.repeat(n, 1)[:T].contiguous()
    g, gh = torch.ones(T, 64, device=DEV), torch.full((T,), -0.5, device=DEV)
    stats = lib.token_scores(z, y, save_stats=True)[4]
    d = lib.token_scores_backward(g, gh, z, y, stats)
    one = _check_grad(lib, z8, y8, g[:6], gh[:6], stats[:6].contiguous(), 1.0, BF)
    assert torch.equal(d, one.repeat(n, 1)[:T])


def test_the_gradient_of_a_row_of_2_28_words(lib):
    """Equal logits, whose gradient is known: more columns than the work-groups' usual share of a row reaches."""
    V = (1 << 28) + 5000
    _case("one row", V)
    z, y = torch.zeros(1, V, device=DEV), torch.tensor([[0, V - 1, V - 1]], dtype=torch.int32, device=DEV)
    _, H, _, _, stats = lib.token_scores(z, y, save_stats=True)
    assert abs(H.item() - np.log(V)) < 1e-3
    d = lib.token_scores_backward(torch.tensor([[1.0, 2.0, 4.0]], device=DEV), None, z, y, stats, out=z)[0]
    assert abs(d[0].item() - 1) < 1e-6 and abs(d[-1].item() - 6) < 1e-6
    lo, hi = torch.aminmax(d[1:-1])
    assert abs(lo.item() * V / 7 + 1) < 1e-4 and abs(hi.item() * V / 7 + 1) < 1e-4


def test_gradients_past_the_cache_are_streamed(lib):
    _case("streamed")
    T, V, m = 2100, 33001, 2
    z = _logits(8, V, BF, 7).repeat(263, 1)[:T].contiguous()
    y = _tokens(8, V, m, 7).repeat(263, 1)[:T].contiguous()
    g, gh = torch.ones(T, m, device=DEV), torch.full((T,), -0.5, device=DEV)
    stats = lib.token_scores(z, y, save_stats=True)[4]
    d = lib.token_scores_backward(g, gh, z, y, stats)
    one = _check_grad(lib, z[:8], y[:8], g[:8], gh[:8], stats[:8].contiguous(), 1.0, BF)
    assert torch.equal(d, one.repeat(263, 1)[:T])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [300, 1500, 5000, 40000, 140000])
def test_ties(lib, V, dtype):
    # rows of one value, of two, of few distinct ones, signed zeros, and with the best words side by side
    _case("ties", V, dtype)
    z = torch.zeros(9, V)
    z[1, V // 2] = 1.0
    z[2, ::3] = 1.0
    z[3] = torch.arange(V) % 5
    z[4, ::2] = -0.0
    z[5] = -1e30
    z[5, 7] = 3.0
    z[6] = torch.linspace(-8, 8, V)
    z[7] = torch.linspace(8, -8, V)
    z[8, V - 70:] = 2.0
    z = z.to(dtype).to(DEV)
    for n in (1, 20, 64):
        _check(lib, z, None, n, 1.0)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [200, 3000, 40000, 140000])
def test_masked_words(lib, V, dtype):
    # a grammar that leaves three, or one, or all but three words; masks of -inf and of the type's lowest value; rows
    # without a distribution; a masked token's own log-probability
    _case("masked", V, dtype)
    z = _logits(10, V, dtype, 9).clone()
    low = torch.finfo(dtype).min
    inf = float("inf")
    kept = torch.tensor([3, V // 2, V - 1], device=DEV)
    for i, mask in ((0, -inf), (1, low)):
        row = z[i].clone()
        z[i] = mask
        z[i, kept] = row[kept]
    z[2] = -inf
    z[2, V - 2] = 5.0
    z[3, kept] = -inf
    z[4] = -inf
    z[5, 9] = float("nan")
    z[6, 9] = inf
    z[7] = low
    z[8] = torch.finfo(dtype).max
    y = torch.zeros(10, 2, dtype=torch.int32, device=DEV)
    y[:, 0], y[:, 1] = 3, V // 3
    for n in (1, 5, 64):
        out = _check(lib, z, y, n, 1.0)
    ok = [0, 1, 2, 3, 7, 8, 9]
    assert out[2][0, :3].sort().values.tolist() == sorted(kept.tolist()) and (out[2][0, 3:] == -1).all()
    g, gh = torch.linspace(-1, 1, 20).view(10, 2).to(DEV), torch.linspace(1, 2, 10).to(DEV)
    sub = torch.tensor(ok, device=DEV)
    _check_grad(lib, z[sub].contiguous(), y[sub].contiguous(), g[sub].contiguous(), gh[sub].contiguous(),
                out[4][sub].contiguous(), 1.0, dtype)
    d = lib.token_scores_backward(g, gh, z, y, out[4])
    assert torch.isnan(d[4]).all() and torch.isnan(d[5]).all() and torch.isnan(d[6]).all()
    # a row whose coefficients are 0 has no gradient, whatever it holds
    g[4:7], gh[4:7] = 0, 0
    assert not lib.token_scores_backward(g, gh, z, y, out[4])[4:7].any()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("level,tau", [(400.0, 1.0), (-400.0, 1.0), (0.0, 30.0), (1000.0, 0.01), (0.0, 1e-6)])
def test_levels_and_temperatures(lib, level, tau, dtype):
    _case("levels", level, tau, dtype)
    for V in (1000, 40000, 140000):
        z = (_logits(4, V, F32, 3) + level).to(dtype)
        y = _tokens(4, V, 2, 3)
        out = _check(lib, z, y, 8, tau)
        g, gh = torch.linspace(-1, 1, 8).view(4, 2).to(DEV), torch.linspace(1, 2, 4).to(DEV)
        _check_grad(lib, z, y, g, gh, out[4], float(np.float32(tau)), dtype)


def test_peaked_rows_have_little_entropy(lib):
    _case("peaked")
    z = torch.full((3, 32000), -60.0, device=DEV)
    z[0, 5], z[1, 5], z[2, 5] = 60.0, 0.0, -59.0
    out = _check(lib, z, None, 3, 1.0)
    assert (out[1] >= 0).all() and float(out[1][0]) < 1e-6


def test_order_does_not_change_results(lib):
    # the list of the best words fills in any order: the same bits each time, and as two calls on two streams
    _case("repeated")
    z, y = _logits(600, 32000, BF, 13), _tokens(600, 32000, 1, 13)
    want = lib.token_scores(z, y, top=64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            a = lib.token_scores(z, y, top=64)
        b = lib.token_scores(z, y, top=64)
        torch.cuda.synchronize()
        for got in (a, b):
            assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_captured_step(lib):
    _case("captured")
    z, y = _logits(40, 5000, BF, 14).clone(), _tokens(40, 5000, 3, 14)
    g, gh = torch.randn(40, 3, device=DEV), torch.randn(40, device=DEV)

    def step():
        logp, ent, ids, top, stats = lib.token_scores(z, y, top=20, save_stats=True)
        return logp, ent, ids, top, lib.token_scores_backward(g, gh, z, y, stats)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for n in range(4):
        z.copy_(torch.randn(40, 5000, generator=torch.Generator().manual_seed(n)).to(BF))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), n


def test_no_rows(lib):
    z = torch.zeros(0, 100, dtype=BF, device=DEV)
    y = torch.zeros(0, 2, dtype=torch.int32, device=DEV)
    logp, ent, ids, top, stats = lib.token_scores(z, y, top=3, save_stats=True)
    assert logp.shape == (0, 2) and ent.shape == (0,) and ids.shape == (0, 3) and stats.shape == (0, 3)
    assert lib.token_scores_backward(logp, ent, z, y, stats).shape == (0, 100)


def test_past_2_31_elements(lib):
    _case("past 2^31 elements")
    T, V = 66000, 33000
    small, y8 = _logits(8, V, BF, 15), _tokens(8, V, 2, 15)
    z = torch.empty(T, V, dtype=BF, device=DEV)
    z.view(T // 8, 8, V)[:] = small
    y = y8.repeat(T // 8, 1).contiguous()
    out = lib.token_scores(z, y, top=5, save_stats=True)
    want = lib.token_scores(small.repeat(40, 1).contiguous(), y8.repeat(40, 1).contiguous(), top=5, save_stats=True)
    for a, b in zip(out, want):
        assert torch.equal(a[-320:], b) and torch.equal(a[:320], b)
    g, gh = torch.ones(T, 2, device=DEV), torch.ones(T, device=DEV)
    d = lib.token_scores_backward(g, gh, z, y, out[4], out=z)
    assert torch.equal(d[-8:], d[:8]) and torch.equal(d[T // 2 // 8 * 8:][:8], d[:8])
    _check_grad(lib, small, y8, g[:8], gh[:8], out[4][:8].contiguous(), 1.0, BF)
    assert torch.equal(d[:8], lib.token_scores_backward(g[:8], gh[:8], small, y8, out[4][:8].contiguous()))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [2048, 4096, 10000, 40000, 140000])
def test_many_words_of_the_last_value(lib, V, dtype):
    # the n-th best is one of very many equal words: at the row's end, behind better ones, in one lane's pieces alone, one
    # step of the type away from as many others, at both signs; and strong words that all lie in one group
    _case("last value", V, dtype)
    g = torch.Generator().manual_seed(V)
    z = (torch.randn(8, V, generator=g) - 8).to(dtype).float()
    z[0, 3 * V // 4:] = 1.0
    z[1, 3 * V // 4:] = 1.0
    z[1, [5, V // 2, V - 1]] = 2.0
    z[2] = -1.0
    z[2, V // 2:] = -1.0 - torch.finfo(dtype).eps  # the next value down
    z[2, ::97] = -0.5
    z[3, torch.arange(V) // 8 % 64 == 7] = 3.0
    z[4] = torch.where(torch.arange(V) % 2 == 0, 2.0, 2.0 + 2 * torch.finfo(dtype).eps)
    lane = torch.nonzero(torch.arange(V) // 8 % 64 == 9)[:, 0]
    z[5, lane] = torch.linspace(1, 2, len(lane))
    z[6] = -torch.finfo(dtype).max
    z[6, V - 30:] = torch.linspace(0, 1, 30)
    z[7, :V // 2] = 0.0
    z[7, 1:V // 2:2] = -0.0
    z = z.to(dtype).to(DEV)
    for n in (1, 7, 64):
        _check(lib, z, None, n, 1.0)
    # as one of many rows, where other threads have them
    many = z.repeat(40, 1).contiguous()
    a, b = lib.token_scores(many, top=64), lib.token_scores(z, top=64)
    for i in (0, 39):
        assert torch.equal(a[2][8 * i:8 * i + 8], b[2]) and torch.allclose(a[3][8 * i:8 * i + 8], b[3], rtol=0, atol=1e-4)


def test_two_streams_at_once(lib):
    _case("two streams")
    sets = [(_logits(64, 40001, BF, 41), _tokens(64, 40001, 33, 41)), (_logits(64, 33000, F32, 42), _tokens(64, 33000, 2, 42))]

    def call(z, y):
        out = lib.token_scores(z, y, top=20, save_stats=True)
        return *out, lib.token_scores_backward(torch.ones_like(out[0]), torch.full_like(out[1], -0.5), z, y, out[4])

    want = [call(*s) for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                got.append(call(*s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
