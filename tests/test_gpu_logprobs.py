"""GPU parity of the label log-probabilities, the preference loss and the
policy loss against the float64 reference, at the sizes, strides, masks and
values where they can go wrong.

Tolerances.  u = 2^-24 is fp32's half step.  With t = tau (z - max z) and S
the sum of exp t over V words:

* an exponent is off by at most 4 u |t| (the difference, the product's
  constant twice, the product), so ln S is off by 4 u E_p|t| <= 4 u ln V, as
  E_p|t| = entropy - ln S <= ln V; the sum of at most V/256 + 24 terms in a
  row by (V/256 + 24) u, the hardware's exp2 and the logarithms by 8 u (1 + ln S);
  the label's own term by 3 u |t_y|, the last difference by u |logp|:
  |d logp| <= u (4 ln V + V/256 + 32 + 8 ln V + 3 |t_y| + |logp|) = B.
* p is off by p (6 u |ln p| + B) with p |ln p| <= 1/e, so a gradient
  g tau ([v = y] - p) by |g tau| (3 u + p B) + 4 u |its value|, and its rounding
  to the output's type by half a step, finfo.eps / 2 of its value.
"""

import numpy as np
import pytest
import torch

from gpu_util import DEV
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def _case(*args):
    print("case:", *args, flush=True)


def _logits(T, V, dtype, seed, ld=None, offset=0, std=3.0):
    """T x V logits as a slice of a wider matrix that starts `offset` elements in; labels with uncounted ones."""
    ld = V if ld is None else ld
    g = torch.Generator().manual_seed(seed)
    buf = (torch.randn(T * ld + offset, generator=g) * std).to(dtype).to(DEV)
    z = buf[offset:].view(T, ld)[:, :V]
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    if T > 3:
        y[1::7] = -100
        y[3::11] = V
    return z, y.to(DEV)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _logp_bound(z, y, logp, tau):
    V = z.shape[1]
    ty = np.array([tau * abs(z[i, c] - z[i].max()) if 0 <= c < V and np.isfinite(z[i, c]) else 0.0
                   for i, c in enumerate(y)])
    lv = np.log(V) + 1
    return U * (12 * lv + V / 256 + 32 + 3 * ty + np.where(np.isfinite(logp), np.abs(logp), 0))


def _grad_bound(ref, g, tau, bound, dtype):
    half = torch.finfo(dtype).eps / 2
    gt = np.abs(g * tau)[:, None]
    p = np.minimum(1.0, np.abs(ref) / np.maximum(gt, 1e-300) + (np.abs(ref) > 0.5 * gt))
    return gt * (3 * U + p * bound[:, None]) + (4 * U + half) * np.abs(ref) + 1e-37


SIZES = [(1, 1), (1, 2), (2, 7), (3, 8), (5, 9), (33, 200), (4, 255), (9, 2048), (7, 2049), (6, 4099), (5, 8191),
         (4, 16385), (3, 32000), (3, 32769), (2, 50021), (2, 65537), (2, 131072), (2, 131077), (1, 262147)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,V", SIZES)
def test_logprobs_and_gradient_parity(lib, T, V, dtype):
    _case("logprobs", T, V, dtype)
    tau = 1.0 if V % 2 else 0.75
    z, y = _logits(T, V, dtype, 11 + V)
    logp, stats = lib.token_logprobs(z, y, inv_temperature=tau, save_stats=True)
    zh, yh = _f64(z), y.cpu().numpy()
    ref = S.label_logprobs(zh, yh, tau)
    bound = _logp_bound(zh, yh, ref, tau)
    assert np.all(np.abs(_f64(logp) - ref) <= bound)
    assert np.array_equal(_f64(lib.token_logprobs(z, y, inv_temperature=tau)), _f64(logp))
    g = torch.randn(T, generator=torch.Generator().manual_seed(V)).to(DEV)
    dz = lib.token_logprobs_backward(g, z, y, stats, inv_temperature=tau)
    assert dz.shape == z.shape and dz.dtype == dtype
    want = S.label_logprobs_grad(zh, yh, _f64(g), tau)
    assert np.all(np.abs(_f64(dz) - want) <= _grad_bound(want, _f64(g), tau, bound, dtype))


# (ld, offset of the first element): odd strides, odd starts, a padded head
LAYOUTS = [(1000, 1), (1001, 0), (1003, 5), (1008, 0), (1024, 3), (4000, 7)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("ld,offset", LAYOUTS)
def test_strides_and_starts(lib, ld, offset, dtype):
    # any layout is within the bounds (pieces are cut at 16-byte boundaries, so
    # a row's sum has another order where it starts elsewhere); an output's
    # layout does not change a bit; the whole stride of the gradient's rows is
    # written, nothing before or behind it
    _case("strides", ld, offset, dtype)
    T, V = 21, 1000
    z, y = _logits(T, V, dtype, 5, ld, offset)
    logp, stats = lib.token_logprobs(z, y, save_stats=True)
    zh, yh = _f64(z), y.cpu().numpy()
    ref = S.label_logprobs(zh, yh)
    bound = _logp_bound(zh, yh, ref, 1.0)
    assert np.all(np.abs(_f64(logp) - ref) <= bound)
    g = torch.linspace(-1, 1, T).to(DEV)
    g[4] = 0
    want = lib.token_logprobs_backward(g, z, y, stats)
    ref = S.label_logprobs_grad(zh, yh, _f64(g))
    assert np.all(np.abs(_f64(want) - ref) <= _grad_bound(ref, _f64(g), 1.0, bound, dtype))
    buf = torch.full((T * ld + offset + 64,), 7.0, dtype=dtype, device=DEV)
    out = buf[offset:offset + T * ld].view(T, ld)
    got = lib.token_logprobs_backward(g, z, y, stats, out=out[:, :V])
    assert torch.equal(got, want) and torch.equal(out[:, :V], want)
    assert torch.all(out[:, V:] == 0)
    assert torch.all(buf[:offset] == 7) and torch.all(buf[offset + T * ld:] == 7)
    adv = torch.linspace(-2, 2, T).to(DEV)
    l0, k0, p0, d0 = lib.policy_loss(z, y, adv)
    assert torch.equal(p0, logp)
    out.fill_(7.0)
    l1, k1, p1, d1 = lib.policy_loss(z, y, adv, out=out[:, :V])
    assert torch.equal(l0, l1) and torch.equal(p0, p1) and torch.equal(d0, d1) and torch.all(out[:, V:] == 0)
    assert torch.all(buf[:offset] == 7) and torch.all(buf[offset + T * ld:] == 7)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [1000, 32000, 70001, 300000])
def test_in_place(lib, V, dtype):
    _case("in place", V, dtype)
    T = 9
    z, y = _logits(T, V, dtype, 6)
    adv = torch.linspace(-2, 2, T).to(DEV)
    logp, stats = lib.token_logprobs(z, y, save_stats=True)
    want = lib.token_logprobs_backward(adv, z, y, stats)
    a, b = z.clone(), z.clone()
    assert lib.token_logprobs_backward(adv, a, y, stats, out=a) is a
    assert torch.equal(a, want)
    loss, _, lp, dz = lib.policy_loss(z, y, adv)
    loss1, _, lp1, dz1 = lib.policy_loss(b, y, adv, out=b)
    assert torch.equal(dz1, dz) and torch.equal(loss, loss1) and torch.equal(lp, lp1) and torch.equal(lp, logp)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [37, 5000, 40000, 140000])
def test_masked_and_extreme_values(lib, V, dtype):
    _case("extreme", V, dtype)
    inf, low = float("inf"), torch.finfo(dtype).min
    z, _ = _logits(10, V, dtype, 8)
    y = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, -100, V], dtype=torch.int32, device=DEV)
    z[0, 1::2] = -inf               # masked words
    z[1, 1:] = -inf                 # the label is masked too (and all but one word): logp = -inf
    z[2, :] = low                   # nothing but the type's lowest value: uniform
    z[3, :] = -inf                  # nothing left: NaN
    z[4, V - 1] = float("nan")
    z[5, V // 2] = inf
    z[6, :] = -inf
    z[6, 6] = low                   # one word left, at the lowest value: certain
    z[7, :] *= 1000                 # one word takes it all
    z[8, :] = float("nan")          # not counted: its logits are not read
    z[9, :] = float("nan")
    for tau in (1.0, 2.0):
        logp, stats = lib.token_logprobs(z, y, inv_temperature=tau, save_stats=True)
        got = _f64(logp)
        zh, yh = _f64(z), y.cpu().numpy()
        ref = S.label_logprobs(zh[[0, 7]], yh[[0, 7]], tau)
        tol = _logp_bound(zh[[0, 7]], yh[[0, 7]], ref, tau)
        assert np.all(np.abs(got[[0, 7]] - ref) <= tol)
        assert got[1] == -np.inf
        assert abs(got[2] + np.log(V)) <= U * (V / 256 + 32) * 12
        assert np.all(np.isnan(got[[3, 4, 5]])) and got[6] == 0 and got[8] == 0 and got[9] == 0
        g = torch.ones(10, device=DEV)
        dz = _f64(lib.token_logprobs_backward(g, z, y, stats, inv_temperature=tau))
        want = S.label_logprobs_grad(zh[[0, 2, 7]], yh[[0, 2, 7]], np.ones(3), tau)
        bound = np.concatenate([tol[:1], [U * (V / 256 + 32) * 12], tol[1:]])
        assert np.all(np.abs(dz[[0, 2, 7]] - want) <= _grad_bound(want, np.ones(3), tau, bound, dtype))
        assert dz[1, 1] == tau and dz[1, 0] == -tau      # IEEE: p of the one word left is 1
        assert np.all(dz[6] == 0) and np.all(dz[8:] == 0)
        g.zero_()                                        # no gradient wanted: zeros whatever the logits are
        assert torch.all(lib.token_logprobs_backward(g, z, y, stats, inv_temperature=tau) == 0)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 5000, 30000, 150000])
@pytest.mark.parametrize("size,tau", [(1e6, 1.0), (3e8, 1.0), (1e25, 1.0), (1e3, 1e9), (1.0, 1e12), (1e30, 1e30),
                                      (1e6, 1e-6), (1.0, 1e-30), (1.0, 3.3e38), (1.0, 1e-40)])
def test_large_logits_and_temperatures(lib, V, dtype, size, tau):
    # exponents far past 2^20, where the maximum's own rounding is a large
    # exponent; a maximum that the top few share
    _case("large", V, dtype, size, tau)
    z, _ = _logits(4, V, dtype, 3)
    z[1] = z[1].abs() + 1
    z[3] = 1
    z[3, : V // 2] = 1 - 2.0 ** -7
    z = (z.double() * size).to(dtype)
    z[0, 5:9] = z[0].max()
    y = torch.tensor([6, 3, V - 1, 1], dtype=torch.int32, device=DEV)
    tau = float(np.float32(tau))
    logp, stats = lib.token_logprobs(z, y, inv_temperature=tau, save_stats=True)
    zh, yh = _f64(z), y.cpu().numpy()
    with np.errstate(over="ignore"):
        ref = S.label_logprobs(zh, yh, tau)
        ref = np.where(np.abs(ref) > 3.4e38, -np.inf, ref)
    got = _f64(logp)
    ok = np.isfinite(ref)
    assert np.array_equal(got[~ok], ref[~ok])
    tol = _logp_bound(zh[ok], yh[ok], ref[ok], tau)
    assert np.all(np.abs(got[ok] - ref[ok]) <= tol)
    g = torch.linspace(0.5, 1, 4).to(DEV)
    dz = _f64(lib.token_logprobs_backward(g, z, y, stats, inv_temperature=tau))
    want = S.label_logprobs_grad(zh, yh, _f64(g), tau)
    keep = ok & (np.abs(want).max(1) < 1e38)
    bound = np.full(int(keep.sum()), U * (12 * (np.log(V) + 1) + V / 256 + 32))   # of ln S alone
    assert np.all(np.abs(dz[keep] - want[keep]) <= _grad_bound(want[keep], _f64(g)[keep], tau, bound, dtype))
    if tau == 1.0:
        pol = lib.policy_loss(z, y, torch.ones(4, device=DEV))
        assert torch.equal(pol[2], logp)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_a_single_token_of_a_padded_head(lib, dtype):
    # one row: the gradient's padding is written as for many
    z, y = _logits(1, 1000, dtype, 4, ld=1024)
    logp, stats = lib.token_logprobs(z, y, save_stats=True)
    dY = torch.full((1, 1024), 3.0, dtype=dtype, device=DEV)
    d = lib.token_logprobs_backward(torch.ones(1, device=DEV), z, y, stats, out=dY[:, :1000])
    want = lib.token_logprobs_backward(torch.ones(1, device=DEV), z.contiguous(), y, stats)
    assert torch.equal(dY[:, :1000], want) and torch.all(dY[:, 1000:] == 0) and torch.equal(d, want)
    dY.fill_(3.0)
    lib.policy_loss(z, y, torch.ones(1, device=DEV), out=dY[:, :1000])
    assert torch.all(dY[:, 1000:] == 0)
    tight = torch.full((1002,), 3.0, dtype=dtype, device=DEV)
    lib.token_logprobs_backward(torch.ones(1, device=DEV), z, y, stats, out=tight[:1000].view(1, 1000))
    assert torch.equal(tight[:1000], want[0]) and torch.all(tight[1000:] == 3)


def test_more_than_2_31_elements(lib):
    _case("2^31 elements")
    T, V = 16500, 131072
    z = torch.zeros(T, V, dtype=BF, device=DEV)
    rows = torch.tensor([0, 8191, 16383, 16384, T - 1], device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    z[rows] = torch.randn(5, V, device=DEV, generator=g).to(BF)
    y = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    y[rows] = torch.tensor([0, 5, V - 1, 77, 1234], dtype=torch.int32, device=DEV)
    logp, stats = lib.token_logprobs(z, y, save_stats=True)
    some = z[rows].contiguous()
    assert torch.equal(logp[rows], lib.token_logprobs(some, y[rows].contiguous()))
    d = torch.full((T,), 0.5, device=DEV)
    want = lib.token_logprobs_backward(d[:5].contiguous(), some, y[rows].contiguous(), stats[rows].contiguous())
    got = lib.token_logprobs_backward(d, z, y, stats, out=z)
    assert torch.equal(got[rows], want)
    assert int((got[:8191] != 0).any(1).sum()) == 1 and int((got != 0).any(1).sum()) == 5


def test_no_tokens(lib):
    z = torch.zeros(0, 50, device=DEV)
    y = torch.zeros(0, dtype=torch.int32, device=DEV)
    logp, stats = lib.token_logprobs(z, y, save_stats=True)
    assert logp.shape == (0,) and lib.token_logprobs_backward(logp, z, y, stats).shape == (0, 50)
    assert all(t.shape[0] == 0 for t in lib.policy_loss(z, y, logp))
    cu = torch.zeros(5, dtype=torch.int32, device=DEV)
    loss, reward, d = lib.preference_loss(logp, y, 50, cu, 0.1)
    assert np.allclose(_f64(loss), np.log(2), atol=1e-7) and torch.all(reward == 0) and d.shape == (0,)
    loss, reward, d = lib.preference_loss(torch.ones(3, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV), 5,
                                          cu[:1], 0.1)
    assert loss.shape == (0,) and torch.all(d == 0)


# ------------------------------------------------------- preference loss --
# Given log-probabilities, everything is fp64 and rounded once to fp32: half a
# step, and the inputs' cancellation in fp64 (1e-12).

@pytest.mark.parametrize("kind,average,smooth,margin", [
    ("sigmoid", False, 0.0, 0.0), ("sigmoid", False, 0.1, 0.0), ("sigmoid", True, 0.5, 0.3), ("hinge", False, 0.0, 0.0),
    ("hinge", True, 0.0, -0.2), ("squared", True, 0.0, 0.0), ("squared", False, 0.0, 0.1)])
@pytest.mark.parametrize("with_ref", [False, True])
def test_preference_parity(lib, kind, average, smooth, margin, with_ref):
    _case("preference", kind, average, smooth, margin, with_ref)
    r = np.random.Generator(np.random.PCG64(9))
    cu = [2, 2, 3, 40, 41, 700, 1000, 3000, 3300]       # an empty sequence, one token, uneven ones; tokens outside
    T, P, V = 3310, 4, 50
    logp = (-3 * r.random(T)).astype(np.float32)
    ref = (logp + 0.3 * r.normal(size=T)).astype(np.float32) if with_ref else None
    y = r.integers(-1, V + 1, T).astype(np.int32)
    w = np.array([0.25, 0.0, 1.5, -1.0], np.float32)
    dev = lambda a: None if a is None else torch.from_numpy(np.asarray(a)).to(DEV)  # noqa: E731
    args = dict(kind=kind, average=average, label_smoothing=smooth, margin=margin)
    loss, reward, d = lib.preference_loss(dev(logp), dev(y), V, dev(np.array(cu, np.int32)), 0.1, ref_logp=dev(ref),
                                          weight=dev(w), **args)
    beta, smooth, margin = np.float32(0.1), np.float32(smooth), np.float32(margin)
    want = S.preference(logp, y, V, cu, float(beta), ref, kind, average, float(smooth), float(margin), w)
    for got, ref64 in zip((loss, reward, d), want):
        assert np.all(np.abs(_f64(got) - ref64) <= U * np.abs(ref64) + 1e-10 * (np.abs(ref64) + 1e-3))
    only = lib.preference_loss(dev(logp), dev(y), V, dev(np.array(cu, np.int32)), 0.1, ref_logp=dev(ref),
                               need_grad=False, **args)
    assert only[2] is None and torch.equal(only[0], loss) and torch.equal(only[1], reward)


def test_preference_of_many_pairs_and_one_long_one(lib):
    _case("preference sizes")
    r = np.random.Generator(np.random.PCG64(10))
    for P, T in ((300, 5000), (1, 40001)):
        cu = np.concatenate([[0], np.sort(r.integers(0, T, 2 * P - 1)), [T]]).astype(np.int32)
        logp = (-2 * r.random(T)).astype(np.float32)
        y = np.where(r.random(T) < 0.2, -100, 3).astype(np.int32)
        loss, reward, d = lib.preference_loss(*(torch.from_numpy(a).to(DEV) for a in (logp, y)), 7,
                                              torch.from_numpy(cu).to(DEV), 0.05)
        for got, ref in zip((loss, reward, d), S.preference(logp, y, 7, cu, float(np.float32(0.05)))):
            assert np.all(np.abs(_f64(got) - ref) <= U * np.abs(ref) + 1e-10 * (np.abs(ref) + 1e-3))


def test_preference_of_extreme_margins(lib):
    # one side certain: the loss is the margin or 0 and no NaN comes of it; a
    # chosen sequence that cannot be (-inf) has an infinite loss
    logp = torch.tensor([-1e4, -1.0, -1.0, -1e4, -float("inf"), -1.0], device=DEV)
    y = torch.zeros(6, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 1, 2, 2, 3, 4, 4], dtype=torch.int32, device=DEV)
    loss, reward, d = lib.preference_loss(logp, y, 1, cu, 1.0)
    assert loss.tolist()[:2] == [9999.0, 0.0] and d.tolist()[:4] == [-1.0, 0.0, 1.0, 0.0]
    cu = torch.tensor([4, 5, 6], dtype=torch.int32, device=DEV)
    loss, reward, d = lib.preference_loss(logp, y, 1, cu, 1.0)
    assert loss.item() == float("inf") and d.tolist() == [0, 0, 0, 0, -1.0, 1.0]


def test_a_pair_of_weight_zero_has_no_gradient(lib):
    logp = torch.tensor([-float("inf"), -1.0, -1.0, -2.0], device=DEV)
    y = torch.zeros(4, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32, device=DEV)
    for kind in ("sigmoid", "hinge", "squared"):
        loss, _, d = lib.preference_loss(logp, y, 1, cu, 0.5, kind=kind, weight=torch.tensor([0.0, 1.0], device=DEV))
        assert loss[0] == float("inf") and d[0] == 0 and d[2] == 0 and torch.isfinite(d).all()


def test_a_label_of_probability_zero_has_infinite_kl(lib):
    z = torch.zeros(1, 9, device=DEV)
    z[0, 3] = -float("inf")
    y = torch.tensor([3], dtype=torch.int32, device=DEV)
    loss, kl, logp, _ = lib.policy_loss(z, y, torch.ones(1, device=DEV), old_logp=torch.full((1,), -2.0, device=DEV),
                                        ref_logp=torch.full((1,), -2.0, device=DEV), kl_coef=0.1)
    assert kl.item() == float("inf") and loss.item() == float("inf") and logp.item() == -float("inf")


def test_offsets_out_of_range_are_clamped(lib):
    logp = -torch.ones(10, device=DEV)
    y = torch.zeros(10, dtype=torch.int32, device=DEV)
    cu = torch.tensor([-5, 4, 2_000_000_000], dtype=torch.int32, device=DEV)
    loss, reward, d = lib.preference_loss(logp, y, 1, cu, 0.1)
    want = S.preference(-np.ones(10), [0] * 10, 1, [0, 4, 10], float(np.float32(0.1)))
    assert np.allclose(_f64(reward), want[1], rtol=1e-7) and np.allclose(_f64(d), want[2], rtol=1e-7)


# ----------------------------------------------------------- policy loss --

@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(1, 5), (40, 300), (65, 4099), (17, 32000), (5, 70001), (3, 140000)])
@pytest.mark.parametrize("full", [False, True])
def test_policy_parity(lib, T, V, dtype, full):
    _case("policy", T, V, dtype, full)
    tau = 1.25 if full else 1.0
    z, y = _logits(T, V, dtype, 21 + V)
    zh, yh = _f64(z), y.cpu().numpy()
    lp = S.label_logprobs(zh, yh, tau)
    bound = _logp_bound(zh, yh, lp, tau)
    r = np.random.Generator(np.random.PCG64(T + V))
    adv = r.normal(size=T).astype(np.float32)
    old = ref = w = None
    if full:
        off = 0.3 * r.normal(size=T)   # no ratio within reach of an error of the clip's edges
        for edge in (np.log(0.9), np.log(1.3)):
            off = np.where(np.abs(off - edge) < 0.01, off + 0.02, off)
        old, ref = ((lp - off).astype(np.float32), (lp + 0.3 * r.normal(size=T)).astype(np.float32))
        w = r.random(T).astype(np.float32)
        w[:1] = 0
    dev = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
    loss, kl, logp, dz = lib.policy_loss(z, y, dev(adv), dev(old), dev(ref), dev(w), clip_low=0.1, clip_high=0.3,
                                         kl_coef=0.2 if full else 0.0, inv_temperature=tau)
    assert np.all(np.abs(_f64(logp) - lp) <= bound)
    assert torch.equal(logp, lib.token_logprobs(z, y, inv_temperature=tau))
    wl, wk, wg = S.policy(lp, yh, V, adv.astype(np.float64), old, ref, w, float(np.float32(0.1)),
                          float(np.float32(0.3)), float(np.float32(0.2)) if full else 0.0)
    # the ratio and the KL term's exponential are off by the log-probability's
    # error, relative, and some steps of their own
    c = (yh >= 0) & (yh < V)
    e = bound + 8 * U + U * np.abs(lp)
    ratio = np.where(c, np.exp(lp - old) if full else 1.0, 0)
    ek = np.where(c, np.exp(ref - lp) if full else 0.0, 0)
    dl = ratio * np.abs(adv) * e + 4 * U * np.abs(wl)
    dk = (ek + 1) * e * 2
    assert np.all(np.abs(_f64(kl) - wk) <= dk)
    assert np.all(np.abs(_f64(loss) - wl) <= dl + 0.2 * dk)
    dg = (ratio * np.abs(adv) * e + 0.2 * dk + 4 * U * (np.abs(adv) * ratio + ek)) * (1 if w is None else w)
    want = S.label_logprobs_grad(zh, yh, wg, tau)
    unit = S.label_logprobs_grad(zh, yh, np.ones(T), tau)
    assert np.all(np.abs(_f64(dz) - want) <= _grad_bound(want, wg, tau, bound, dtype) * 1.001
                  + np.abs(unit) * (dg * (1 + torch.finfo(dtype).eps))[:, None])
    again = lib.policy_loss(z, y, dev(adv), dev(old), dev(ref), dev(w), clip_low=0.1, clip_high=0.3,
                            kl_coef=0.2 if full else 0.0, inv_temperature=tau, need_grad=False)
    assert again[3] is None and all(torch.equal(a, b) for a, b in zip(again[:3], (loss, kl, logp)))


def test_policy_without_weight_leaves_nan_rows_out(lib):
    # a zero weight takes a token's gradient out, whatever its logits hold
    z, y = _logits(6, 3000, F32, 2)
    y[:] = 1
    z[2] = float("nan")
    w = torch.tensor([1, 1, 0, 1, 0, 1.0], device=DEV)
    loss, _, _, dz = lib.policy_loss(z, y, torch.ones(6, device=DEV), weight=w)
    assert torch.isnan(loss[2]) and torch.all(dz[[2, 4]] == 0) and torch.isfinite(dz).all()


# ---------------------------------------------- streams, graphs, repeats --

def test_another_stream_and_repeats(lib):
    _case("stream")
    z, y = _logits(300, 32000, BF, 1)
    g = torch.linspace(-1, 1, 300).to(DEV)
    logp, stats = lib.token_logprobs(z, y, save_stats=True)
    dz = lib.token_logprobs_backward(g, z, y, stats)
    pol = lib.policy_loss(z, y, g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(3):
            logp1, stats1 = lib.token_logprobs(z, y, save_stats=True)
            dz1 = lib.token_logprobs_backward(g, z, y, stats1)
            pol1 = lib.policy_loss(z, y, g)
    side.synchronize()
    assert torch.equal(logp, logp1) and torch.equal(stats, stats1) and torch.equal(dz, dz1)
    assert all(torch.equal(a, b) for a, b in zip(pol, pol1))


def test_captured_step_replays(lib):
    # forward, loss and backward captured once; two graphs of the same calls
    # share nothing, and every replay follows the logits it finds
    _case("graph")
    T, V = 128, 5001
    z, y = _logits(T, V, BF, 31)
    other, _ = _logits(T, V, BF, 32)
    first = z.clone()
    cu = torch.tensor([0, 30, 64, 100, 128], dtype=torch.int32, device=DEV)
    adv = torch.linspace(-1, 1, T).to(DEV)

    def step():
        logp, stats = lib.token_logprobs(z, y, save_stats=True)
        loss, reward, d = lib.preference_loss(logp, y, V, cu, 0.1)
        return (loss, reward, lib.token_logprobs_backward(d, z, y, stats)) + lib.policy_loss(z, y, adv)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step())
    for rep in range(4):
        z.copy_(first if rep % 2 == 0 else other)
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graphs[rep % 2].replay()
        graphs[1 - rep % 2].replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, want)), rep


@pytest.mark.parametrize("tau", [0.6934478282928467, 0.6936106085777283])
@pytest.mark.parametrize("T,V,dtype", [(4096, 8191, F32), (4096, 70001, BF)], ids=["f32", "bf16"])
def test_logprobs_do_not_drift(lib, T, V, dtype, tau):
    # temperatures whose scale tau log2 e rounds by most, 2^-24 of it, either way: exponents taken with it alone put
    # ln S off by 2^-24 E_p|t|, 1.3e-7 here, the same way in every token.  Of the mean over T tokens are left the
    # results' roundings (half steps of 2^-21 for -16 < logp < -8, 2^-21 / sqrt 3 a token, six standard deviations) and of the
    # hardware's exp2 as much as half a step one way.
    _case("drift", T, V, dtype, tau)
    g = torch.Generator(device=DEV).manual_seed(V)
    z = torch.randn(T, V, device=DEV, generator=g).to(dtype)
    y = torch.randint(0, V, (T,), device=DEV, generator=g, dtype=torch.int32)
    logp = lib.token_logprobs(z, y, tau)
    want = torch.cat([(r.double() * tau).log_softmax(1)[torch.arange(len(r), device=DEV), i.long()]
                      for r, i in zip(z.split(256), y.split(256))])
    assert abs((logp.double() - want).mean().item()) <= U + 6 * 2.0 ** -21 / (3 * T) ** 0.5


# a row in one wave, in 256, 512 and 1024 threads' registers of each width, and in pieces
FORMS = [(BF, v) for v in (2001, 4001, 8150, 14001, 20009, 24500, 32011, 40007, 48011, 65530, 70001, 98000, 131071,
                           140000)] + [(F32, v) for v in (1003, 12003, 20011, 32000, 48011, 65535, 70001)]


@pytest.mark.parametrize("dtype,V", FORMS, ids=lambda x: str(x).split(".")[-1])
def test_every_form_of_a_row(lib, dtype, V):
    # more rows than a CU has to itself, with a policy of its own (ratio 1: the
    # gradient of -A r is -A) beside the log-probabilities; in place as well
    _case("forms", dtype, V)
    T, tau = 261, 0.8
    g = torch.Generator(device=DEV).manual_seed(V)
    z = (2 * torch.randn(T, V, device=DEV, generator=g)).to(dtype)
    z[7, 5:] = -float("inf")
    y = torch.randint(0, V, (T,), device=DEV, generator=g, dtype=torch.int32)
    y[::9], y[1], y[2], y[7] = -1, 0, V - 1, 3
    adv = torch.randn(T, device=DEV, generator=g)
    logp, stats = lib.token_logprobs(z, y, tau, save_stats=True)
    dz = lib.token_logprobs_backward(adv, z, y, stats, tau)
    loss, _, plogp, pdz = lib.policy_loss(z, y, -adv, inv_temperature=tau)
    zz = z.clone()
    assert torch.equal(lib.token_logprobs_backward(adv, zz, y, stats, tau, out=zz), dz)
    zz.copy_(z)
    assert torch.equal(lib.policy_loss(zz, y, -adv, inv_temperature=tau, out=zz)[3], pdz)
    tau = float(np.float32(tau))
    for r in range(0, T, 29):
        t = tau * (z[r:r + 29].double() - z[r:r + 29].double().amax(1, keepdim=True))
        yy = y[r:r + 29].long()
        c = yy >= 0
        ty = t.gather(1, yy.clamp(min=0)[:, None])[:, 0]
        want = torch.where(c, ty - t.logsumexp(1), 0)
        bound = U * (12 * (np.log(V) + 1) + V / 256 + 32 + 3 * ty.abs() + want.abs())
        p = t.softmax(1)
        onehot = torch.zeros_like(p).scatter_(1, yy.clamp(min=0)[:, None], 1.0)
        a = adv[r:r + 29].double()
        dwant = (a * tau * c)[:, None] * (onehot - p)
        half = torch.finfo(dtype).eps / 2
        dbound = (a.abs() * tau)[:, None] * (3 * U + p * bound[:, None]) + (4 * U + half) * dwant.abs() + 1e-37
        for lp, d in ((logp, dz), (plogp, pdz)):
            assert ((lp[r:r + 29].double() - want).abs() <= bound).all()
            assert ((d[r:r + 29].double() - dwant).abs() <= dbound).all()
    assert torch.equal(loss, torch.where(y >= 0, adv, 0))


def test_more_rows_than_a_launch_takes(lib):
    _case("2^20 + 37 rows")
    T, cut = (1 << 20) + 37, 1 << 20
    g = torch.Generator(device=DEV).manual_seed(1)
    z = torch.randn(T, 9, device=DEV, generator=g).bfloat16()
    y = torch.randint(-1, 9, (T,), device=DEV, generator=g, dtype=torch.int32)
    adv = torch.randn(T, device=DEV, generator=g)

    def calls(z, y, adv):
        logp, stats = lib.token_logprobs(z, y, save_stats=True)
        return (logp, stats, lib.token_logprobs_backward(adv, z, y, stats)) + lib.policy_loss(z, y, adv)

    for got, a, b in zip(calls(z, y, adv), calls(z[:cut], y[:cut], adv[:cut]),
                         calls(z[cut:].clone(), y[cut:].clone(), adv[cut:].clone())):
        assert torch.equal(got[:cut], a) and torch.equal(got[cut:], b)


def test_logits_past_4_gib(lib):
    # element offsets past 2^31, byte offsets past 2^32: the last rows give what they give alone
    T, V = 17000, 131072
    _case("large offsets", T, V)
    z = torch.empty(T, V, dtype=BF, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    z[-3:] = torch.randn(3, V, device=DEV, generator=g).to(BF)
    y = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    y[-3:] = torch.tensor([5, V - 1, 77777], dtype=torch.int32, device=DEV)
    adv = torch.ones(T, device=DEV)
    few = z[-3:].clone()
    logp, stats = lib.token_logprobs(z, y, save_stats=True)
    flogp, fstats = lib.token_logprobs(few, y[-3:].clone(), save_stats=True)
    assert torch.equal(logp[-3:], flogp) and torch.equal(stats[-3:], fstats) and torch.all(logp[:-3] == 0)
    assert torch.isfinite(flogp).all()
    dz = lib.token_logprobs_backward(adv, z, y, stats)
    assert torch.equal(dz[-3:], lib.token_logprobs_backward(adv[-3:], few, y[-3:].clone(), fstats))
    assert not dz[:-3].any()
    pdz = lib.policy_loss(z, y, adv, out=dz)[3]
    assert torch.equal(pdz[-3:], lib.policy_loss(few, y[-3:].clone(), adv[-3:])[3]) and not pdz[:-3].any()
