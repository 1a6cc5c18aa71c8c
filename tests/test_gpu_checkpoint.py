"""GPU parity of the 8-bit activation checkpoint (bit for bit against its
definition) and of the backward that starts from it.

The restored input is bf16, so the backward from a checkpoint has to give the
bits of the ordinary backward on the restored input, with the T that the
forward made of the input itself.  Against float64: U = dY B is rounded to
bf16 (2^-8 of it) after an fp32 sum of d terms, dA = s U^T x^ is an fp32 sum of M
terms and rounded: |d dA| <= s sum_m (|U| 2^-8 + d 2^-24 sum |dY||B|) |x^| +
M 2^-24 s sum |U||x^| + 2^-8 |dA|, element by element.
"""

import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import DEV, Layer, bf16_dev, bits_host
from oracle import checkpoint_oracle as K

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _case(*args):
    print("case:", *args, flush=True)


def _input(M, k, seed):
    """Normal activations with strong channels, zero blocks, ties and the ends of the type's range."""
    r = np.random.Generator(np.random.PCG64(seed))
    x = r.normal(size=(M, k))
    x[:, r.integers(0, k, size=max(1, k // 100))] *= 50.0
    b = O.bf16_rne_bits_from_f64(x).reshape(M, k // 64, 64)
    rows = r.permutation(M)
    extremes = [0.0, 2.0 ** -133, 2.0 ** -130, 2.0 ** -126, 2.0 ** -101, 2.0 ** -100, 2.0 ** -99, 1.0, 254.0,
                3.3895313892515355e38]
    for i, size in enumerate(extremes[:M]):
        block = size * r.uniform(-1, 1, size=64)
        block[5] = size
        block[9] = size / 2      # a tie
        b[rows[i], r.integers(k // 64)] = O.bf16_rne_bits_from_f64(block)
    return b.reshape(M, k)


def _same(got, want):
    """Equal bf16 bits, any NaN for a NaN, and no zero's sign."""
    a, b = O.bf16_bits_to_f64(got), O.bf16_bits_to_f64(want)
    return np.array_equal(a, b, equal_nan=True)


@pytest.mark.parametrize("M,k", [(1, 64), (2, 128), (31, 192), (32, 256), (33, 448), (64, 512), (65, 576), (100, 1088),
                                 (1001, 4160), (4096, 512), (7, 22016)])
def test_save_and_load_bit_for_bit(lib, M, k):
    _case("save", M, k)
    b = _input(M, k, 3 * M + k)
    X = bf16_dev(b)
    ck = lib.checkpoint_save(X)
    codes, a = K.encode(b)
    assert np.array_equal(ck.codes.cpu().numpy(), codes)
    assert np.array_equal(ck.absmax[:, :M].t().double().cpu().numpy(), a)
    assert _same(bits_host(lib.checkpoint_load(ck)), K.decode(codes, a))
    # into given buffers: the same, and no further
    buf = torch.full((M + 1, k), 5, dtype=torch.int8, device=DEV)
    out = lib.Checkpoint(M, k, buf[:M], torch.full_like(ck.absmax, 7.0))
    assert lib.checkpoint_save(X, out=out) is out
    assert torch.equal(out.codes, ck.codes) and torch.equal(out.absmax[:, :M], ck.absmax[:, :M])
    assert torch.all(buf[M] == 5)
    dst = torch.full((M + 1, k), 5.0, dtype=BF, device=DEV)
    lib.checkpoint_load(out, out=dst[:M])
    assert _same(bits_host(dst[:M]), K.decode(codes, a)) and torch.all(dst[M] == 5)


def test_every_pair_of_mantissas(lib):
    # a block's constant and one of its values over all mantissas of bf16 and the exponents in which a code is not 0
    _case("mantissas")
    a = np.arange(128, 256)
    x = np.arange(128, 256)
    blocks = []
    for e in range(0, 9):
        v = np.zeros((128, 128, 64))
        for j in range(2):
            part = np.zeros((128, 64))
            part[:, 0] = a
            rows = np.repeat(part[:, None], 2, axis=1)
            rows[:, 0, 1:] = x[:63] * 2.0 ** -e
            rows[:, 1, 1:] = x[63:126] * 2.0 ** -e
            v[:, :2] = rows
        v[:, 2, 0], v[:, 2, 1:3] = a, x[126:] * 2.0 ** -e
        v[:, :3][np.abs(v[:, :3]) > a[:, None, None]] = 0
        blocks.append(v[:, :3].reshape(-1, 64))
    b = O.bf16_rne_bits_from_f64(np.concatenate(blocks))
    codes, c = K.encode(b)
    ck = lib.checkpoint_save(bf16_dev(b))
    assert np.array_equal(ck.codes.cpu().numpy(), codes)
    assert _same(bits_host(lib.checkpoint_load(ck)), K.decode(codes, c))


def test_every_code(lib):
    _case("codes")
    codes = np.tile(np.arange(-127, 129)[:256].astype(np.int8).reshape(4, 64), (64, 1)).reshape(64, 256)
    a = O.bf16_bits_to_f64(np.random.default_rng(1).integers(0, 0x7F80, size=(64, 4)).astype(np.uint16))
    am = torch.from_numpy(a.T.copy()).to(BF).to(DEV).contiguous()
    ck = lib.Checkpoint(64, 256, torch.from_numpy(codes.copy()).to(DEV), am)
    assert _same(bits_host(lib.checkpoint_load(ck)), K.decode(codes, a))


def test_blocks_without_a_scale(lib):
    _case("non-finite blocks")
    x = np.ones((40, 256))
    x[3, 70], x[3, 130], x[20, 255], x[39, 0] = np.nan, np.inf, -np.inf, np.nan
    X = torch.from_numpy(x).to(BF).to(DEV)
    back = lib.checkpoint_load(lib.checkpoint_save(X)).double().cpu().numpy()
    bad = ~np.isfinite(x).reshape(40, 4, 64).all(axis=2).repeat(64, axis=1)
    assert np.isnan(back[bad]).all() and np.all(back[~bad] == 1)


# (d, k, r, M, nsec): one tile and less, odd tokens and ranks, both strip widths, every number of rank blocks
LAYERS = [(16, 64, 1, 1, 1), (48, 64, 3, 31, 1), (64, 192, 8, 33, 1), (256, 256, 8, 32, 1), (272, 320, 17, 65, 1),
          (1040, 832, 5, 301, 1), (512, 512, 33, 128, 1), (256, 1024, 64, 257, 1), (8192, 8448, 16, 70, 1),
          (8192, 8256, 40, 290, 1), (8192, 8192, 64, 45, 1), (512, 256, 16, 100, 2), (768, 576, 32, 77, 3),
          (1024, 512, 64, 90, 2), (1024, 128, 48, 50, 4)]


def _layer(lib, d, k, r, M, nsec, seed):
    g = torch.Generator().manual_seed(seed)
    ds = d // nsec
    w = lib.quantize_sections([(torch.randn(ds, k, generator=g) * 0.02).to(DEV) for _ in range(nsec)])
    A = (torch.randn(nsec * r, k, generator=g) * k ** -0.5).to(BF).to(DEV)
    B = (torch.randn(d, r, generator=g) * 0.05).to(BF).to(DEV)
    X = bf16_dev(_input(M, k, seed)[:, :])
    X = torch.where(X.float().abs() < 1e30, X, torch.zeros_like(X))  # sums stay finite
    dY = torch.randn(M, d, generator=g).to(BF).to(DEV)
    return w, A, B, X, dY


@pytest.mark.parametrize("d,k,r,M,nsec", LAYERS)
def test_step_is_the_ordinary_one_on_the_restored_input(lib, d, k, r, M, nsec):
    _case("step", d, k, r, M, nsec)
    w, A, B, X, dY = _layer(lib, d, k, r, M, nsec, d + k + r + M)
    alpha = 24.0
    fwd = lib.forward if nsec == 1 else lib.forward_sections
    bwd = lib.backward if nsec == 1 else lib.backward_sections
    Y0, T0 = fwd(X, w, A, B, alpha, save_t=True)
    Y, T, ck = lib.forward_checkpoint(X, w, A, B, alpha)
    assert torch.equal(Y, Y0)
    ldt = -(-M // 64) * 64
    assert torch.equal(T.view(-1, ldt)[:, :M], T0.view(-1, ldt)[:, :M])
    saved = lib.checkpoint_save(X)
    assert torch.equal(ck.codes, saved.codes) and torch.equal(ck.absmax[:, :M], saved.absmax[:, :M])
    Xr = lib.checkpoint_load(ck)
    ck.absmax[:, M:] = float("nan")  # the padding takes no part
    want = bwd(dY, Xr, w, A, B, alpha, T_saved=T)
    got = lib.backward_checkpoint(dY, ck, w, A, B, alpha, T)
    for name, a, b in zip(("dX", "dA", "dB"), got, want):
        assert torch.equal(a, b), name
    no_dx = lib.backward_checkpoint(dY, ck, w, A, B, alpha, T, need_dx=False)
    assert no_dx[0] is None and torch.equal(no_dx[1], got[1]) and torch.equal(no_dx[2], got[2])
    # against float64
    s = float(np.float32(alpha / r))
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    x, g, b, ds = f(Xr), f(dY), f(B), d // nsec
    for p in range(nsec):
        gp, bp = g[:, p * ds:(p + 1) * ds], b[p * ds:(p + 1) * ds]
        U, Uabs = gp @ bp, np.abs(gp) @ np.abs(bp)
        ref = s * (U.T @ x)
        off = s * ((np.abs(U) * 2.0 ** -8 + (d + 8) * 2.0 ** -24 * Uabs).T @ np.abs(x)
                   + (M + 8) * 2.0 ** -24 * (np.abs(U).T @ np.abs(x))) * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(ref)
        assert np.all(np.abs(f(got[1][p * r:(p + 1) * r]) - ref) <= off + 1e-30)


def test_frozen_path_needs_no_checkpoint(lib):
    _case("r = 0")
    w, _, _, X, dY = _layer(lib, 256, 256, 8, 40, 1, 1)
    Y, T, ck = lib.forward_checkpoint(X, w)
    assert T is None and torch.equal(Y, lib.forward(X, w))
    assert torch.equal(ck.codes, lib.checkpoint_save(X).codes)
    dX, dA, dB = lib.backward_checkpoint(dY, ck, w)
    assert dA is None and dB is None and torch.equal(dX, lib.backward(dY, X, w)[0])
    assert torch.equal(dX, lib.backward_checkpoint(dY, None, w)[0])


@pytest.mark.parametrize("d,k,r,M", [(256, 256, 8, 33), (272, 320, 16, 130)])
def test_dropout_from_a_checkpoint(lib, d, k, r, M):
    _case("dropout", d, k, r, M)
    w, A, B, X, dY = _layer(lib, d, k, r, M, 1, 5)
    keep = (torch.rand(M, k, generator=torch.Generator().manual_seed(2)) > 0.1).to(torch.uint8).to(DEV)
    Xd = torch.empty_like(X)
    _, T = lib.forward_dropout(X, w, A, B, 16.0, keep, 0.1, save_t=True, xd_out=Xd)
    ck = lib.checkpoint_save(Xd)
    want = lib.backward_dropout(dY, X, w, A, B, 16.0, keep, 0.1, T_saved=T, Xd_saved=lib.checkpoint_load(ck))
    got = lib.backward_checkpoint(dY, ck, w, A, B, 16.0, T, keep=keep, p=0.1)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_block_without_a_scale_reaches_its_own_columns_only(lib):
    _case("NaN block in the backward")
    w, A, B, X, dY = _layer(lib, 64, 256, 4, 50, 1, 6)
    T = lib.forward(X, w, A, B, 8.0, save_t=True)[1]
    ck = lib.checkpoint_save(X)
    clean = lib.backward_checkpoint(dY, ck, w, A, B, 8.0, T)
    X[49, 130] = float("inf")
    got = lib.backward_checkpoint(dY, lib.checkpoint_save(X), w, A, B, 8.0, T)
    assert torch.isnan(got[1][:, 128:192]).all()
    assert torch.equal(got[1][:, :128], clean[1][:, :128]) and torch.equal(got[1][:, 192:], clean[1][:, 192:])
    assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])


def test_no_tokens(lib):
    _case("M = 0")
    w, A, B, X, dY = _layer(lib, 64, 128, 4, 3, 1, 7)
    Y, T, ck = lib.forward_checkpoint(X[:0], w, A, B, 8.0)
    assert Y.shape == (0, 64) and ck.codes.shape == (0, 128) and lib.checkpoint_load(ck).shape == (0, 128)
    dX, dA, dB = lib.backward_checkpoint(dY[:0], ck, w, A, B, 8.0, T)
    assert dX.shape == (0, 128) and not dA.any() and not dB.any()


def test_refusals_on_the_gpu(lib):
    w, A, B, X, dY = _layer(lib, 64, 128, 4, 3, 1, 8)
    Y, T, ck = lib.forward_checkpoint(X, w, A, B, 8.0)
    bad = [lambda: lib.backward_checkpoint(dY, ck, w, A, B, 8.0),                        # no T
           lambda: lib.backward_checkpoint(dY, None, w, A, B, 8.0, T),
           lambda: lib.backward_checkpoint(dY, ck, w, A, B, 8.0, T[:, :3]),
           lambda: lib.backward_checkpoint(dY[:2], ck, w, A, B, 8.0, T),
           lambda: lib.backward_checkpoint(dY, ck, w, A[:, :64], B, 8.0, T),
           lambda: lib.backward_checkpoint(dY, ck, w, A, B.float(), 8.0, T),
           lambda: lib.backward_checkpoint(dY, ck, w, A, None, 8.0, T),
           lambda: lib.backward_checkpoint(dY, ck, w, A, B, 8.0, T, keep=torch.ones(3, 64, device=DEV)),
           lambda: lib.checkpoint_save(X.float()), lambda: lib.checkpoint_save(X[:, :64]),
           lambda: lib.checkpoint_save(X, out=lib.Checkpoint.empty(4, 128, DEV)),
           lambda: lib.checkpoint_load(ck, out=torch.empty(2, 128, dtype=BF, device=DEV)),
           lambda: lib.forward_checkpoint(X, w, A, B, 8.0, out=torch.empty(3, 32, dtype=BF, device=DEV)),
           lambda: lib.forward_checkpoint(X, w, A, B, 8.0, ck=lib.Checkpoint.empty(3, 192, DEV))]
    for f in bad:
        with pytest.raises(ValueError):
            f()


def test_streams_and_graphs(lib):
    # a step on another stream, and replayed from a graph between eager ones whose inputs change in place
    _case("stream and graph")
    w, A, B, X, dY = _layer(lib, 256, 512, 16, 200, 1, 9)

    def step():
        Y, T, ck = lib.forward_checkpoint(X, w, A, B, 8.0)
        return (Y, ck.codes, lib.checkpoint_load(ck), *lib.backward_checkpoint(dY, ck, w, A, B, 8.0, T))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for n in range(4):
        X.copy_(torch.randn(200, 512, generator=torch.Generator().manual_seed(n)).to(BF))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), n


def test_more_than_2_31_bytes(lib):
    # codes that end just below 2^31, an input of twice that
    _case("largest")
    M, k = 33_554_431, 64
    X = torch.empty(M, k, dtype=BF, device=DEV)
    X.view(-1)[:1 << 20] = torch.randn(1 << 20, device=DEV).to(BF)
    n = 1 << 20
    while n < M * k:  # copies of the first part, each two tokens on
        m = min(n, M * k - n)
        X.view(-1)[n:n + m] = X.view(-1)[:m]
        n += m
    last = torch.randn(100, k, device=DEV).to(BF)
    X[-100:] = last
    ck = lib.checkpoint_save(X)
    small = lib.checkpoint_save(last)
    assert torch.equal(ck.codes[-100:], small.codes) and torch.equal(ck.absmax[:, M - 100:M], small.absmax[:, :100])
    first = lib.checkpoint_save(X[:16384])
    assert torch.equal(ck.codes[16384 * 100:16384 * 101], first.codes)
    back = lib.checkpoint_load(ck)
    assert torch.equal(back[-100:], lib.checkpoint_load(small))
    assert torch.equal(back[16384 * 2000:16384 * 2001], lib.checkpoint_load(first))


def test_many_tokens(lib):
    # 2^30 codes of narrow rows: the reduction's offsets and its last, ragged tokens
    _case("many tokens")
    M, d, k, r = (1 << 24) - 37, 16, 64, 4
    g = torch.Generator().manual_seed(4)
    w = lib.quantize((torch.randn(d, k, generator=g) * 0.02).to(DEV))
    A, B = torch.randn(r, k, generator=g).to(BF).to(DEV), torch.randn(d, r, generator=g).to(BF).to(DEV)
    X = torch.randn(M, k, device=DEV).to(BF)
    dY = torch.randn(M, d, device=DEV).to(BF)
    Y, T, ck = lib.forward_checkpoint(X, w, A, B, 4.0)
    lib.checkpoint_load(ck, out=X)
    want = lib.backward(dY, X, w, A, B, 4.0, T_saved=T, need_dx=False)
    got = lib.backward_checkpoint(dY, ck, w, A, B, 4.0, T, need_dx=False)
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2]) and torch.isfinite(got[1].float()).all()


def test_the_longest_row(lib):
    # a single token of as many columns as there may be: its constants take twice the codes' bytes
    _case("longest row")
    k = (1 << 31) - 64
    X = torch.ones(1, k, dtype=BF, device=DEV)
    last = torch.randn(1, 4096, device=DEV).to(BF)
    X[:, -4096:] = last
    ck = lib.checkpoint_save(X)
    small = lib.checkpoint_save(last)
    assert torch.equal(ck.codes[:, -4096:], small.codes) and torch.equal(ck.absmax[-64:, 0], small.absmax[:, 0])
    assert bool((ck.codes[:, :1 << 20] == 127).all()) and bool((ck.codes[:, (k - 8192) // 64 * 64:-4096] == 127).all())
    X.zero_()
    lib.checkpoint_load(ck, out=X)
    assert torch.equal(X[:, -4096:], lib.checkpoint_load(small)) and bool((X[:, :1 << 20] == 1).all())
