"""Every tile of the token-rich kernels by name, whatever the shape's own: forward tiles of 256 x 256, 128 x 256,
128 x 128 and 64 x 128, dX tiles of 256 x 256, 128 x 128, 64 x 128 and 64 x 64 (``QLORA_TILE``).  Each output is the
same sum in the same order, so all give the same bits, and those of the shape's own choice; one of them is compared
with float64."""

import pytest
import torch

from gpu_util import DEV, Layer, bits_host, rel

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# a name that a kernel lacks (the forward's 64 x 64, dX's 128 x 256) leaves the choice to the shape
TILES = ["128", "256", "256x256", "128x256", "128x128", "64x128", "64x64"]


def _layer(lib, ds, k, r, M, nsec=1):
    g = torch.Generator().manual_seed(ds + k + M)
    w = lib.quantize_sections([(torch.randn(ds, k, generator=g) * 0.02).to(DEV) for _ in range(nsec)])
    X, dY = torch.randn(M, k, generator=g).to(BF).to(DEV), torch.randn(M, nsec * ds, generator=g).to(BF).to(DEV)
    A = (torch.randn(nsec * r, k, generator=g) * 0.05).to(BF).to(DEV) if r else None
    B = (torch.randn(nsec * ds, r, generator=g) * 0.05).to(BF).to(DEV) if r else None
    return w, X, dY, A, B


def _all_alike(monkeypatch, step):
    monkeypatch.delenv("QLORA_TILE", raising=False)
    want = [t for t in step() if t is not None]
    for tile in TILES:
        print("tile:", tile, flush=True)
        monkeypatch.setenv("QLORA_TILE", tile)
        got = [t for t in step() if t is not None]
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want)), tile
    return want


# the first three take dX tiles of 64 x 128 by themselves; then odd ends of rows and columns, one K step and many, ranks
# that end inside a load, a column more than a tile has, fewer tokens than any tile
SHAPES = [(80, 576, 8, 2500), (96, 640, 5, 2500), (1040, 4160, 5, 1001), (272, 320, 17, 130), (16, 64, 1, 129),
          (48, 192, 64, 200), (528, 1088, 24, 520), (1040, 2112, 33, 1100), (2064, 448, 0, 300), (304, 64, 8, 4100)]


@pytest.mark.parametrize("d,k,r,M", SHAPES)
def test_every_tile(lib, monkeypatch, d, k, r, M):
    print("case:", d, k, r, M, flush=True)
    w, X, dY, A, B = _layer(lib, d, k, r, M)

    def step():
        Y, T = lib.forward(X, w, A, B, 16.0, save_t=True) if r else (lib.forward(X, w), None)
        return Y, *lib.backward(dY, X, w, A, B, 16.0, T_saved=T)

    _all_alike(monkeypatch, step)


@pytest.mark.parametrize("d,k,r,M", [(80, 576, 8, 2500), (96, 640, 5, 2500), (272, 320, 16, 130), (528, 1088, 33, 520)])
def test_every_tile_under_dropout(lib, monkeypatch, d, k, r, M):
    print("case:", "dropout", d, k, r, M, flush=True)
    w, X, dY, A, B = _layer(lib, d, k, r, M)
    keep = (torch.rand(M, k, generator=torch.Generator().manual_seed(1)) > 0.1).to(torch.uint8).to(DEV)

    def step():
        return lib.forward_dropout(X, w, A, B, 16.0, keep, 0.1), *lib.backward_dropout(dY, X, w, A, B, 16.0, keep, 0.1)

    _all_alike(monkeypatch, step)


@pytest.mark.parametrize("nsec,ds,k,r,M", [(3, 256, 320, 16, 130), (2, 768, 1088, 32, 520), (4, 256, 576, 48, 2500)])
def test_every_tile_of_sections(lib, monkeypatch, nsec, ds, k, r, M):
    print("case:", "sections", nsec, ds, k, r, M, flush=True)
    w, X, dY, A, B = _layer(lib, ds, k, r, M, nsec)

    def step():
        Y, T, ck = lib.forward_checkpoint(X, w, A, B, 16.0)
        return Y, *lib.backward_sections(dY, X, w, A, B, 16.0), *lib.backward_checkpoint(dY, ck, w, A, B, 16.0, T)

    _all_alike(monkeypatch, step)


@pytest.mark.parametrize("tile", ["64x128", "64x64"])
def test_small_tiles_against_the_oracle(lib, monkeypatch, tile):
    print("case:", "oracle", tile, flush=True)
    monkeypatch.setenv("QLORA_TILE", tile)
    L = Layer(lib, 272, 320, 8, 130)
    Y, T = lib.forward(L.X, L.w, L.A, L.B, L.alpha, save_t=True)
    dX, dA, dB = lib.backward(L.dY, L.X, L.w, L.A, L.B, L.alpha, T_saved=T)
    want = L.oracle_bwd()
    assert rel(bits_host(Y), L.oracle_fwd()[0]) <= 1e-2 and rel(bits_host(dX), want[0]) <= 1e-2
    assert rel(bits_host(dA), want[1]) <= 2e-2 and rel(bits_host(dB), want[2]) <= 2e-2
