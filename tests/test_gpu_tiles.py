"""The token-rich kernels of shapes that fill no 256-wide tile: the sizes of
their tiles differ with the number of them, the bits do not (each output is the
same sum in the same order).  ``QLORA_TILE=128`` is the one tile of 128 rows."""

import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# (d, k, r, M): forward tiles of 64 and 128 rows by 128 columns, 128 by 256; dX tiles of 64 x 64, 64 x 128, 128 x 128
SHAPES = [(272, 320, 8, 65), (272, 320, 5, 127), (16, 192, 16, 130), (4992, 448, 8, 400), (528, 1088, 24, 520),
          (1040, 2112, 64, 1100), (4112, 4160, 16, 70), (10960, 64, 3, 257), (304, 64, 0, 4100), (144, 4160, 33, 1001)]


def _layer(lib, d, k, r, M):
    g = torch.Generator().manual_seed(d + k + M)
    w = lib.quantize((torch.randn(d, k, generator=g) * 0.02).to(DEV))
    X, dY = torch.randn(M, k, generator=g).to(BF).to(DEV), torch.randn(M, d, generator=g).to(BF).to(DEV)
    A = (torch.randn(r, k, generator=g) * 0.05).to(BF).to(DEV) if r else None
    B = (torch.randn(d, r, generator=g) * 0.05).to(BF).to(DEV) if r else None
    return w, X, dY, A, B


@pytest.mark.parametrize("d,k,r,M", SHAPES)
def test_every_tile_gives_the_same_bits(lib, monkeypatch, d, k, r, M):
    print("case:", d, k, r, M, flush=True)
    w, X, dY, A, B = _layer(lib, d, k, r, M)

    def step():
        Y, T = lib.forward(X, w, A, B, 16.0, save_t=True) if r else (lib.forward(X, w), None)
        return Y, *[t for t in lib.backward(dY, X, w, A, B, 16.0, T_saved=T) if t is not None]

    got = step()
    monkeypatch.setenv("QLORA_TILE", "128")
    want = step()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("d,k,r,M", [(272, 320, 8, 130), (528, 1088, 24, 520), (1040, 2112, 16, 1100)])
def test_every_tile_drops_the_same(lib, monkeypatch, d, k, r, M):
    print("case:", "dropout", d, k, r, M, flush=True)
    w, X, dY, A, B = _layer(lib, d, k, r, M)
    keep = (torch.rand(M, k, generator=torch.Generator().manual_seed(1)) > 0.1).to(torch.uint8).to(DEV)

    def step():
        return lib.forward_dropout(X, w, A, B, 16.0, keep, 0.1), *lib.backward_dropout(dY, X, w, A, B, 16.0, keep, 0.1)

    got = step()
    monkeypatch.setenv("QLORA_TILE", "128")
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


@pytest.mark.parametrize("dsec,k,r,M", [(256, 320, 16, 130), (768, 1088, 32, 520)])
def test_every_tile_of_sections(lib, monkeypatch, dsec, k, r, M):
    print("case:", "sections", dsec, k, r, M, flush=True)
    g = torch.Generator().manual_seed(M)
    w = lib.quantize_sections([(torch.randn(dsec, k, generator=g) * 0.02).to(DEV) for _ in range(3)])
    X, dY = torch.randn(M, k, generator=g).to(BF).to(DEV), torch.randn(M, 3 * dsec, generator=g).to(BF).to(DEV)
    A = (torch.randn(3 * r, k, generator=g) * 0.05).to(BF).to(DEV)
    B = (torch.randn(3 * dsec, r, generator=g) * 0.05).to(BF).to(DEV)

    def step():
        return lib.forward_sections(X, w, A, B, 16.0), *lib.backward_sections(dY, X, w, A, B, 16.0)

    got = step()
    monkeypatch.setenv("QLORA_TILE", "128")
    assert all(torch.equal(a, b) for a, b in zip(got, step()))
