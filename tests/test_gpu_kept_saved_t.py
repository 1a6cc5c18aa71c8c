"""The T that a backward from a checkpoint takes is the one of its own forward: its rows are as long as that
forward's tokens, rounded up to 64, so that of another number of tokens or ranks every rank but the first would be read
from wrong places."""

import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _layer(lib, M, nsec=1, r=4):
    g = torch.Generator().manual_seed(M)
    w = lib.quantize_sections([(torch.randn(256, 128, generator=g) * 0.02).to(DEV) for _ in range(nsec)])
    A = (torch.randn(nsec * r, 128, generator=g) * 0.1).to(BF).to(DEV)
    B = (torch.randn(nsec * 256, r, generator=g) * 0.1).to(BF).to(DEV)
    X, dY = torch.randn(M, 128, generator=g).to(BF).to(DEV), torch.randn(M, nsec * 256, generator=g).to(BF).to(DEV)
    return w, A, B, X, dY


@pytest.mark.parametrize("nsec,r", [(1, 4), (2, 16)])
def test_another_forwards_t_is_refused(lib, nsec, r):
    print("case: T of another forward", nsec, r, flush=True)
    w, A, B, X, dY = _layer(lib, 200, nsec, r)
    T = lib.forward_checkpoint(X, w, A, B, 8.0)[1]
    M = 70
    _, own, ck = lib.forward_checkpoint(X[:M].contiguous(), w, A, B, 8.0)
    assert own.shape == (nsec * r, 128) and T.shape == (nsec * r, 256)
    g = dY[:M].contiguous()
    more = torch.cat([own, own])
    for bad in (T, T.view(-1), more, more.view(-1), own.view(-1)[:-1], own.view(128, -1), own.view(2, -1, 128)):
        with pytest.raises(ValueError, match="T_saved"):
            lib.backward_checkpoint(g, ck, w, A, B, 8.0, bad)
    # the forward's own, also as the vector that the ordinary forward returns
    fwd = lib.forward if nsec == 1 else lib.forward_sections
    flat = fwd(X[:M].contiguous(), w, A, B, 8.0, save_t=True)[1]
    want = lib.backward_checkpoint(g, ck, w, A, B, 8.0, own)
    for good in (own.view(-1), flat):
        assert all(torch.equal(a, b) for a, b in zip(lib.backward_checkpoint(g, ck, w, A, B, 8.0, good), want))


def test_no_tokens_take_the_forwards_t(lib):
    w, A, B, X, dY = _layer(lib, 3)
    ck = lib.checkpoint_save(X[:0])
    for T in (lib.forward_checkpoint(X[:0], w, A, B, 8.0)[1], torch.empty(1, dtype=BF, device=DEV)):
        assert not lib.backward_checkpoint(dY[:0], ck, w, A, B, 8.0, T)[1].any()
