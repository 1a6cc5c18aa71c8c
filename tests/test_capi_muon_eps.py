"""The orthogonalised update refuses an eps whose reciprocal fp32 cannot hold (host checks, no GPU needed; the device
pointers are fake addresses that are never dereferenced)."""

import pytest

E_ALPHA, E_NULL = 6, 1


@pytest.mark.parametrize("eps,ok", [(1e-45, False), (1e-38, False), (9e-31, False), (1e-30, True), (1e-7, True)])
def test_eps(lib, eps, ok):
    s = lib.lib().qlora_muon_step(None, None, None, None, 1, 16, 4096, 1e-3, 0.95, 1, 0.0, 1.0, eps, 5, None, None, 0,
                                  None)
    assert s == (E_NULL if ok else E_ALPHA)
