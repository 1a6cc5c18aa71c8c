"""A NaN makes its row one without a distribution wherever it stands: among masked words too, where the thread that
reads it has no finite word of its own.  Such rows are made of a few finite words, NaNs and masks (-inf)."""

import pytest
import torch

from gpu_util import DEV
from test_gpu_scores import _check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _rows(V, dtype, offset):
    """Six rows without a distribution and one, the last, with: what is not said here is masked."""
    nan = float("nan")
    buf = torch.full((7 * V + offset,), -float("inf"))
    z = buf[offset:].view(7, V)
    some = torch.linspace(-3, 3, 70)
    z[0, 9], z[0, V - 70:] = nan, some       # a NaN long before the row's words
    z[1], z[1, V - 70:] = nan, some          # nothing but NaNs before them
    z[2, V - 1], z[2, :70] = nan, some       # the last word
    z[3, V // 2], z[3, 3] = nan, 1.0
    z[4, 0], z[4, V // 3] = nan, 1.0         # the first one
    z[5] = nan
    z[6, V // 2], z[6, V - 1] = 0.5, 1.5
    return buf.to(dtype).to(DEV)[offset:].view(7, V)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("copies", [1, 40])
@pytest.mark.parametrize("V,offset", [(200, 0), (3000, 0), (9001, 3), (40000, 0), (70001, 1), (140000, 0), (300007, 0)])
def test_a_nan_among_masked_words(lib, V, offset, copies, dtype):
    print("case: NaN among masks", V, offset, copies, dtype, flush=True)
    z = _rows(V, dtype, offset)
    if copies > 1:  # as many rows, which other kernels read
        z = z.repeat(copies, 1)
    y = torch.tensor([V - 1, V // 2], dtype=torch.int32, device=DEV).repeat(len(z), 1)
    if copies == 1:
        out = _check(lib, z, y, 5, 1.0)
    else:
        out = lib.token_scores(z, y, top=5, save_stats=True)
    bad = torch.arange(len(z), device=DEV) % 7 != 6
    for t in (out[0], out[1], out[3]):
        assert torch.isnan(t[bad]).all() and not torch.isnan(t[~bad]).any()
    assert (out[2][bad] == -1).all() and (out[2][~bad][:, :2] == torch.tensor([V - 1, V // 2], device=DEV)).all()
    g, gh = torch.ones(len(z), 2, device=DEV), torch.ones(len(z), device=DEV)
    d = lib.token_scores_backward(g, gh, z, y, out[4])
    assert torch.isnan(d[bad]).all() and not torch.isnan(d[~bad]).any()
