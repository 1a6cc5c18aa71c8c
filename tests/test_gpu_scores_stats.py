"""Statistics of rows of logits serve a gradient of other tokens than the forward's (a teacher's words beside the
label), except where the forward read nothing of a row: such a row has none, and a gradient that needs them is NaN,
not one of some other distribution."""

import pytest
import torch

from gpu_util import DEV
from test_gpu_scores import _check_grad, _logits

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [300, 5000, 40000, 140000])
def test_other_tokens_than_the_forwards(lib, V, dtype):
    print("case: other tokens", V, dtype, flush=True)
    T = 6
    z = _logits(T, V, dtype, V + 1)
    labels = torch.tensor([3, -100, V - 1, V, 7, -1], dtype=torch.int32, device=DEV)
    unread = torch.tensor([False, True, False, True, False, True], device=DEV)
    teacher = torch.tensor([[1, 2], [4, 5], [V - 1, 0], [6, 8], [-1, -1], [-1, -1]], dtype=torch.int32, device=DEV)
    stats = lib.token_scores(z, labels, save_stats=True)[4]
    g, gh = torch.linspace(0.5, 1, 2 * T).view(T, 2).to(DEV), torch.linspace(-1, -0.5, T).to(DEV)
    d = lib.token_scores_backward(g, gh, z, teacher, stats)
    assert torch.isnan(d[[1, 3]]).all()      # not read, needed
    assert not d[[4, 5]].any()               # nothing counts: no statistics are needed
    read = torch.nonzero(~unread)[:, 0]
    one = _check_grad(lib, z[read].contiguous(), teacher[read].contiguous(), g[read].contiguous(), gh[read].contiguous(),
                      stats[read].contiguous(), 1.0, dtype)
    assert torch.equal(d[read], one)
    # without coefficients there is no gradient and nothing to ask for
    g[[1, 3]], gh[[1, 3]] = 0, 0
    assert not lib.token_scores_backward(g, gh, z, teacher, stats)[[1, 3]].any()
    # the forward's own tokens never need a row that it did not read
    own = lib.token_scores_backward(g[:, 0].contiguous(), gh, z, labels, stats)
    assert not own[unread].any() and torch.isfinite(own.float()).all()
