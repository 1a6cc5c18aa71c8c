"""What lies between the rows of an output of the losses' gradients: padding is
written with them, other rows of the caller's tensor are not."""

import pytest
import torch


def _args(T, V, dtype=torch.float32, device="cpu"):
    return (torch.zeros(T, device=device), torch.zeros(T, V, dtype=dtype, device=device),
            torch.zeros(T, dtype=torch.int32, device=device), torch.zeros(T, 2, device=device))


def _slices(T, V, device="cpu"):
    """Outputs of T rows between whose rows other rows of the same tensor lie."""
    yield torch.zeros(T, 3, V, device=device)[:, 0]                      # one position of every sequence
    yield torch.zeros(2 * T, V, device=device)[::2]                      # every other row
    yield torch.zeros(2 * T, V + 24, device=device)[::2, :V]             # of a padded head
    yield torch.zeros(T, 2, V + 24, device=device)[:, 0, :V]
    yield torch.zeros(T, 4, V, device=device)[:, 1:3][:, 0]
    yield torch.zeros(T + 1, V + 400, device=device)[:T, 100:100 + V]    # columns of the next row
    yield torch.zeros(T, 3, V, 1, device=device)[:, 0, :, 0]
    yield torch.zeros(2 * T, 2 * V, dtype=torch.bfloat16, device=device).view(torch.float32)[::2]


def test_other_rows_between_the_outputs_rows_are_refused(lib):
    # (host tensors: refused before anything is launched)
    T, V = 5, 1000
    g, z, y, st = _args(T, V)
    for out in _slices(T, V):
        with pytest.raises(ValueError, match="other rows"):
            lib.token_logprobs_backward(g, z, y, st, out=out)
    both = torch.zeros(T, 3, V)[:, 1]
    with pytest.raises(ValueError, match="other rows"):
        lib.token_logprobs_backward(g, both, y, st, out=both)            # in place as well
    with torch.inference_mode():
        with pytest.raises(ValueError, match="other rows"):
            lib.token_logprobs_backward(g, z, y, st, out=torch.zeros(T, 3, V)[:, 0])


def test_paddings_are_taken(lib):
    # ... of a wider matrix, of its first rows, of a flat buffer, of another type's
    T, V = 5, 1000
    g, z, y, st = _args(T, V)
    outs = [torch.zeros(T, 1024)[:, :V], torch.zeros(T + 3, 1400)[1:T + 1, :V], torch.zeros(T, V),
            torch.zeros(T * 4000).view(T, 4000)[:, :V], torch.zeros(1100 * T).as_strided((T, V), (1100, 1)),
            torch.zeros(T, 2048, dtype=torch.bfloat16).view(torch.float32)[:, :V], torch.zeros(T, 1, 1024)[:, 0, :V],
            torch.zeros(3, T, 1024)[1, :, :V], torch.zeros(T, V, 1)[:, :, 0], torch.zeros(T, 1024).detach()[:, :V],
            torch.nn.Parameter(torch.zeros(T, 1024)).data[:, :V], torch.zeros(1000, 64).view(-1)[:T * V].view(T, V),
            torch.zeros(1000, 64).view(-1)[:T * 1024].view(T, 1024)[:, :V],
            torch.zeros(2 * T, 2 * V).view(-1)[77:77 + T * V].view(T, V)]
    with torch.inference_mode():
        outs.append(torch.zeros(T, 1024)[:, :V])
    for out in outs:
        with pytest.raises(ValueError, match="on a GPU"):
            lib.token_logprobs_backward(g, z, y, st, out=out)


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
def test_one_row_leaves_its_neighbours(lib, in_place):
    # the stride of a single row is not a padding's: the first position of a batch of one
    V, S = 1000, 4
    full = torch.full((1, S, V), 3.0, device="cuda")
    z = torch.randn(1, V, device="cuda")
    y = torch.tensor([7], dtype=torch.int32, device="cuda")
    one = torch.ones(1, device="cuda")
    logp, stats = lib.token_logprobs(z, y, save_stats=True)
    want = lib.token_logprobs_backward(one, z, y, stats)
    out = full[:1, 0]
    if in_place:
        out.copy_(z)
    src = out if in_place else z
    lib.token_logprobs_backward(one, src, y, stats, out=out)
    assert torch.equal(out, want) and (full[0, 1:] == 3).all()
    if in_place:
        out.copy_(z)
    lib.policy_loss(src, y, -one, out=out)
    assert torch.equal(out, want) and (full[0, 1:] == 3).all()


@pytest.mark.gpu
def test_one_row_of_a_padded_head_is_written_whole(lib):
    # ... whatever else the tensor holds that it is a row of: the first position of a batch of one
    V, S = 1000, 4
    z, y = torch.randn(1, V, device="cuda"), torch.tensor([7], dtype=torch.int32, device="cuda")
    one = torch.ones(1, device="cuda")
    logp, stats = lib.token_logprobs(z, y, save_stats=True)
    want = lib.token_logprobs_backward(one, z, y, stats)
    for at in (0, 2):
        full = torch.full((1, S, 1024), 3.0, device="cuda")
        lib.token_logprobs_backward(one, z, y, stats, out=full[:, at, :V])
        assert torch.equal(full[0, at, :V], want[0]) and (full[0, at, V:] == 0).all()
        assert (full[0, :at] == 3).all() and (full[0, at + 1:] == 3).all()
    full = torch.full((3, 2000), 3.0, device="cuda")
    lib.token_logprobs_backward(one, z, y, stats, out=full[1:2, 100:100 + V])    # amid a row: nothing but its words
    assert torch.equal(full[1:2, 100:100 + V], want) and (full[1, :100] == 3).all() and (full[1, 100 + V:] == 3).all()
    assert (full[::2] == 3).all()


@pytest.mark.gpu
def test_one_row_needs_no_stride(lib):
    # a batch of one whose positions are 2^30 elements long, as far as the stride says
    V = 1000
    big = torch.empty((1 << 30) + 8192, dtype=torch.bfloat16, device="cuda")
    row = big.as_strided((1, V), (1 << 30, 1), 64)
    row.copy_(torch.randn(1, V, device="cuda"))
    y = torch.tensor([7], dtype=torch.int32, device="cuda")
    assert torch.equal(lib.token_logprobs(row, y), lib.token_logprobs(row.clone(), y))
