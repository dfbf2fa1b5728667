"""GPU tests of the few-row products and the experts' operators at the ends of their ranges: sizes
that the helpers have to refuse before anything is allocated or cut to 32 bits."""
import pytest

pytestmark = pytest.mark.gpu


def wide(rows, cols, dtype):
    """A [rows, cols] view of one element."""
    import torch
    return torch.zeros(1, 1, dtype=dtype, device="cuda").expand(rows, cols)


@pytest.mark.parametrize("num_experts", [-5, 0, 1025, 2 ** 31, 2 ** 32 + 3])
def test_counts_of_experts(num_experts):
    import fp4_sparse_dense_b200 as sq
    import torch
    ids = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    with pytest.raises(sq.SharqError):
        sq.sort_tokens(ids, num_experts)


@pytest.mark.parametrize("T,k", [(2 ** 32, 1), (2 ** 32 + 2, 1), (2 ** 30, 1), (2 ** 29, 2), (4, 2 ** 32 + 1), (3, 0)])
def test_counts_of_assignments(T, k):
    """2^32 + 2 tokens are not 2."""
    import fp4_sparse_dense_b200 as sq
    import torch
    with pytest.raises(sq.SharqError):
        sq.sort_tokens(wide(T, k, torch.int32), 4)


@pytest.mark.parametrize("H", [2 ** 31, 2 ** 32 + 8])
def test_lengths_of_rows(H):
    import fp4_sparse_dense_b200 as sq
    import torch
    ids = torch.zeros(1, 1, dtype=torch.int64, device="cuda")
    t, _ = sq.sort_tokens(ids, 1)
    x = wide(1, H, torch.bfloat16)
    w = torch.ones(1, 1, device="cuda")
    for call in (lambda: sq.sort_tokens(ids, 1, x), lambda: sq.sort_tokens_backward(x, t),
                 lambda: sq.combine_tokens(x, t, w), lambda: sq.combine_tokens_backward(x, x, t, w)):
        with pytest.raises(ValueError):
            call()


def test_lengths_that_32_bits_hold_but_the_kernels_do_not():
    import fp4_sparse_dense_b200 as sq
    import torch
    H = 2 ** 31 - 65535
    ids = torch.zeros(1, 1, dtype=torch.int64, device="cuda")
    t, _ = sq.sort_tokens(ids, 1)
    x = torch.empty(1, H, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(sq.SharqError):
        sq.combine_tokens(x, t, out=x)


def test_numbers_of_rows():
    import fp4_sparse_dense_b200 as sq
    import torch
    w = sq.quantize_weight(torch.zeros(256, 128, dtype=torch.bfloat16, device="cuda"))
    for rows in (2 ** 31, 2 ** 32 + 1):
        with pytest.raises(ValueError):
            sq.matvec(wide(rows, 256, torch.bfloat16), w)
