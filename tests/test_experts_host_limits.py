"""Refusals at the limits of the experts' operators, and what importing the package takes (no GPU
is touched)."""
import ctypes

import pytest

from tests.test_abi import sq  # noqa: F401  (builds the library)
from tests.test_experts_host import BF16, F16, F32, P, UNSUPPORTED, tokens


@pytest.mark.parametrize("H", [2 ** 31 - 65535, 2 ** 31 - 8192, 2 ** 31 - 1])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_rows_beyond_a_32_bit_column_are_refused(sq, H, dtype):  # noqa: F811
    """The row moves step a 32-bit column past the row's end: in a row of nearly 2^31 elements it
    would turn negative and start again before the row."""
    b = ctypes.byref(tokens(sq, T=1, k=1))
    assert sq.sharq_sort_tokens(P, 64, b, P, H, H, dtype, P, H, None) == UNSUPPORTED
    assert sq.sharq_sort_tokens_backward(P, H, H, dtype, b, P, H, None) == UNSUPPORTED
    assert sq.sharq_combine_tokens(P, H, H, dtype, b, P, P, H, None) == UNSUPPORTED
    assert sq.sharq_combine_tokens_backward(P, H, P, H, H, dtype, b, P, P, H, P, None) == UNSUPPORTED
    # the longest row passes these checks: the next one, alignment, answers
    n = 2 ** 31 - 65536
    assert sq.sharq_combine_tokens(P + 1, n, n, dtype, b, P, P, n, None) == 3
