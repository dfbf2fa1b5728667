"""Refusals at the limits of the experts' operators, and what importing the package takes (no GPU
is touched)."""
import ctypes
import os
import subprocess
import sys

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


def run_python(code):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return r.stdout


NO_TORCH = """
import sys
class NoTorch:
    def find_spec(self, name, path=None, target=None):
        if name.split(".")[0] == "torch":
            raise ModuleNotFoundError(name)
sys.meta_path.insert(0, NoTorch())
"""

SIZES = """
import ctypes
import fp4_sparse_dense_b200 as sq
sz = sq.sharq_weight_bytes()
assert sq.sharq_weight_sizes(256, 128, sq.Config().c(), ctypes.byref(sz)) == 0 and sz.codes == 16384
t = sq.sharq_tokens(None, None, None, 0, 1, 1)
assert sq.sharq_sort_tokens(None, 64, ctypes.byref(t), None, 0, 0, 1, None, 0, None) == 1
"""


def test_the_package_imports_without_torch(sq):  # noqa: F811
    """The C names and the size queries need no torch; the tensor helpers are named all the same."""
    run_python(NO_TORCH + SIZES + "from fp4_sparse_dense_b200 import *\nassert matvec and SortedTokens")


def test_importing_the_package_does_not_import_torch(sq):  # noqa: F811
    run_python("import sys\n" + SIZES + "assert 'torch' not in sys.modules")


def test_helpers_refuse_cpu_tensors_on_a_cpu_build_of_torch(sq):  # noqa: F811
    """A build without CUDA has neither of the queries that the helpers use."""
    run_python("""
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import fp4_sparse_dense_b200 as sq
try:
    sq.matvec(torch.zeros(1, 256, dtype=torch.bfloat16), None)
except ValueError as e:
    assert "CUDA" in str(e)
else:
    raise AssertionError
""")


@pytest.mark.parametrize("first", ["sq.SortedTokens(i(5), i(4), i(2, 2), 2, 2, 4).c",
                                   "sq.ExpertWeights(None, None, None, torch.zeros(4), 256, 128, 1, sq.Config()).c"])
def test_structs_check_their_buffers_before_any_call(sq, first):  # noqa: F811
    """The checks work whatever is called first: these refuse CPU tensors and missing buffers."""
    run_python("""
import torch
import fp4_sparse_dense_b200 as sq
i = lambda *s: torch.zeros(*s, dtype=torch.int32)
try:
    %s()
except ValueError:
    pass
""" % first)


def plan(sq, M, E, K):  # noqa: F811
    tile_rows, splits = ctypes.c_int32(), ctypes.c_int32()
    assert sq.sharq_matvec_plan(M, E, K, ctypes.byref(tile_rows), ctypes.byref(splits)) == 0
    return tile_rows.value, splits.value


def test_plan_of_the_products(sq):  # noqa: F811
    """Up to 16 rows (8 per expert on average) stream, over as few CTAs as hold their activations;
    the rest go to the tiles, in slots of 16 rows where no more are expected."""
    for M, E, K, want in ((1, 0, 4096, (0, 1)), (8, 0, 4096, (0, 1)), (16, 0, 4096, (0, 2)), (17, 0, 256, (32, 0)), (1 << 21, 0, 256, (32, 0)),
                          (8, 0, 14336, (0, 4)), (1, 0, 57344, (0, 2)), (16, 0, 19456, (0, 8)), (16, 0, 19712, (16, 0)),
                          (1, 8, 4096, (0, 1)), (64, 8, 14336, (0, 4)), (65, 8, 4096, (32, 0)), (8, 1, 51200, (16, 0)),
                          (9, 1, 51200, (32, 0))):
        assert plan(sq, M, E, K) == want, (M, E, K)


def test_plan_refuses(sq):  # noqa: F811
    a, b = ctypes.c_int32(), ctypes.c_int32()
    f, r = sq.sharq_matvec_plan, ctypes.byref
    for M, E, K in ((0, 0, 256), (1, -1, 256), (1, 0, 128), (1, 0, 300), (1, 0, 0)):
        assert f(M, E, K, r(a), r(b)) == 1
    assert f(1, 0, 256, None, r(b)) == 1 and f(1, 0, 256, r(a), None) == 1


# ------------------------------------------------------------------ buffers of a weight

def stacked(**other):
    import torch

    import fp4_sparse_dense_b200 as sq
    E, K, N = 3, 256, 128
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    f = dict(codes=u8(E * N * K // 2), scales_dense=u8(E * N * K // 16), scales_sparse=u8(E * N * K // 32),
             tensor_scale=torch.zeros(E, 4))
    f.update(other)
    return sq.ExpertWeights(*f.values(), K, N, E, sq.Config())


def test_stacked_scales_have_to_be_contiguous(sq):  # noqa: F811
    """A column range of a wider matrix holds as many numbers, elsewhere."""
    import torch
    assert stacked().c().E == 3
    with pytest.raises(ValueError):
        stacked(tensor_scale=torch.zeros(3, 8)[:, :4]).c()
    with pytest.raises(ValueError):
        stacked(tensor_scale=torch.zeros(4, 3).t()).c()


@pytest.mark.parametrize("name", ["scales_dense", "scales_sparse", "tensor_scale"])
def test_buffers_of_a_weight_are_on_one_device(sq, name):  # noqa: F811
    """A pointer of another device never reaches a kernel."""
    w = stacked()
    setattr(w, name, getattr(w, name).to("meta"))
    with pytest.raises(ValueError):
        w.c()
    one = stacked().expert(1)
    assert one.c().K == 256
    setattr(one, name, getattr(one, name).to("meta"))
    with pytest.raises(ValueError):
        one.c()
