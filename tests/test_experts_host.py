"""Refusals of the few-row products and the experts' operators (no GPU is touched: every
check comes before the device is looked at)."""
import ctypes

import pytest
import torch

from tests.test_abi import sq  # noqa: F401  (builds the library)

P = 1 << 20  # an address that is never dereferenced
INVALID, UNSUPPORTED, MISALIGNED = 1, 2, 3
F16, BF16, F32 = 0, 1, 2


def weight(sq, K=256, N=128, cfg=None, **kw):
    f = dict(codes=P, scales_dense=P, scales_sparse=P, tensor_scale=P, K=K, N=N,
             cfg=(cfg or sq.Config()).c())
    f.update(kw)
    return sq.sharq_weight(*f.values())


def experts(sq, K=256, N=128, E=4, **kw):
    f = dict(codes=P, scales_dense=P, scales_sparse=P, tensor_scale=P, K=K, N=N, E=E,
             cfg=sq.Config().c())
    f.update(kw)
    return sq.sharq_expert_weights(*f.values())


def tokens(sq, T=8, k=2, E=4, **kw):
    f = dict(offsets=P, order=P, place=P, T=T, k=k, E=E)
    f.update(kw)
    return sq.sharq_tokens(*f.values())


def call_matvec(sq, w, X=P, ldx=256, M=1, dtype=BF16, Y=P, ldy=128, y_dtype=BF16):
    return sq.sharq_matvec(X, ldx, M, dtype, ctypes.byref(w), Y, ldy, y_dtype, None)


@pytest.mark.parametrize("kw,want", [
    (dict(X=None), INVALID), (dict(Y=None), INVALID), (dict(M=-1), INVALID),
    (dict(dtype=F32), INVALID), (dict(dtype=7), INVALID), (dict(y_dtype=3), INVALID),
    (dict(ldx=255), INVALID), (dict(ldx=248), INVALID), (dict(ldy=127), INVALID),
    (dict(ldx=257), MISALIGNED), (dict(ldx=260), MISALIGNED), (dict(X=P + 2), MISALIGNED),
    (dict(Y=P + 8), MISALIGNED), (dict(M=(1 << 21) + 1), UNSUPPORTED),
])
def test_matvec_refuses(sq, kw, want):  # noqa: F811
    assert call_matvec(sq, weight(sq), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(K=128), INVALID), (dict(K=320), INVALID), (dict(N=64), INVALID), (dict(K=0), INVALID),
    (dict(codes=None), INVALID), (dict(scales_sparse=None), INVALID),
    (dict(tensor_scale=None), INVALID), (dict(codes=P + 4), MISALIGNED),
    (dict(scales_sparse=P + 4), MISALIGNED), (dict(tensor_scale=P + 2), MISALIGNED),
])
def test_matvec_refuses_weights(sq, kw, want):  # noqa: F811
    assert call_matvec(sq, weight(sq, **kw), ldx=512, ldy=512) == want


def test_matvec_reads_one_scale_view(sq):  # noqa: F811
    """Pair masks need the sparse view only, the others the dense view only."""
    none = sq.Config.from_names("nvfp4", "none")
    assert call_matvec(sq, weight(sq, cfg=none, scales_dense=None)) == INVALID
    assert call_matvec(sq, weight(sq, cfg=none, scales_sparse=None, codes=P + 1)) == MISALIGNED
    assert call_matvec(sq, weight(sq, scales_dense=None, codes=P + 1)) == MISALIGNED


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(E=0), INVALID), (dict(E=1025), UNSUPPORTED),
    (dict(T=1 << 28, k=4), UNSUPPORTED), (dict(offsets=None), INVALID),
    (dict(order=None), INVALID), (dict(place=None), INVALID), (dict(place=P + 2), MISALIGNED),
    (dict(offsets=P + 1), MISALIGNED),
])
def test_tokens_refused_everywhere(sq, kw, want):  # noqa: F811
    t = tokens(sq, **kw)
    b = ctypes.byref(t)
    w = ctypes.byref(experts(sq, E=t.E))
    assert sq.sharq_sort_tokens(P, 64, b, None, 0, 0, BF16, None, 0, None) == want
    assert sq.sharq_sort_tokens_backward(P, 8, 8, BF16, b, P, 8, None) == want
    assert sq.sharq_combine_tokens(P, 8, 8, BF16, b, P, P, 8, None) == want
    assert sq.sharq_combine_tokens_backward(P, 8, P, 8, 8, BF16, b, P, P, 8, P, None) == want
    assert sq.sharq_expert_matvec(P, 256, 0, BF16, b, w, P, 128, BF16, None) == want


def test_sort_refuses(sq):  # noqa: F811
    b = ctypes.byref(tokens(sq))
    sort = sq.sharq_sort_tokens
    assert sort(None, 64, b, None, 0, 0, BF16, None, 0, None) == INVALID
    assert sort(P, 16, b, None, 0, 0, BF16, None, 0, None) == INVALID
    assert sort(P + 4, 64, b, None, 0, 0, BF16, None, 0, None) == MISALIGNED
    assert sort(P, 64, b, P, 8, 0, BF16, P, 8, None) == INVALID      # H
    assert sort(P, 64, b, P, 7, 8, BF16, P, 8, None) == INVALID      # ldx
    assert sort(P, 64, b, P, 8, 8, BF16, P, 7, None) == INVALID      # ld_rows
    assert sort(P, 64, b, P, 8, 8, BF16, None, 8, None) == INVALID   # rows
    assert sort(P, 64, b, P, 8, 8, 3, P, 8, None) == INVALID         # dtype
    assert sort(P, 64, b, P + 1, 8, 8, BF16, P, 8, None) == MISALIGNED
    assert sort(P, 64, b, P, 8, 8, F32, P + 2, 8, None) == MISALIGNED


def test_combine_refuses(sq):  # noqa: F811
    b = ctypes.byref(tokens(sq))
    f, g = sq.sharq_combine_tokens, sq.sharq_combine_tokens_backward
    assert f(None, 8, 8, BF16, b, P, P, 8, None) == INVALID
    assert f(P, 8, 8, BF16, b, P, None, 8, None) == INVALID
    assert f(P, 8, 8, BF16, b, P + 2, P, 8, None) == MISALIGNED
    assert f(P, 8, 8, BF16, b, P, P, 7, None) == INVALID
    assert g(P, 8, P, 8, 8, BF16, b, None, P, 8, P, None) == INVALID   # weights
    assert g(P, 8, P, 8, 8, BF16, b, P, P, 8, None, None) == INVALID   # d_weights
    assert g(P, 8, P, 8, 8, BF16, b, P, P, 8, P + 2, None) == MISALIGNED
    assert g(P, 8, P + 1, 8, 8, BF16, b, P, P, 8, P, None) == MISALIGNED
    assert g(P, 4, P, 8, 8, BF16, b, P, P, 8, P, None) == INVALID


def test_expert_matvec_refuses(sq):  # noqa: F811
    b = ctypes.byref(tokens(sq))
    f = sq.sharq_expert_matvec
    assert f(P, 256, 0, BF16, b, ctypes.byref(experts(sq, E=5)), P, 128, BF16, None) == INVALID
    w = ctypes.byref(experts(sq))
    assert f(P, 256, 2, BF16, b, w, P, 128, BF16, None) == INVALID
    assert f(None, 256, 0, BF16, b, w, P, 128, BF16, None) == INVALID
    assert f(P, 256, 0, F32, b, w, P, 128, BF16, None) == INVALID
    assert f(P, 252, 0, BF16, b, w, P, 128, BF16, None) == INVALID
    assert f(P, 260, 0, BF16, b, w, P, 128, BF16, None) == MISALIGNED
    assert f(P, 256, 0, BF16, b, ctypes.byref(experts(sq, N=96)), P, 128, BF16, None) == INVALID
    many = ctypes.byref(tokens(sq, T=1 << 19, k=2))
    assert f(P, 256, 0, BF16, many, w, P, 128, BF16, None) == UNSUPPORTED


def test_expert_matvec_refuses_outputs_beyond_32_bits(sq):  # noqa: F811
    """The copies' coordinate counts the outputs of all experts."""
    t, n = ctypes.byref(tokens(sq, E=1024)), 1 << 21
    w = ctypes.byref(experts(sq, E=1024, N=n))
    assert sq.sharq_expert_matvec(P, 256, 0, BF16, t, w, P, n, BF16, None) == UNSUPPORTED


# ------------------------------------------------------------------ the tensor-level helpers

def test_cpu_tensors_are_refused(sq):  # noqa: F811
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    ids = torch.zeros(2, 2, dtype=torch.int64)
    t = sq.SortedTokens(torch.zeros(5, dtype=torch.int32), torch.zeros(4, dtype=torch.int32),
                        torch.zeros(2, 2, dtype=torch.int32), 2, 2, 4)
    for call in (lambda: sq.matvec(x, None), lambda: sq.sort_tokens(ids, 4, x),
                 lambda: sq.expert_matvec(x, None, t), lambda: sq.combine_tokens(x, t),
                 lambda: sq.combine_tokens_backward(x, x, t, None),
                 lambda: sq.quantize_experts(torch.zeros(1, 256, 128))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_quantize_experts_shape(sq):  # noqa: F811
    with pytest.raises(ValueError, match="E, K, N"):
        sq.quantize_experts(torch.zeros(256, 128))


def test_expert_buffers_are_checked(sq):  # noqa: F811
    """ExpertWeights and SortedTokens reject buffers of the wrong size or layout, and give
    each expert its part."""
    E, K, N = 3, 256, 128
    code, scale = N * K // 2, N * K // 16

    def make(codes=E * code, dense=E * scale, sparse=E * scale // 2, ts=4 * E):
        return sq.ExpertWeights(torch.zeros(codes, dtype=torch.uint8), torch.zeros(dense, dtype=torch.uint8),
                                torch.zeros(sparse, dtype=torch.uint8), torch.zeros(ts), K, N, E, sq.Config())

    w = make()
    assert w.c().E == E
    one = w.expert(2)
    assert one.codes.data_ptr() == w.codes.data_ptr() + 2 * code
    assert one.scales_dense.data_ptr() == w.scales_dense.data_ptr() + 2 * scale
    assert one.scales_sparse.data_ptr() == w.scales_sparse.data_ptr() + scale
    assert one.tensor_scale.data_ptr() == w.tensor_scale.data_ptr() + 32
    for e in (-1, 3):
        with pytest.raises(IndexError):
            w.expert(e)
    for kw in (dict(codes=code), dict(dense=scale), dict(sparse=1), dict(ts=E)):
        with pytest.raises(ValueError):
            make(**kw).c()
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError):
        sq.SortedTokens(torch.zeros(4, **i32), torch.zeros(4, **i32), torch.zeros(2, 2, **i32), 2, 2, 4).c()
    with pytest.raises(ValueError):
        sq.SortedTokens(torch.zeros(5), torch.zeros(4, **i32), torch.zeros(2, 2, **i32), 2, 2, 4).c()
