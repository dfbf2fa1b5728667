"""GPU parity of the few-row products' streaming kernel at its own limits: every row count it
takes, units by the hundred per CTA, clusters along K, activations whose spread leaves f16.

Tolerances: those of test_gpu_e_matvec.py (see there): every product is exact, an accumulator
takes eight MMAs, the sums are joined in float32."""
import numpy as np
import pytest

from oracle import formats as F
from tests.gpu_helpers import to_device
from tests.test_gpu_e_matvec import VIEWS, check, make_weight, tdt
from tests.test_gpu_f_experts import check_experts, dev, make_experts, route, sorted_np
from workloads import BF16, F16, heavy_activations

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", range(1, 18))
@pytest.mark.parametrize("fmt,mask", VIEWS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_row_counts(M, fmt, mask, dtype):
    import fp4_sparse_dense_b200 as sq
    rng = np.random.default_rng(M)
    w, w64 = make_weight(rng, 768, 256, fmt, mask)
    x = heavy_activations(rng, M, 768, dtype=F16 if dtype == "f16" else BF16)
    check(sq.matvec(to_device(x), w, out_dtype=tdt("f32")), x.values.astype(np.float64), w64, "f32")


@pytest.mark.parametrize("M,K", [(1, 57344), (3, 28672), (8, 14336), (8, 28672), (12, 8192), (16, 4096), (16, 14336)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_long_k(M, K, dtype):
    """Activations that one CTA holds, that a cluster of two, four or eight holds, or that none does."""
    import fp4_sparse_dense_b200 as sq
    rng = np.random.default_rng(M + K)
    w, w64 = make_weight(rng, K, 256, "nvfp4", "pair48")
    x = heavy_activations(rng, M, K, dtype=F16 if dtype == "f16" else BF16)
    check(sq.matvec(to_device(x), w, out_dtype=tdt("f32")), x.values.astype(np.float64), w64, "f32")


@pytest.mark.parametrize("M", [1, 5, 13, 20])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_wide_spread_in_a_step(M, fmt):
    """bf16 rows whose step holds 1e30 beside 1e-8: outputs that see only the small ones keep them."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(M)
    K, N = 512, 128
    w, w64 = make_weight(rng, K, N, fmt, "pair48")
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    x[::2] *= 1e-8
    x[::2, 130] = 1e30
    x[::2, 131] = -1e-38
    y = sq.matvec(x, w, out_dtype=torch.float32)
    check(y, x.double().cpu().numpy(), w64, "f32")
    free = np.flatnonzero(w64[:, 130] == 0)
    assert free.size
    got, x64 = y.cpu().numpy()[::2][:, free].astype(np.float64), x.double().cpu().numpy()[::2]
    want, scale = x64 @ w64[free].T, np.abs(x64) @ np.abs(w64[free].T)
    assert (np.abs(got - want) <= (K + 8) * 2.0 ** -23 * scale).all()


@pytest.mark.parametrize("M", [3, 11])
def test_units_by_the_hundred(M):
    """Ten thousand units of 32 outputs: more than a phase of each CTA. Outputs sampled."""
    import fp4_sparse_dense_b200 as sq
    import torch
    K, N = 256, 128 * 2500
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    w = sq.empty_weight(K, N, sq.Config.from_names("nvfp4", "none"))
    w.codes.copy_(torch.randint(0, 256, (w.codes.numel(),), dtype=torch.uint8, device="cuda", generator=g))
    w.scales_dense.copy_(torch.randint(40, 72, (w.scales_dense.numel(),), dtype=torch.uint8, device="cuda", generator=g))
    w.tensor_scale[0] = 1.0
    x = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    y = sq.matvec(x, w, out_dtype=torch.float32)
    rows = np.unique(np.concatenate([np.arange(0, N, 997), np.arange(N - 64, N)]))
    at_rows = torch.from_numpy(rows).cuda()
    codes = w.codes.view(N, K // 2)[at_rows].cpu().numpy()
    codes = np.stack((codes & 15, codes >> 4), axis=-1).reshape(len(rows), K)
    C = K // 16
    cols = np.arange(C)[None, :]
    at = ((rows[:, None] // 128) * (C // 4) + cols // 4) * 512 + (rows[:, None] % 32) * 16 + \
        (rows[:, None] // 32 % 4) * 4 + cols % 4
    raw = w.scales_dense[torch.from_numpy(at).cuda()].cpu().numpy()
    w64 = F.e2m1_decode(codes) * np.repeat(F.e4m3_decode(raw), 16, axis=1)
    check(y[:, at_rows], x.double().cpu().numpy(), w64, "f32")


@pytest.mark.parametrize("T,k,E,K,N", [(20, 4, 10, 512, 4096), (100, 1, 9, 256, 1024), (9, 8, 64, 1024, 256),
                                       (70, 2, 12, 4096, 128), (3, 2, 1024, 256, 128)])
@pytest.mark.parametrize("fmt,dtype", [("nvfp4", "bf16"), ("mxfp4", "f16"), ("mxfp4", "bf16")])
def test_experts(T, k, E, K, N, fmt, dtype):
    import fp4_sparse_dense_b200 as sq
    import torch
    if E > 64:
        w, w64 = make_experts(np.random.default_rng(1), 4, K, N, fmt, "pair48")
        stack = [None if t is None else t.view(4, -1).repeat(E // 4, 1)
                 for t in (w.codes, w.scales_dense, w.scales_sparse, w.tensor_scale)]
        w, w64 = sq.ExpertWeights(*stack, K, N, E, w.cfg), np.tile(w64, (E // 4, 1, 1))
    else:
        w, w64 = make_experts(np.random.default_rng(1), E, K, N, fmt, "pair48")
    rng = np.random.default_rng(T + E)
    ids = route(rng, T, k, E, 0.15)
    x = heavy_activations(rng, T, K, dtype=F16 if dtype == "f16" else BF16)
    t, _ = sq.sort_tokens(dev(ids), E)
    y = torch.full((T * k, N), 9.0, device="cuda")
    sq.expert_matvec(to_device(x), w, t, gather=True, out=y)
    offsets, order, _ = sorted_np(ids, E)
    check_experts(y, x.values.astype(np.float64), w64, offsets, order // k, "f32")
    assert (y[offsets[E]:] == 9).all()


def test_status_is_clear():
    import fp4_sparse_dense_b200 as sq
    assert sq.sharq_device_status() == 0
