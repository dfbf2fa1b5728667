"""GPU parity of the few-row products on MXFP4 weights whose blocks differ: blocks of zeros (scale
byte 0 beside ordinary ones), scales many binades apart, and infinite activations on them.

Tolerances: those of test_gpu_e_matvec.py. Where a step is added up block by block its
accumulators take no more MMAs than counted there, and each block's sum joins by one more float32
addition: 3 per 128 of K, which the count of one MMA per 16 of K (17 * 2^-23 each) covers eight
times over. Rows are compared one by one, so a row that only sees small blocks is held to them."""
import numpy as np
import pytest

from oracle import formats as F
from oracle import layouts as L
from oracle import sharq as S
from tests.gpu_helpers import cfg_of, to_device, upload_weight
from tests.test_gpu_e_matvec import check, tdt, weight64
from workloads import BF16, F16, heavy_activations

pytestmark = pytest.mark.gpu

ROWS = [1, 6, 8, 9, 12, 16, 20]


def quantised(w, mask="pair48"):
    """An MXFP4 weight of the float32 values w [K, N], and its float64 values [N, K]."""
    K, N = w.shape
    qw = S.quantize_weight(w, "mxfp4", mask)
    return upload_weight(S.weight_buffers(qw), K, N, cfg_of("mxfp4", mask)), weight64(qw)


def with_scales(rng, raw):
    """An MXFP4 weight of random codes with the scale bytes raw [N, K / 32]."""
    N, K = raw.shape[0], raw.shape[1] * 32
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    buf = {"codes": L.pack_nibbles(codes).reshape(-1), "tensor_scale": np.array([1.0], np.float32),
           "scales_dense": L.to_scale_layout(raw), "scales_sparse": L.to_scale_layout(raw)}
    w64 = F.e2m1_decode(codes) * np.repeat(F.e8m0_decode(raw), 32, axis=1)
    return upload_weight(buf, K, N, cfg_of("mxfp4", "pair48")), w64


def with_zeros(rng, K, N, zeros):
    w = (rng.standard_normal((K, N)) * 0.02).astype(np.float32)
    b = w.reshape(K // 32, 32, N)
    if zeros == "one":
        b[3, :, 5] = 0
    elif zeros == "first":
        b[4, :, 7] = 0
    elif zeros == "each":
        for n in range(N):
            b[rng.integers(0, K // 32), :, n] = 0
    elif zeros == "padded":
        w[K - 160:] = 0
    elif zeros == "most":
        b *= rng.random((K // 32, 1, N)) < 0.3
        for n in range(0, N, 3):
            b[:, :, n] = 0
    elif zeros == "far":
        b[1::4] *= np.float32(2.0 ** -30)
        b[2::4, :, ::2] *= np.float32(2.0 ** 20)
        b[5, :, 9] = 0
    return quantised(w)


ZEROS = ["one", "first", "each", "padded", "most", "far"]


@pytest.mark.parametrize("zeros", ZEROS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M", ROWS)
def test_blocks_of_zeros(M, dtype, zeros):
    import fp4_sparse_dense_b200 as sq
    rng = np.random.default_rng(M)
    K, N = 768, 128
    w, w64 = with_zeros(rng, K, N, zeros)
    x = heavy_activations(rng, M, K, dtype=F16 if dtype == "f16" else BF16)
    check(sq.matvec(to_device(x), w, out_dtype=tdt("f32")), x.values.astype(np.float64), w64, "f32")


@pytest.mark.parametrize("zeros", ZEROS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M", ROWS)
def test_infinities_beside_blocks_of_zeros(M, dtype, zeros):
    """An infinite activation gives an infinity where the weight is not 0 and NaN where it is, as
    in a float32 product, and stays in its row."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(M)
    K, N = 768, 128
    w, w64 = with_zeros(rng, K, N, zeros)
    x = heavy_activations(rng, M, K, dtype=F16 if dtype == "f16" else BF16)
    for r, k, s in ((0, 100, 1), (M - 1, 130, -1), (M // 2, K - 40, 1)):
        xi = to_device(x)
        xi[r, k] = s * float("inf")
        y = sq.matvec(xi, w, out_dtype=torch.float32).cpu().numpy()
        col = w64[:, k]
        want = np.where(col == 0, np.nan, np.copysign(np.inf, col * s))
        assert np.array_equal(y[r], want, equal_nan=True), (r, k)
        rest = [i for i in range(M) if i != r]
        check(torch.from_numpy(y[rest]), x.values[rest].astype(np.float64), w64, "f32") if rest else None


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("apart", [13, 14, 15, 23, 24, 40, 100])
@pytest.mark.parametrize("M", [3, 11, 20])
def test_scales_apart(M, apart, dtype):
    """Blocks up to `apart` binades from each other, among them the largest and the smallest of
    the spread in every output; every third row sees one block of each step only."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(apart)
    K, N = 512, 128
    low = 127 - apart // 2
    raw = rng.integers(low, low + apart + 1, (N, K // 32)).astype(np.uint8)
    ends = raw.reshape(N, -1, 4)
    ends[:, :, 1], ends[:, :, 2] = low, low + apart
    w, w64 = with_scales(rng, raw)
    x = heavy_activations(rng, M, K, dtype=F16 if dtype == "f16" else BF16)
    v = to_device(x)
    for r in range(0, M, 3):
        keep = np.arange(K) // 32 % 4 == 1 + r % 2
        v[r, torch.from_numpy(~keep).cuda()] = 0
    y = sq.matvec(v, w, out_dtype=tdt("f32"))
    v64 = v.double().cpu().numpy()
    for r in range(M):
        check(y[r:r + 1], v64[r:r + 1], w64, "f32")


@pytest.mark.parametrize("M", [2, 8, 13, 20])
def test_scales_apart_beside_a_wide_row(M):
    """Rows that see only blocks of scale 2^-107 beside others of 2^53, in a call with a row whose
    activations do not fit f16."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(M)
    K, N = 512, 128
    raw = np.full((N, K // 32), 180, np.uint8)
    raw[:, 1::4] = 20
    w, w64 = with_scales(rng, raw)
    x = torch.from_numpy(rng.standard_normal((M, K))).to(torch.bfloat16)
    small = torch.from_numpy(np.arange(K) // 32 % 4 == 1)
    x[1:, ~small] = 0
    x[0] = 0
    x[0, 40], x[0, 5] = 1e30, 1e-8
    x64 = x.double().numpy()
    y = sq.matvec(x.cuda(), w, out_dtype=torch.float32)
    for r in range(M):
        check(y[r:r + 1], x64[r:r + 1], w64, "f32")


@pytest.mark.parametrize("x_size,w_size", [(1e37, 0.02), (1e36, 1e-15), (1e-37, 1e20), (1e-30, 1e25), (1e30, 1e-30),
                                           (1e-38, 1e38), (1e3, 1e-38)])
@pytest.mark.parametrize("M", [1, 8, 12, 20])
def test_large_and_small_magnitudes(M, x_size, w_size):
    """bf16 activations and MXFP4 weights anywhere in their range: what a float32 product holds,
    the call holds."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(M)
    K, N = 512, 128
    w, w64 = quantised((rng.standard_normal((K, N)) * w_size).clip(-3e38, 3e38).astype(np.float32))
    x = torch.from_numpy(rng.standard_normal((M, K)) * x_size).to(torch.bfloat16)
    x64 = x.double().numpy()
    assert np.abs(x64 @ w64.T).max() < 2.0 ** 127 and np.abs(x64 @ w64.T).min() > 2.0 ** -126
    check(sq.matvec(x.cuda(), w, out_dtype=torch.float32), x64, w64, "f32")


@pytest.mark.parametrize("kind", ["f16", "bf16", "bf16 beside a wide row"])
@pytest.mark.parametrize("neighbours", ["apart", "alike"])
def test_unit_rows_return_every_scale(kind, neighbours):
    """x = e_k picks column k of the weight, exactly, at every E8M0 scale of a finite float32 weight,
    subnormal values among them: with f16 operands, block by block, and with bf16 operands."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(3)
    K, N = 512, 128
    if neighbours == "apart":
        raw = (np.arange(N * K // 32) % 253).astype(np.uint8).reshape(N, K // 32)
    else:  # a step's four blocks within two binades
        raw = (np.arange(N * K // 128) % 250).repeat(4).reshape(N, K // 32) + rng.integers(0, 3, (N, K // 32))
    w, w64 = with_scales(rng, raw.astype(np.uint8))
    dt = torch.float16 if kind == "f16" else torch.bfloat16
    eye = torch.eye(K, dtype=dt, device="cuda")
    wide = torch.zeros(1, K, dtype=dt, device="cuda")
    if kind.endswith("wide row"):
        wide[0, 3], wide[0, 4] = 1e30, 1e-8
    for k in range(0, K, 11):
        y = sq.matvec(torch.cat((wide, eye[k:k + 11])), w, out_dtype=torch.float32)[1:]
        assert np.array_equal(y.cpu().numpy().astype(np.float64), w64.T[k:k + 11]), k
