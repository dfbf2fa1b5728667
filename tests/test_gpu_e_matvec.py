"""GPU parity of the few-row product (16-bit activations, FP4 weights) against float64.

Tolerances. All products are exact in the kernel (E2M1 * scale: at most 6 significant bits;
fp16 activations enter as two bf16), so only sums and the output round. One MMA adds 16
products to its accumulator; terms below the 24th bit of the largest are cut, so it is off by
at most 17 * 2^-23 of the sum of magnitudes, and there are at most K / 16 of them in a row, then
fewer than 32 float32 additions and two multiplications:

    |y - y64| <= (K / 16 + 34) * 17 * 2^-23 * sum_k |x w| + |y64| * eps(out) / 2 (+ fp16's
    smallest step / 2).

Errors of that many roundings rarely point the same way: the float32 output is also held to
1e-5 relative Frobenius error, the bound of the linear layer, which accumulates alike."""
import numpy as np
import pytest

from oracle import formats as F
from oracle import layouts as L
from oracle import sharq as S
from tests.gpu_helpers import cfg_of, rel_fro, to_device, upload_weight
from workloads import BF16, F16, gaussian_weight, heavy_activations

pytestmark = pytest.mark.gpu

VIEWS = [("nvfp4", "pair48"), ("nvfp4", "none"), ("nvfp4", "elem24"), ("mxfp4", "pair48"),
         ("mxfp4", "none")]
EPS = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}  # half a step, relative


def tdt(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def weight64(qw):
    """float64 [N, K], tensor scale included."""
    return S.weight_values(qw) * (float(qw.s_gw) if qw.fmt == "nvfp4" else 1.0)


def make_weight(rng, K, N, fmt, mask):
    w = gaussian_weight(rng, K, N)
    qw = S.quantize_weight(w.values, fmt, mask)
    return upload_weight(S.weight_buffers(qw), K, N, cfg_of(fmt, mask)), weight64(qw)


def check(y, x64, w64, out):
    y = y.double().cpu().numpy()
    want = x64 @ w64.T
    K = w64.shape[1]
    bound = (K / 16 + 34) * 17 * 2.0 ** -23 * (np.abs(x64) @ np.abs(w64).T)
    bound += np.abs(want) * EPS[out] * 1.01 + (2.0 ** -25 if out == "f16" else 0)
    assert np.isfinite(y).all()
    worst = np.max(np.abs(y - want) - bound)
    assert worst <= 0, worst
    if out == "f32":
        assert rel_fro(y, want) <= 1e-5


@pytest.mark.parametrize("fmt,mask", VIEWS)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"),
                                       ("f16", "f32"), ("bf16", "f16"), ("f16", "bf16")])
@pytest.mark.parametrize("M,K,N", [(1, 256, 128), (3, 512, 384), (8, 1024, 128), (9, 768, 256)])
def test_parity(fmt, mask, dtype, out, M, K, N):
    import fp4_sparse_dense_b200 as sq
    rng = np.random.default_rng(M + K + N)
    w, w64 = make_weight(rng, K, N, fmt, mask)
    x = heavy_activations(rng, M, K, dtype=F16 if dtype == "f16" else BF16)
    y = sq.matvec(to_device(x), w, out_dtype=tdt(out))
    assert y.dtype == tdt(out) and list(y.shape) == [M, N]
    check(y, x.values.astype(np.float64), w64, out)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 16, 17, 24, 31, 32, 33, 65, 100])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_row_counts(M, dtype):
    import fp4_sparse_dense_b200 as sq
    rng = np.random.default_rng(M)
    w, w64 = make_weight(rng, 512, 256, "nvfp4", "pair48")
    x = heavy_activations(rng, M, 512, dtype=F16 if dtype == "f16" else BF16)
    y = sq.matvec(to_device(x), w, out_dtype=tdt("f32"))
    check(y, x.values.astype(np.float64), w64, "f32")


@pytest.mark.parametrize("K,N", [(4096, 1024), (14336, 256), (256, 4096), (2816, 640)])
@pytest.mark.parametrize("M", [1, 5, 20])
def test_layer_shapes(K, N, M):
    import fp4_sparse_dense_b200 as sq
    rng = np.random.default_rng(K + N + M)
    w, w64 = make_weight(rng, K, N, "mxfp4", "pair48")
    x = heavy_activations(rng, M, K)
    check(sq.matvec(to_device(x), w, out_dtype=tdt("f32")), x.values.astype(np.float64), w64, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt,mask", VIEWS)
def test_unit_rows_return_the_weight(fmt, mask, dtype):
    """x = e_k picks column k of the dequantised weight, exactly: one product, zeros beside it,
    one rounding by the tensor scale."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(5)
    K, N = 256, 128
    w, w64 = make_weight(rng, K, N, fmt, mask)
    y = sq.matvec(torch.eye(K, dtype=tdt(dtype), device="cuda"), w, out_dtype=torch.float32)
    assert np.array_equal(y.cpu().numpy(), w64.T.astype(np.float32))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_scale_byte(dtype):
    """Every E4M3 scale (0 ... 0x7E) and every E8M0 scale of a finite float32 weight, with
    every code: the exact value, subnormal and largest ones among them."""
    import fp4_sparse_dense_b200 as sq
    import torch
    K, N = 512, 128
    rng = np.random.default_rng(6)
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    for fmt, mask, block, top in (("nvfp4", "none", 16, 0x7F), ("nvfp4", "pair48", 32, 0x7F),
                                  ("mxfp4", "none", 32, 252)):
        raw = (np.arange(N * K // block) % top).astype(np.uint8).reshape(N, K // block)
        vals = F.e4m3_decode(raw) if fmt == "nvfp4" else F.e8m0_decode(raw)
        w64 = F.e2m1_decode(codes) * np.repeat(vals, block, axis=1)
        buf = {"codes": L.pack_nibbles(codes).reshape(-1), "tensor_scale": np.array([1.0], np.float32)}
        buf["scales_dense"] = L.to_scale_layout(raw if block == 16 or fmt == "mxfp4" else np.repeat(raw, 2, 1))
        buf["scales_sparse"] = L.to_scale_layout(raw)
        w = upload_weight(buf, K, N, cfg_of(fmt, mask))
        y = sq.matvec(torch.eye(K, dtype=tdt(dtype), device="cuda"), w, out_dtype=torch.float32)
        assert np.array_equal(y.cpu().numpy().astype(np.float64), w64.T), (fmt, mask)


def test_small_and_large_halves():
    """fp16 activations from the smallest subnormal to the largest value are exact operands."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(7)
    K, N = 256, 128
    w, w64 = make_weight(rng, K, N, "nvfp4", "pair48")
    bits = rng.integers(0, 0x7C00, (24, K)).astype(np.uint16) | (rng.integers(0, 2, (24, K)) << 15).astype(np.uint16)
    x = torch.from_numpy(bits.view(np.float16).copy()).cuda()
    x[0] = 0
    x[0, 3] = 2.0 ** -24
    x[1] = 0
    x[1, 200] = 65504
    y = sq.matvec(x, w, out_dtype=torch.float32)
    check(y, x.double().cpu().numpy(), w64, "f32")
    assert np.array_equal(y[0].cpu().numpy(), (w64[:, 3] * 2.0 ** -24).astype(np.float32))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_infinities_and_nan_stay_in_their_row(dtype):
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(8)
    K, N = 512, 128
    w, w64 = make_weight(rng, K, N, "nvfp4", "pair48")
    x = to_device(heavy_activations(rng, 6, K, dtype=F16 if dtype == "f16" else BF16))
    clean = sq.matvec(x, w, out_dtype=torch.float32)
    x2 = x.clone()
    x2[1, 17], x2[3, 400], x2[4, 5] = float("inf"), float("nan"), float("-inf")
    y = sq.matvec(x2, w, out_dtype=torch.float32).cpu().numpy()
    for r in (0, 2, 5):
        assert np.array_equal(y[r], clean[r].cpu().numpy())
    assert np.isnan(y[3]).all()
    for r, k, s in ((1, 17, 1), (4, 5, -1)):
        col = w64[:, k]
        assert np.isnan(y[r][col == 0]).all()
        assert np.array_equal(y[r][col != 0], np.sign(col[col != 0]) * s * np.inf)


def test_strides_and_views():
    """Rows of a wider matrix, an odd pitch, an offset start and a transposed X; the output a
    column range of a wider matrix whose other columns stay."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(9)
    K, N, M = 256, 128, 5
    w, w64 = make_weight(rng, K, N, "nvfp4", "none")
    x = to_device(heavy_activations(rng, M, K))
    want = sq.matvec(x, w, out_dtype=torch.float32)
    for pitch, off in ((K + 64, 8), (K + 3, 0), (K + 8, 1), (2 * K, K)):
        big = torch.full((M, pitch + off), float("nan"), dtype=x.dtype, device="cuda")
        big[:, off:off + K] = x
        assert torch.equal(sq.matvec(big[:, off:off + K], w, out_dtype=torch.float32), want)
    assert torch.equal(sq.matvec(x.t().contiguous().t(), w, out_dtype=torch.float32), want)
    assert torch.equal(sq.matvec(x[:1].expand(3, K), w, out_dtype=torch.float32), want[:1].expand(3, N))
    big = torch.full((M + 1, N + 36), 7.0, device="cuda")
    y = sq.matvec(x, w, out=big[:M, 4:4 + N])
    assert y.data_ptr() == big.data_ptr() + 16
    assert torch.equal(big[:M, 4:4 + N], want)
    assert (big[:, :4] == 7).all() and (big[:, 4 + N:] == 7).all() and (big[M] == 7).all()


def test_no_rows():
    import fp4_sparse_dense_b200 as sq
    import torch
    w, _ = make_weight(np.random.default_rng(1), 256, 128, "nvfp4", "pair48")
    y = sq.matvec(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), w)
    assert list(y.shape) == [0, 128]


def test_repeatable_and_row_independent():
    """The same bits every time, and a row's result does not depend on the rows beside it
    within its group."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(10)
    w, _ = make_weight(rng, 4096, 512, "nvfp4", "pair48")
    x = to_device(heavy_activations(rng, 8, 4096))
    y = sq.matvec(x, w, out_dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(sq.matvec(x, w, out_dtype=torch.float32), y)
    assert torch.equal(sq.matvec(x[:3], w, out_dtype=torch.float32), y[:3])


def test_other_stream_and_graph():
    """On a side stream beside work on the main one, and captured: a replay reads the inputs of
    that moment."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(11)
    w, w64 = make_weight(rng, 1024, 256, "nvfp4", "pair48")
    x1, x2 = (to_device(heavy_activations(rng, 4, 1024)) for _ in range(2))
    want1, want2 = (sq.matvec(x, w, out_dtype=torch.float32) for x in (x1, x2))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y1 = sq.matvec(x1, w, out_dtype=torch.float32, stream=side)
    y2 = sq.matvec(x2, w, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(y1, want1) and torch.equal(y2, want2)

    x, y = x1.clone(), torch.zeros(4, 256, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sq.matvec(x, w, out=y)
        z = y * 2
        sq.matvec(x, w, out=y)
    for src, want in ((x2, want2), (x1, want1)):
        x.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(z, 2 * want)


def test_beside_linear_on_one_stream():
    """Chains of matvec and the prepared linear layer on one stream, each reading what the one
    before wrote, and a weight re-quantised by this library in between."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(12)
    K = N = 512
    wa, wb = gaussian_weight(rng, K, N), gaussian_weight(rng, K, N)
    w64 = [weight64(S.quantize_weight(v.values)) for v in (wa, wb)]
    w = sq.quantize_weight(to_device(wa))
    x = heavy_activations(rng, 2, K)
    xd, da, db = to_device(x), to_device(wa), to_device(wb)
    for _ in range(10):
        sq.quantize_weight(da, out=w)
        h = sq.matvec(xd, w)
        first = sq.linear(sq.prepare(h), w, out_dtype=torch.float32)
        sq.quantize_weight(db, out=w)
        h2 = sq.matvec(xd, w, out_dtype=torch.float32)
        check(h, x.values.astype(np.float64), w64[0], "bf16")
        check(h2, x.values.astype(np.float64), w64[1], "f32")
        p = S.prepare(h.float().cpu().numpy())
        assert rel_fro(first.cpu().numpy(), S.linear(p, S.quantize_weight(wa.values))) <= 1e-5
    assert sq.sharq_device_status() == 0


def test_refusals_of_the_helper():
    import fp4_sparse_dense_b200 as sq
    import torch
    w, _ = make_weight(np.random.default_rng(1), 256, 128, "nvfp4", "pair48")
    ok = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        sq.matvec(ok.float(), w)
    with pytest.raises(TypeError):
        sq.matvec(ok, w, out_dtype=torch.float64)
    for bad in (ok[0], ok[:, :128], torch.zeros(2, 512, dtype=torch.bfloat16, device="cuda")):
        with pytest.raises(ValueError):
            sq.matvec(bad, w)
    for out in (torch.zeros(3, 128, device="cuda"), torch.zeros(2, 64, device="cuda"),
                torch.zeros(128, 2, device="cuda").t(), torch.zeros(2, 128)):
        with pytest.raises(ValueError):
            sq.matvec(ok, w, out=out)
    with pytest.raises(sq.SharqError):
        sq.matvec(ok, w, out=torch.zeros(2, 133, device="cuda")[:, 1:129])
