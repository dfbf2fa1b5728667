"""GPU parity of the few-row products where the tensor-core kernel takes them (more than eight
rows of a weight): row counts around its slots of 16 and 32 rows, more tiles than run at once, K
split over a cluster, ragged experts, and buffers beyond 32-bit offsets.

Tolerances: those of test_gpu_e_matvec.py. This kernel's accumulators take at most K / 16 MMAs
in all, as counted there, and its sums are joined by fewer float32 additions."""
import numpy as np
import pytest

from oracle import formats as F
from oracle import sharq as S
from tests.gpu_helpers import to_device
from tests.test_gpu_e_matvec import VIEWS, check, make_weight, tdt
from tests.test_gpu_f_experts import check_experts, dev, make_experts, route, sorted_np
from workloads import BF16, F16, heavy_activations

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,mask", VIEWS)
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("f16", "f32"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("M,K,N", [(9, 256, 128), (16, 512, 384), (17, 1280, 128), (33, 768, 256)])
def test_parity(fmt, mask, dtype, out, M, K, N):
    import fp4_sparse_dense_b200 as sq
    rng = np.random.default_rng(M + K + N)
    w, w64 = make_weight(rng, K, N, fmt, mask)
    x = heavy_activations(rng, M, K, dtype=F16 if dtype == "f16" else BF16)
    check(sq.matvec(to_device(x), w, out_dtype=tdt(out)), x.values.astype(np.float64), w64, out)


@pytest.mark.parametrize("M", [10, 15, 23, 24, 25, 31, 32, 40, 48, 63, 64, 65, 97, 300, 1000])
def test_row_counts(M):
    import fp4_sparse_dense_b200 as sq
    rng = np.random.default_rng(M)
    w, w64 = make_weight(rng, 512, 128, "nvfp4", "none")
    x = heavy_activations(rng, M, 512)
    check(sq.matvec(to_device(x), w, out_dtype=tdt("f32")), x.values.astype(np.float64), w64, "f32")


@pytest.mark.parametrize("M,K,N", [(20, 256, 51200),    # 400 tiles: two rounds of the CTAs
                                   (70, 256, 25600),    # three slots, 600 tiles
                                   (12, 4096, 128),     # one tile: K over eight CTAs
                                   (32, 1792, 256),     # 14 steps over two
                                   (20, 14336, 640), (9, 14336, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_tiles_and_clusters(M, K, N, dtype):
    import fp4_sparse_dense_b200 as sq
    rng = np.random.default_rng(K + N)
    w, w64 = make_weight(rng, K, N, "mxfp4" if K == 1792 else "nvfp4", "pair48")
    x = heavy_activations(rng, M, K, dtype=F16 if dtype == "f16" else BF16)
    check(sq.matvec(to_device(x), w, out_dtype=tdt("f32")), x.values.astype(np.float64), w64, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_infinities_and_nan_stay_in_their_row(dtype, fmt):
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(8)
    K, N, M = 512, 128, 20
    w, w64 = make_weight(rng, K, N, fmt, "pair48")
    x = to_device(heavy_activations(rng, M, K, dtype=F16 if dtype == "f16" else BF16))
    clean = sq.matvec(x, w, out_dtype=torch.float32)
    x2 = x.clone()
    x2[1, 17], x2[13, 400], x2[19, 5] = float("inf"), float("nan"), float("-inf")
    y = sq.matvec(x2, w, out_dtype=torch.float32).cpu().numpy()
    for r in set(range(M)) - {1, 13, 19}:
        assert np.array_equal(y[r], clean[r].cpu().numpy())
    assert np.isnan(y[13]).all()
    for r, k, s in ((1, 17, 1), (19, 5, -1)):
        col = w64[:, k]
        assert np.isnan(y[r][col == 0]).all()
        assert np.array_equal(y[r][col != 0], np.sign(col[col != 0]) * s * np.inf)


@pytest.mark.parametrize("T,k,E,drop", [(400, 2, 40, 0.1), (50, 1, 1, 0.0), (300, 4, 9, 0.5), (40, 8, 33, 0.0)])
@pytest.mark.parametrize("fmt,dtype", [("nvfp4", "bf16"), ("mxfp4", "f16")])
def test_ragged_experts(T, k, E, drop, fmt, dtype):
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(T + E)
    K, N = 512, 256
    w, w64 = make_experts(rng, E, K, N, fmt, "pair48")
    ids = route(rng, T, k, E, drop)
    x = heavy_activations(rng, T, K, dtype=F16 if dtype == "f16" else BF16)
    t, _ = sq.sort_tokens(dev(ids), E)
    y = torch.full((T * k, N), 9.0, device="cuda")
    sq.expert_matvec(to_device(x), w, t, gather=True, out=y)
    offsets, order, _ = sorted_np(ids, E)
    check_experts(y, x.values.astype(np.float64), w64, offsets, order // k, "f32")
    assert (y[offsets[E]:] == 9).all()


def test_graphs_on_two_streams_and_repeats():
    """Two captured chains of products replayed at once give the eager run's bits, every time."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(3)
    K = N = 1024
    w, _ = make_weight(rng, K, N, "nvfp4", "pair48")
    xs = [to_device(heavy_activations(rng, 24, K)) for _ in range(2)]

    def chain(x):
        y = sq.matvec(x, w)
        return sq.matvec(y[:4], w), sq.matvec(y, w, out_dtype=torch.float32)

    want = [chain(x) for x in xs]
    for a, b in zip(chain(xs[0]), want[0]):
        assert torch.equal(a, b)
    graphs = []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = chain(x)
        graphs.append((g, out, torch.cuda.Stream()))
    for _ in range(5):
        torch.cuda.synchronize()
        for g, _, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, out, _), exp in zip(graphs, want):
            assert torch.equal(out[0], exp[0]) and torch.equal(out[1], exp[1])
    assert sq.sharq_device_status() == 0


def test_beside_the_prepared_linear_on_another_stream():
    """Both use tensor memory; a CTA of one waits for the other's to leave, none for ever."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(4)
    K = N = 1024
    w, _ = make_weight(rng, K, N, "nvfp4", "pair48")
    x = to_device(heavy_activations(rng, 512, K))
    few = x[:32].contiguous()
    want, want2 = sq.linear(sq.prepare(x), w), sq.matvec(few, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(30):
        a = sq.matvec(few, w, stream=side)
        b = sq.linear(sq.prepare(x), w)
        outs.append((a, b))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, want2) and torch.equal(b, want)
    assert sq.sharq_device_status() == 0


@pytest.mark.parametrize("M", [2, 20])
def test_weight_beyond_32_bit_offsets(M):
    """A weight of 2.2 GB of codes: outputs sampled from its start, middle and end."""
    import fp4_sparse_dense_b200 as sq
    import torch
    K, N = 16384, 128 * 2112
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    w = sq.empty_weight(K, N, sq.Config.from_names("nvfp4", "none"))
    w.codes.copy_(torch.randint(0, 256, (w.codes.numel(),), dtype=torch.uint8, device="cuda", generator=g))
    w.scales_dense.copy_(torch.randint(40, 72, (w.scales_dense.numel(),), dtype=torch.uint8, device="cuda", generator=g))
    w.tensor_scale[0] = 1.0
    x = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    y = sq.matvec(x, w, out_dtype=torch.float32)
    rows = np.concatenate([np.arange(0, 40), np.arange(N // 2, N // 2 + 40), np.arange(N - 40, N)])
    codes = w.codes.view(N, K // 2)[torch.from_numpy(rows).cuda()].cpu().numpy()
    codes = np.stack((codes & 15, codes >> 4), axis=-1).reshape(len(rows), K)
    C = K // 16
    cols = np.arange(C)[None, :]
    at = ((rows[:, None] // 128) * (C // 4) + cols // 4) * 512 + (rows[:, None] % 32) * 16 + \
        (rows[:, None] // 32 % 4) * 4 + cols % 4
    raw = w.scales_dense[torch.from_numpy(at).cuda()].cpu().numpy()
    w64 = F.e2m1_decode(codes) * np.repeat(F.e4m3_decode(raw), 16, axis=1)
    check(y[:, torch.from_numpy(rows).cuda()], x.double().cpu().numpy(), w64, "f32")


def test_rows_beyond_32_bit_offsets():
    """2.2e9 gathered elements: the last token's rows and their way back."""
    import fp4_sparse_dense_b200 as sq
    import torch
    T, k, H = 65600, 2, 16448
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    ids[:, 1] = 1
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.arange(T, device="cuda").remainder(251).to(torch.bfloat16).unsqueeze(1).expand(T, H))
    t, rows = sq.sort_tokens(ids, 2, x)
    assert rows.numel() > 2 ** 31
    for p in (0, T - 1, T, 2 * T - 1):
        assert (rows[p] == float((p % T) % 251)).all()
    y = sq.combine_tokens(rows, t)
    for i in (0, T // 2, T - 1):
        assert (y[i] == float(torch.tensor(2.0 * (i % 251)).to(torch.bfloat16))).all()


def test_more_assignments_than_a_round_of_the_gradient():
    """70 assignments per token: the weights' gradient in two rounds."""
    import fp4_sparse_dense_b200 as sq
    rng = np.random.default_rng(6)
    T, k, E, H = 5, 70, 100, 264
    ids = route(rng, T, k, E, 0.2)
    t, _ = sq.sort_tokens(dev(ids), E)
    _, _, place = sorted_np(ids, E)
    rows, dy = rng.standard_normal((T * k, H)).astype(np.float32), rng.standard_normal((T, H)).astype(np.float32)
    w = rng.standard_normal((T, k)).astype(np.float32)
    d_rows, d_w = sq.combine_tokens_backward(dev(dy), dev(rows), t, dev(w))
    d_rows, d_w = d_rows.cpu().numpy(), d_w.cpu().numpy()
    for i in range(T):
        for j in range(k):
            if place[i, j] < 0:
                assert d_w[i, j] == 0
                continue
            prod = dy[i].astype(np.float64) * rows[place[i, j]]
            assert abs(d_w[i, j] - prod.sum()) <= (H + 1) * 2.0 ** -24 * np.abs(prod).sum()
            assert np.array_equal(d_rows[place[i, j]], w[i, j] * dy[i])
