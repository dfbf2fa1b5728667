"""GPU parity of the few-row products on every way through them that the sizes choose: experts whose
K is split over a cluster, and few rows of a K so long that the tensor-memory kernel takes them in
slots of 16. Each case asks the library which kernel takes it, so that a changed rule cannot leave
one of them untested unseen.

Tolerances: those of test_gpu_e_matvec.py. The weights are random codes and scales, decoded here."""
import ctypes

import numpy as np
import pytest

from oracle import formats as F
from oracle import layouts as L
from tests.gpu_helpers import cfg_of, to_device, upload_weight
from tests.test_gpu_e_matvec import VIEWS, check, tdt
from tests.test_gpu_f_experts import check_experts, dev, sorted_np
from workloads import BF16, F16, heavy_activations

pytestmark = pytest.mark.gpu


def plan(M, E, K):
    import fp4_sparse_dense_b200 as sq
    tile_rows, splits = ctypes.c_int32(), ctypes.c_int32()
    assert sq.sharq_matvec_plan(M, E, K, ctypes.byref(tile_rows), ctypes.byref(splits)) == 0
    return tile_rows.value, splits.value


def random_weight(rng, K, N, fmt, mask):
    """A weight of random codes and scales, and its float64 values [N, K]."""
    block = 16 if fmt == "nvfp4" and mask in ("none", "elem24") else 32
    codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
    raw = rng.integers(*((40, 72) if fmt == "nvfp4" else (118, 126)), (N, K // block)).astype(np.uint8)
    vals = F.e4m3_decode(raw) if fmt == "nvfp4" else F.e8m0_decode(raw)
    buf = {"codes": L.pack_nibbles(codes).reshape(-1), "tensor_scale": np.array([1.0], np.float32),
           "scales_dense": L.to_scale_layout(raw if block == 16 or fmt == "mxfp4" else np.repeat(raw, 2, 1)),
           "scales_sparse": L.to_scale_layout(raw)}
    return (upload_weight(buf, K, N, cfg_of(fmt, mask)),
            F.e2m1_decode(codes) * np.repeat(vals, block, axis=1))


def random_experts(rng, E, K, N, fmt, mask):
    import fp4_sparse_dense_b200 as sq
    import torch
    ws, w64 = zip(*(random_weight(rng, K, N, fmt, mask) for _ in range(E)))
    stack = [None if getattr(ws[0], name) is None else torch.stack([getattr(w, name).view(-1) for w in ws])
             for name in ("codes", "scales_dense", "scales_sparse", "tensor_scale")]
    return sq.ExpertWeights(*stack, K, N, E, ws[0].cfg), w64


LONG = [(16, 19712), (16, 28672), (13, 28672), (9, 36864), (8, 53248), (2, 204800)]


@pytest.mark.parametrize("M,K", LONG)
@pytest.mark.parametrize("fmt,mask", [v for v in VIEWS if v[1] != "elem24"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_slots_of_sixteen_rows(M, K, fmt, mask, dtype):
    import fp4_sparse_dense_b200 as sq
    assert plan(M, 0, K) == (16, 0)
    rng = np.random.default_rng(M)
    N = 128 if K > 100000 else 384
    w, w64 = random_weight(rng, K, N, fmt, mask)
    x = heavy_activations(rng, M, K, dtype=F16 if dtype == "f16" else BF16)
    check(sq.matvec(to_device(x), w, out_dtype=tdt("f32")), x.values.astype(np.float64), w64, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_infinities_and_nan_in_slots_of_sixteen_rows(dtype, fmt):
    import fp4_sparse_dense_b200 as sq
    import torch
    M, K, N = 14, 28672, 256
    assert plan(M, 0, K) == (16, 0)
    rng = np.random.default_rng(1)
    w, w64 = random_weight(rng, K, N, fmt, "pair48")
    x = to_device(heavy_activations(rng, M, K, dtype=F16 if dtype == "f16" else BF16))
    clean = sq.matvec(x, w, out_dtype=torch.float32)
    x2 = x.clone()
    x2[1, 17], x2[7, 20001], x2[13, K - 1] = float("inf"), float("nan"), float("-inf")
    y = sq.matvec(x2, w, out_dtype=torch.float32).cpu().numpy()
    for r in set(range(M)) - {1, 7, 13}:
        assert np.array_equal(y[r], clean[r].cpu().numpy())
    assert np.isnan(y[7]).all()
    for r, k, s in ((1, 17, 1), (13, K - 1, -1)):
        col = w64[:, k]
        assert np.array_equal(y[r], np.where(col == 0, np.nan, np.copysign(np.inf, col * s)), equal_nan=True)


def run_experts(counts, drop, K, N, fmt, mask, dtype, want_plan, k=1):
    """Rows of each expert as in `counts`, `drop` dropped ones among them, in a random order; sorted
    rows and gathered tokens give the same bits."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(sum(counts) + K)
    E, n = len(counts), sum(counts) + drop
    assert n % k == 0 and plan(n, E, K) == want_plan
    w, w64 = random_experts(rng, E, K, N, fmt, mask)
    ids = np.concatenate([np.full(c, e) for e, c in enumerate(counts)] + [np.full(drop, -1)]).astype(np.int64)
    ids = rng.permutation(ids).reshape(-1, k)
    x = heavy_activations(rng, n // k, K, dtype=F16 if dtype == "f16" else BF16)
    xd = to_device(x)
    t, rows = sq.sort_tokens(dev(ids), E, xd, rows=torch.full((n, K), float("nan"), dtype=xd.dtype, device="cuda"))
    y = torch.full((n, N), 9.0, device="cuda")
    sq.expert_matvec(xd, w, t, gather=True, out=y)
    z = torch.full((n, N), 9.0, device="cuda")
    sq.expert_matvec(rows, w, t, out=z)
    assert torch.equal(y, z)
    offsets, order, _ = sorted_np(ids, E)
    check_experts(y, x.values.astype(np.float64), w64, offsets, order // k, "f32")
    assert (y[offsets[E]:] == 9).all()
    assert sq.sharq_device_status() == 0


# a decoded token's and a small batch's down projection: K over a cluster
@pytest.mark.parametrize("fmt,mask", [("nvfp4", "none"), ("nvfp4", "pair48"), ("mxfp4", "pair48")])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts,drop,k,K,N,splits", [
    ([0, 1, 0, 0, 0, 1, 0, 0], 0, 2, 14336, 512, 4),      # one token, 2 of 8 experts
    ([1, 0, 0], 1, 2, 14336, 4096, 4),                    # one of its two choices dropped
    ([8] * 8, 0, 1, 14336, 256, 4),                       # a full slot each
    ([30, 0, 1, 9, 8, 0, 7, 1], 6, 2, 14336, 256, 4),     # four slots of one expert, empty ones
    ([3, 17, 0, 2], 0, 1, 6400, 1024, 2),
    ([5, 0, 11, 8], 4, 4, 28672, 384, 8),
    ([1, 7, 15], 1, 1, 49152, 1024, 8),                    # sums of few units at a time: phases
])
def test_experts_over_a_cluster(counts, drop, k, K, N, splits, fmt, mask, dtype):
    run_experts(counts, drop, K, N, fmt, mask, dtype, (0, splits), k)


@pytest.mark.parametrize("fmt,mask", [("nvfp4", "none"), ("nvfp4", "pair48"), ("mxfp4", "pair48")])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts,drop", [([8, 8, 8, 8], 0), ([20, 0, 12, 0], 0), ([0, 1, 0], 2), ([0, 0, 33, 0, 1], 2)])
def test_experts_in_slots_of_sixteen_rows(counts, drop, fmt, mask, dtype):
    run_experts(counts, drop, 51200, 128, fmt, mask, dtype, (16, 0))


@pytest.mark.parametrize("fmt,dtype", [("nvfp4", "bf16"), ("mxfp4", "f16")])
def test_experts_in_slots_of_thirty_two_rows(fmt, dtype):
    run_experts([40, 1, 0, 33], 2, 1024, 256, fmt, "pair48", dtype, (32, 0))


def layer(sq, x, ids, probs, E, up, down, bufs):
    """The steps of a layer of experts into buffers that are used again in every call."""
    t, rows = sq.sort_tokens(ids, E, x, rows=bufs["rows"], out=bufs["tokens"])
    h = sq.expert_matvec(rows, up, t, out=bufs["h"])
    y = sq.expert_matvec(h, down, t, out=bufs["y"])
    return sq.combine_tokens(y, t, probs, out=bufs["out"])


@pytest.mark.parametrize("T,k,E,K,N", [(9, 2, 8, 14336, 256),     # products over clusters, one launch sorts
                                       (700, 2, 200, 512, 256),   # a cluster sorts, the rows' kernel behind it
                                       (600, 2, 5, 512, 256)])    # the tensor-memory kernel
def test_chains_on_reused_buffers(T, k, E, K, N):
    """One call after the other on the same buffers, without a wait between them, and the same
    captured and replayed on two streams at once: the bits of calls that were waited for."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(T)
    cfg = cfg_of("nvfp4", "none")
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    up, down = (sq.quantize_experts(torch.randn(E, *s, device="cuda", generator=g).mul_(0.02).to(torch.bfloat16), cfg)
                for s in ((K, N), (N, K)))

    def buffers():
        bf = dict(dtype=torch.bfloat16, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        tokens = sq.SortedTokens(torch.zeros(E + 1, **i32), torch.zeros(T * k, **i32), torch.zeros(T, k, **i32), T, k, E)
        return dict(rows=torch.zeros(T * k, K, **bf), tokens=tokens, h=torch.zeros(T * k, N, **bf),
                    y=torch.zeros(T * k, K, **bf), out=torch.zeros(T, K, **bf))

    data = []
    for i in range(4):
        ids = rng.integers(-1 if i % 2 else 0, E, (T, k))
        if i == 3:
            ids[:] = -1  # nothing kept: the rows before stay in the buffers, the output is 0
        data.append((to_device(heavy_activations(rng, T, K)), dev(ids), dev(rng.random((T, k)).astype(np.float32))))
    bufs, want = buffers(), []
    for d in data:
        torch.cuda.synchronize()
        want.append(layer(sq, *d, E, up, down, bufs).clone())
        torch.cuda.synchronize()
    assert (want[3] == 0).all() and not (want[0] == 0).all()

    got = [layer(sq, *data[i], E, up, down, bufs).clone() for i in (0, 2, 3, 1, 0, 3, 2, 1) * 3]
    for y, i in zip(got, (0, 2, 3, 1, 0, 3, 2, 1) * 3):
        assert torch.equal(y, want[i])

    graphs = []
    for _ in range(2):
        state, b = tuple(v.clone() for v in data[0]), buffers()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer(sq, *state, E, up, down, b)
        graphs.append((graph, state, b["out"], torch.cuda.Stream()))
    for pair in ((0, 1), (3, 2), (1, 3), (2, 0)):
        torch.cuda.synchronize()
        for (graph, state, _, s), i in zip(graphs, pair):
            with torch.cuda.stream(s):
                for dst, src in zip(state, data[i]):
                    dst.copy_(src)
                graph.replay()
        torch.cuda.synchronize()
        for (_, _, out, _), i in zip(graphs, pair):
            assert torch.equal(out, want[i])
    assert sq.sharq_device_status() == 0
