"""GPU tests of the experts' operators: the sort by expert, the rows' way there and back with
its gradients, and the experts' products, each against plain numpy in 64 bits.

Tolerances. Sorted orders and moved rows are exact. A combination of k rows in float32 is off
by at most (k + 1) * 2^-24 of sum |w r| (a product and an addition per term) before its one
rounding (half a step: bf16 2^-8, fp16 2^-11, float32 2^-24, relative; fp16 also half its
smallest step, 2^-25); a dot product over H by at most (H + 1) * 2^-24 of sum |a b|. The
products' bound is the few-row product's."""
import numpy as np
import pytest

from oracle import sharq as S
from tests.gpu_helpers import to_device
from tests.test_gpu_e_matvec import EPS, check, tdt, weight64
from workloads import BF16, F16, gaussian_weight, heavy_activations

pytestmark = pytest.mark.gpu


def sorted_np(ids, E):
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[order], np.arange(E + 1), side="left")
    place = np.empty(flat.size, np.int64)
    place[order] = np.arange(flat.size)
    place[key == E] = -1
    return offsets, order, place.reshape(ids.shape)


def route(rng, T, k, E, drop=0.0):
    ids = np.argsort(rng.random((T, E)) + 0.3 * rng.random(E), axis=1)[:, :k].astype(np.int64) \
        if k <= E else rng.integers(0, E, (T, k))
    ids[rng.random((T, k)) < drop] = -1
    return ids


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def plan_equal(t, ids, E):
    offsets, order, place = sorted_np(ids, E)
    assert np.array_equal(t.offsets.cpu().numpy(), offsets)
    assert np.array_equal(t.order.cpu().numpy(), order)
    assert np.array_equal(t.place.cpu().numpy().reshape(place.shape), place)
    return offsets, order, place


# ------------------------------------------------------------------ the sort

@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 2, 8), (1, 8, 256), (5, 3, 4), (31, 1, 2), (32, 1, 2),
                                   (33, 4, 60), (700, 6, 60), (1024, 1, 1024), (1025, 2, 1000),
                                   (4096, 2, 8), (8191, 8, 128), (20000, 3, 17), (3, 40, 7)])
@pytest.mark.parametrize("bits", [32, 64])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_sort(T, k, E, bits, drop):
    import fp4_sparse_dense_b200 as sq
    import torch
    ids = route(np.random.default_rng(T + k + E), T, k, E, drop)
    t, rows = sq.sort_tokens(dev(ids, torch.int32 if bits == 32 else torch.int64), E)
    assert rows is None
    plan_equal(t, ids, E)


def test_sort_ids_outside():
    """Ids below, at and far beyond the experts' range are dropped, none wraps around."""
    import fp4_sparse_dense_b200 as sq
    import torch
    ids = np.array([[0, 7, 8], [-1, 2 ** 40 + 3, -2 ** 40], [2 ** 32 + 1, 2 ** 31, 7], [-2 ** 63, 2 ** 63 - 1, 3]])
    plan_equal(sq.sort_tokens(dev(ids), 8)[0], ids, 8)
    small = np.array([[0, 7, 8], [-1, 2 ** 31 - 1, -2 ** 31]])
    plan_equal(sq.sort_tokens(dev(small, torch.int32), 8)[0], small, 8)


@pytest.mark.parametrize("value", [-1, 0, 5])
def test_sort_all_alike(value):
    """One expert has everything, or all is dropped."""
    import fp4_sparse_dense_b200 as sq
    ids = np.full((2050, 3), value, np.int64)
    plan_equal(sq.sort_tokens(dev(ids), 6)[0], ids, 6)


def test_sort_duplicates_in_a_token():
    import fp4_sparse_dense_b200 as sq
    ids = np.random.default_rng(0).integers(0, 3, (50, 5))
    plan_equal(sq.sort_tokens(dev(ids), 3)[0], ids, 3)


def test_sort_into_given_buffers_and_views():
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(1)
    first, second = (route(rng, 64, 4, 16) for _ in range(2))
    t, _ = sq.sort_tokens(dev(first), 16)
    again, _ = sq.sort_tokens(dev(second), 16, out=t)
    assert again is t
    plan_equal(t, second, 16)
    wide = dev(np.concatenate((first, second), axis=1))
    plan_equal(sq.sort_tokens(wide[:, 4:], 16)[0], second, 16)
    with pytest.raises(ValueError):
        sq.sort_tokens(dev(first[:32]), 16, out=t)
    with pytest.raises(TypeError):
        sq.sort_tokens(dev(first).to(torch.int16), 16)


ROWS = [(1, 2, 8, 4096), (7, 4, 16, 2050), (33, 3, 5, 129), (64, 2, 8, 1), (5, 2, 4, 8), (100, 6, 60, 2056),
        (9, 1, 3, 20), (300, 2, 4, 36)]


@pytest.mark.parametrize("T,k,E,H", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_rows_there_and_back(T, k, E, H, dtype, drop):
    """sort with its rows, the gather's gradient, the combination and its gradients; rows
    behind the last kept assignment keep what they held, and nothing of them is read."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(T + H)
    dt = tdt(dtype)
    ids = route(rng, T, k, E, drop)
    n, tiny = T * k, 2.0 ** -25 if dtype == "f16" else 0.0
    x = dev(rng.standard_normal((T, H)), dt)
    rows = torch.full((n, H), float("nan"), dtype=dt, device="cuda")
    t, got = sq.sort_tokens(dev(ids), E, x, rows=rows)
    assert got is rows
    offsets, order, place = plan_equal(t, ids, E)
    m = offsets[E]
    assert torch.equal(rows[:m], x[dev(order[:m] // k)])
    assert torch.isnan(rows[m:]).all()
    kept = place >= 0

    d_rows = dev(rng.standard_normal((n, H)), dt)
    d_rows[m:] = float("nan")
    d64 = d_rows.double().cpu().numpy()
    want, mag = np.zeros((T, H)), np.zeros((T, H))
    for j in range(k):
        r = np.where(kept[:, j:j + 1], d64[place[:, j]], 0)
        want += r
        mag += np.abs(r)
    dx = sq.sort_tokens_backward(d_rows, t).double().cpu().numpy()
    assert (np.abs(dx - want) <= (k + 1) * 2.0 ** -24 * mag + np.abs(want) * EPS[dtype] * 1.01 + tiny).all()

    w = rng.standard_normal((T, k)).astype(np.float32)
    wn = np.where(kept, w, np.nan)  # a dropped assignment's weight is not read
    y = sq.combine_tokens(d_rows, t, dev(wn.astype(np.float32))).double().cpu().numpy()
    want, mag = np.zeros((T, H)), np.zeros((T, H))
    for j in range(k):
        r = np.where(kept[:, j:j + 1], d64[place[:, j]] * w[:, j:j + 1], 0)
        want += r
        mag += np.abs(r)
    assert (np.abs(y - want) <= (k + 1) * 2.0 ** -24 * mag + np.abs(want) * EPS[dtype] * 1.01 + tiny).all()

    dy = dev(rng.standard_normal((T, H)), dt)
    dy64 = dy.double().cpu().numpy()
    keep = torch.full((n, H), 3.0, dtype=dt, device="cuda")
    gr, gw = sq.combine_tokens_backward(dy, d_rows, t, dev(wn.astype(np.float32)), d_rows=keep)
    assert gr is keep and (keep[m:] == 3).all()
    gr, gw = gr.double().cpu().numpy(), gw.cpu().numpy()
    for j in range(k):
        k_j, p_j = kept[:, j], place[:, j]
        want = w[k_j, j:j + 1].astype(np.float64) * dy64[k_j]
        got = gr[p_j[k_j]]
        # w dy in float32 (half a step of 2^-24), then one rounding
        assert (np.abs(got - want) <= np.abs(want) * (EPS[dtype] * 1.01 + 2.0 ** -24) + tiny).all()
        a, b = dy64[k_j], d64[p_j[k_j]]
        dot, mag = (a * b).sum(1), np.abs(a * b).sum(1)
        assert (np.abs(gw[k_j, j] - dot) <= (H + 1) * 2.0 ** -24 * mag).all()
        assert (gw[~k_j, j] == 0).all()


def test_gradients_against_differences():
    """Gradient of L = sum(combine(sort(x) * c, w) * v) against the loss's own differences. L is
    linear in x and in w, so its difference quotient over a step of 1 is the derivative itself
    up to rounding: with values of up to 8 bits every product and sum here is exact in
    float32."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(3)
    T, k, E, H = 6, 3, 5, 12
    ids = dev(route(rng, T, k, E, 0.2))
    small = lambda *s: dev(rng.integers(-8, 9, s).astype(np.float32))  # noqa: E731
    x, w, c, v = small(T, H), small(T, k), small(T * k, H), small(T, H)

    def loss(x, w):
        t, rows = sq.sort_tokens(ids, E, x, rows=torch.zeros(T * k, H, device="cuda"))
        return float((sq.combine_tokens(rows * c, t, w) * v).sum()), t, rows

    base, t, rows = loss(x, w)
    d_rows = torch.zeros(T * k, H, device="cuda")
    _, d_w = sq.combine_tokens_backward(v, rows * c, t, w, d_rows=d_rows)
    dx = sq.sort_tokens_backward(d_rows * c, t)
    for i in range(T):
        for h in range(H):
            step = x.clone()
            step[i, h] += 1
            assert loss(step, w)[0] - base == float(dx[i, h])
        for j in range(k):
            step = w.clone()
            step[i, j] += 1
            assert loss(x, step)[0] - base == float(d_w[i, j])


def test_infinities_in_kept_and_dropped_rows():
    import fp4_sparse_dense_b200 as sq
    import torch
    ids = np.array([[0, 1], [1, -1], [-1, -1]])
    rows = torch.tensor([[1.0, float("inf")], [2.0, 3.0], [float("nan"), 4.0]] + [[float("nan")] * 2] * 3,
                        device="cuda")
    t, _ = sq.sort_tokens(dev(ids), 2)
    y = sq.combine_tokens(rows, t).cpu().numpy()   # token 0: rows 0 and 1, token 1: row 2
    assert y[0, 0] == 3 and y[0, 1] == np.inf and np.isnan(y[1, 0]) and y[1, 1] == 4
    assert (y[2] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_rows(dtype):
    """Rows inside wider matrices, on both sides, an expanded gradient, a transposed input."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(4)
    T, k, E, H = 20, 2, 4, 64
    dt = tdt(dtype)
    ids = dev(route(rng, T, k, E, 0.2))
    x = dev(rng.standard_normal((T, H)), dt)
    zero = lambda: torch.zeros(T * k, H, dtype=dt, device="cuda")  # noqa: E731
    t, rows = sq.sort_tokens(ids, E, x, rows=zero())
    for pitch, off in ((H + 8, 0), (H + 5, 3), (H + 2, 2)):
        big = torch.zeros(T, pitch + off, dtype=dt, device="cuda")
        big[:, off:off + H] = x
        dst = torch.full((T * k, pitch + off), 5.0, dtype=dt, device="cuda")
        dst[:, off:off + H] = 0
        sq.sort_tokens(ids, E, big[:, off:off + H], rows=dst[:, off:off + H])
        assert torch.equal(dst[:, off:off + H], rows)
        assert (dst[:, :off] == 5).all() and (dst[:, off + H:] == 5).all()
        out = torch.full((T, pitch + off), 5.0, dtype=dt, device="cuda")
        sq.combine_tokens(dst[:, off:off + H], t, out=out[:, off:off + H])
        assert torch.equal(out[:, off:off + H], sq.combine_tokens(rows, t))
        assert (out[:, :off] == 5).all() and (out[:, off + H:] == 5).all()
    assert torch.equal(sq.sort_tokens(ids, E, x.t().contiguous().t(), rows=zero())[1], rows)
    w = dev(rng.random((T, k)).astype(np.float32))
    one = torch.ones((), dtype=dt, device="cuda").expand(T, H)
    a = sq.combine_tokens_backward(one, rows, t, w, d_rows=zero())
    b = sq.combine_tokens_backward(one.contiguous(), rows, t, w, d_rows=zero())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # in place: the gradient of the rows over the rows themselves
    own = rows.clone()
    c = sq.combine_tokens_backward(one, own, t, w, d_rows=own)
    m = int(t.offsets[E])
    assert torch.equal(own[:m], b[0][:m]) and torch.equal(c[1], b[1])


def test_no_tokens():
    import fp4_sparse_dense_b200 as sq
    import torch
    ids = torch.empty(0, 2, dtype=torch.int64, device="cuda")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    t, rows = sq.sort_tokens(ids, 4, x)
    assert (t.offsets == 0).all() and list(rows.shape) == [0, 64]
    w = torch.empty(0, 2, device="cuda")
    assert list(sq.combine_tokens(rows, t, w).shape) == [0, 64]
    assert list(sq.sort_tokens_backward(rows, t).shape) == [0, 64]
    assert [list(g.shape) for g in sq.combine_tokens_backward(x, rows, t, w)] == [[0, 64], [0, 2]]
    ew = sq.quantize_experts(torch.zeros(4, 256, 128, dtype=torch.bfloat16, device="cuda"))
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    assert list(sq.expert_matvec(e, ew, t).shape) == [0, 128]
    assert sq.sharq_device_status() == 0


# ------------------------------------------------------------------ the experts' products

def make_experts(rng, E, K, N, fmt, mask):
    import fp4_sparse_dense_b200 as sq
    import torch
    cfg = sq.Config.from_names(fmt, mask)
    ws = [gaussian_weight(rng, K, N, sigma=0.02 * (1 + e % 3)) for e in range(E)]
    w = sq.quantize_experts(torch.stack([to_device(v) for v in ws]), cfg)
    return w, [weight64(S.quantize_weight(v.values, fmt, mask)) for v in ws]


def check_experts(y, x64, w64, offsets, rows_of, out):
    for e in range(len(w64)):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            check(y[lo:hi], x64[rows_of[lo:hi]], w64[e], out)


@pytest.mark.parametrize("fmt,mask", [("nvfp4", "pair48"), ("nvfp4", "none"), ("mxfp4", "pair48")])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("T,k,E,drop", [(1, 2, 8, 0.0), (1, 1, 1, 0.0), (11, 2, 4, 0.3), (40, 3, 5, 0.0),
                                        (70, 2, 2, 0.5), (6, 4, 33, 0.1)])
def test_expert_products(fmt, mask, dtype, out, T, k, E, drop):
    """Sorted rows and gathered tokens give the same rows, bit for bit; empty experts, experts
    of more rows than a tile, and rows behind the last left as they were."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(T + E)
    K, N = 512, 256
    w, w64 = make_experts(rng, E, K, N, fmt, mask)
    ids = route(rng, T, k, E, drop)
    x = heavy_activations(rng, T, K, dtype=F16 if dtype == "f16" else BF16)
    xd = to_device(x)
    t, rows = sq.sort_tokens(dev(ids), E, xd, rows=torch.full((T * k, K), float("nan"), dtype=xd.dtype, device="cuda"))
    offsets, order, _ = sorted_np(ids, E)
    y = torch.full((T * k, N), 9.0, dtype=tdt(out), device="cuda")
    sq.expert_matvec(xd, w, t, gather=True, out=y)
    z = torch.full((T * k, N), 9.0, dtype=tdt(out), device="cuda")
    sq.expert_matvec(rows, w, t, out=z)
    assert torch.equal(y, z)
    assert (y[offsets[E]:] == 9).all()
    check_experts(y, x.values.astype(np.float64), w64, offsets, order // k, out)


@pytest.mark.parametrize("counts", [[0, 0, 100, 0], [33, 0, 0, 1], [1, 31, 32, 64], [0, 0, 0, 0]])
def test_uneven_experts(counts):
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(sum(counts))
    K, N = 256, 128
    w, w64 = make_experts(rng, 4, K, N, "nvfp4", "pair48")
    ids = np.concatenate([np.full(c, e) for e, c in enumerate(counts)] + [np.full(3, -1)])
    ids = rng.permutation(ids).reshape(-1, 1)
    x = heavy_activations(rng, len(ids), K)
    t, _ = sq.sort_tokens(dev(ids), 4)
    y = torch.zeros(len(ids), N, device="cuda")
    sq.expert_matvec(to_device(x), w, t, gather=True, out=y)
    offsets, order, _ = sorted_np(ids, 4)
    check_experts(y, x.values.astype(np.float64), w64, offsets, order, "f32")
    assert (y[offsets[4]:] == 0).all()


def test_many_experts_few_rows():
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(2)
    E, K, N, T, k = 300, 256, 128, 4, 8
    w, w64 = make_experts(rng, E, K, N, "nvfp4", "pair48")
    ids = route(rng, T, k, E)
    t, _ = sq.sort_tokens(dev(ids), E)
    x = heavy_activations(rng, T, K)
    y = sq.expert_matvec(to_device(x), w, t, gather=True, out_dtype=torch.float32)
    offsets, order, _ = sorted_np(ids, E)
    check_experts(y, x.values.astype(np.float64), w64, offsets, order // k, "f32")


def moe(sq, x, ids, probs, E, up, down, t_out=None):
    import torch
    t, _ = sq.sort_tokens(ids, E, out=t_out)
    h = sq.expert_matvec(x, up, t, gather=True)
    a, b = h.float().chunk(2, dim=1)
    h = (torch.nn.functional.silu(a) * b).to(x.dtype)
    return sq.combine_tokens(sq.expert_matvec(h, down, t), t, probs)


@pytest.mark.parametrize("T", [1, 13])
def test_layer_of_experts(T):
    """sort -> gate|up -> activation -> down -> combine, against float64 with the same roundings
    of the intermediate rows: each bf16 rounding moves a value by at most 2^-8, three of them
    lie on the way, so 4 * 2^-8 of the norm bounds the result's error."""
    import fp4_sparse_dense_b200 as sq
    rng = np.random.default_rng(T)
    K, N, E, k = 512, 256, 6, 2
    up, up64 = make_experts(rng, E, K, 2 * N, "nvfp4", "pair48")
    down, down64 = make_experts(rng, E, N, K, "mxfp4", "pair48")
    ids = route(rng, T, k, E)
    probs = rng.random((T, k)).astype(np.float32)
    x = heavy_activations(rng, T, K)
    y = moe(sq, to_device(x), dev(ids), dev(probs), E, up, down).double().cpu().numpy()
    want = np.zeros((T, K))
    for i in range(T):
        for j in range(k):
            h = up64[ids[i, j]] @ x.values[i].astype(np.float64)
            a, b = h[:N], h[N:]
            want[i] += probs[i, j] * (down64[ids[i, j]] @ (a / (1 + np.exp(-a)) * b))
    assert np.linalg.norm(y - want) <= 4 * 2.0 ** -8 * np.linalg.norm(want)


def test_layer_of_experts_captured():
    """The whole layer in a CUDA graph, replayed on new tokens and new choices, and two graphs
    replayed at once on two streams: the bits of the eager run."""
    import fp4_sparse_dense_b200 as sq
    import torch
    rng = np.random.default_rng(20)
    K, N, E, k, T = 512, 256, 6, 2, 9
    up, _ = make_experts(rng, E, K, 2 * N, "nvfp4", "none")
    down, _ = make_experts(rng, E, N, K, "nvfp4", "pair48")
    data = [(to_device(heavy_activations(rng, T, K)), dev(route(rng, T, k, E, 0.2)),
             dev(rng.random((T, k)).astype(np.float32))) for _ in range(3)]
    want = [moe(sq, *d, E, up, down) for d in data]
    graphs = []
    for _ in range(2):
        x, ids, probs = (v.clone() for v in data[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = moe(sq, x, ids, probs, E, up, down)
        graphs.append((g, (x, ids, probs), y))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for a, b in ((0, 1), (2, 0), (1, 2)):
        for (g, state, y), i, s in zip(graphs, (a, b), streams):
            for dst, src in zip(state, data[i]):
                dst.copy_(src)
        torch.cuda.synchronize()
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][2], want[a]) and torch.equal(graphs[1][2], want[b])
    assert sq.sharq_device_status() == 0


def test_refusals_of_the_helpers():
    import fp4_sparse_dense_b200 as sq
    import torch
    ids = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    t, rows = sq.sort_tokens(ids, 3, x)
    w = sq.quantize_experts(torch.zeros(3, 256, 128, dtype=torch.bfloat16, device="cuda"))
    two = sq.quantize_experts(torch.zeros(2, 256, 128, dtype=torch.bfloat16, device="cuda"))
    probs = torch.zeros(4, 2, device="cuda")
    with pytest.raises(sq.SharqError):
        sq.sort_tokens(ids, 1025)
    with pytest.raises(ValueError):
        sq.sort_tokens(ids[0], 3)
    with pytest.raises(ValueError):
        sq.sort_tokens(ids, 3, x[:3])
    with pytest.raises(ValueError):
        sq.sort_tokens(ids, 3, x, rows=rows[:7])
    with pytest.raises(TypeError):
        sq.sort_tokens(ids, 3, x, rows=rows.float())
    with pytest.raises(ValueError):
        sq.sort_tokens(ids, 3, rows=rows)
    with pytest.raises(ValueError):
        sq.expert_matvec(rows, two, t)
    with pytest.raises(ValueError):
        sq.expert_matvec(rows, w, t, gather=True)   # 8 rows where 4 tokens are expected
    with pytest.raises(TypeError):
        sq.expert_matvec(rows.float(), w, t)
    with pytest.raises(TypeError):
        sq.combine_tokens(rows, t, probs.double())
    with pytest.raises(ValueError):
        sq.combine_tokens(rows, t, probs[:3])
    with pytest.raises(ValueError):
        sq.combine_tokens(x, t, probs)
    with pytest.raises(TypeError):
        sq.combine_tokens_backward(x.float(), rows, t, probs)
    with pytest.raises(ValueError):
        sq.combine_tokens_backward(x, rows, t, probs, d_weights=torch.zeros(4, 3, device="cuda"))
