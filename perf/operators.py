"""Measured cases of the 16-bit-activation operators on FP4 weights.

Four operators: the few-row product with 4-bit weights (`matvec`), tokens sorted by expert
(`sort_tokens`, and its gradient), the experts' products on the sorted rows (`expert_matvec`)
and the rows combined back into tokens (`combine_tokens`, and its gradient). `run` computes a
case with elementary torch operations in float32, or, where `own` is true, with the
package's entry points; `exact` computes it in float64.

Weight buffers have the layouts of include/sharq.h: codes [N][K/2] (even k in the low
nibble), scales in 512-byte chunks of 128 rows x 4 blocks.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases

def listed():
    def mv(name, M, K, N, fmt, block, dtype, out):
        return {"name": name, "op": "matvec", "M": M, "K": K, "N": N, "fmt": fmt,
                "block": block, "dtype": dtype, "out": out}

    def tok(name, op, T, k, E, H, dtype, ids, drop):
        return {"name": name, "op": op, "T": T, "k": k, "E": E, "H": H, "dtype": dtype,
                "ids": ids, "drop": drop}

    def ex(name, T, k, E, K, N, fmt, block, dtype, out, gather, drop):
        return {"name": name, "op": "expert_matvec", "T": T, "k": k, "E": E, "K": K, "N": N,
                "fmt": fmt, "block": block, "dtype": dtype, "out": out, "gather": gather,
                "drop": drop}

    return [
        # the attention output projection of one decoded token: the call's latency counts
        mv("o_proj, 1 token", 1, 4096, 4096, "nvfp4", 32, "bf16", "bf16"),
        # the fused gate|up projection of one token, plain NVFP4 weights: the weight stream counts
        mv("gate_up, 1 token", 1, 4096, 28672, "nvfp4", 16, "bf16", "bf16"),
        # the down projection of a small decode batch, MXFP4, fp16 activations
        mv("down, 8 tokens", 8, 14336, 4096, "mxfp4", 32, "f16", "f16"),
        # the fused q|k|v projection of an odd decode batch, float32 out (before rotary)
        mv("qkv, 21 tokens", 21, 4096, 6144, "nvfp4", 32, "bf16", "f32"),
        # the router's sort of one decoded token: launch latency only
        tok("sort, 1 token", "sort_tokens", 1, 2, 8, 4096, "bf16", "int64", 0.0),
        # the sort of a long prefill, two of eight experts, all rows gathered
        tok("sort, 8192 tokens", "sort_tokens", 8192, 2, 8, 4096, "bf16", "int64", 0.0),
        # the gradient of the gather in training, many small experts, some tokens over capacity
        tok("sort gradient, 1777 tokens", "sort_tokens_backward", 1777, 6, 60, 2048, "bf16", "int32", 0.05),
        # gate|up of the two experts that one decoded token uses
        ex("experts gate_up, 1 token", 1, 2, 8, 4096, 28672, "nvfp4", 32, "bf16", "bf16", True, 0.0),
        # the down projections of a decode batch over many small experts
        ex("64 experts down, 48 tokens", 48, 8, 64, 1024, 2048, "mxfp4", 32, "bf16", "bf16", False, 0.0),
        # the down projections of a larger decode batch; a quarter of the experts' rows live on another rank
        ex("experts down, 70 tokens", 70, 2, 8, 14336, 4096, "nvfp4", 16, "f16", "f32", False, 0.25),
        # rows of a small decode batch back to tokens, an odd hidden size
        tok("combine, 7 tokens", "combine_tokens", 7, 4, 16, 2050, "f16", "int64", 0.0),
        # the gradient of the combination over a training batch, some assignments dropped
        tok("combine gradient, 4096 tokens", "combine_tokens_backward", 4096, 2, 8, 4096, "bf16", "int64", 0.05),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("matvec", "matvec", "expert_matvec", "expert_matvec", "sort_tokens",
                     "sort_tokens_backward", "combine_tokens", "combine_tokens_backward"))
    fmt, block = rng.choice((("nvfp4", 16), ("nvfp4", 32), ("mxfp4", 32)))
    if op == "matvec":
        K, N = 256 * _log(rng, 1, 56), 128 * _log(rng, 1, 224)
        while K * N > 4096 * 28672:
            N = 128 * max(1, N // 256)
        dtype = rng.choice(("bf16", "f16"))
        return {"op": op, "M": _log(rng, 1, 32), "K": K, "N": N, "fmt": fmt, "block": block,
                "dtype": dtype, "out": rng.choice((dtype, "f32"))}
    E = _log(rng, 2, 64 if op == "expert_matvec" else 256)
    k = rng.randint(1, min(8, E))
    drop = rng.choice((0.0, 0.0, 0.05, 0.5))
    if op == "expert_matvec":
        K, N = 256 * _log(rng, 1, 56), 128 * _log(rng, 1, 112)
        while E * K * N > 8 * 14336 * 4096:
            N, K = 128 * max(1, N // 256), 256 * max(1, K // 512)
        dtype = rng.choice(("bf16", "f16"))
        return {"op": op, "T": _log(rng, 1, 70), "k": k, "E": E, "K": K, "N": N, "fmt": fmt,
                "block": block, "dtype": dtype, "out": rng.choice((dtype, "f32")),
                "gather": rng.random() < 0.5, "drop": drop}
    H, dtype = _log(rng, 16, 8192), rng.choice(("bf16", "f16", "f32"))
    T = _log(rng, 1, 8192)
    while T * k * H * (4 if dtype == "f32" else 2) > 4096 * 2 * 4096 * 2:
        T = T // 2
    return {"op": op, "T": max(1, T), "k": k, "E": E, "H": H, "dtype": dtype,
            "ids": rng.choice(("int32", "int64")), "drop": drop}


# ------------------------------------------------------------------ the inputs

def _activations(g, rows, cols, dtype):
    """Heavy-tailed activations with outlier channels: Student-t(4), 0.5 % of the elements
    twenty to fifty times larger (fp16: a tenth of that, inside its range)."""
    z = torch.randn(rows, cols, device="cuda", generator=g)
    chi = torch.zeros_like(z)
    for _ in range(4):
        chi += torch.randn(rows, cols, device="cuda", generator=g).square()
    x = z / (chi / 4).sqrt()
    big = torch.rand(rows, cols, device="cuda", generator=g)
    u = torch.rand(rows, cols, device="cuda", generator=g)
    x = torch.where(big < 0.005, x * (20 + 30 * u), x).clamp(-6e4, 6e4)
    return x.to(DTYPES[dtype])


def _tile(s):
    """Scales [N][C] in the 128 x 4 chunks of the weight layout (C padded to 4 by K % 256)."""
    N, C = s.shape
    return s.view(N // 128, 4, 32, C // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _untile(b, N, C):
    return b.view(N // 128, C // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(N, C)


def _weight(g, K, N, fmt, block):
    """One quantised weight of ~N(0, 0.02) values: codes [N, K/2], tiled scales of `block`
    elements, and for NVFP4 the dense view of 16-element blocks and the tensor scale."""
    w = torch.randn(N, K // block, block, device="cuda", generator=g) * 0.02
    amax = w.abs().amax(-1)
    if fmt == "nvfp4":
        ts = w.abs().max() / 2688
        sf = (amax / 6 / ts).to(torch.float8_e4m3fn)
        step = sf.float() * ts
        raw = sf.view(torch.uint8)
    else:
        ts = torch.ones((), device="cuda")
        e = torch.floor(torch.log2(amax.clamp_min(1e-30))) - 2
        step = torch.exp2(e)
        raw = (e + 127).to(torch.uint8)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    v = w / step.clamp_min(1e-30).unsqueeze(-1)
    code = torch.bucketize(v.abs(), mids).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    code = code.view(N, K // 2, 2)
    codes = code[..., 0] | (code[..., 1] << 4)
    sparse = _tile(raw)
    dense = sparse if fmt == "mxfp4" or block == 16 else _tile(raw.repeat_interleave(2, dim=1))
    tscale = torch.zeros(4, device="cuda")
    tscale[0] = ts
    tscale[1] = ts * 2688
    return codes.reshape(-1), dense, sparse, tscale


def _route(g, T, k, E, ids, drop):
    """Router choices of T tokens: k distinct experts of E, of uneven popularity; a share
    `drop` of the assignments is dropped (-1)."""
    logits = torch.randn(T, E, device="cuda", generator=g) + torch.randn(E, device="cuda", generator=g)
    top = logits.topk(k, dim=1)
    gone = torch.rand(T, k, device="cuda", generator=g) < drop
    experts = torch.where(gone, -1, top.indices)
    return experts.to(torch.int32 if ids == "int32" else torch.int64), top.values.softmax(1).float()


def _sorted(experts, E):
    """Stable order of the assignments by expert (dropped ones last): offsets, order, place."""
    e = experts.reshape(-1).long()
    n = e.numel()
    e = torch.where((e >= 0) & (e < E), e, E)
    order = torch.argsort(e, stable=True)
    counts = (e.unsqueeze(0) == torch.arange(E, device=e.device).unsqueeze(1)).sum(1)
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    place = torch.empty(n, dtype=torch.int64, device=e.device)
    place[order] = torch.arange(n, device=e.device)
    place = torch.where(e < E, place, -1)
    return offsets.int(), order.int(), place.int().view(experts.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, s = case, dict(case)
    op = c["op"]
    sq = None
    if own:
        import fp4_sparse_dense_b200 as sq
    if op == "matvec":
        s["x"] = _activations(g, c["M"], c["K"], c["dtype"])
        s["codes"], s["dense"], s["sparse"], s["tscale"] = _weight(g, c["K"], c["N"], c["fmt"], c["block"])
    else:
        s["experts"], s["weights"] = _route(g, c["T"], c["k"], c["E"], c.get("ids", "int64"), c["drop"])
        n = c["T"] * c["k"]
        if op != "sort_tokens":
            s["offsets"], s["order"], s["place"] = _sorted(s["experts"], c["E"])
            if own:
                s["tokens"] = sq.SortedTokens(s["offsets"], s["order"], s["place"], c["T"], c["k"], c["E"])
    if op == "expert_matvec":
        s["x"] = _activations(g, c["T"] if c["gather"] else n, c["K"], c["dtype"])
        parts = [_weight(g, c["K"], c["N"], c["fmt"], c["block"]) for _ in range(c["E"])]
        s["codes"], s["dense"], s["sparse"], s["tscale"] = (torch.stack(p) for p in zip(*parts))
        # rows behind the last expert's are not written: a user's buffer keeps what it had
        s["y"] = torch.zeros(n, c["N"], dtype=DTYPES[c["out"]], device="cuda")
    elif op == "sort_tokens":
        s["x"] = _activations(g, c["T"], c["H"], c["dtype"])
        s["rows"] = torch.zeros(n, c["H"], dtype=DTYPES[c["dtype"]], device="cuda")
    elif op == "sort_tokens_backward":
        s["d_rows"] = torch.randn(n, c["H"], device="cuda", generator=g).to(DTYPES[c["dtype"]])
    elif op in ("combine_tokens", "combine_tokens_backward"):
        s["rows"] = _activations(g, n, c["H"], c["dtype"])
        if op == "combine_tokens_backward":
            s["dy"] = torch.randn(c["T"], c["H"], device="cuda", generator=g).to(DTYPES[c["dtype"]])
            s["d_rows"] = torch.zeros_like(s["rows"])
    if own and "codes" in s:
        # plain NVFP4 weights (16-element blocks) have one scale view, those of the pair mask two
        cfg = sq.Config.from_names(c["fmt"], "none" if c["block"] == 16 else "pair48")
        sparse = None if c["block"] == 16 else s["sparse"]
        if op == "matvec":
            s["w"] = sq.QuantWeight(s["codes"], s["dense"], sparse, s["tscale"], c["K"], c["N"], cfg)
        else:
            s["w"] = sq.ExpertWeights(s["codes"], s["dense"], sparse, s["tscale"], c["K"], c["N"], c["E"], cfg)
    return s


# ------------------------------------------------------------------ the plain forms

def _dequantised(s, codes, scales):
    """float32 weight [..., N, K] without the tensor scale, from stacked codes and scales."""
    N, K, B = s["N"], s["K"], s["block"]
    lead = codes.numel() // (N * K // 2)
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    byte = torch.arange(256, device="cuda")
    pairs = torch.stack((lut[byte & 15], lut[byte >> 4]), dim=1)
    w = pairs[codes.view(-1).int()].view(lead * N, K // B, B)
    raw = _untile(scales.reshape(-1), lead * N, K // B)
    sf = raw.view(torch.float8_e4m3fn).float() if s["fmt"] == "nvfp4" else torch.exp2(raw.float() - 127)
    return (w * sf.unsqueeze(-1)).view(lead, N, K)


def _plain(s):
    op = s["op"]
    if op == "matvec":
        w = _dequantised(s, s["codes"], s["sparse"])[0]
        return ((s["x"].float() @ w.t()) * s["tscale"][0]).to(DTYPES[s["out"]])
    T, k, E = s["T"], s["k"], s["E"]
    n = T * k
    if op == "sort_tokens":
        offsets, order, place = _sorted(s["experts"], E)
        kept = torch.arange(n, device="cuda") < offsets[E]
        rows = torch.where(kept.unsqueeze(1), s["x"][order.long() // k], torch.zeros_like(s["rows"]))
        return {"offsets": offsets, "order": order, "place": place, "rows": rows}
    place = s["place"].long()
    kept = place >= 0
    if op == "expert_matvec":
        w = _dequantised(s, s["codes"], s["sparse"])
        e = torch.where(kept, s["experts"].long(), E).reshape(-1)
        at = torch.where(kept, place, n).reshape(-1)
        # each expert's rows in a padded batch; a dropped assignment's go to a batch entry behind the last
        start = torch.cat((s["offsets"].long(), s["offsets"].new_full((1,), n).long()))
        inside = torch.where(e < E, at - start[e], 0)
        token = torch.arange(n, device="cuda") // k
        src = s["x"][token] if s["gather"] else s["x"][at.clamp_max(n - 1)]
        batch = torch.zeros(E + 1, T, s["K"], device="cuda")
        batch[e, inside] = src.float()
        y = torch.bmm(batch[:E], w.transpose(1, 2)) * s["tscale"][:, 0].view(E, 1, 1)
        out = torch.zeros(n + 1, s["N"], dtype=DTYPES[s["out"]], device="cuda")
        out[at] = torch.where((e < E).unsqueeze(1), y[e.clamp_max(E - 1), inside], 0.0).to(out.dtype)
        return out[:n]
    if op == "sort_tokens_backward":
        d = s["d_rows"][place.clamp_min(0)].float()
        return torch.where(kept.unsqueeze(2), d, 0.0).sum(1).to(s["d_rows"].dtype)
    rows = torch.where(kept.unsqueeze(2), s["rows"][place.clamp_min(0)].float(), 0.0)
    if op == "combine_tokens":
        w = torch.where(kept, s["weights"], 0.0)
        return (rows * w.unsqueeze(2)).sum(1).to(s["rows"].dtype)
    dy = s["dy"].float()
    d_weights = (rows * dy.unsqueeze(1)).sum(2)
    d_rows = torch.zeros(n + 1, s["H"], dtype=s["rows"].dtype, device="cuda")
    d_rows[torch.where(kept, place, n)] = (s["weights"].unsqueeze(2) * dy.unsqueeze(1)).to(d_rows.dtype)
    return {"d_rows": d_rows[:n], "d_weights": d_weights}


def run(state):
    if not own:
        return _plain(state)
    import fp4_sparse_dense_b200 as sq
    s, op = state, state["op"]
    if op == "matvec":
        return sq.matvec(s["x"], s["w"], out_dtype=DTYPES[s["out"]])
    if op == "expert_matvec":
        return sq.expert_matvec(s["x"], s["w"], s["tokens"], gather=s["gather"], out=s["y"])
    if op == "sort_tokens":
        t, rows = sq.sort_tokens(s["experts"], s["E"], s["x"], rows=s["rows"])
        return {"offsets": t.offsets, "order": t.order, "place": t.place, "rows": rows}
    if op == "sort_tokens_backward":
        return sq.sort_tokens_backward(s["d_rows"], s["tokens"])
    if op == "combine_tokens":
        return sq.combine_tokens(s["rows"], s["tokens"], s["weights"])
    d_rows, d_weights = sq.combine_tokens_backward(s["dy"], s["rows"], s["tokens"], s["weights"],
                                                   d_rows=s["d_rows"])
    return {"d_rows": d_rows, "d_weights": d_weights}


# ------------------------------------------------------------------ the work

def work(case):
    """Each input read once, each output written once. Expert weights: those of the experts
    that uniformly chosen assignments are expected to reach."""
    c, op = case, case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if op == "matvec":
        wb = c["K"] * c["N"] / 2 + c["K"] * c["N"] / c["block"]
        return {"bytes": wb + c["M"] * c["K"] * 2 + c["M"] * c["N"] * size[c["out"]],
                "flops": 2 * c["M"] * c["K"] * c["N"]}
    n = c["T"] * c["k"] * (1 - c["drop"])
    if op == "expert_matvec":
        wb = c["K"] * c["N"] / 2 + c["K"] * c["N"] / c["block"]
        used = c["E"] * (1 - (1 - c["k"] * (1 - c["drop"]) / c["E"]) ** c["T"])
        rows = min(c["T"], n) if c["gather"] else n
        return {"bytes": used * wb + rows * c["K"] * 2 + n * c["N"] * size[c["out"]],
                "flops": 2 * n * c["K"] * c["N"]}
    row = c["H"] * size[c["dtype"]]
    plan = c["T"] * c["k"] * 4
    if op == "sort_tokens":
        ids = c["T"] * c["k"] * (4 if c["ids"] == "int32" else 8)
        return {"bytes": c["T"] * row + n * row + ids + 2 * plan + 4 * (c["E"] + 1), "flops": 0}
    if op in ("sort_tokens_backward", "combine_tokens"):
        w = plan if op == "combine_tokens" else 0
        return {"bytes": n * row + c["T"] * row + plan + w, "flops": 2 * n * c["H"]}
    return {"bytes": 2 * n * row + c["T"] * row + 3 * plan, "flops": 3 * n * c["H"]}


# ------------------------------------------------------------------ in 64 bits

def _weight64(codes, scales, K, N, fmt, block):
    """[N, K] float64 weight from the definitions of E2M1 (bias 1), E4M3 (bias 7) and E8M0."""
    c = codes.reshape(N, K // 2)
    c = torch.stack((c % 16, c // 16), dim=-1).reshape(N, K)
    e, m = ((c // 2) % 4).double(), (c % 2).double()
    mag = torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
    w = torch.where(c >= 8, -mag, mag)
    # chunk (row group, column group) of 512 bytes: row r, column c at (r%32)*16 + (r//32%4)*4 + c%4
    C = K // block
    r = torch.arange(N, device="cuda").unsqueeze(1)
    b = torch.arange(C, device="cuda").unsqueeze(0)
    at = ((r // 128) * (C // 4) + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4
    raw = scales.reshape(-1)[at].double()
    if fmt == "mxfp4":
        sf = torch.exp2(raw - 127)
    else:
        ex, fr = torch.floor(raw / 8) % 16, raw % 8
        sf = torch.where(ex > 0, (1 + fr / 8) * torch.exp2(ex - 7), fr / 8 * 2.0 ** -6)
    return w * sf.repeat_interleave(block, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "matvec":
        w = _weight64(s["codes"], s["sparse"], s["K"], s["N"], s["fmt"], s["block"])
        return s["tscale"][0].double() * torch.einsum("mk,nk->mn", s["x"].double(), w)
    T, k, E = s["T"], s["k"], s["E"]
    n = T * k
    ids = s["experts"].reshape(-1).tolist()
    order = [a for e in range(E) for a in range(n) if ids[a] == e] if n * E < 200000 else \
        sorted((a for a in range(n) if 0 <= ids[a] < E), key=lambda a: (ids[a], a))
    last = [a for a in range(n) if not 0 <= ids[a] < E]
    at = torch.tensor(order, dtype=torch.int64, device="cuda")  # assignment of each sorted row
    m = len(order)
    if op == "sort_tokens":
        rows = torch.zeros(n, s["H"], dtype=torch.float64, device="cuda")
        rows[:m] = s["x"].double()[torch.div(at, k, rounding_mode="floor")]
        place = [-1] * n
        for p, a in enumerate(order):
            place[a] = p
        offsets = [sum(1 for a in ids if 0 <= a < e) for e in range(E + 1)]
        return {"offsets": torch.tensor(offsets), "order": torch.tensor(order + last),
                "place": torch.tensor(place), "rows": rows}
    token = torch.div(at, k, rounding_mode="floor")
    if op == "expert_matvec":
        out = torch.zeros(n, s["N"], dtype=torch.float64, device="cuda")
        lo = 0
        for e in range(E):
            hi = lo + sum(1 for a in order[lo:] if ids[a] == e)
            if hi > lo:
                x = s["x"][token[lo:hi]] if s["gather"] else s["x"][lo:hi]
                w = _weight64(s["codes"][e], s["sparse"][e], s["K"], s["N"], s["fmt"], s["block"])
                out[lo:hi] = s["tscale"][e, 0].double() * torch.einsum("mk,nk->mn", x.double(), w)
            lo = hi
        return out
    if op == "sort_tokens_backward":
        d = torch.zeros(T, s["H"], dtype=torch.float64, device="cuda")
        return d.index_add_(0, token, s["d_rows"][:m].double())
    weight = s["weights"].double().reshape(-1)[at].unsqueeze(1)
    if op == "combine_tokens":
        y = torch.zeros(T, s["H"], dtype=torch.float64, device="cuda")
        return y.index_add_(0, token, weight * s["rows"][:m].double())
    dy = s["dy"].double()[token]
    d_rows = torch.zeros(n, s["H"], dtype=torch.float64, device="cuda")
    d_rows[:m] = weight * dy
    d_weights = torch.zeros(n, dtype=torch.float64, device="cuda")
    d_weights[at] = (dy * s["rows"][:m].double()).sum(1)
    return {"d_rows": d_rows, "d_weights": d_weights}
