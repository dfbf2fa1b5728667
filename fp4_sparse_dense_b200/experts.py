"""Few-row products with 16-bit activations on FP4 weights, and the experts' operators.

Tensor-level helpers over ``sharq_matvec``, ``sharq_sort_tokens``, ``sharq_expert_matvec``,
``sharq_combine_tokens`` and their gradients (include/sharq.h). A decoded batch runs through a
layer of experts as

    tokens, _ = sort_tokens(experts, num_experts)         # router's choices [T, k]
    h = expert_matvec(x, gate_up, tokens, gather=True)    # [T * k, N], in expert order
    y = expert_matvec(act(h), down, tokens)
    out = combine_tokens(y, tokens, weights)              # [T, H]

Every call runs on the device of its tensors and on ``stream`` (default: that device's
current stream); outputs it allocates belong to that stream. Bad arguments raise ValueError
or TypeError here, or SharqError with the C status. What a call writes (``out``, ``rows``,
``d_rows``, ``d_weights``) overlaps nothing that it reads, except that ``d_rows`` may be
``rows``. No call records an autograd graph: its outputs do not require gradients, and the
gradients are calls of their own.
"""
from __future__ import annotations

from ctypes import byref
from dataclasses import dataclass

from . import (BF16, Config, F16, F32, QuantWeight, _CStructCache, _one_device, _ptr, _torch,
               check, quantize_weight)
from ._abi import (
    sharq_combine_tokens as _combine_tokens, sharq_combine_tokens_backward as _combine_tokens_backward,
    sharq_expert_matvec as _expert_matvec, sharq_expert_weights, sharq_matvec as _matvec,
    sharq_sort_tokens as _sort_tokens, sharq_tokens, sharq_weight_bytes, sharq_weight_sizes,
)

# bound by _load: importing the package takes neither torch nor a CUDA build of it
torch = _current_device = _current_stream = None
_DTYPE = {}

_INVALID_ARG, _UNSUPPORTED = 1, 2  # sharq_status
_INT32_MAX = 2 ** 31 - 1


def _load():
    """Binds torch and its two cheapest queries on first use (a CPU build has no queries, and no
    CUDA tensors to ask about)."""
    global torch, _current_device, _current_stream
    t = _torch()
    _DTYPE.update({t.bfloat16: BF16, t.float16: F16, t.float32: F32})
    _current_device = getattr(t._C, "_cuda_getDevice", None)
    _current_stream = getattr(t._C, "_cuda_getCurrentRawStream", None)
    torch = t


def _elsewhere(device, stream) -> bool:
    """Whether the call has to switch to `stream` or to the tensors' device first."""
    return stream is not None or device.index != _current_device()


def _on(device, stream):
    """Context in which the tensors' device and `stream` are current, so that allocations and
    copies of the call happen there too."""
    if stream is None:
        return torch.cuda.device(device)
    if stream.device != device:
        raise ValueError(f"stream on {stream.device}, tensors on {device}")
    return torch.cuda.stream(stream)


def _cuda(name, x, device=None):
    if torch is None:
        _load()
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and x.device != device:
        raise ValueError(f"{name} is on {x.device}, expected {device}")


def _code(name, x) -> int:
    c = _DTYPE.get(x.dtype)
    if c is None:
        raise TypeError(f"unsupported dtype {x.dtype} of {name} (need bfloat16, float16 or float32)")
    return c


def _code16(name, x) -> int:
    if x.dtype is torch.bfloat16:
        return BF16
    if x.dtype is torch.float16:
        return F16
    raise TypeError(f"unsupported dtype {x.dtype} of {name} (need bfloat16 or float16)")


def _matrix(name, x, rows, cols, device):
    """Checks a [rows, cols] matrix with unit column stride and returns its row pitch."""
    _cuda(name, x, device)
    if x.dim() != 2 or x.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], got {list(x.shape)}")
    if x.is_contiguous():
        return cols
    ld, unit = x.stride()
    if rows <= 1:
        ld = cols
    if (cols > 1 and unit != 1) or ld < cols:
        raise ValueError(f"{name} must have unit column stride and rows that do not overlap")
    return ld


def _readable(name, x, align16=False):
    """An input matrix as the kernels read it, and its row pitch: unit column stride, rows that
    do not overlap (an expanded or transposed view is copied), and for the products 16-byte
    rows."""
    if x.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got {list(x.shape)}")
    rows, cols = x.shape
    if rows > _INT32_MAX or cols > _INT32_MAX:  # ctypes would cut them to 32 bits
        raise ValueError(f"{name} must be smaller than 2^31 rows and columns, got {list(x.shape)}")
    if x.is_contiguous():
        ld, ok = cols, True
    else:
        ld, unit = x.stride()
        if rows <= 1:
            ld = cols
        ok = (cols <= 1 or unit == 1) and ld >= cols
    if align16 and (ld % 8 or x.data_ptr() % 16):
        ok = False
    if ok:
        return x, rows, cols, ld
    return x.clone(memory_format=torch.contiguous_format), rows, cols, cols


def _new(like, rows, cols, dtype=None):
    """An empty matrix on the device of `like`, in its dtype by default (new_empty takes half a
    microsecond less than torch.empty with a device)."""
    if dtype is None:
        return like.new_empty((rows, cols))
    return like.new_empty((rows, cols), dtype=dtype)


# ------------------------------------------------------------------ the few-row product

def matvec(X, w: QuantWeight, out=None, out_dtype=None, stream=None):
    """Y[M x N] = X[M x K] deq(w) with the activations left in 16 bits (``sharq_matvec``).

    X: CUDA tensor [M x K], bf16 or fp16 (rows may be strided). Y is `out` (its first element
    16-byte aligned), or a new tensor of `out_dtype` (default: X's; also float32). For the few
    rows of a decode step, where the weight's bytes set the time; the activations are not
    quantised. For many rows ``prepare`` + ``linear`` is faster.

    The weight may be loaded before the kernel launched just before has completed, unless that
    was ``quantize_weight``. A kernel of one's own that writes w's buffers in place must not come
    directly before this call; copies, or a write ordered through an event, are fine.
    """
    _cuda("X", X)
    device = X.device
    if _elsewhere(device, stream):
        with _on(device, stream):
            return matvec(X, w, out, out_dtype)
    code = _code16("X", X)
    X, M, K, ldx = _readable("X", X, align16=True)
    N = w.N
    if K != w.K:
        raise ValueError(f"X must be [M, {w.K}], got {list(X.shape)}")
    if w.codes.device != device:
        raise ValueError(f"w is on {w.codes.device}, expected {device}")
    if out is None:
        out = _new(X, M, N, out_dtype)
        ldy = N
    else:
        ldy = _matrix("out", out, M, N, device)
    if M == 0:
        return out
    check(_matvec(X.data_ptr(), ldx, M, code, byref(w.c()), out.data_ptr(), ldy,
                  _code("out", out), _current_stream(device.index)))
    return out


# ------------------------------------------------------------------ experts' weights

@dataclass
class ExpertWeights(_CStructCache):
    """E quantised weights [K x N] of one configuration, stacked (``sharq_expert_weights``):
    `tensor_scale` is float32 [E, 4]; the other buffers hold E times the bytes of a
    ``QuantWeight``'s."""
    codes: object
    scales_dense: object
    scales_sparse: object
    tensor_scale: object
    K: int
    N: int
    E: int
    cfg: Config

    def _make_c(self) -> sharq_expert_weights:
        torch = _torch()
        sz = self._bytes()
        for name in ("codes", "scales_dense", "scales_sparse"):
            t, n = getattr(self, name), getattr(sz, name)
            if n and (t is None or t.numel() * t.element_size() != self.E * n or not t.is_contiguous()):
                raise ValueError(f"{name} must be contiguous and hold {self.E} x {n} bytes")
        t = self.tensor_scale
        if t.dtype != torch.float32 or t.numel() != 4 * self.E or not t.is_contiguous():
            raise ValueError(f"tensor_scale must be contiguous float32 [{self.E}, 4]")
        _one_device(self)
        return sharq_expert_weights(_ptr(self.codes), _ptr(self.scales_dense),
                                    _ptr(self.scales_sparse), _ptr(self.tensor_scale),
                                    self.K, self.N, self.E, self.cfg.c())

    def _bytes(self) -> sharq_weight_bytes:
        sz = sharq_weight_bytes()
        check(sharq_weight_sizes(self.K, self.N, self.cfg.c(), byref(sz)))
        return sz

    def expert(self, e: int) -> QuantWeight:
        """Expert e as a QuantWeight that shares these buffers (for ``linear``, ``matvec``)."""
        if not 0 <= e < self.E:
            raise IndexError(f"expert {e} of {self.E}")
        sz = self._bytes()

        def part(t, n):
            return t.view(-1)[e * n:(e + 1) * n] if n else None

        return QuantWeight(part(self.codes, sz.codes), part(self.scales_dense, sz.scales_dense),
                           part(self.scales_sparse, sz.scales_sparse),
                           self.tensor_scale.view(-1)[4 * e:4 * e + 4], self.K, self.N, self.cfg)


def quantize_experts(W, cfg: Config = Config(), stream=None) -> ExpertWeights:
    """W: CUDA tensor [E x K x N] (bf16/fp16) -> the experts' FP4 payloads, each as
    ``quantize_weight`` gives it."""
    if W.dim() != 3:
        raise ValueError(f"W must be [E, K, N], got {list(W.shape)}")
    _cuda("W", W)
    if _elsewhere(W.device, stream):
        with _on(W.device, stream):
            return quantize_experts(W, cfg)
    E, K, N = W.shape
    one = sharq_weight_bytes()
    check(sharq_weight_sizes(K, N, cfg.c(), byref(one)))

    def stack(n):
        return torch.empty(E, n, dtype=torch.uint8, device=W.device) if n else None

    out = ExpertWeights(stack(one.codes), stack(one.scales_dense), stack(one.scales_sparse),
                        torch.zeros(E, 4, dtype=torch.float32, device=W.device), K, N, E, cfg)
    for e in range(E):
        quantize_weight(W[e], cfg, out=out.expert(e))
    return out


# ------------------------------------------------------------------ tokens and experts

@dataclass
class SortedTokens(_CStructCache):
    """T tokens' assignments in expert order (``sharq_tokens``); int32 tensors `offsets`
    [E + 1], `order` [T * k] and `place` [T, k], as ``sort_tokens`` fills them."""
    offsets: object
    order: object
    place: object
    T: int
    k: int
    E: int

    def _make_c(self) -> sharq_tokens:
        torch = _torch()
        _assignments(self.T, self.k, self.E)
        n = self.T * self.k
        for name, want in (("offsets", self.E + 1), ("order", n), ("place", n)):
            t = getattr(self, name)
            if t.dtype != torch.int32 or t.numel() != want or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous int32 with {want} elements")
            _cuda(name, t, self.offsets.device)
        return sharq_tokens(_ptr(self.offsets), _ptr(self.order), _ptr(self.place),
                            self.T, self.k, self.E)


def _assignments(T, k, E):
    """Raises what the C call answers to these sizes: before anything of them is allocated, and
    before ctypes cuts them to 32 bits."""
    if T < 0 or k < 1 or E < 1:
        check(_INVALID_ARG)
    if E > 1024 or T * k >= 1 << 30:
        check(_UNSUPPORTED)


def _empty_tokens(T, k, E, like) -> SortedTokens:
    """SortedTokens over one new buffer; its parts fit by construction, so the C struct is made
    here without the checks of _make_c."""
    n = T * k
    plan = like.new_empty(2 * n + E + 1, dtype=torch.int32)
    order, place, offsets = plan.split_with_sizes((n, n, E + 1))
    t = object.__new__(SortedTokens)
    p = plan.data_ptr()
    t.__dict__.update(offsets=offsets, order=order, place=place.view(T, k), T=T, k=k, E=E,
                      _c=sharq_tokens(p + 8 * n, p, p + 4 * n, T, k, E))
    return t


def sort_tokens(experts, num_experts: int, X=None, rows=None, out: SortedTokens | None = None,
                stream=None):
    """Stable order of the assignments `experts` [T, k] (int32 or int64; an id outside
    [0, num_experts) is dropped) by expert. Returns (SortedTokens, rows): with X [T x H] the
    rows gathered in that order ([T * k, H], `rows` if given), else None. Rows behind the last
    kept assignment are left as they were (undefined in a new `rows`)."""
    _cuda("experts", experts)
    device = experts.device
    if _elsewhere(device, stream):
        with _on(device, stream):
            return sort_tokens(experts, num_experts, X, rows, out)
    if experts.dim() != 2:
        raise ValueError(f"experts must be [T, k], got {list(experts.shape)}")
    if experts.dtype is torch.int64:
        bits = 64
    elif experts.dtype is torch.int32:
        bits = 32
    else:
        raise TypeError(f"unsupported dtype {experts.dtype} of experts (need int32 or int64)")
    T, k = experts.shape
    _assignments(T, k, num_experts)
    if not experts.is_contiguous():
        experts = experts.contiguous()
    if out is None:
        out = _empty_tokens(T, k, num_experts, experts)
    elif (out.T, out.k, out.E) != (T, k, num_experts):
        raise ValueError(f"out is for T, k, E = {out.T}, {out.k}, {out.E}")
    else:
        _cuda("out.offsets", out.offsets, device)
    x_ptr = rows_ptr = None
    ldx = ld_rows = H = code = 0
    if X is not None:
        _cuda("X", X, device)
        X, n, H, ldx = _readable("X", X)
        if n != T:
            raise ValueError(f"X must be [{T}, H], got {list(X.shape)}")
        code = _code("X", X)
        if rows is None:
            rows = _new(X, T * k, H)
            ld_rows = H
        else:
            ld_rows = _matrix("rows", rows, T * k, H, device)
            if rows.dtype != X.dtype:
                raise TypeError(f"rows is {rows.dtype}, X is {X.dtype}")
        x_ptr, rows_ptr = X.data_ptr(), rows.data_ptr()
    elif rows is not None:
        raise ValueError("rows without X")
    check(_sort_tokens(experts.data_ptr(), bits, byref(out.c()), x_ptr, ldx, H, code, rows_ptr,
                       ld_rows, _current_stream(device.index)))
    return out, rows


def sort_tokens_backward(d_rows, tokens: SortedTokens, out=None, stream=None):
    """Gradient of sort_tokens' gather: dX [T x H] from d_rows [T * k, H]."""
    return combine_tokens(d_rows, tokens, None, out, stream)


def expert_matvec(X, w: ExpertWeights, tokens: SortedTokens, gather: bool = False, out=None,
                  out_dtype=None, stream=None):
    """Y[p] = X row of sorted row p times its expert's weight (``sharq_expert_matvec``), the
    activations left in 16 bits. X: the sorted rows [T * k, K], or with gather=True the tokens
    [T, K]. Returns Y [T * k, N] (`out`, its first element 16-byte aligned, or a new tensor of
    `out_dtype`, default X's); rows behind the last kept assignment are left as they were
    (undefined in a new tensor)."""
    _cuda("X", X)
    device = X.device
    if _elsewhere(device, stream):
        with _on(device, stream):
            return expert_matvec(X, w, tokens, gather, out, out_dtype)
    if w.E != tokens.E:
        raise ValueError(f"{w.E} expert weights, tokens sorted over {tokens.E}")
    code = _code16("X", X)
    n = tokens.T * tokens.k
    X, rows, K, ldx = _readable("X", X, align16=True)
    if rows != (tokens.T if gather else n) or K != w.K:
        raise ValueError(f"X must be [{tokens.T if gather else n}, {w.K}], got {list(X.shape)}")
    if w.codes.device != device or tokens.offsets.device != device:
        raise ValueError(f"w is on {w.codes.device}, tokens on {tokens.offsets.device}, expected {device}")
    if out is None:
        out = _new(X, n, w.N, out_dtype)
        ldy = w.N
    else:
        ldy = _matrix("out", out, n, w.N, device)
    if n == 0:
        return out
    check(_expert_matvec(X.data_ptr(), ldx, 1 if gather else 0, code, byref(tokens.c()),
                         byref(w.c()), out.data_ptr(), ldy, _code("out", out),
                         _current_stream(device.index)))
    return out


def _weights(weights, tokens, device):
    _cuda("weights", weights, device)
    if weights.dtype is not torch.float32:
        raise TypeError(f"unsupported dtype {weights.dtype} of weights (need float32)")
    if weights.shape != (tokens.T, tokens.k):
        raise ValueError(f"weights must be [{tokens.T}, {tokens.k}], got {list(weights.shape)}")
    return weights if weights.is_contiguous() else weights.contiguous()


def combine_tokens(rows, tokens: SortedTokens, weights=None, out=None, stream=None):
    """Y[t] = sum_j weights[t, j] rows[place[t, j]] over the kept assignments
    (``sharq_combine_tokens``): [T x H] in the dtype of `rows` [T * k, H]. weights: float32
    [T, k], or None for 1."""
    _cuda("rows", rows)
    device = rows.device
    if _elsewhere(device, stream):
        with _on(device, stream):
            return combine_tokens(rows, tokens, weights, out)
    rows, n, H, ld_rows = _readable("rows", rows)
    if n != tokens.T * tokens.k:
        raise ValueError(f"rows must be [{tokens.T * tokens.k}, H], got {list(rows.shape)}")
    code = _code("rows", rows)
    if tokens.offsets.device != device:
        raise ValueError(f"tokens on {tokens.offsets.device}, expected {device}")
    if weights is not None:
        weights = _weights(weights, tokens, device)
    if out is None:
        out = _new(rows, tokens.T, H)
        ldy = H
    else:
        ldy = _matrix("out", out, tokens.T, H, device)
        if out.dtype != rows.dtype:
            raise TypeError(f"out is {out.dtype}, rows is {rows.dtype}")
    check(_combine_tokens(rows.data_ptr(), ld_rows, H, code, byref(tokens.c()),
                                    None if weights is None else weights.data_ptr(),
                                    out.data_ptr(), ldy, _current_stream(device.index)))
    return out


def combine_tokens_backward(dY, rows, tokens: SortedTokens, weights, d_rows=None, d_weights=None,
                            stream=None):
    """Gradients of combine_tokens: (d_rows [T * k, H] in the dtype of `rows`, d_weights
    float32 [T, k]). Rows of d_rows behind the last kept assignment are left as they were
    (undefined in a new tensor); a dropped assignment's weight gets 0."""
    _cuda("dY", dY)
    device = dY.device
    if _elsewhere(device, stream):
        with _on(device, stream):
            return combine_tokens_backward(dY, rows, tokens, weights, d_rows, d_weights)
    T, k = tokens.T, tokens.k
    dY, n, H, ld_dy = _readable("dY", dY)
    _cuda("rows", rows, device)
    rows, m, h, ld_rows = _readable("rows", rows)
    if n != T or m != T * k or h != H:
        raise ValueError(f"dY must be [{T}, H] and rows [{T * k}, H], got {list(dY.shape)} and {list(rows.shape)}")
    code = _code("rows", rows)
    if dY.dtype != rows.dtype:
        raise TypeError(f"dY is {dY.dtype}, rows is {rows.dtype}")
    if tokens.offsets.device != device:
        raise ValueError(f"tokens on {tokens.offsets.device}, expected {device}")
    weights = _weights(weights, tokens, device)
    if d_rows is None:
        d_rows = _new(rows, T * k, H)
        ld_d = H
    else:
        ld_d = _matrix("d_rows", d_rows, T * k, H, device)
        if d_rows.dtype != rows.dtype:
            raise TypeError(f"d_rows is {d_rows.dtype}, rows is {rows.dtype}")
    if d_weights is None:
        d_weights = _new(weights, T, k)
    elif d_weights.dtype != torch.float32 or list(d_weights.shape) != [T, k] or not d_weights.is_contiguous():
        raise ValueError(f"d_weights must be contiguous float32 [{T}, {k}]")
    else:
        _cuda("d_weights", d_weights, device)
    check(_combine_tokens_backward(
        dY.data_ptr(), ld_dy, rows.data_ptr(), ld_rows, H, code, byref(tokens.c()),
        weights.data_ptr(), d_rows.data_ptr(), ld_d, d_weights.data_ptr(), _current_stream(device.index)))
    return d_rows, d_weights
