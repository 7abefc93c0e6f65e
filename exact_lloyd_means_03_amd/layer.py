"""Python entry points of a layer of 8-bit experts (include/kmeans.h, last
part): norms with the residual's addition, 8-bit codes, the gate, the plan of a
dispatch, and products with 8-bit matrices.

8-bit codes are torch.float8_e4m3fn tensors with float32 scales for blocks of
128 columns (rows) or 128 x 128 (matrices).  What is differentiable is handed to
torch's autograd where an input requires a gradient, as in api.py.
"""
from __future__ import annotations

import functools

import torch

from . import _lib
from .api import _DT, _bytes, _grads, _no_buffers, _no_gradient, _ptr, _stream, _tensor, kmeans_combine

E4M3 = torch.float8_e4m3fn
BLOCK = 128


def _blocks(n):
    return -(-n // BLOCK)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _output(t, name, dev, dtype, shape):
    """The caller's output, or a new one (the least of torch's ways to make one)."""
    if t is not None:
        return _tensor(t, name, dev, dtype, shape)
    strides, n = (), 1
    for size in reversed(shape):
        strides = (n, *strides)
        n *= size
    return torch.empty_strided(shape, strides, dtype=dtype, device=dev)


_entry = {}


def _call(name, dev, *args):
    """The entry point on the current stream of dev, with dev current (kernels are launched on the current device)."""
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(_lib.load(), name)
    if dev.index is None or dev.index == _current_device():
        st = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _stream(dev))
    if st:
        _lib.check(st, name)


@functools.lru_cache(1024)
def _bytes_of(query, *sizes):
    """A workspace query of the library (sizes and types alone decide it)."""
    return getattr(_lib.load(), query)(*sizes)


def _workspace(ws, dev, query, *sizes):
    """The caller's workspace, or one of the size asked for (None: none is needed)."""
    if ws is not None:
        return _tensor(ws, "workspace", dev, torch.uint8, None)
    n = _bytes_of(query, *sizes)
    return torch.empty(n, dtype=torch.uint8, device=dev) if n else None


def _ws_args(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel())


# 8-bit codes ---------------------------------------------------------------

def kmeans_quantize(x, rows: int = 1, codes=None, scales=None):
    """8-bit codes of x [M, K] or [B, M, K] by blocks of `rows` x 128 elements:
    rows 1 for the rows of a product, 128 for its matrices.  Returns (codes of
    x's shape, float32 scales [.., ceil(M / rows), ceil(K / 128)]); the values
    are codes * scales."""
    _tensor(x, "x", None, None, None)
    if x.dim() not in (2, 3):
        raise ValueError("x must be [M, K] or [B, M, K]")
    if rows not in (1, BLOCK):
        raise ValueError("rows must be 1 or 128")
    if _grads(x):
        _no_gradient("kmeans_quantize", x=x)
    dev, shape = x.device, tuple(x.shape)
    M, K = shape[-2:]
    codes = _output(codes, "codes", dev, E4M3, shape)
    scales = _output(scales, "scales", dev, torch.float32, (*shape[:-2], -(-M // rows), _blocks(K)))
    _call("kmeans_quantize", dev, x.data_ptr(), _DT[x.dtype], shape[0] if len(shape) == 3 else 1, M, K, rows,
          codes.data_ptr(), scales.data_ptr())
    return codes, scales


# Norm ----------------------------------------------------------------------

def _norm_inputs(x, weight, residual, name):
    _tensor(x, name, None, None, None)
    if x.dim() != 2:
        raise ValueError(f"{name} must be [T, d]")
    dev, d = x.device, x.shape[1]
    if weight is not None:
        _tensor(weight, "weight", dev, torch.float32 if weight.dtype == torch.float32 else x.dtype, (d,))
    if residual is not None:
        _tensor(residual, "residual", dev, x.dtype, tuple(x.shape))
    return dev, x.dtype, x.shape[0], d


def _weight_args(weight, dt):
    return _ptr(weight), _DT[dt if weight is None else weight.dtype]


def kmeans_norm(x, weight=None, eps: float = 1e-6, residual=None, y=None, h=None):
    """Root-mean-square norm of the rows of h = x + residual: y = h * weight /
    sqrt(mean(h^2) + eps) from the unrounded sum.  x, residual [T, d], weight [d]
    of x's dtype or float32 (None: ones).  Returns (y, h); without a residual h
    is x itself.  Differentiable in x, residual and weight."""
    dev, dt, T, d = _norm_inputs(x, weight, residual, "x")
    if _grads(x, weight, residual):
        _no_buffers("kmeans_norm", y, h)
        y, h = _Norm.apply(x, weight, eps, residual)
        return y, x if residual is None else h
    y = _output(y, "y", dev, dt, (T, d))
    if residual is None:
        h = x
    else:
        h = _output(h, "h", dev, dt, (T, d))
    _call("kmeans_norm", dev, x.data_ptr(), _DT[dt], T, d, _ptr(residual), *_weight_args(weight, dt), eps,
          None if residual is None else h.data_ptr(), y.data_ptr(), None, None)
    return y, h


def kmeans_norm_quantize(x, weight=None, eps: float = 1e-6, residual=None, codes=None, scales=None, h=None):
    """kmeans_norm whose y is rounded to 8-bit codes, for an 8-bit product.
    Returns (codes [T, d], scales [T, ceil(d / 128)], h).  No gradient: train
    through kmeans_norm and the product of its rows."""
    dev, dt, T, d = _norm_inputs(x, weight, residual, "x")
    if _grads(x, weight, residual):
        _no_gradient("kmeans_norm_quantize", x=x, weight=weight, residual=residual)
    codes = _output(codes, "codes", dev, E4M3, (T, d))
    scales = _output(scales, "scales", dev, torch.float32, (T, _blocks(d)))
    if residual is None:
        h = x
    else:
        h = _output(h, "h", dev, dt, (T, d))
    _call("kmeans_norm", dev, x.data_ptr(), _DT[dt], T, d, _ptr(residual), *_weight_args(weight, dt), eps,
          None if residual is None else h.data_ptr(), None, codes.data_ptr(), scales.data_ptr())
    return codes, scales, h


def norm_grad_workspace(T: int, d: int, dtype: torch.dtype, device) -> torch.Tensor:
    """A workspace for kmeans_norm_grad at these shapes."""
    return _bytes(_lib.load().kmeans_norm_grad_workspace_bytes(T, d, _DT[dtype]), device)


def kmeans_norm_grad(grad, h, weight=None, eps: float = 1e-6, grad_residual=None, grad_x=None, grad_weight=None, ws=None):
    """Gradients of kmeans_norm at the h it returned, for grad = dy and
    grad_residual = dh (None: nothing else uses h).  Returns (grad_x, the
    gradient of x and of the residual; grad_weight of weight's dtype, None
    without a weight)."""
    dev, dt, T, d = _norm_inputs(h, weight, grad_residual, "h")
    _tensor(grad, "grad", dev, dt, (T, d))
    if _grads(grad, h, weight, grad_residual):
        _no_gradient("kmeans_norm_grad", grad=grad, h=h, weight=weight, grad_residual=grad_residual)
    grad_x = _output(grad_x, "grad_x", dev, dt, (T, d))
    if weight is None:
        grad_weight = None
    else:
        grad_weight = _output(grad_weight, "grad_weight", dev, weight.dtype, (d,))
        ws = _workspace(ws, dev, "kmeans_norm_grad_workspace_bytes", T, d, _DT[dt])
    _call("kmeans_norm_grad", dev, grad.data_ptr(), h.data_ptr(), _DT[dt], T, d, _ptr(grad_residual),
          *_weight_args(weight, dt), eps, grad_x.data_ptr(), _ptr(grad_weight), *_ws_args(ws))
    return grad_x, grad_weight


# Gate ----------------------------------------------------------------------

def _logits(logits):
    _tensor(logits, "logits", None, None, None)
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    return logits.device, logits.shape[0], logits.shape[1]


def gate_workspace(T: int, E: int, device) -> torch.Tensor:
    """A workspace for kmeans_gate at these shapes."""
    return _bytes(_lib.load().kmeans_gate_workspace_bytes(T, E), device)


def kmeans_gate(logits, top: int, normalize: bool = True, experts=None, weights=None, counts=None, shares=None, loss=None,
                ws=None):
    """Tokens choose experts: logits [T, E] -> (experts [T, top] int32, the
    largest logits' first, -1 where only -inf is left; weights [T, top] float32,
    the softmax over the chosen (normalize) or over all; counts [E + 1] int32,
    the choices of every expert and the rows that are not all -inf; shares [E]
    float32, the mean probabilities; loss [] float32, E * <shares, shares of the
    choices>).  Differentiable in logits, through weights and loss."""
    dev, T, E = _logits(logits)
    if _grads(logits):
        _no_buffers("kmeans_gate", experts, weights, counts, shares, loss)
        return _Gate.apply(logits, top, normalize, ws)
    # (each a tensor of its own: parts of one allocation would be views, which autograd does
    # not let a caller scale in place, and a loss that is kept would keep the choices)
    experts = _output(experts, "experts", dev, torch.int32, (T, top))
    weights = _output(weights, "weights", dev, torch.float32, (T, top))
    counts = _output(counts, "counts", dev, torch.int32, (E + 1,))
    shares = _output(shares, "shares", dev, torch.float32, (E,))
    loss = _output(loss, "loss", dev, torch.float32, ())
    ws = _workspace(ws, dev, "kmeans_gate_workspace_bytes", T, E)
    _call("kmeans_gate", dev, logits.data_ptr(), _DT[logits.dtype], T, E, top, int(normalize), experts.data_ptr(),
          weights.data_ptr(), counts.data_ptr(), shares.data_ptr(), loss.data_ptr(), *_ws_args(ws))
    return experts, weights, counts, shares, loss


def kmeans_gate_grad(logits, experts, counts, grad_weights=None, grad_loss=None, normalize: bool = True, grad_logits=None):
    """Gradient of kmeans_gate's logits for the choices it made: grad_weights
    [T, top] float32, grad_loss [] float32 (None: none)."""
    dev, T, E = _logits(logits)
    _tensor(experts, "experts", dev, torch.int32, None)
    if experts.dim() != 2 or experts.shape[0] != T:
        raise ValueError("experts must be [T, top] int32")
    top = experts.shape[1]
    _tensor(counts, "counts", dev, torch.int32, (E + 1,))
    if grad_weights is not None:
        _tensor(grad_weights, "grad_weights", dev, torch.float32, (T, top))
    if grad_loss is not None:
        _tensor(grad_loss, "grad_loss", dev, torch.float32, ())
    if _grads(logits, grad_weights, grad_loss):
        _no_gradient("kmeans_gate_grad", logits=logits, grad_weights=grad_weights, grad_loss=grad_loss)
    grad_logits = _output(grad_logits, "grad_logits", dev, logits.dtype, (T, E))
    _call("kmeans_gate_grad", dev, logits.data_ptr(), _DT[logits.dtype], T, E, top, int(normalize), experts.data_ptr(),
          counts.data_ptr(), _ptr(grad_weights), _ptr(grad_loss), grad_logits.data_ptr())
    return grad_logits


def plan_workspace(T: int, top: int, E: int, device) -> torch.Tensor:
    """A workspace for kmeans_plan at these shapes."""
    return _bytes(_lib.load().kmeans_plan_workspace_bytes(T, top, E), device)


def kmeans_plan(experts, E: int, plan=None, ws=None):
    """The plan of kmeans_dispatch without its rows: experts [T, top] int32 ->
    (offsets [E + 1], slots [T, top], order [T * top]); kmeans_block_product
    gathers the rows by its order."""
    _tensor(experts, "experts", None, torch.int32, None)
    if experts.dim() != 2:
        raise ValueError("experts must be [T, top] int32")
    T, top = experts.shape
    dev = experts.device
    offsets, slots, order = (None, None, None) if plan is None else plan
    offsets = _output(offsets, "offsets", dev, torch.int32, (E + 1,))
    slots = _output(slots, "slots", dev, torch.int32, (T, top))
    order = _output(order, "order", dev, torch.int32, (T * top,))
    ws = _workspace(ws, dev, "kmeans_plan_workspace_bytes", T, top, E)
    _call("kmeans_plan", dev, experts.data_ptr(), T, top, E, offsets.data_ptr(), slots.data_ptr(), order.data_ptr(),
          *_ws_args(ws))
    return offsets, slots, order


# Products with 8-bit matrices ----------------------------------------------

def block_product_workspace(S: int, E: int, M: int, K: int, device) -> torch.Tensor:
    """A workspace for kmeans_block_product at these shapes."""
    return _bytes(_lib.load().kmeans_block_product_workspace_bytes(S, E, M, K), device)


def block_product_grad_workspace(S: int, E: int, M: int, K: int, device) -> torch.Tensor:
    """A workspace for kmeans_block_product_grad at these shapes."""
    return _bytes(_lib.load().kmeans_block_product_grad_workspace_bytes(S, E, M, K), device)


def _matrices(codes, scales, dev):
    _tensor(codes, "codes", dev, E4M3, None)
    if codes.dim() not in (2, 3):
        raise ValueError("codes must be [E, M, K] or [M, K]")
    E, (M, K) = codes.shape[0] if codes.dim() == 3 else 1, codes.shape[-2:]
    _tensor(scales, "scales", dev, torch.float32, None)
    if scales.numel() != E * _blocks(M) * _blocks(K) or tuple(scales.shape[-2:]) != (_blocks(M), _blocks(K)):
        raise ValueError("scales must be [E, ceil(M / 128), ceil(K / 128)]")
    return E, M, K


def _rows8(x, x_scales, name, inner):
    """x as codes and scales: given, or made from 16 or 32 bits."""
    if x.shape[1] != inner:
        raise ValueError(f"{name} must have {inner} columns, got {x.shape[1]}")
    if x.dtype != E4M3:
        if x_scales is not None:
            raise ValueError(f"scales of {name} go with 8-bit codes, not with {x.dtype}")
        return kmeans_quantize(x)
    if x_scales is None:
        raise ValueError(f"8-bit codes of {name} need their scales")
    _tensor(x_scales, f"scales of {name}", x.device, torch.float32, (x.shape[0], _blocks(inner)))
    return x, x_scales


def _rows_tensor(x, name):
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    _tensor(x, name, None, E4M3 if x.dtype == E4M3 else None, None)
    if x.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    return x.device


def _result_dtype(x, dtype, out):
    if out is not None:
        dtype = out.dtype if dtype is None else dtype
    elif dtype is None:
        dtype = torch.bfloat16 if x.dtype == E4M3 else x.dtype
    if dtype not in _DT:
        raise TypeError(f"results of dtype {dtype} are not float32 / float16 / bfloat16")
    return dtype


def kmeans_block_product(x, x_scales, codes, scales, offsets=None, order=None, dtype=None, out=None, ws=None):
    """Rows times 8-bit matrices: out[p] = X[p] W[e]^T, e the expert whose
    segment offsets[e] : offsets[e + 1] holds p (offsets None: one matrix), X = x
    * x_scales and W = codes * scales by blocks of 128 and 128 x 128.

    x [S, K]: 8-bit codes with x_scales [S, ceil(K / 128)], or float32 / float16 /
    bfloat16 with x_scales None, rounded to codes by the call.  codes [E, M, K]
    (or [M, K]), scales [E, ceil(M / 128), ceil(K / 128)].  order [S] int32 of
    kmeans_plan: x has T rows (S = T * top) and row p of the product is row
    order[p] // top of x, zeros for -1.  Returns [S, M] of `dtype` (None: x's, or
    bfloat16 from codes); rows past offsets[E] are zeros.

    Differentiable in x where it is no codes; the matrices are held.  The backward
    pass is an 8-bit product too: the rounding of x to codes is passed through, the
    gradient that comes in is itself rounded to codes (kmeans_block_product_grad),
    and with an order every choice's row of the result is rounded to x's type
    before a token's rows are added in float32."""
    dev = _rows_tensor(x, "x")
    E, M, K = _matrices(codes, scales, dev)
    T, top, S = x.shape[0], 1, x.shape[0]
    if order is not None:
        _tensor(order, "order", dev, torch.int32, None)
        S = order.numel()
        if order.dim() != 1 or (S % T if T else S) != 0:
            raise ValueError("order must be [T * top] int32")
        top = max(S // T, 1) if T else 1
    if offsets is not None:
        _tensor(offsets, "offsets", dev, torch.int32, (E + 1,))
    elif E != 1:
        raise ValueError("offsets are needed for more than one expert")
    dtype = _result_dtype(x, dtype, out)
    if _grads(x, x_scales, codes, scales):
        if x.dtype == E4M3:
            _no_gradient("kmeans_block_product", x=x, x_scales=x_scales)
        _no_gradient("kmeans_block_product", x_scales=x_scales, codes=codes, scales=scales)
        _no_buffers("kmeans_block_product", out)
        return _BlockProduct.apply(x, x_scales, codes, scales, offsets, order, dtype, ws)
    x, x_scales = _rows8(x, x_scales, "x", K)
    out = _output(out, "out", dev, dtype, (S, M))
    ws = _workspace(ws, dev, "kmeans_block_product_workspace_bytes", S, E, M, K)
    _call("kmeans_block_product", dev, x.data_ptr(), x_scales.data_ptr(), S, codes.data_ptr(), scales.data_ptr(), E, M, K,
          _ptr(offsets), _ptr(order), top, out.data_ptr(), _DT[dtype], *_ws_args(ws))
    return out


def kmeans_block_product_grad(grad, grad_scales, codes, scales, offsets=None, dtype=None, out=None, ws=None):
    """Gradient of kmeans_block_product's rows: out[p] = G[p] W[e] for grad
    [S, M], 8-bit codes with grad_scales [S, ceil(M / 128)] or wider with None
    (rounded to codes by the call) -> [S, K]."""
    dev = _rows_tensor(grad, "grad")
    E, M, K = _matrices(codes, scales, dev)
    S = grad.shape[0]
    if offsets is not None:
        _tensor(offsets, "offsets", dev, torch.int32, (E + 1,))
    elif E != 1:
        raise ValueError("offsets are needed for more than one expert")
    dtype = _result_dtype(grad, dtype, out)
    if _grads(grad, grad_scales, codes, scales):
        _no_gradient("kmeans_block_product_grad", grad=grad, grad_scales=grad_scales, codes=codes, scales=scales)
    grad, grad_scales = _rows8(grad, grad_scales, "grad", M)
    out = _output(out, "out", dev, dtype, (S, K))
    ws = _workspace(ws, dev, "kmeans_block_product_grad_workspace_bytes", S, E, M, K)
    _call("kmeans_block_product_grad", dev, grad.data_ptr(), grad_scales.data_ptr(), S, codes.data_ptr(),
          scales.data_ptr(), E, M, K, _ptr(offsets), out.data_ptr(), _DT[dtype], *_ws_args(ws))
    return out


# What autograd records (forward runs with recording off) --------------------

class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, eps, residual):
        y, h = kmeans_norm(x, weight, eps, residual)
        ctx.eps, ctx.added = eps, residual is not None
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(h, weight)
        return y, h if ctx.added else None

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, grad_h):
        h, weight = ctx.saved_tensors
        if grad is None:
            return grad_h, None, None, grad_h
        wanted = weight if ctx.needs_input_grad[1] else None
        gx, gw = _norm_grads(grad.contiguous(), h, weight, ctx.eps, None if grad_h is None else grad_h.contiguous(),
                             wanted is not None)
        return gx, gw, None, gx if ctx.added else None


def _norm_grads(grad, h, weight, eps, grad_residual, weighted):
    """kmeans_norm_grad, without the weight's gradient where it is not wanted."""
    if weight is None or weighted:
        return kmeans_norm_grad(grad, h, weight, eps, grad_residual)
    dev, dt = h.device, h.dtype
    gx = torch.empty_like(h)
    _call("kmeans_norm_grad", dev, grad.data_ptr(), h.data_ptr(), _DT[dt], *h.shape, _ptr(grad_residual),
          *_weight_args(weight, dt), eps, gx.data_ptr(), None, None, 0)
    return gx, None


class _Gate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top, normalize, ws):
        experts, weights, counts, shares, loss = kmeans_gate(logits, top, normalize, ws=ws)
        ctx.normalize = normalize
        ctx.mark_non_differentiable(experts, counts, shares)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(logits, experts, counts)
        return experts, weights, counts, shares, loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _e, grad_weights, _c, _s, grad_loss):
        logits, experts, counts = ctx.saved_tensors
        if grad_weights is not None:
            grad_weights = grad_weights.contiguous()
        return kmeans_gate_grad(logits, experts, counts, grad_weights, grad_loss, ctx.normalize), None, None, None


class _BlockProduct(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, x_scales, codes, scales, offsets, order, dtype, ws):
        ctx.T, ctx.dtype = x.shape[0], x.dtype
        ctx.save_for_backward(codes, scales, offsets, order)
        return kmeans_block_product(x, x_scales, codes, scales, offsets, order, dtype, ws=ws)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        codes, scales, offsets, order = ctx.saved_tensors
        rows = kmeans_block_product_grad(grad.contiguous(), None, codes, scales, offsets, ctx.dtype)
        if order is not None:
            # the rows back at the tokens that they were gathered from (of x's type, as a
            # dispatched layer has them: half the bytes of float32 rows for 16-bit tokens)
            S = order.numel()
            if S == 0:
                return rows.new_zeros((ctx.T, rows.shape[1])), *[None] * 7
            slots = torch.full((S + 1,), -1, dtype=torch.int32, device=order.device)
            slots[torch.where((order >= 0) & (order < S), order, S).long()] = torch.arange(
                S, dtype=torch.int32, device=order.device)
            rows = kmeans_combine(rows, slots[:S].view(ctx.T, -1))
        return rows, *[None] * 7
