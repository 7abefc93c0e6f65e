"""Python entry points with the C ABI's names (argument marshalling, and the
operators' gradients handed to torch's autograd).

Tensors are torch tensors on the GPU: torch provides the device memory and
the stream (the current stream of the tensors' device).  Every step of the
computation runs in the HIP kernels of libkmeans_mi355x.so.
"""
from __future__ import annotations

import ctypes

import torch
import torch.autograd.forward_ad as _forward

from . import _lib

_DT = {torch.float32: _lib.KM_F32, torch.float16: _lib.KM_F16, torch.bfloat16: _lib.KM_BF16}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dev_tensor(t, name, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _points(x):
    _dev_tensor(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be [B, N, d]")
    if x.dtype not in _DT:
        raise TypeError(f"x dtype {x.dtype} is not float32 / float16 / bfloat16")
    return x.shape


# The current stream's handle; building torch's Stream object for it takes
# about as long as launching a kernel.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev):
    if _raw_stream is not None and dev.index is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def workspace_bytes(B: int, N: int, d: int, K: int, dtype: torch.dtype) -> int:
    n = _lib.load().kmeans_workspace_bytes(B, N, d, K, _DT[dtype])
    if n == 0 and B * N * d * K > 0:
        _lib.check(2, "kmeans_workspace_bytes")
    return int(n)


def workspace(B: int, N: int, d: int, K: int, dtype: torch.dtype, device) -> torch.Tensor:
    """A device workspace large enough for every entry point at these shapes."""
    n = workspace_bytes(B, N, d, K, dtype)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _ws(ws, B, N, d, K, dtype, device):
    if ws is None:
        ws = workspace(B, N, d, K, dtype, device)
    _dev_tensor(ws, "workspace", torch.uint8)
    return ws


def kmeans_assign(x, centroids, weights=None, labels=None, min_dist=None, objective=None, ws=None):
    """Nearest centroid of every point.  Returns (labels, min_dist, objective);
    min_dist / objective are None unless tensors are passed in (or True)."""
    B, N, d = _points(x)
    _dev_tensor(centroids, "centroids", torch.float32)
    if centroids.dim() != 3 or centroids.shape[0] != B or centroids.shape[2] != d:
        raise ValueError("centroids must be [B, K, d] float32")
    K = centroids.shape[1]
    dev = x.device
    if weights is not None:
        _dev_tensor(weights, "weights", torch.float32, (B, N))
    labels = torch.empty((B, N), dtype=torch.int32, device=dev) if labels is None else \
        _dev_tensor(labels, "labels", torch.int32, (B, N))
    if min_dist is True:
        min_dist = torch.empty((B, N), dtype=torch.float32, device=dev)
    elif min_dist is not None:
        _dev_tensor(min_dist, "min_dist", torch.float32, (B, N))
    if objective is True:
        objective = torch.empty((B,), dtype=torch.float64, device=dev)
    elif objective is not None:
        _dev_tensor(objective, "objective", torch.float64, (B,))
    ws = _ws(ws, B, N, d, K, x.dtype, dev)
    st = _lib.load().kmeans_assign(_ptr(x), _DT[x.dtype], B, N, d, _ptr(centroids), K, _ptr(weights),
                                   _ptr(labels), _ptr(min_dist), _ptr(objective), _ptr(ws), ws.numel(),
                                   _stream(dev))
    _lib.check(st, "kmeans_assign")
    return labels, min_dist, objective


def kmeans_sort_labels(labels, K: int, ws=None):
    """Counting argsort of labels [B, N] int32.  Returns (counts, offsets, perm)."""
    _dev_tensor(labels, "labels", torch.int32)
    if labels.dim() != 2:
        raise ValueError("labels must be [B, N]")
    B, N = labels.shape
    dev = labels.device
    counts = torch.empty((B, K), dtype=torch.int32, device=dev)
    offsets = torch.empty((B, K + 1), dtype=torch.int32, device=dev)
    perm = torch.empty((B, N), dtype=torch.int32, device=dev)
    ws = _ws(ws, B, N, 2, K, torch.float32, dev)
    st = _lib.load().kmeans_sort_labels(_ptr(labels), B, N, K, _ptr(counts), _ptr(offsets), _ptr(perm),
                                        _ptr(ws), ws.numel(), _stream(dev))
    _lib.check(st, "kmeans_sort_labels")
    return counts, offsets, perm


def kmeans_update(x, labels, c_old, weights=None, c_new=None, counts=None, ws=None):
    """Centroids as the (weighted) means of their points; empty clusters keep
    c_old.  Returns (c_new, counts)."""
    B, N, d = _points(x)
    _dev_tensor(labels, "labels", torch.int32, (B, N))
    _dev_tensor(c_old, "c_old", torch.float32)
    if c_old.dim() != 3 or c_old.shape[0] != B or c_old.shape[2] != d:
        raise ValueError("c_old must be [B, K, d] float32")
    K = c_old.shape[1]
    dev = x.device
    if weights is not None:
        _dev_tensor(weights, "weights", torch.float32, (B, N))
    c_new = torch.empty_like(c_old) if c_new is None else _dev_tensor(c_new, "c_new", torch.float32, c_old.shape)
    counts = torch.empty((B, K), dtype=torch.int32, device=dev) if counts is None else \
        _dev_tensor(counts, "counts", torch.int32, (B, K))
    ws = _ws(ws, B, N, d, K, x.dtype, dev)
    st = _lib.load().kmeans_update(_ptr(x), _DT[x.dtype], _ptr(weights), B, N, d, _ptr(labels), K,
                                   _ptr(c_old), _ptr(c_new), _ptr(counts), _ptr(ws), ws.numel(), _stream(dev))
    _lib.check(st, "kmeans_update")
    return c_new, counts


def kmeans_fit(x, init, n_iter: int, weights=None, centroids=None, labels=None, counts=None,
               objective=None, ws=None, assign_events=None):
    """n_iter Lloyd iterations from init.  Returns (centroids, labels, counts,
    objective [B, n_iter] float64).  assign_events: None, or 2 * n_iter
    recorded torch.cuda.Event objects (enable_timing=True) of the tensors'
    device; event 2t is re-recorded right before iteration t's assignment
    kernels and event 2t + 1 right after them (kmeans_fit_timed)."""
    B, N, d = _points(x)
    _dev_tensor(init, "init", torch.float32)
    if init.dim() != 3 or init.shape[0] != B or init.shape[2] != d:
        raise ValueError("init must be [B, K, d] float32")
    K = init.shape[1]
    dev = x.device
    if weights is not None:
        _dev_tensor(weights, "weights", torch.float32, (B, N))
    centroids = torch.empty_like(init) if centroids is None else \
        _dev_tensor(centroids, "centroids", torch.float32, init.shape)
    labels = torch.empty((B, N), dtype=torch.int32, device=dev) if labels is None else \
        _dev_tensor(labels, "labels", torch.int32, (B, N))
    counts = torch.empty((B, K), dtype=torch.int32, device=dev) if counts is None else \
        _dev_tensor(counts, "counts", torch.int32, (B, K))
    objective = torch.empty((B, max(n_iter, 0)), dtype=torch.float64, device=dev) if objective is None else \
        _dev_tensor(objective, "objective", torch.float64, (B, n_iter))
    ws = _ws(ws, B, N, d, K, x.dtype, dev)
    if assign_events is None:
        st = _lib.load().kmeans_fit(_ptr(x), _DT[x.dtype], _ptr(weights), B, N, d, K, _ptr(init), int(n_iter),
                                    _ptr(centroids), _ptr(labels), _ptr(counts), _ptr(objective), _ptr(ws),
                                    ws.numel(), _stream(dev))
        _lib.check(st, "kmeans_fit")
        return centroids, labels, counts, objective
    if len(assign_events) != 2 * n_iter:
        raise ValueError(f"assign_events must hold 2 * n_iter = {2 * n_iter} events")
    handles = []
    for e in assign_events:
        h = getattr(e, "cuda_event", 0)
        if not h:
            raise ValueError("assign_events must be torch.cuda.Event objects recorded once (so that they exist)")
        handles.append(h)
    arr = (ctypes.c_void_p * len(handles))(*handles)
    st = _lib.load().kmeans_fit_timed(_ptr(x), _DT[x.dtype], _ptr(weights), B, N, d, K, _ptr(init), int(n_iter),
                                      _ptr(centroids), _ptr(labels), _ptr(counts), _ptr(objective), arr, _ptr(ws),
                                      ws.numel(), _stream(dev))
    _lib.check(st, "kmeans_fit_timed")
    return centroids, labels, counts, objective


def kmeans_fit_static(x, init, n_iter: int, weights=None, centroids=None, labels=None, counts=None,
                      objective=None):
    """kmeans_fit without a workspace: the library's static per-device scratch
    (kmeans_fit_static_max_bytes() bytes) serves instead, so the call
    allocates nothing itself (pass every output tensor to allocate nothing
    here either).  Returns (centroids, labels, counts, objective)."""
    B, N, d = _points(x)
    _dev_tensor(init, "init", torch.float32)
    if init.dim() != 3 or init.shape[0] != B or init.shape[2] != d:
        raise ValueError("init must be [B, K, d] float32")
    K = init.shape[1]
    dev = x.device
    if weights is not None:
        _dev_tensor(weights, "weights", torch.float32, (B, N))
    centroids = torch.empty_like(init) if centroids is None else \
        _dev_tensor(centroids, "centroids", torch.float32, init.shape)
    labels = torch.empty((B, N), dtype=torch.int32, device=dev) if labels is None else \
        _dev_tensor(labels, "labels", torch.int32, (B, N))
    counts = torch.empty((B, K), dtype=torch.int32, device=dev) if counts is None else \
        _dev_tensor(counts, "counts", torch.int32, (B, K))
    objective = torch.empty((B, max(n_iter, 0)), dtype=torch.float64, device=dev) if objective is None else \
        _dev_tensor(objective, "objective", torch.float64, (B, n_iter))
    st = _lib.load().kmeans_fit_static(_ptr(x), _DT[x.dtype], _ptr(weights), B, N, d, K, _ptr(init), int(n_iter),
                                       _ptr(centroids), _ptr(labels), _ptr(counts), _ptr(objective), _stream(dev))
    _lib.check(st, "kmeans_fit_static")
    return centroids, labels, counts, objective


def kmeans_optimal_1d(x, K: int, weights=None, centroids=None, labels=None, counts=None, objective=None, ws=None):
    """Globally optimal weighted 1D k-means of every row of x [B, N] (or
    [B, N, 1]).  Returns (centroids [B, K] float32 ascending, labels [B, N]
    int32, counts [B, K] int32, objective [B] float64)."""
    _dev_tensor(x, "x")
    if x.dim() == 3 and x.shape[2] == 1:
        B, N = x.shape[0], x.shape[1]
    elif x.dim() == 2:
        B, N = x.shape
    else:
        raise ValueError("x must be [B, N] or [B, N, 1]")
    if x.dtype not in _DT:
        raise TypeError(f"x dtype {x.dtype} is not float32 / float16 / bfloat16")
    dev = x.device
    if weights is not None:
        _dev_tensor(weights, "weights", torch.float32, (B, N))
    centroids = torch.empty((B, K), dtype=torch.float32, device=dev) if centroids is None else \
        _dev_tensor(centroids, "centroids", torch.float32, (B, K))
    labels = torch.empty((B, N), dtype=torch.int32, device=dev) if labels is None else \
        _dev_tensor(labels, "labels", torch.int32, (B, N))
    counts = torch.empty((B, K), dtype=torch.int32, device=dev) if counts is None else \
        _dev_tensor(counts, "counts", torch.int32, (B, K))
    objective = torch.empty((B,), dtype=torch.float64, device=dev) if objective is None else \
        _dev_tensor(objective, "objective", torch.float64, (B,))
    L = _lib.load()
    if ws is None:
        n = L.kmeans_optimal_1d_workspace_bytes(B, N, K)
        ws = torch.empty(max(int(n), 256), dtype=torch.uint8, device=dev)
    _dev_tensor(ws, "workspace", torch.uint8)
    st = L.kmeans_optimal_1d(_ptr(x), _DT[x.dtype], _ptr(weights), B, N, K, _ptr(centroids), _ptr(labels),
                             _ptr(counts), _ptr(objective), _ptr(ws), ws.numel(), _stream(dev))
    _lib.check(st, "kmeans_optimal_1d")
    return centroids, labels, counts, objective


def kmeans_fit_stream(x_host, init, n_iter: int, weights=None, chunk: int = 1 << 22, centroids=None, labels=None,
                      counts=None, objective=None, ws=None):
    """n_iter Lloyd iterations of one problem whose points x_host [N, d] (or
    [1, N, d]) stay in host memory (a CPU tensor, ideally pinned), streamed
    to the GPU in chunks of `chunk` points.  init [K, d] (or [1, K, d])
    float32 on the GPU.  Returns (centroids [K, d], labels [N] (None unless
    True or a tensor is passed), counts [K], objective [n_iter] float64)."""
    if not isinstance(x_host, torch.Tensor) or x_host.is_cuda:
        raise ValueError("x_host must be a CPU tensor")
    if not x_host.is_contiguous():
        raise ValueError("x_host must be contiguous")
    if x_host.dim() == 3 and x_host.shape[0] == 1:
        x_host = x_host[0]
    if x_host.dim() != 2:
        raise ValueError("x_host must be [N, d]")
    if x_host.dtype not in _DT:
        raise TypeError(f"x dtype {x_host.dtype} is not float32 / float16 / bfloat16")
    N, d = x_host.shape
    _dev_tensor(init, "init", torch.float32)
    if init.dim() == 3 and init.shape[0] == 1:
        init = init[0]
    if init.dim() != 2 or init.shape[1] != d:
        raise ValueError("init must be [K, d] float32")
    K = init.shape[0]
    dev = init.device
    if weights is not None:
        if not isinstance(weights, torch.Tensor) or weights.is_cuda or weights.dtype != torch.float32 \
                or tuple(weights.shape) != (N,) or not weights.is_contiguous():
            raise ValueError("weights must be a contiguous float32 CPU tensor [N]")
    centroids = torch.empty_like(init) if centroids is None else \
        _dev_tensor(centroids, "centroids", torch.float32, init.shape)
    if labels is True:
        labels = torch.empty((N,), dtype=torch.int32, device=dev)
    elif labels is not None:
        _dev_tensor(labels, "labels", torch.int32, (N,))
    counts = torch.empty((K,), dtype=torch.int32, device=dev) if counts is None else \
        _dev_tensor(counts, "counts", torch.int32, (K,))
    objective = torch.empty((max(n_iter, 0),), dtype=torch.float64, device=dev) if objective is None else \
        _dev_tensor(objective, "objective", torch.float64, (n_iter,))
    L = _lib.load()
    if ws is None:
        # 0 for arguments the entry point rejects: it then reports why
        n = L.kmeans_stream_workspace_bytes(N, d, K, _DT[x_host.dtype], chunk)
        ws = torch.empty(max(int(n), 256), dtype=torch.uint8, device=dev)
    _dev_tensor(ws, "workspace", torch.uint8)
    st = L.kmeans_fit_stream(_ptr(x_host), _DT[x_host.dtype], _ptr(weights), N, d, K, _ptr(init), int(n_iter),
                             _ptr(centroids), _ptr(labels), _ptr(counts), _ptr(objective), int(chunk), _ptr(ws),
                             ws.numel(), _stream(dev))
    _lib.check(st, "kmeans_fit_stream")
    return centroids, labels, counts, objective


def emeans_steps(N: int, batch: int, epochs: int) -> int:
    """Number of e-means steps: epochs times the batches of one pass."""
    return epochs * ((N + batch - 1) // batch) if N > 0 else 0


def kmeans_emeans(x, init, batch: int, epochs: int, alpha0: float, floor_frac: float = 0.1, dead_frac: float = 0.0,
                  eps: float = 1e-3, uniforms=None, centroids=None, labels=None, counts=None, objective=None,
                  ws=None):
    """e-means (moving-average mini-batch k-means) of one problem x [N, d]
    (or [1, N, d]) on the GPU from init [K, d] float32.  uniforms [T, K]
    float32 on the GPU (T = emeans_steps(N, batch, epochs)) are the split
    draws, needed when dead_frac > 0.  Returns (centroids [K, d], labels [N]
    (None unless True or a tensor is passed), counts [K], objective [T]
    float64)."""
    _dev_tensor(x, "x")
    if x.dim() == 3 and x.shape[0] == 1:
        x = x[0]
    if x.dim() != 2:
        raise ValueError("x must be [N, d]")
    if x.dtype not in _DT:
        raise TypeError(f"x dtype {x.dtype} is not float32 / float16 / bfloat16")
    N, d = x.shape
    _dev_tensor(init, "init", torch.float32)
    if init.dim() == 3 and init.shape[0] == 1:
        init = init[0]
    if init.dim() != 2 or init.shape[1] != d:
        raise ValueError("init must be [K, d] float32")
    K = init.shape[0]
    dev = x.device
    T = emeans_steps(N, batch, epochs) if batch >= 1 and epochs >= 1 else 0
    if uniforms is not None:
        _dev_tensor(uniforms, "uniforms", torch.float32, (T, K))
    centroids = torch.empty_like(init) if centroids is None else \
        _dev_tensor(centroids, "centroids", torch.float32, init.shape)
    if labels is True:
        labels = torch.empty((N,), dtype=torch.int32, device=dev)
    elif labels is not None:
        _dev_tensor(labels, "labels", torch.int32, (N,))
    counts = torch.empty((K,), dtype=torch.int32, device=dev) if counts is None else \
        _dev_tensor(counts, "counts", torch.int32, (K,))
    objective = torch.empty((T,), dtype=torch.float64, device=dev) if objective is None else \
        _dev_tensor(objective, "objective", torch.float64, (T,))
    L = _lib.load()
    if ws is None:
        # 0 for arguments the entry point rejects: it then reports why
        n = L.kmeans_emeans_workspace_bytes(N, d, K, _DT[x.dtype], int(batch))
        ws = torch.empty(max(int(n), 256), dtype=torch.uint8, device=dev)
    _dev_tensor(ws, "workspace", torch.uint8)
    st = L.kmeans_emeans(_ptr(x), _DT[x.dtype], N, d, K, _ptr(init), int(batch), int(epochs), float(alpha0),
                         float(floor_frac), float(dead_frac), float(eps), _ptr(uniforms), _ptr(centroids),
                         _ptr(labels), _ptr(counts), _ptr(objective), _ptr(ws), ws.numel(), _stream(dev))
    _lib.check(st, "kmeans_emeans")
    return centroids, labels, counts, objective


# Labels and codebooks inside a model --------------------------------------
# A call may be a few microseconds of GPU work, so these wrappers check each
# tensor once and keep to the checks that the C ABI cannot make.

def _tensor(t, name, dev, dtype, shape):
    """t checked against a device, a dtype (None: any the library has) and a
    shape (None: any); dev None: any GPU."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is None:
        if t.dtype not in _DT:
            raise TypeError(f"{name} dtype {t.dtype} is not float32 / float16 / bfloat16")
    elif t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _output(t, name, dev, dtype, shape):
    return torch.empty(shape, dtype=dtype, device=dev) if t is None else _tensor(t, name, dev, dtype, shape)


def _grads(*tensors):
    """Whether autograd records a call of these inputs (None among them).  Forward-mode
    tangents, which no operator takes along, are refused."""
    if getattr(_forward, "_current_level", 0) >= 0:  # (dual tensors live inside a dual_level)
        _no_tangents(tensors)
    for t in tensors:
        if t is not None and t.requires_grad:
            return torch.is_grad_enabled()
    return False


def _no_tangents(tensors):
    # (a dual tensor does not require a gradient, and results would pass for constants)
    for t in tensors:
        if t is not None and _forward.unpack_dual(t).tangent is not None:
            raise ValueError("the operators have no forward-mode derivatives: pass the primal of a dual tensor "
                             "(torch.autograd.forward_ad.unpack_dual)")


def _no_gradient(name, **tensors):
    # a result without history would lose these tensors' gradients without a word
    for arg, t in tensors.items():
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} has no gradient of {arg}: pass {arg}.detach(), or call it under torch.no_grad()")


def _no_buffers(name, *buffers):
    if any(b is not None for b in buffers):
        raise ValueError(f"{name} cannot write to given tensors where autograd records it: pass none, or call it "
                         "under torch.no_grad()")


def _bytes(n, device):
    return torch.empty(max(int(n), 256), dtype=torch.uint8, device=device)


def kmeans_lookup(table, labels, scale: float = 1.0, out=None):
    """scale * table[b, labels[b, i]] for every label: table [B, V, d], labels
    [B, N] int32 -> [B, N, d]; labels outside [0, V) give rows of zeros.
    Differentiable in table."""
    _tensor(table, "table", None, None, None)
    if table.dim() != 3:
        raise ValueError("table must be [B, V, d]")
    B, V, d = table.shape
    dev = table.device
    _tensor(labels, "labels", dev, torch.int32, None)
    if labels.dim() != 2 or labels.shape[0] != B:
        raise ValueError("labels must be [B, N] int32")
    if _grads(table):
        _no_buffers("kmeans_lookup", out)
        return _Lookup.apply(table, labels, scale)
    N = labels.shape[1]
    out = _output(out, "out", dev, table.dtype, (B, N, d))
    st = _lib.load().kmeans_lookup(table.data_ptr(), _DT[table.dtype], B, V, d, labels.data_ptr(), N, scale,
                                   out.data_ptr(), _stream(dev))
    if st:
        _lib.check(st, "kmeans_lookup")
    return out


def lookup_grad_workspace(B: int, N: int, d: int, V: int, dtype: torch.dtype, device) -> torch.Tensor:
    """A workspace for kmeans_lookup_grad at these shapes."""
    return _bytes(_lib.load().kmeans_lookup_grad_workspace_bytes(B, N, d, V, _DT[dtype]), device)


def kmeans_lookup_grad(grad, labels, V: int, scale: float = 1.0, out=None, ws=None):
    """Gradient of kmeans_lookup's table: scale times the sum of grad's rows
    per label.  grad [B, N, d], labels [B, N] int32 -> [B, V, d] of grad's
    dtype, or of out's (grad's dtype or float32)."""
    _tensor(grad, "grad", None, None, None)
    if grad.dim() != 3:
        raise ValueError("grad must be [B, N, d]")
    if _grads(grad):
        _no_gradient("kmeans_lookup_grad", grad=grad)
    B, N, d = grad.shape
    dev = grad.device
    _tensor(labels, "labels", dev, torch.int32, (B, N))
    if out is None:
        out = torch.empty((B, V, d), dtype=grad.dtype, device=dev)
    else:
        _tensor(out, "out", dev, None, (B, V, d))
    ws = lookup_grad_workspace(B, N, d, V, grad.dtype, dev) if ws is None else \
        _tensor(ws, "workspace", dev, torch.uint8, None)
    st = _lib.load().kmeans_lookup_grad(grad.data_ptr(), _DT[grad.dtype], B, N, d, labels.data_ptr(), V, scale,
                                        out.data_ptr(), _DT[out.dtype], ws.data_ptr(), ws.numel(), _stream(dev))
    if st:
        _lib.check(st, "kmeans_lookup_grad")
    return out


def dispatch_workspace(T: int, top: int, E: int, device) -> torch.Tensor:
    """A workspace for kmeans_dispatch at these shapes."""
    return _bytes(_lib.load().kmeans_dispatch_workspace_bytes(T, top, E), device)


def kmeans_dispatch(x, experts, E: int, rows=None, plan=None, ws=None):
    """Tokens sorted by expert: x [T, d], experts [T, top] int32 (outside
    [0, E): dropped).  Returns (rows [T * top, d], offsets [E + 1], slots
    [T, top], order [T * top]): expert e's rows are rows[offsets[e] :
    offsets[e + 1]], rows[slots[t, k]] = x[t], order[p] = t * top + k, and the
    rows from offsets[E] on are zeros with order -1; dropped choices have slot
    -1.  plan: (offsets, slots, order) tensors to write.  Differentiable in x;
    its gradient is kmeans_combine(grad_rows, slots, None)."""
    _tensor(x, "x", None, None, None)
    if x.dim() != 2:
        raise ValueError("x must be [T, d]")
    T, d = x.shape
    dev = x.device
    _tensor(experts, "experts", dev, torch.int32, None)
    if experts.dim() != 2 or experts.shape[0] != T:
        raise ValueError("experts must be [T, top] int32")
    if _grads(x):
        _no_buffers("kmeans_dispatch", rows, plan)
        return _Dispatch.apply(x, experts, E, ws)
    top = experts.shape[1]
    rows = _output(rows, "rows", dev, x.dtype, (T * top, d))
    offsets, slots, order = (None, None, None) if plan is None else plan
    offsets = _output(offsets, "offsets", dev, torch.int32, (E + 1,))
    slots = _output(slots, "slots", dev, torch.int32, (T, top))
    order = _output(order, "order", dev, torch.int32, (T * top,))
    ws = dispatch_workspace(T, top, E, dev) if ws is None else _tensor(ws, "workspace", dev, torch.uint8, None)
    st = _lib.load().kmeans_dispatch(x.data_ptr(), _DT[x.dtype], T, d, experts.data_ptr(), top, E, rows.data_ptr(),
                                     offsets.data_ptr(), slots.data_ptr(), order.data_ptr(), ws.data_ptr(),
                                     ws.numel(), _stream(dev))
    if st:
        _lib.check(st, "kmeans_dispatch")
    return rows, offsets, slots, order


def _sorted_rows(rows, slots):
    _tensor(rows, "rows", None, None, None)
    dev = rows.device
    _tensor(slots, "slots", dev, torch.int32, None)
    if slots.dim() != 2:
        raise ValueError("slots must be [T, top] int32")
    T, top = slots.shape
    if rows.dim() != 2 or rows.shape[0] != T * top:
        raise ValueError("rows must be [T * top, d]")
    return T, top, rows.shape[1], dev


def kmeans_combine(rows, slots, weights=None, out=None):
    """Sorted rows back at their tokens: out[t] = sum_k weights[t, k] *
    rows[slots[t, k]] (weights None: all 1), slots -1 adding nothing.
    Differentiable in rows and weights."""
    T, top, d, dev = _sorted_rows(rows, slots)
    if weights is not None:
        _tensor(weights, "weights", dev, torch.float32, (T, top))
    if _grads(rows, weights):
        _no_buffers("kmeans_combine", out)
        return _Combine.apply(rows, slots, weights)
    out = _output(out, "out", dev, rows.dtype, (T, d))
    st = _lib.load().kmeans_combine(rows.data_ptr(), _DT[rows.dtype], T, d, top, slots.data_ptr(), _ptr(weights),
                                    out.data_ptr(), _stream(dev))
    if st:
        _lib.check(st, "kmeans_combine")
    return out


def kmeans_combine_grad(grad, rows, slots, order, weights, grad_rows=None, grad_weights=None):
    """Gradients of kmeans_combine: (grad_rows [T * top, d] = weights * grad at
    every slot, zeros from offsets[E] on; grad_weights [T, top] float32 = <grad,
    row>, 0 for a dropped choice)."""
    T, top, d, dev = _sorted_rows(rows, slots)
    _tensor(grad, "grad", dev, rows.dtype, (T, d))
    _tensor(order, "order", dev, torch.int32, (T * top,))
    _tensor(weights, "weights", dev, torch.float32, (T, top))
    if _grads(grad, rows, weights):
        _no_gradient("kmeans_combine_grad", grad=grad, rows=rows, weights=weights)
    grad_rows = _output(grad_rows, "grad_rows", dev, rows.dtype, (T * top, d))
    grad_weights = _output(grad_weights, "grad_weights", dev, torch.float32, (T, top))
    st = _lib.load().kmeans_combine_grad(grad.data_ptr(), rows.data_ptr(), _DT[rows.dtype], T, d, top,
                                         slots.data_ptr(), order.data_ptr(), weights.data_ptr(),
                                         grad_rows.data_ptr(), grad_weights.data_ptr(), _stream(dev))
    if st:
        _lib.check(st, "kmeans_combine_grad")
    return grad_rows, grad_weights


def kmeans_pack_codes(labels, codes=None):
    """4-bit labels [M, K] int32 (as kmeans_fit labels the scalar rows of a
    weight matrix, K <= 16 clusters) laid out for kmeans_codes_product:
    uint8 [ceil(M / 16), ceil(K / 128), 1024]."""
    _tensor(labels, "labels", None, torch.int32, None)
    if labels.dim() != 2:
        raise ValueError("labels must be [M, K] int32")
    M, K = labels.shape
    dev = labels.device
    codes = _output(codes, "codes", dev, torch.uint8, (-(-M // 16), -(-K // 128), 1024))
    st = _lib.load().kmeans_pack_codes(labels.data_ptr(), M, K, codes.data_ptr(), _stream(dev))
    if st:
        _lib.check(st, "kmeans_pack_codes")
    return codes


def codes_workspace(S: int, E: int, M: int, K: int, dtype: torch.dtype, device) -> torch.Tensor:
    """A workspace for kmeans_codes_product_grad at these shapes (the product
    itself needs none)."""
    return _bytes(_lib.load().kmeans_codes_workspace_bytes(S, E, M, K, _DT[dtype]), device)


def _codes_call(name, x, codes, table, M, K, scales, group, offsets, out, n_out, ws):
    dev, dt, S = x.device, x.dtype, x.shape[0]
    _tensor(codes, "codes", dev, torch.uint8, None)
    tiles = (-(-M // 16), -(-K // 128), 1024)
    shape = tuple(codes.shape)
    if len(shape) == 4:
        E, shape = shape[0], shape[1:]
    elif len(shape) == 3:
        E = 1
    else:
        raise ValueError("codes must be [E, ceil(M / 16), ceil(K / 128), 1024] (or without E)")
    if shape != tiles:
        raise ValueError(f"codes must be tiles {tiles}, got {shape}")
    _tensor(table, "table", dev, dt, None)
    shape = tuple(table.shape)
    rows = shape[-2] if len(shape) > 1 else 0
    if (rows != M and rows != 1) or shape[-1] != 16 or table.numel() != E * rows * 16:
        raise ValueError("table must be [E, M, 16] or [E, 1, 16]")
    if scales is not None:
        groups = -(-K // group) if group > 0 else 0
        _tensor(scales, "scales", dev, dt, None)
        if tuple(scales.shape[-2:]) != (M, groups) or scales.numel() != E * M * groups:
            raise ValueError("scales must be [E, M, ceil(K / group)]")
    if offsets is not None:
        _tensor(offsets, "offsets", dev, torch.int32, (E + 1,))
    elif E != 1:
        raise ValueError("offsets are needed for more than one expert")
    if _grads(x, table, scales):
        _no_gradient(name, table=table, scales=scales)
        if name == "kmeans_codes_product_grad":
            _no_gradient(name, grad=x)
        else:
            _no_buffers(name, out)
            return _Product.apply(x, codes, table, M, scales, group, offsets)
    out = _output(out, "out", dev, dt, (S, n_out))
    if ws is not None:
        _tensor(ws, "workspace", dev, torch.uint8, None)
    elif name == "kmeans_codes_product_grad":
        ws = codes_workspace(S, E, M, K, dt, dev)
    st = getattr(_lib.load(), name)(x.data_ptr(), _DT[dt], S, codes.data_ptr(), table.data_ptr(), rows, _ptr(scales),
                                    group, E, M, K, _ptr(offsets), out.data_ptr(), _ptr(ws),
                                    0 if ws is None else ws.numel(), _stream(dev))
    if st:
        _lib.check(st, name)
    return out


def kmeans_codes_product(x, codes, table, M: int, scales=None, group: int = 0, offsets=None, out=None, ws=None):
    """Rows times 4-bit matrices: out[p, m] = sum_k x[p, k] * scales[e, m, k //
    group] * table[e, m, code[e, m, k]], e the expert whose segment
    offsets[e] : offsets[e + 1] holds p (offsets None: one matrix).  x [S, K]
    float16 / bfloat16, codes of kmeans_pack_codes (stacked over the experts),
    table [E, M, 16] or [E, 1, 16] and scales [E, M, ceil(K / group)] of x's
    dtype.  Returns [S, M]; rows past offsets[E] are zeros.  Differentiable in
    x; the codebooks and scales are held."""
    _tensor(x, "x", None, None, None)
    if x.dim() != 2:
        raise ValueError("x must be [S, K]")
    return _codes_call("kmeans_codes_product", x, codes, table, M, x.shape[1], scales, group, offsets, out, M, ws)


def kmeans_codes_product_grad(grad, codes, table, K: int, scales=None, group: int = 0, offsets=None, out=None, ws=None):
    """Gradient of kmeans_codes_product's x: grad [S, M] -> [S, K]."""
    _tensor(grad, "grad", None, None, None)
    if grad.dim() != 2:
        raise ValueError("grad must be [S, M]")
    return _codes_call("kmeans_codes_product_grad", grad, codes, table, grad.shape[1], K, scales, group, offsets, out,
                       K, ws)


# What autograd records of a call whose input requires a gradient: the call
# itself and, backwards, the entry point of its gradient.  (forward runs with
# recording off.)

class _Lookup(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, labels, scale):
        ctx.save_for_backward(labels)
        ctx.V, ctx.scale = table.shape[1], scale
        return kmeans_lookup(table, labels, scale)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        return kmeans_lookup_grad(grad.contiguous(), ctx.saved_tensors[0], ctx.V, ctx.scale), None, None


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, experts, E, ws):
        rows, *plan = kmeans_dispatch(x, experts, E, ws=ws)
        ctx.mark_non_differentiable(*plan)
        ctx.save_for_backward(plan[1])
        return (rows, *plan)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, *_):
        return kmeans_combine(grad.contiguous(), ctx.saved_tensors[0], None), None, None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, slots, weights):
        ctx.save_for_backward(rows, slots, weights)
        return kmeans_combine(rows, slots, weights)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        rows, slots, weights = ctx.saved_tensors
        S = slots.numel()
        # the dispatch's order, of which the gradient reads where it is -1
        flat = slots.view(-1)
        order = torch.full((S + 1,), -1, dtype=torch.int32, device=slots.device)
        order.index_fill_(0, torch.where((flat >= 0) & (flat < S), flat, S).long(), 0)
        ones = torch.ones(slots.shape, device=slots.device) if weights is None else weights
        grad_rows, grad_weights = kmeans_combine_grad(grad.contiguous(), rows, slots, order[:S], ones)
        return grad_rows, None, None if weights is None else grad_weights


class _Product(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, codes, table, M, scales, group, offsets):
        ctx.save_for_backward(codes, table, scales, offsets)
        ctx.K, ctx.group = x.shape[1], group
        return kmeans_codes_product(x, codes, table, M, scales, group, offsets)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        codes, table, scales, offsets = ctx.saved_tensors
        return (kmeans_codes_product_grad(grad.contiguous(), codes, table, ctx.K, scales, ctx.group, offsets),
                *[None] * 6)
