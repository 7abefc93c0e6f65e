"""The entry points of a layer of 8-bit experts on a machine without a GPU: sizes
of their workspaces, and invalid arguments refused on the host before any HIP
call."""
import ctypes as C

import pytest

FAKE = C.c_void_p(0x1000)  # never dereferenced: every case fails before any HIP call
WS = C.c_void_p(0x100000)
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from exact_lloyd_means_03_amd import _lib
    return _lib.load()


def _call(fn, defaults):
    def call(**kw):
        a = dict(defaults)
        assert set(kw) <= set(a)
        a.update(kw)
        return fn(*a.values())
    return call


def test_quantize_rejects(lib):
    call = _call(lib.kmeans_quantize, dict(x=FAKE, xt=BF16, B=2, M=10, K=64, rows=1, codes=FAKE, scales=FAKE, stream=None))
    for name in ("x", "codes", "scales"):
        assert call(**{name: None}) == 1 and name.encode() in lib.kmeans_last_error()
    assert call(xt=3) == 2 and call(rows=2) == 1 and call(rows=0) == 1
    assert call(B=-1) == 1 and call(M=-1) == 1 and call(K=0) == 1
    assert call(B=70000) == 2 and call(K=(1 << 20) + 1) == 2 and call(M=1 << 31) == 2 and call(B=65535, M=1 << 20) == 2
    assert call(rows=128, M=(1 << 20) + 1) == 2
    assert call(B=0, x=None, codes=None, scales=None) == 0  # nothing to do, nothing enqueued


def test_norm_rejects(lib):
    call = _call(lib.kmeans_norm, dict(x=FAKE, xt=F16, T=10, d=64, residual=FAKE, weight=FAKE, wt=F16, eps=1e-6, h=FAKE,
                                       y=FAKE, codes=None, scales=None, stream=None))
    assert call(x=None) == 1 and call(y=None) == 1 and b"exactly one" in lib.kmeans_last_error()
    assert call(codes=FAKE, scales=FAKE) == 1 and call(codes=FAKE) == 1 and call(y=None, codes=FAKE) == 1
    assert call(xt=7) == 2 and call(wt=BF16) == 2 and call(wt=9) == 2
    assert call(T=-1) == 1 and call(d=0) == 1 and call(T=1 << 31) == 2 and call(d=32769) == 2 and call(xt=F32, wt=F32, d=16385) == 2
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    assert call(T=0, x=None, y=None) == 0


def test_norm_grad_rejects(lib):
    q = lib.kmeans_norm_grad_workspace_bytes
    assert q(1000, 512, BF16) >= 512 * 4 and q(1000, 512, BF16) % 256 == 0
    assert q(1000, 0, BF16) == 0 and q(-1, 8, BF16) == 0 and q(10, 40000, F16) == 0 and q(10, 8, 5) == 0
    call = _call(lib.kmeans_norm_grad, dict(grad=FAKE, h=FAKE, xt=F16, T=1000, d=64, grad_residual=None, weight=FAKE, wt=F16,
                                            eps=0.0, grad_x=FAKE, grad_weight=FAKE, ws=WS, ws_bytes=1 << 30, stream=None))
    for name in ("grad", "h", "grad_x"):
        assert call(**{name: None}) == 1 and name.encode() in lib.kmeans_last_error()
    assert call(ws=None) == 1 and call(ws=C.c_void_p(0x100010)) == 1 and call(ws_bytes=256) == 3
    assert call(wt=BF16) == 2 and call(weight=None, wt=BF16) == 2 and call(d=50000) == 2 and call(T=-2) == 1


def test_gate_rejects(lib):
    q = lib.kmeans_gate_workspace_bytes
    assert q(5000, 64) >= 64 * 8 and q(5000, 64) % 256 == 0 and q(24, 64) == q(0, 8) == 0
    assert q(-1, 8) == 0 and q(5, 0) == 0 and q(5, 4097) == 0
    call = _call(lib.kmeans_gate, dict(logits=FAKE, xt=F32, T=100, E=8, top=2, normalize=1, experts=FAKE, weights=FAKE,
                                       counts=FAKE, shares=FAKE, loss=FAKE, ws=WS, ws_bytes=1 << 30, stream=None))
    for name in ("logits", "experts", "weights", "counts", "shares", "loss"):
        assert call(**{name: None}) == 1 and name.encode() in lib.kmeans_last_error()
    assert call(top=0) == 1 and call(top=9) == 1 and call(E=100, top=65) == 2 and call(E=0) == 1 and call(E=5000) == 2
    assert call(T=-1) == 1 and call(T=1 << 31) == 2 and call(T=1 << 30, top=2) == 2 and call(xt=8) == 2
    assert call(T=1000, ws=None) == 1 and call(T=1000, ws_bytes=16) == 3
    grad = _call(lib.kmeans_gate_grad, dict(logits=FAKE, xt=F32, T=100, E=8, top=2, normalize=1, experts=FAKE, counts=FAKE,
                                            grad_weights=FAKE, grad_loss=FAKE, grad_logits=FAKE, stream=None))
    for name in ("logits", "experts", "counts", "grad_logits"):
        assert grad(**{name: None}) == 1 and name.encode() in lib.kmeans_last_error()
    assert grad(top=9) == 1 and grad(T=-1) == 1 and grad(xt=4) == 2


def test_plan_rejects(lib):
    assert lib.kmeans_plan_workspace_bytes(100, 2, 8) == lib.kmeans_dispatch_workspace_bytes(100, 2, 8)
    assert lib.kmeans_plan_workspace_bytes(100000, 2, 64) == lib.kmeans_dispatch_workspace_bytes(100000, 2, 64) > 0
    call = _call(lib.kmeans_plan, dict(experts=FAKE, T=10000, top=2, E=8, offsets=FAKE, slots=FAKE, order=FAKE, ws=WS,
                                       ws_bytes=1 << 30, stream=None))
    for name in ("experts", "offsets", "slots", "order"):
        assert call(**{name: None}) == 1 and name.encode() in lib.kmeans_last_error()
    assert call(E=0) == 1 and call(E=4097) == 2 and call(top=0) == 1 and call(T=1 << 30) == 2
    assert call(ws=None) == 1 and call(ws_bytes=16) == 3


def test_block_products_reject(lib):
    for grad in (False, True):
        q = lib.kmeans_block_product_grad_workspace_bytes if grad else lib.kmeans_block_product_workspace_bytes
        assert q(8, 1, 64, 128) % 256 == 0
        assert q(-1, 1, 64, 128) == 0 and q(8, 0, 64, 128) == 0 and q(8, 1, 0, 128) == 0 and q(8, 1, 64, (1 << 20) + 1) == 0
        d = dict(x=FAKE, xs=FAKE, S=8, codes=FAKE, scales=FAKE, E=2, M=64, K=128, offsets=FAKE)
        if not grad:
            d |= dict(order=None, top=1)
        d |= dict(out=FAKE, ot=BF16, ws=WS, ws_bytes=1 << 30, stream=None)
        call = _call(lib.kmeans_block_product_grad if grad else lib.kmeans_block_product, d)
        for name in ("x", "xs", "codes", "scales", "offsets", "out"):
            assert call(**{name: None}) == 1, name
        assert call(ot=3) == 2 and call(S=-1) == 1 and call(M=0) == 1 and call(K=0) == 1 and call(E=0) == 1
        assert call(E=5000) == 2 and call(S=(1 << 20) + 1) == 2 and call(M=(1 << 20) + 1) == 2
        if not grad:
            assert call(order=FAKE, top=3) == 1 and b"multiple of top" in lib.kmeans_last_error()
            assert call(order=FAKE, top=0) == 1


def test_python_wrappers_want_gpu_tensors():
    import torch
    import exact_lloyd_means_03_amd as km
    x = torch.zeros((4, 128))
    q = torch.zeros((4, 128), dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones((4, 1))
    for call in (lambda: km.kmeans_quantize(x), lambda: km.kmeans_norm(x), lambda: km.kmeans_norm_quantize(x),
                 lambda: km.kmeans_norm_grad(x, x), lambda: km.kmeans_gate(x, 2),
                 lambda: km.kmeans_gate_grad(x, s.int(), s.int()), lambda: km.kmeans_plan(s.int(), 4),
                 lambda: km.kmeans_block_product(q, s, q, s[:1]), lambda: km.kmeans_block_product_grad(q, s, q, s[:1])):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError, match="Tensor"):
        km.kmeans_block_product(None, s, q, s)
