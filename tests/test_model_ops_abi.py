"""The entry points on labels and codebooks inside a model, on a machine
without a GPU: sizes of their workspaces, and invalid arguments refused on the
host before any HIP call."""
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


def test_lookup_rejects(lib):
    call = _call(lib.kmeans_lookup, dict(table=FAKE, xt=F16, B=1, V=10, d=8, labels=FAKE, N=5, scale=1.0, out=FAKE,
                                         stream=None))
    assert call(table=None) == 1 and b"table" in lib.kmeans_last_error()
    assert call(labels=None) == 1 and call(out=None) == 1
    assert call(V=0) == 1 and call(d=0) == 1 and call(N=-1) == 1 and call(B=-1) == 1
    assert call(xt=3) == 2 and b"dtype" in lib.kmeans_last_error()
    assert call(B=70000) == 2 and call(V=(1 << 30) + 1) == 2 and call(N=1 << 31) == 2
    assert call(B=65535, N=1 << 20) == 2  # 2^31 rows or more
    assert call(N=1 << 30, d=1 << 20) == 2


def test_lookup_grad_rejects(lib):
    q = lib.kmeans_lookup_grad_workspace_bytes
    # the sorted keys and indices, and two float32 slots for each piece of rows
    assert q(1, 100000, 64, 50000, F16) >= 2 * 100000 * 4 + 100000 // 256 * 2 * 64 * 4
    assert q(1, 100000, 64, 50000, F16) % 256 == 0
    assert q(1, 10, 0, 5, F16) == 0 and q(1, 10, 4, 0, F16) == 0 and q(1, -1, 4, 5, F16) == 0 and q(1, 10, 4, 5, 9) == 0
    call = _call(lib.kmeans_lookup_grad, dict(grad=FAKE, xt=F16, B=1, N=50, d=8, labels=FAKE, V=10, scale=1.0, out=FAKE,
                                              gt=F16, ws=WS, ws_bytes=1 << 30, stream=None))
    assert call(gt=BF16) == 2 and call(gt=7) == 2 and call(xt=-1) == 2
    assert call(xt=F32, gt=F16) == 2
    assert call(grad=None) == 1 and call(labels=None) == 1 and call(out=None) == 1
    assert call(ws=None) == 1 and call(ws=C.c_void_p(0x100010)) == 1 and call(ws_bytes=64) == 3
    assert call(V=-4) == 1 and call(d=0) == 1


def test_dispatch_rejects(lib):
    q = lib.kmeans_dispatch_workspace_bytes
    assert q(100, 2, 8) == 0             # sorted in the launch that copies
    assert q(100000, 2, 64) >= 2 * 64 * 4
    assert q(100000, 2, 5000) == 0 and q(-1, 2, 8) == 0
    call = _call(lib.kmeans_dispatch, dict(x=FAKE, xt=BF16, T=10000, d=8, experts=FAKE, top=2, E=8, rows=FAKE,
                                           offsets=FAKE, slots=FAKE, order=FAKE, ws=WS, ws_bytes=1 << 30, stream=None))
    for name in ("x", "experts", "rows", "offsets", "slots", "order"):
        assert call(**{name: None}) == 1 and name.encode() in lib.kmeans_last_error()
    assert call(E=0) == 1 and call(E=4097) == 2
    assert call(top=0) == 1 and call(T=-1) == 1 and call(T=1 << 30, top=2) == 2
    assert call(d=0) == 1 and call(xt=4) == 2
    assert call(ws=None) == 1 and call(ws_bytes=16) == 3


def test_combine_rejects(lib):
    call = _call(lib.kmeans_combine, dict(rows=FAKE, xt=F32, T=10, d=8, top=2, slots=FAKE, weights=FAKE, out=FAKE,
                                          stream=None))
    assert call(rows=None) == 1 and call(slots=None) == 1 and call(out=None) == 1
    assert call(top=0) == 1 and call(d=0) == 1 and call(T=-1) == 1 and call(xt=9) == 2
    grad = _call(lib.kmeans_combine_grad, dict(grad=FAKE, rows=FAKE, xt=F32, T=10, d=8, top=2, slots=FAKE, order=FAKE,
                                               weights=FAKE, grows=FAKE, gweights=FAKE, stream=None))
    for name in ("grad", "rows", "slots", "order", "weights", "grows", "gweights"):
        assert grad(**{name: None}) == 1
    assert grad(T=1 << 31) == 2 and grad(xt=-2) == 2


def test_codes_reject(lib):
    assert lib.kmeans_codes_bytes(1, 1) == 1024
    assert lib.kmeans_codes_bytes(17, 129) == 4 * 1024
    assert lib.kmeans_codes_bytes(0, 5) == 0 and lib.kmeans_codes_bytes(5, (1 << 20) + 1) == 0
    pack = _call(lib.kmeans_pack_codes, dict(labels=FAKE, M=16, K=16, codes=FAKE, stream=None))
    assert pack(labels=None) == 1 and pack(codes=None) == 1 and pack(codes=C.c_void_p(0x1008)) == 1
    assert pack(M=0) == 1 and pack(K=(1 << 20) + 1) == 2
    q = lib.kmeans_codes_workspace_bytes
    assert q(1, 1, 4096, 4096, BF16) % 256 == 0
    assert q(1, 1, 0, 4096, BF16) == 0 and q(1, 1, 16, 16, F32) == 0
    defaults = dict(x=FAKE, xt=F16, S=8, codes=FAKE, table=FAKE, table_rows=64, scales=FAKE, group=64, E=2, M=64, K=128,
                    offsets=FAKE, out=FAKE, ws=WS, ws_bytes=1 << 30, stream=None)
    for fn in (lib.kmeans_codes_product, lib.kmeans_codes_product_grad):
        call = _call(fn, defaults)
        for name in ("x", "codes", "table", "out", "offsets"):
            assert call(**{name: None}) == 1, name
        assert call(xt=F32) == 2 and call(xt=5) == 2
        assert call(table_rows=2) == 1 and b"table_rows" in lib.kmeans_last_error()
        assert call(group=48) == 2 and call(group=16) == 2 and call(group=160) == 2 and call(group=0) == 1
        assert call(codes=C.c_void_p(0x1004)) == 1
        assert call(S=-1) == 1 and call(M=0) == 1 and call(E=0) == 1 and call(E=5000) == 2
        assert call(S=1 << 21) == 2  # more token tiles than a launch has
    # the gradient of few rows adds partial sums in the workspace
    n = q(1, 1, 4096, 4096, F16)
    assert n >= 2 * 4096 * 4
    assert _call(lib.kmeans_codes_product_grad, defaults)(S=1, E=1, M=4096, K=4096, table_rows=1, offsets=None,
                                                          ws_bytes=256) == 3


def test_python_wrappers_want_gpu_tensors():
    import torch
    import exact_lloyd_means_03_amd as km
    i32 = torch.zeros((1, 3), dtype=torch.int32)
    for call in (lambda: km.kmeans_lookup(torch.zeros(1, 4, 8), i32),
                 lambda: km.kmeans_lookup_grad(torch.zeros(1, 3, 8), i32, 4),
                 lambda: km.kmeans_dispatch(torch.zeros(1, 8), i32, 4),
                 lambda: km.kmeans_combine(torch.zeros(3, 8), i32),
                 lambda: km.kmeans_pack_codes(i32)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError, match="Tensor"):
        km.kmeans_lookup(None, i32)


def test_rows_of_a_4_bit_product(lib):
    # 2^20 rows (131072 tokens of 8 choices) pass the check of sizes, with any number of
    # experts: the next check refuses; one more row does not
    misaligned = C.c_void_p(0x1004)
    for fn in (lib.kmeans_codes_product, lib.kmeans_codes_product_grad):
        for E in (1, 4096):
            call = _call(fn, dict(x=FAKE, xt=F16, S=1 << 20, codes=misaligned, table=FAKE, table_rows=64, scales=None,
                                  group=0, E=E, M=64, K=128, offsets=FAKE, out=FAKE, ws=WS, ws_bytes=1 << 30,
                                  stream=None))
            assert call() == 1 and b"codes" in lib.kmeans_last_error()
            assert call(S=(1 << 20) + 1) == 2 and b"2^20" in lib.kmeans_last_error()


def test_many_choices_are_sorted_in_passes_of_their_own(lib):
    # (no workspace: one launch, whose blocks read every label once for eight choices)
    q = lib.kmeans_dispatch_workspace_bytes
    assert q(512, 8, 64) == 0 and q(64, 16, 64) == 0 and q(8, 24, 64) == 0 and q(0, 4096, 8) == 0
    assert q(256, 16, 64) > 0 and q(64, 17, 64) > 0 and q(1, 64, 64) > 0 and q(1, 4096, 256) > 0
