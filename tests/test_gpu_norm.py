"""kmeans_norm, kmeans_norm_quantize, kmeans_norm_grad and kmeans_quantize
against their formulas in float64.

Bounds (u32 = 2^-24, u the output type's half step).  A row's sum of squares has
at most 64 terms a lane and 6 + 16 additions over lanes and waves, all positive:
off by 96 u32 of itself with the terms' own roundings, its root by 48.  With the
sum h (1), the mean, eps, root and inverse (4), and two products: y is off by 64
u32 of itself before it is rounded.  grad_x has r^3 and two sums of signed terms,
the terms over absolute values: 256 u32 of (|r u| + |h| r^3 mean |u h|), rounded
once.  grad_weight adds T terms in some order: (T + 96) u32 of sum |g h r|.
A code is within half a step of e4m3: 2^-4 of itself, or 2^-10 below 2^-6.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -140, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -130}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
E4M3 = torch.float8_e4m3fn

# every number of waves and chunks of a row, with odd ends
SHAPES = [(1, 1), (3, 7), (2, 8), (5, 127), (4, 128), (33, 129), (64, 1000), (7, 2048), (2, 4099), (3, 8192), (2, 16384),
          (2050, 64), (2049, 515), (2100, 1031), (2055, 2050), (2048, 4096), (0, 16)]


@pytest.fixture(scope="module")
def km():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import exact_lloyd_means_03_amd as km
    km.load()
    return km


def _rows(shape, dtype, seed, std=1.0, off=0):
    """Random rows, `off` elements after an aligned address."""
    g = torch.Generator().manual_seed(seed)
    n = math.prod(shape)
    flat = torch.empty(n + off, dtype=dtype, device="cuda")
    flat[off:] = (torch.randn(n, generator=g) * std).to(dtype)
    return flat[off:].view(shape)


def _guarded(shape, dtype, off=0):
    """An output inside a larger buffer, and the buffer's bytes outside it."""
    n = math.prod(shape)
    whole = torch.full((n + off + 64,), 7.0, device="cuda").to(dtype)
    return whole[off:off + n].view(shape), lambda: torch.cat([whole[:off], whole[off + n:]]).float()


def _reference(x, residual, weight, eps):
    h = x.double() if residual is None else x.double() + residual.double()
    r = 1.0 / (h.square().mean(1, keepdim=True) + eps).sqrt()
    y = h * r
    return h, r, y if weight is None else y * weight.double()


def _near(got, want, bound, what):
    off = (got.double() - want).abs()
    assert got.shape == want.shape and torch.isfinite(got.float()).all(), what
    assert (off <= bound).all(), f"{what}: {(off - bound).max().item()} over the bound"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d", SHAPES)
def test_norm(km, dtype, T, d):
    off = 1 if d % 2 else 0
    for add, wt in ((True, dtype), (False, torch.float32), (True, None)):
        x, eps = _rows((T, d), dtype, 1, 2.0, off), 1e-5
        residual = _rows((T, d), dtype, 2, 1.0, off) if add else None
        weight = None if wt is None else (1.0 + 0.2 * _rows((d,), torch.float32, 3)).to(wt)
        y, y_rest = _guarded((T, d), dtype, off)
        h, h_rest = _guarded((T, d), dtype, off)
        got, got_h = km.kmeans_norm(x, weight, eps, residual=residual, y=y, h=h if add else None)
        want_h, _, want = _reference(x, residual, weight, eps)
        _near(got, want, (U[dtype] + 64 * U32) * want.abs() + TINY[dtype], "y")
        if add:
            _near(got_h, want_h, (U[dtype] + 2 * U32) * want_h.abs() + TINY[dtype], "h")
        else:
            assert got_h is x
        assert (y_rest() == 7).all() and (h_rest() == 7).all()


def _check_codes(codes, scales, want, rel, what):
    """Codes and scales of rows whose exact values `want` are known to `rel` of themselves."""
    T, d = want.shape
    assert codes.dtype == E4M3 and codes.shape == want.shape and scales.shape == (T, -(-d // 128))
    pad = torch.nn.functional.pad(want, (0, -d % 128)).view(T, -(-d // 128), 128)
    s = (pad.abs().amax(-1) / 448).clamp(min=2.0 ** -100)
    assert ((scales.double() - s).abs() <= (rel + 2 * U32) * s).all(), what
    q = want / scales.double().repeat_interleave(128, 1)[:, :d]
    half = torch.maximum(q.abs() * 2.0 ** -4, torch.full_like(q, 2.0 ** -10))
    off = (codes.float().double() - q).abs()
    assert (off <= half * (1 + 1e-6) + (rel + 4 * U32) * q.abs()).all(), f"{what}: {(off - half).max().item()}"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d", SHAPES)
def test_norm_quantize(km, dtype, T, d):
    off = 3 if d % 2 else 0
    for add in (True, False):
        x, residual = _rows((T, d), dtype, 4, 2.0, off), _rows((T, d), dtype, 5, 1.0, off) if add else None
        weight = (1.0 + 0.2 * _rows((d,), torch.float32, 6)).to(dtype)
        codes, codes_rest = _guarded((T, d), E4M3, off)
        scales, scales_rest = _guarded((T, -(-d // 128)), torch.float32, off)
        q, s, h = km.kmeans_norm_quantize(x, weight, 1e-6, residual=residual, codes=codes, scales=scales)
        want_h, _, want = _reference(x, residual, weight, 1e-6)
        _check_codes(q, s, want, 64 * U32, f"add={add}")
        if add:
            _near(h, want_h, (U[dtype] + 2 * U32) * want_h.abs() + TINY[dtype], "h")
        assert (codes_rest() == 7).all() and (scales_rest() == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,B", [(1, 1, 1), (3, 7, 1), (5, 128, 2), (130, 129, 1), (127, 1000, 3), (256, 384, 1),
                                   (1, 5000, 1), (300, 4, 1), (0, 8, 1)])
def test_quantize(km, dtype, M, K, B):
    off = 1 if K % 2 else 0
    x = _rows((B, M, K), dtype, 7, 3.0, off)
    if M > 2:
        x[0, 1] = 0.0
    for rows in (1, 128):
        codes, codes_rest = _guarded((B, M, K), E4M3, off)
        scales, scales_rest = _guarded((B, -(-M // rows), -(-K // 128)), torch.float32, off)
        km.kmeans_quantize(x, rows, codes=codes, scales=scales)
        assert (codes_rest() == 7).all() and (scales_rest() == 7).all()
        for b in range(B):
            if rows == 1:
                _check_codes(codes[b], scales[b], x[b].double(), 0.0, "rows")
                continue
            pad = torch.nn.functional.pad(x[b].double(), (0, -K % 128, 0, -M % 128))
            blocks = pad.view(pad.shape[0] // 128, 128, -(-K // 128), 128).abs().amax((1, 3)) / 448
            s = blocks.clamp(min=2.0 ** -100)
            assert ((scales[b].double() - s).abs() <= 2 * U32 * s).all()
            q = x[b].double() / scales[b].double().repeat_interleave(128, 0)[:M].repeat_interleave(128, 1)[:, :K]
            half = torch.maximum(q.abs() * 2.0 ** -4, torch.full_like(q, 2.0 ** -10))
            assert ((codes[b].float().double() - q).abs() <= half * (1 + 1e-6) + 4 * U32 * q.abs()).all()


def test_quantize_one_problem_of_two_dimensions(km):
    x = _rows((200, 300), torch.bfloat16, 8)
    a, b = km.kmeans_quantize(x, 128), km.kmeans_quantize(x[None], 128)
    assert a[0].shape == (200, 300) and a[1].shape == (2, 3)
    assert torch.equal(a[0].view(torch.uint8), b[0][0].view(torch.uint8)) and torch.equal(a[1], b[1][0])


@pytest.mark.parametrize("dtype", DTYPES)
def test_extreme_values(km, dtype):
    big = torch.finfo(dtype).max
    x = torch.zeros((8, 300), dtype=dtype, device="cuda")
    x[1, :] = big
    x[2, 5] = float("inf")
    x[3, 150] = float("nan")
    x[4, :] = torch.finfo(dtype).tiny
    x[5, 299] = -big
    codes, scales = km.kmeans_quantize(x)
    v = codes.float() * scales.repeat_interleave(128, 1)[:, :300]
    assert (v[0] == 0).all() and (scales[0] == 2.0 ** -100).all()
    assert ((v[1].double() - big).abs() <= 2 * U32 * big).all()
    assert v[2, :128].isnan().all() and (v[2, 128:] == 0).all()
    assert v[3, 128:256].isnan().all() and (v[3, :128] == 0).all() and (v[3, 256:] == 0).all()
    tiny = torch.finfo(dtype).tiny
    if tiny / 448 > 2.0 ** -100:
        assert ((v[4].double() - tiny).abs() <= 2 * U32 * tiny).all()
    else:  # below the smallest scale: zeros
        assert (v[4] == 0).all()
    assert abs(v[5, 299].item() + big) <= 2 * U32 * big and (v[5, :299] == 0).all()
    # a norm: an infinite row is NaN or 0 by the formula, its neighbours are not touched
    y, _ = km.kmeans_norm(x[2:6].clone(), None, 1e-6)
    assert y[0, 5].isnan() and (y[0, :5] == 0).all() and y[1].isnan().all()
    zero, _ = km.kmeans_norm(x[:1].clone(), None, 0.0)
    assert zero.isnan().all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d", SHAPES)
def test_norm_grad(km, dtype, T, d):
    off = 1 if d % 2 else 0
    for more, wt in ((True, dtype), (False, torch.float32), (True, None)):
        g, h = _rows((T, d), dtype, 11, 0.3, off), _rows((T, d), dtype, 12, 2.0, off)
        gr = _rows((T, d), dtype, 13, 1.0, off) if more else None
        weight = None if wt is None else (1.0 + 0.2 * _rows((d,), torch.float32, 14)).to(wt)
        gx, rest = _guarded((T, d), dtype, off)
        got, gw = km.kmeans_norm_grad(g, h, weight, 1e-5, grad_residual=gr, grad_x=gx)
        hd, gd = h.double(), g.double()
        r = 1.0 / (hd.square().mean(1, keepdim=True) + 1e-5).sqrt()
        u = gd if weight is None else gd * weight.double()
        want = r * u - hd * r ** 3 * (u * hd).mean(1, keepdim=True)
        size = (r * u).abs() + hd.abs() * r ** 3 * (u * hd).abs().mean(1, keepdim=True)
        if more:
            want, size = want + gr.double(), size + gr.double().abs()
        _near(got, want, U[dtype] * want.abs() + 256 * U32 * size + TINY[dtype], "grad_x")
        assert (rest() == 7).all()
        if weight is None:
            assert gw is None
            continue
        assert gw.dtype == weight.dtype
        wgw, size = (gd * hd * r).sum(0), (gd * hd * r).abs().sum(0)
        _near(gw, wgw, U[weight.dtype] * wgw.abs() + (T + 96) * U32 * size + TINY[weight.dtype], "grad_weight")


@pytest.mark.parametrize("dtype,T,d", [(torch.bfloat16, 3, 32768), (torch.float16, 2, 20001), (torch.float32, 2, 12345),
                                       (torch.bfloat16, 1500, 16384), (torch.bfloat16, 1100, 8200)])
def test_long_rows(km, dtype, T, d):
    # (a lane's sums are longer: 64 terms more, and as many more rows a block)
    g, h, w = _rows((T, d), dtype, 1, 0.3), _rows((T, d), dtype, 2), (1.0 + 0.2 * _rows((d,), torch.float32, 3)).to(dtype)
    gx, gw = km.kmeans_norm_grad(g, h, w, 1e-5)
    hd, gd = h.double(), g.double()
    r = 1.0 / (hd.square().mean(1, keepdim=True) + 1e-5).sqrt()
    u = gd * w.double()
    want = r * u - hd * r ** 3 * (u * hd).mean(1, keepdim=True)
    size = (r * u).abs() + hd.abs() * r ** 3 * (u * hd).abs().mean(1, keepdim=True)
    _near(gx, want, U[dtype] * want.abs() + 384 * U32 * size + TINY[dtype], "grad_x")
    wgw, size = (gd * hd * r).sum(0), (gd * hd * r).abs().sum(0)
    _near(gw, wgw, U[dtype] * wgw.abs() + (T + 160) * U32 * size + TINY[dtype], "grad_weight")
    y, _ = km.kmeans_norm(h, w, 1e-5)
    _near(y, hd * r * w.double(), (U[dtype] + 96 * U32) * (hd * r * w.double()).abs() + TINY[dtype], "y")
    q, s, _ = km.kmeans_norm_quantize(h, w, 1e-5)
    _check_codes(q, s, hd * r * w.double(), 96 * U32, "codes")


@pytest.mark.parametrize("size", [2.0 ** -50, 2.0 ** 50])
def test_grad_of_large_and_small_rows(km, size):
    # grad_x falls as the rows grow: h = size * v has 1 / size times v's (powers of two: the
    # same bits), also where r^3 is out of float32's range
    g, v = _rows((5, 300), torch.float32, 41, 0.3), _rows((5, 300), torch.float32, 42)
    weight = 1.0 + 0.2 * _rows((300,), torch.float32, 43)
    one, gw1 = km.kmeans_norm_grad(g, v, weight, 0.0)
    gx, gw = km.kmeans_norm_grad(g, v * size, weight, 0.0)
    assert torch.equal(gx * size, one) and torch.equal(gw, gw1)


def test_grad_by_differences(km):
    # along a direction v: (f(h + e v) - f(h - e v)) / 2 e of f = <g, y>, in float32 sums of
    # 40 x 160 terms of size 1 (off by 6400 u32 / 2 e = 0.02 at e = 1/100) and a third-order
    # term of e^2 |v|^3 in a function whose derivatives are of size 1 / |h| (0.01)
    g, h, v = (_rows((40, 160), torch.float32, s) for s in (21, 22, 23))
    weight = 1.0 + 0.2 * _rows((160,), torch.float32, 24)
    dw = _rows((160,), torch.float32, 25)
    gx, gw = km.kmeans_norm_grad(g, h, weight, 1e-6)

    def f(e, along_weight):
        y, _ = km.kmeans_norm(h if along_weight else h + e * v, weight + e * dw if along_weight else weight, 1e-6)
        return (g.double() * y.double()).sum().item()
    for along, want in ((False, (gx.double() * v.double()).sum().item()), (True, (gw.double() * dw.double()).sum().item())):
        got = (f(0.01, along) - f(-0.01, along)) / 0.02
        assert abs(got - want) <= 0.05 + 1e-3 * abs(want), (along, got, want)


@pytest.mark.parametrize("add", [False, True])
def test_autograd(km, add):
    x, residual = _rows((37, 200), torch.float32, 31), _rows((37, 200), torch.float32, 32)
    weight = 1.0 + 0.2 * _rows((200,), torch.float32, 33)
    gy, gh = _rows((37, 200), torch.float32, 34), _rows((37, 200), torch.float32, 35)
    leaves = [t.clone().requires_grad_() for t in ((x, residual, weight) if add else (x, weight))]
    y, h = km.kmeans_norm(leaves[0], leaves[-1], 1e-6, residual=leaves[1] if add else None)
    ((y * gy).sum() + (h * gh).sum()).backward()
    d = [t.double().requires_grad_() for t in ((x, residual, weight) if add else (x, weight))]
    hd = d[0] + d[1] if add else d[0]
    yd = hd / (hd.square().mean(1, keepdim=True) + 1e-6).sqrt() * d[-1]
    ((yd * gy.double()).sum() + (hd * gh.double()).sum()).backward()
    for a, b in zip(leaves, d):
        assert (a.grad.double() - b.grad).norm() <= 1e-5 * b.grad.norm()
    # the residual's stream alone, and no recording
    if add:
        a, b = x.clone().requires_grad_(), residual.clone().requires_grad_()
        km.kmeans_norm(a, weight, 1e-6, residual=b)[1].sum().backward()
        assert (a.grad == 1).all() and (b.grad == 1).all()
    with torch.no_grad():
        assert not km.kmeans_norm(leaves[0], leaves[-1])[0].requires_grad
    with pytest.raises(ValueError, match="no gradient"):
        km.kmeans_norm_quantize(leaves[0], weight)
    with pytest.raises(ValueError, match="given tensors"):
        km.kmeans_norm(leaves[0], weight, y=torch.empty_like(x))


def test_equal_inputs_equal_bits(km):
    g, h, w = _rows((3000, 1000), torch.bfloat16, 41), _rows((3000, 1000), torch.bfloat16, 42), _rows((1000,), torch.bfloat16, 43)
    first = km.kmeans_norm_grad(g, h, w)
    for _ in range(3):
        again = km.kmeans_norm_grad(g, h, w)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_refusals(km):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        km.kmeans_norm(x, torch.ones(63, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError, match="weight"):
        km.kmeans_norm(x, torch.ones(64, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError, match="residual"):
        km.kmeans_norm(x, None, residual=torch.zeros((5, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        km.kmeans_norm(x[:, ::2])
    with pytest.raises(km.KMeansError, match="eps"):
        km.kmeans_norm(x, None, -1.0)
    with pytest.raises(km.KMeansError, match="64 KB"):
        km.kmeans_norm(torch.zeros((1, 40000), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="rows"):
        km.kmeans_quantize(x, 64)
    with pytest.raises(km.KMeansError, match="workspace"):
        km.kmeans_norm_grad(x, x, torch.ones(64, dtype=torch.bfloat16, device="cuda"),
                            ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
