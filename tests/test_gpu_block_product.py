"""kmeans_block_product and kmeans_block_product_grad against float64.

Bounds (u32 = 2^-24, u the output type's half step).  Codes here are whole numbers
up to 15, so that a block's 128 products and their sums are whole numbers below
2^24 and the matrix instruction is exact; the scales' product, the block's and each
sum over the blocks are off by u32: u |out| + (blocks + 16) u32 sum |X W|.

The instruction sums eight products at a time on a grid of 2^-13 of the largest
one's power of two (as it was seen to): codes of all sizes lose less than 7 * 2^-13
of the largest of eight products besides (test_codes_of_all_sizes).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -140, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -130}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def km():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import exact_lloyd_means_03_amd as km
    km.load()
    return km


def _bytes(v, off=0):
    """The codes nearest to v, `off` bytes after an aligned address."""
    n = v.numel()
    flat = torch.empty(n + off, dtype=torch.uint8, device="cuda")
    flat[off:] = v.clamp(-448, 448).to(E4M3).view(torch.uint8).reshape(-1).cuda()
    return flat[off:].view(E4M3).view(v.shape)


def _codes(shape, seed, off=0):
    """Random whole numbers from -15 to 15 as codes."""
    return _bytes(torch.randint(-15, 16, shape, generator=torch.Generator().manual_seed(seed)).float(), off)


def _all_sizes(shape, seed):
    """Random codes from the smallest to the largest, zeros among them."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-10, 9, shape, generator=g).float())
    v[torch.rand(shape, generator=g) < 0.05] = 0.0
    return _bytes(v)


def _scales(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return (0.01 * (0.5 + torch.rand(shape, generator=g))).cuda()


def _offsets(S, E, kind, seed=3):
    """Segments of S rows among E experts; "tail" leaves rows behind the last one."""
    g = torch.Generator().manual_seed(seed)
    if E == 1 and kind == "even":
        return None
    cuts = torch.sort(torch.randint(0, S + 1, (E - 1,), generator=g))[0]
    if kind == "first":
        cuts[:] = S
    if kind == "last":
        cuts[:] = 0
    end = S - S // 4 if kind == "tail" else S
    return torch.cat([torch.tensor([0]), cuts.clamp(max=end), torch.tensor([end])]).to(torch.int32).cuda()


def _wide(codes, scales, rows):
    return codes.double() * scales.double().repeat_interleave(rows, -2)[..., :codes.shape[-2], :] \
        .repeat_interleave(128, -1)[..., :codes.shape[-1]]


def _reference(x, w, offsets, grad):
    """(out, sum of absolute terms) in float64."""
    S, E = x.shape[0], w.shape[0]
    out = x.new_zeros((S, w.shape[2] if grad else w.shape[1]))
    size = torch.zeros_like(out)
    ends = [0, S] if offsets is None else offsets.tolist()
    for e in range(E):
        a, z = ends[e], ends[e + 1]
        if a < z:
            m = w[e] if grad else w[e].t().contiguous()
            out[a:z], size[a:z] = x[a:z] @ m, x[a:z].abs() @ m.abs()
    return out, size


def _check(got, want, size, blocks, dtype, what="", more=0.0):
    bound = U[dtype] * want.abs() + (blocks + 16) * U32 * size + more + TINY[dtype]
    off = (got.double() - want).abs()
    assert got.dtype == dtype and got.shape == want.shape and torch.isfinite(got.float()).all(), what
    assert (off <= bound).all(), f"{what}: {(off - bound).max().item()} over the bound, {(off > bound).sum().item()} of {off.numel()}"


SHAPES = [  # S, E, M, K, kind of offsets
    (1, 1, 16, 128, "even"), (1, 1, 1, 1, "even"), (3, 1, 7, 5, "even"), (1, 1, 500, 4096, "even"), (17, 1, 130, 129, "even"),
    (16, 1, 128, 256, "even"), (64, 1, 1024, 1040, "even"), (100, 1, 333, 1000, "even"), (130, 1, 256, 512, "even"),
    (300, 1, 512, 384, "even"), (257, 1, 300, 257, "even"), (700, 1, 640, 272, "even"), (1100, 1, 1280, 144, "even"),
    (5, 4, 100, 200, "even"), (64, 16, 200, 640, "even"), (90, 3, 257, 143, "tail"), (500, 8, 384, 256, "tail"),
    (1000, 5, 260, 400, "first"), (1300, 3, 520, 160, "last"), (2000, 7, 264, 144, "tail"), (40, 40, 48, 80, "even"),
    (200, 100, 33, 65, "tail"), (3000, 2, 128, 128, "even"), (0, 2, 64, 64, "even"), (600, 4, 1024, 1024, "even"),
    (4500, 3, 1536, 256, "even"), (2100, 2, 2304, 640, "tail"),
    # every kernel of few rows, every token tile with and without splits, aligned and not
    (1, 1, 4096, 1024, "even"), (2, 1, 8192, 384, "even"), (64, 1, 2048, 1024, "even"), (100, 3, 4096, 512, "tail"),
    (200, 8, 8192, 256, "even"), (150, 1, 2048, 1024, "even"), (520, 2, 1024, 2048, "tail"), (1100, 1, 4096, 640, "even"),
    (2100, 1, 2048, 2048, "even"), (300, 1, 260, 4096, "even"), (130, 1, 4097, 257, "even"), (600, 1, 513, 2049, "even"),
    (40, 1, 700, 2050, "even"), (3000, 1, 1030, 1031, "even"), (9, 2, 15, 9, "even"), (70000, 2, 3, 5, "tail"),
    (1530, 1, 4096, 400, "even"), (1530, 1, 4095, 401, "even"), (1530, 1, 400, 4096, "even"),
    (1, 1, 40, 40000, "even"), (1, 1, 40000, 40, "even"), (33000, 1, 16, 32, "even"),
]


def _outputs(shape, dtype, off):
    whole = torch.full((math.prod(shape) + off + 64,), 7.0, dtype=dtype, device="cuda")
    n = math.prod(shape)
    return whole[off:off + n].view(shape), lambda: torch.cat([whole[:off], whole[off + n:]])


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("S,E,M,K,kind", SHAPES)
def test_product(km, dtype, S, E, M, K, kind):
    x, xs = _codes((S, K), 1), _scales((S, -(-K // 128)), 2)
    w, ws = _codes((E, M, K), 3), _scales((E, -(-M // 128), -(-K // 128)), 4)
    offsets = _offsets(S, E, kind)
    want, size = _reference(_wide(x, xs, 1), _wide(w, ws, 128), offsets, False)
    out, rest = _outputs((S, M), dtype, M % 2)
    got = km.kmeans_block_product(x, xs, w, ws, offsets, dtype=dtype, out=out)
    _check(got, want, size, -(-K // 128), dtype)
    assert (rest() == 7).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("S,E,M,K,kind", SHAPES)
def test_product_grad(km, dtype, S, E, M, K, kind):
    g, gs = _codes((S, M), 5), _scales((S, -(-M // 128)), 6)
    w, ws = _codes((E, M, K), 7), _scales((E, -(-M // 128), -(-K // 128)), 8)
    offsets = _offsets(S, E, kind, 4)
    want, size = _reference(_wide(g, gs, 1), _wide(w, ws, 128), offsets, True)
    out, rest = _outputs((S, K), dtype, K % 2)
    got = km.kmeans_block_product_grad(g, gs, w, ws, offsets, dtype=dtype, out=out)
    _check(got, want, size, -(-M // 128), dtype)
    assert (rest() == 7).all()


@pytest.mark.parametrize("S,M,K", [(1, 96, 512), (40, 80, 384), (300, 256, 256), (64, 128, 1000)])
def test_codes_of_all_sizes(km, S, M, K):
    x, xs = _all_sizes((S, K), 1), _scales((S, -(-K // 128)), 2)
    g, gs = _all_sizes((S, M), 5), _scales((S, -(-M // 128)), 6)
    w, ws = _all_sizes((1, M, K), 3), _scales((1, -(-M // 128), -(-K // 128)), 4)
    wide = _wide(w, ws, 128)
    for rows, blocks, grad in ((_wide(x, xs, 1), -(-K // 128), False), (_wide(g, gs, 1), -(-M // 128), True)):
        want, size = _reference(rows, wide, None, grad)
        m = wide[0] if grad else wide[0].t()
        pad = -rows.shape[1] % 8
        a = torch.nn.functional.pad(rows.abs(), (0, pad)).view(S, -1, 8)
        b = torch.nn.functional.pad(m.abs(), (0, 0, 0, pad)).view(-1, 8, m.shape[1])
        most = torch.zeros_like(want)
        for i in range(a.shape[1]):
            most += (a[:, i, :, None] * b[None, i]).amax(1)
        got = km.kmeans_block_product_grad(g, gs, w, ws, dtype=torch.float32) if grad else \
            km.kmeans_block_product(x, xs, w, ws, dtype=torch.float32)
        _check(got, want, size, blocks, torch.float32, f"grad={grad}", 7 * 2.0 ** -13 * most)


@pytest.mark.parametrize("S,M,K", [(1, 64, 256), (20, 80, 128), (200, 272, 384), (1000, 512, 256)])
def test_codes_that_start_anywhere(km, S, M, K):
    # rows and matrices one byte after an aligned address
    x, xs = _codes((S, K), 1, off=1), _scales((S, -(-K // 128)), 2)
    w, ws = _codes((2, M, K), 3, off=3), _scales((2, -(-M // 128), -(-K // 128)), 4)
    offsets = _offsets(S, 2, "even")
    want, size = _reference(_wide(x, xs, 1), _wide(w, ws, 128), offsets, False)
    _check(km.kmeans_block_product(x, xs, w, ws, offsets), want, size, -(-K // 128), torch.bfloat16)
    g, gs = _codes((S, M), 5, off=5), _scales((S, -(-M // 128)), 6)
    want, size = _reference(_wide(g, gs, 1), _wide(w, ws, 128), offsets, True)
    _check(km.kmeans_block_product_grad(g, gs, w, ws, offsets), want, size, -(-M // 128), torch.bfloat16)


@pytest.mark.parametrize("T,top,E,M,K", [(1, 1, 2, 48, 128), (5, 3, 4, 100, 200), (64, 2, 16, 256, 256), (700, 2, 4, 300, 384),
                                         (1500, 4, 8, 512, 272), (300, 1, 3, 130, 129)])
def test_rows_gathered_by_the_order(km, T, top, E, M, K):
    g = torch.Generator().manual_seed(11)
    experts = torch.randint(-1, E + 1, (T, top), generator=g).to(torch.int32).cuda()
    offsets, slots, order = km.kmeans_plan(experts, E)
    x, xs = _codes((T, K), 12), _scales((T, -(-K // 128)), 13)
    w, ws = _codes((E, M, K), 14), _scales((E, -(-M // 128), -(-K // 128)), 15)
    got = km.kmeans_block_product(x, xs, w, ws, offsets, order=order)
    rows = torch.where((order >= 0)[:, None], _wide(x, xs, 1)[(order // top).clamp(min=0).long()], 0.0)
    want, size = _reference(rows, _wide(w, ws, 128), offsets, False)
    _check(got, want, size, -(-K // 128), torch.bfloat16)
    assert (got[int(offsets[-1]):] == 0).all()
    # an order whose entries are no rows, and an offset past them, read nothing
    odd = order.clone()
    odd[::3] = -5
    odd[1::3] = T * top + 9
    got = km.kmeans_block_product(x, xs, w, ws, offsets, order=odd)
    rows[::3] = 0.0
    rows[1::3] = 0.0
    want, size = _reference(rows, _wide(w, ws, 128), offsets, False)
    _check(got, want, size, -(-K // 128), torch.bfloat16)


def test_offsets_that_are_none(km):
    # whatever they hold, rows stay inside and rows of no expert are zeros
    S, E, M, K = 300, 3, 144, 256
    x, xs = _codes((S, K), 1), _scales((S, 2), 2)
    w, ws = _codes((E, M, K), 3), _scales((E, 2, 2), 4)
    wide, wx = _wide(w, ws, 128), _wide(x, xs, 1)
    for bad, ends in (([0, 200, 100, 250], [0, 200, 200, 250]), ([0, -7, 900, 1200], [0, 0, 300, 300]),
                      ([0, 0, 0, 0], [0, 0, 0, 0])):
        out = km.kmeans_block_product(x, xs, w, ws, torch.tensor(bad, dtype=torch.int32, device="cuda"))
        want, size = _reference(wx, wide, torch.tensor(ends), False)
        _check(out, want, size, 2, torch.bfloat16, str(bad))


def test_from_wider_rows(km):
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        x = torch.randn((70, 300), generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
        w, ws = _codes((130, 300), 3), _scales((2, 3), 4)
        got = km.kmeans_block_product(x, None, w, ws)
        assert got.dtype == dtype
        assert torch.equal(got, km.kmeans_block_product(*km.kmeans_quantize(x), w, ws, dtype=dtype))
        g = torch.randn((70, 130), generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
        got = km.kmeans_block_product_grad(g, None, w, ws)
        assert torch.equal(got, km.kmeans_block_product_grad(*km.kmeans_quantize(g), w, ws, dtype=dtype))


@pytest.mark.parametrize("gather", [False, True])
def test_autograd(km, gather):
    T, top, E, M, K = 90, 2, 4, 200, 260
    g = torch.Generator().manual_seed(21)
    experts = torch.randint(-1, E, (T, top), generator=g).to(torch.int32).cuda()
    offsets, slots, order = km.kmeans_plan(experts, E)
    w, ws = _codes((E, M, K), 22), _scales((E, 2, 3), 23)
    x = torch.randn((T if gather else T * top, K), generator=g).cuda().requires_grad_()
    gy = torch.randn((T * top, M), generator=g).cuda()
    y = km.kmeans_block_product(x, None, w, ws, offsets, order=order if gather else None)
    y.backward(gy)
    rows = km.kmeans_block_product_grad(gy, None, w, ws, offsets)
    want = km.kmeans_combine(rows, slots) if gather else rows
    assert torch.equal(x.grad, want)
    # the rows' gradient is that of the gradient's codes
    gq = _wide(*km.kmeans_quantize(gy), 1)
    exact, size = _reference(gq, _wide(w, ws, 128), offsets, True)
    _check(rows, exact, size, 2, torch.float32, more=7 * 2.0 ** -13 * size)
    with pytest.raises(ValueError, match="no gradient"):
        km.kmeans_block_product(x, None, w, ws.clone().requires_grad_(), offsets)
    with pytest.raises(ValueError, match="given tensors"):
        km.kmeans_block_product(x, None, w, ws, offsets, order=order if gather else None, out=torch.empty_like(gy))


def test_grad_by_differences(km):
    # the product is linear in its rows' values: f(x + v) - f(x - v) = 2 <grad, v> for codes
    # x, v whose sums are codes again (whole numbers up to 8), up to float32 sums
    S, M, K = 60, 144, 256
    g = torch.Generator().manual_seed(31)
    x, v = (torch.randint(-4, 5, (S, K), generator=g).float().cuda() for _ in range(2))
    gy = torch.randint(-4, 5, (S, M), generator=g).float().cuda()
    w, ws, one = _codes((M, K), 32), _scales((2, 2), 33), torch.ones((S, 2), device="cuda")
    grad = km.kmeans_block_product_grad(gy.to(E4M3), one, w, ws, dtype=torch.float32)

    def f(r):
        y = km.kmeans_block_product(r.to(E4M3), one, w, ws, dtype=torch.float32)
        return (y.double() * gy.double()).sum()
    got, want = f(x + v) - f(x - v), 2 * (grad.double() * v.double()).sum()
    size = (gy.abs().double() @ _wide(w, ws, 128).abs() * 8).sum()
    assert abs((got - want).item()) <= 64 * U32 * size.item()


def test_special_codes(km):
    # a NaN code (0x7f) reaches the results of its row or column alone
    S, M, K = 40, 64, 256
    x, xs, w, ws = _codes((S, K), 1), _scales((S, 2), 2), _codes((M, K), 3), _scales((1, 2), 4)
    x.view(torch.uint8)[3, 200] = 0x7f
    w.view(torch.uint8)[17, 5] = 0x7f
    y = km.kmeans_block_product(x, xs, w, ws)
    bad = torch.zeros((S, M), dtype=torch.bool, device="cuda")
    bad[3], bad[:, 17] = True, True
    assert torch.equal(y.isnan(), bad)


@pytest.mark.parametrize("S,M,K", [(20, 40, 9), (20, 40, 200), (20, 48, 256), (600, 256, 256), (600, 256, 200)])
def test_rows_of_none_among_others(km, S, M, K):
    # an order of -1 is a row of zeros, also where the matrix holds a NaN code and an infinite
    # scale; K below 16, unaligned, aligned rows, few and many
    x, xs, w, ws = _codes((S, K), 1), _scales((S, -(-K // 128)), 2), _codes((M, K), 3), _scales((-(-M // 128), -(-K // 128)), 4)
    order = torch.arange(S - 1, -1, -1, dtype=torch.int32, device="cuda")
    order[::3] = -1
    want = km.kmeans_block_product(x[order.clamp(min=0).long()].contiguous(), xs[order.clamp(min=0).long()].contiguous(), w, ws)
    want[::3] = 0
    assert torch.equal(km.kmeans_block_product(x, xs, w, ws, order=order), want)
    w.view(torch.uint8)[5, K - 1] = 0x7f
    ws[-1, 0] = float("inf")
    y = km.kmeans_block_product(x, xs, w, ws, order=order)
    assert (y[::3] == 0).all() and y[1::3, 5].isnan().all()


@pytest.mark.parametrize("T,top", [(0, 2), (4, 0)])
def test_autograd_without_choices(km, T, top):
    x = torch.zeros((T, 256), device="cuda").requires_grad_()
    order = torch.empty(T * top, dtype=torch.int32, device="cuda")
    y = km.kmeans_block_product(x, None, _codes((128, 256), 1), _scales((1, 2), 2), order=order)
    assert y.shape == (0, 128)
    y.sum().backward()
    assert x.grad.shape == x.shape and (x.grad == 0).all()


def test_refusals(km):
    x, xs = _codes((4, 256), 1), _scales((4, 2), 2)
    w, ws = _codes((2, 128, 256), 3), _scales((2, 1, 2), 4)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="offsets"):
        km.kmeans_block_product(x, xs, w, ws)
    with pytest.raises(ValueError, match="scales"):
        km.kmeans_block_product(x, None, w, ws, off)
    with pytest.raises(ValueError, match="scales"):
        km.kmeans_block_product(x, xs, w, ws[:, :, :1].contiguous(), off)
    with pytest.raises(ValueError, match="scales"):
        km.kmeans_block_product(x.float(), xs, w, ws, off)
    with pytest.raises(ValueError, match="columns"):
        km.kmeans_block_product(_codes((4, 128), 1), xs, w, ws, off)
    with pytest.raises(ValueError, match="columns"):
        km.kmeans_block_product_grad(x, xs, w, ws, off)
    with pytest.raises(ValueError, match="order"):
        km.kmeans_block_product(x, xs, w, ws, off, order=torch.zeros(6, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError, match="float32 / float16"):
        km.kmeans_block_product(x, xs, w, ws, off, dtype=torch.float64)
    with pytest.raises(TypeError, match="codes"):
        km.kmeans_block_product(x, xs, w.float(), ws, off)
