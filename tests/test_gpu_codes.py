"""kmeans_pack_codes, kmeans_codes_product and kmeans_codes_product_grad
against plain float64 products.

Bounds: a sum of n products of 16-bit values in float32, the scales applied to
float32 partial sums: |err| <= 2 (n + 16) u32 sum|x W| + u |ref| (the factor 2
and 16 for the roundings inside the matrix instructions, the scales' products
and the join of partial sums).  The gradient rounds the scaled weight to the
16-bit type before the product, so each weight is off by u relative there:
u sum|x W| more.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -130}
DTYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def km():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import exact_lloyd_means_03_amd as km
    km.load()
    return km


def _case(S, E, M, K, group, dtype, rows, seed, used=None):
    g = torch.Generator().manual_seed(seed)
    lab = torch.randint(0, 16, (E, M, K), generator=g).to(torch.int32)
    table = torch.randn((E, M if rows == "each" else 1, 16), generator=g).to(dtype)
    scales = (0.5 + torch.rand((E, M, -(-K // group)), generator=g)).to(dtype) if group else None
    used = S if used is None else used
    cut = torch.randint(0, used + 1, (E - 1,), generator=g).sort()[0]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), cut, torch.tensor([used])]).to(torch.int32)
    W = torch.gather(table.double().expand(E, M, 16), 2, lab.long())
    if group:
        W = W * scales.double().repeat_interleave(group, 2)[..., :K]
    return lab, table, scales, offsets, W


def _packed(km, lab):
    return torch.stack([km.kmeans_pack_codes(m.cuda()) for m in lab])


def _ref(x, W, offsets, grad):
    S = x.shape[0]
    out = torch.zeros((S, W.shape[2] if grad else W.shape[1]), dtype=torch.float64)
    mag = torch.zeros_like(out)
    for e in range(W.shape[0]):
        a, z = int(offsets[e]), int(offsets[e + 1])
        w = W[e] if grad else W[e].t()
        out[a:z] = x[a:z].double() @ w
        mag[a:z] = x[a:z].double().abs() @ w.abs()
    return out, mag


def _close(got, ref, mag, n, dtype, rounded, what):
    got = got.cpu().double()
    tol = 2 * (n + 16) * U32 * mag + U[dtype] * (ref.abs() + 2 * (n + 16) * U32 * mag) + TINY[dtype]
    if rounded:
        tol = tol + U[dtype] * mag * (1 + U[dtype])
    worst = ((got - ref).abs() / tol).max() if got.numel() else 0
    assert worst <= 1, f"{what}: {float(worst):.3g} of the bound"


def test_packed_layout(km):
    M, K = 37, 301
    lab = torch.randint(0, 16, (M, K), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    codes = km.kmeans_pack_codes(lab.cuda()).cpu().numpy()
    words = codes.view(np.uint32).reshape(codes.shape[0], codes.shape[1], 256)
    want = np.zeros((-(-M // 16) * 16, -(-K // 128) * 128), np.uint32)
    want[:M, :K] = lab.numpy()
    m, k = np.meshgrid(np.arange(want.shape[0]), np.arange(want.shape[1]), indexing="ij")
    r, c = m % 16, k % 128
    j, q, i = c // 32, c % 32 // 8, c % 8
    got = words[m // 16, k // 128, (16 * q + r) * 4 + j] >> (8 * (i % 4) + 4 * (i // 4)).astype(np.uint32) & 15
    np.testing.assert_array_equal(got, want)


SHAPES = [  # S, E, M, K, group, rows, used
    (1, 1, 16, 128, 0, "each", None), (1, 1, 1, 1, 0, "each", None), (3, 1, 17, 7, 32, "each", None),
    (1, 1, 300, 1000, 128, "each", None), (16, 1, 64, 130, 64, "shared", None), (17, 1, 100, 257, 32, "each", None),
    (5, 4, 40, 384, 128, "each", None), (33, 8, 48, 200, 64, "each", 20), (64, 3, 130, 512, 256, "shared", None),
    (65, 2, 96, 640, 32, "each", 65), (40, 70, 20, 96, 32, "each", 33), (200, 5, 144, 333, 128, "each", 190),
    (300, 1, 257, 129, 0, "shared", None), (9, 3, 16, 128, 64, "each", 0), (700, 2, 260, 300, 64, "each", 650),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("S,E,M,K,group,rows,used", SHAPES)
def test_products(km, dtype, S, E, M, K, group, rows, used):
    lab, table, scales, offsets, W = _case(S, E, M, K, group, dtype, rows, 2, used)
    g = torch.Generator().manual_seed(3)
    x, gy = torch.randn((S, K), generator=g).to(dtype), torch.randn((S, M), generator=g).to(dtype)
    args = (_packed(km, lab), table.cuda())
    sc = None if scales is None else scales.cuda()
    off = None if E == 1 and used is None else offsets.cuda()
    out = torch.full((S, M), 7.0, dtype=dtype, device="cuda")
    got = km.kmeans_codes_product(x.cuda(), *args, M, sc, group, off, out=out)
    ref, mag = _ref(x, W, offsets, False)
    _close(got, ref, mag, K, dtype, False, "product")
    out = torch.full((S, K), 7.0, dtype=dtype, device="cuda")
    got = km.kmeans_codes_product_grad(gy.cuda(), *args, K, sc, group, off, out=out)
    ref, mag = _ref(gy, W, offsets, True)
    _close(got, ref, mag, M, dtype, group > 0, "gradient")


# One shape for each block the launches choose from (rows x columns of the
# matrix, experts), with ragged rows, columns and tokens.
BLOCKS = [  # S, E, M, K
    (700, 1, 4128, 264), (700, 1, 4100, 640), (300, 1, 5000, 264), (150, 1, 5000, 648), (150, 1, 2600, 264),
    (12, 6, 4200, 264), (12, 1, 6200, 136), (700, 1, 4128, 263), (150, 1, 5000, 517), (9, 1, 300, 1033),
    (500, 1, 200, 8200), (300, 1, 130, 8200), (40, 1, 2000, 300), (1, 1, 3000, 130), (600, 3, 1100, 520),
]


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("S,E,M,K", BLOCKS)
def test_products_of_every_block(km, S, E, M, K, group):
    dtype = torch.float16 if (M + group) % 64 else torch.bfloat16
    lab, table, scales, offsets, W = _case(S, E, M, K, group, dtype, "each", 30, S - S // 9)
    g = torch.Generator().manual_seed(31)
    x, gy = torch.randn((S, K), generator=g).to(dtype), torch.randn((S, M), generator=g).to(dtype)
    args = (_packed(km, lab), table.cuda())
    sc, off = None if scales is None else scales.cuda(), offsets.cuda()
    got = km.kmeans_codes_product(x.cuda(), *args, M, sc, group, off, out=torch.full((S, M), 7.0, dtype=dtype, device="cuda"))
    ref, mag = _ref(x, W, offsets, False)
    _close(got, ref, mag, K, dtype, False, "product")
    got = km.kmeans_codes_product_grad(gy.cuda(), *args, K, sc, group, off, out=torch.full((S, K), 7.0, dtype=dtype, device="cuda"))
    ref, mag = _ref(gy, W, offsets, True)
    _close(got, ref, mag, M, dtype, group > 0, "gradient")
    again = km.kmeans_codes_product_grad(gy.cuda(), *args, K, sc, group, off)
    assert torch.equal(got, again)


@pytest.mark.parametrize("S", [1, 48, 600])
def test_nothing_leaks_from_padding_or_neighbours(km, S):
    # infinite and NaN entries reach exactly the outputs whose formula reads them
    E, M, K, group = 2, 50, 200, 64
    dtype = torch.float16
    lab, table, scales, offsets, _ = _case(S, E, M, K, group, dtype, "each", 4)
    lab[lab == 0] = 1          # code 0 (what padding holds) is used nowhere
    table[:, :, 0] = float("inf")
    x = torch.randn((S, K), generator=torch.Generator().manual_seed(5)).to(dtype)
    gy = torch.randn((S, M), generator=torch.Generator().manual_seed(6)).to(dtype)
    args = (_packed(km, lab), table.cuda())
    for bad in (False, True):
        if bad:
            x[S // 2, 3] = float("inf")
            gy[S // 2, 7] = float("nan")
        y = km.kmeans_codes_product(x.cuda(), *args, M, scales.cuda(), group, offsets.cuda()).cpu()
        gx = km.kmeans_codes_product_grad(gy.cuda(), *args, K, scales.cuda(), group, offsets.cuda()).cpu()
        hit = torch.zeros(S, dtype=torch.bool)
        hit[S // 2] = bad
        assert torch.isfinite(y[~hit]).all() and torch.isfinite(gx[~hit]).all()
        if bad:
            assert not torch.isfinite(y[hit]).any() and not torch.isfinite(gx[hit]).any()


def test_gradient_against_differences(km):
    # L(x) = <product(x), c>, linear in x; powers of two keep x +- h v exact
    S, E, M, K, group = 40, 3, 64, 256, 64
    dtype = torch.float16
    lab, table, scales, offsets, W = _case(S, E, M, K, group, dtype, "each", 7)
    g = torch.Generator().manual_seed(8)
    x = torch.randint(-8, 9, (S, K), generator=g).to(dtype)
    v = torch.randint(-8, 9, (S, K), generator=g).to(dtype)
    c = torch.randn((S, M), generator=g).to(dtype)
    args = (_packed(km, lab), table.cuda())
    f = lambda t: (km.kmeans_codes_product(t.cuda(), *args, M, scales.cuda(), group, offsets.cuda()).cpu().double()  # noqa: E731
                   * c.double()).sum()
    diff = (f(x + v) - f(x - v)) / 2
    gx = km.kmeans_codes_product_grad(c.cuda(), *args, K, scales.cuda(), group, offsets.cuda()).cpu().double()
    want = (gx * v.double()).sum()
    _, mag_y = _ref(x.abs() + v.abs(), W, offsets, False)
    _, mag_g = _ref(c, W, offsets, True)
    # both products round their outputs to the type; the gradient its scaled weights too
    bound = 2 * U[dtype] * (mag_y * c.double().abs()).sum() + 4 * U[dtype] * (mag_g * v.double().abs()).sum()
    assert abs(diff - want) <= bound


def test_fitted_rows(km):
    # a weight matrix clustered row by row to 16 values, then used
    M, K, S = 64, 512, 4
    w = torch.randn((M, K, 1), generator=torch.Generator().manual_seed(9)).cuda()
    lo, hi = w.amin(1, keepdim=True), w.amax(1, keepdim=True)
    init = (lo + (hi - lo) * torch.linspace(0, 1, 16, device="cuda").view(1, 16, 1)).contiguous()
    cen, lab, _, _ = km.kmeans_fit(w, init, 10)
    lab, _, _ = km.kmeans_assign(w, cen)
    table = cen.view(1, M, 16).to(torch.float16)
    x = torch.randn((S, K), generator=torch.Generator().manual_seed(10)).to(torch.float16)
    y = km.kmeans_codes_product(x.cuda(), km.kmeans_pack_codes(lab), table, M)
    W = torch.gather(table[0].cpu().double(), 1, lab.cpu().long())
    ref, mag = _ref(x, W[None], [0, S], False)
    _close(y, ref, mag, K, torch.float16, False, "fitted")


def test_odd_alignment_and_offsets_out_of_order(km):
    # x and out start one element into their storage; offsets that do not
    # ascend or leave the rows are clamped, never followed out of the rows
    S, E, M, K = 30, 3, 33, 131
    dtype = torch.bfloat16
    lab, table, scales, offsets, W = _case(S, E, M, K, 32, dtype, "each", 11)
    x = torch.randn((S * K + 1,), generator=torch.Generator().manual_seed(12)).to(dtype).cuda()[1:].view(S, K)
    args = (_packed(km, lab), table.cuda())
    out = torch.empty((S * M + 1,), dtype=dtype, device="cuda")[1:].view(S, M)
    y = km.kmeans_codes_product(x, *args, M, scales.cuda(), 32, offsets.cuda(), out=out)
    ref, mag = _ref(x.cpu(), W, offsets, False)
    _close(y, ref, mag, K, dtype, False, "odd alignment")
    wild = torch.tensor([0, 25, 10, 99], dtype=torch.int32).cuda()
    y = km.kmeans_codes_product(x, *args, M, scales.cuda(), 32, wild)
    ref, mag = _ref(x.cpu(), W, [0, 25, 25, 30], False)
    _close(y, ref, mag, K, dtype, False, "clamped offsets")


def test_products_in_a_graph(km):
    for S in (4, 300):
        lab, table, scales, offsets, _ = _case(S, 2, 80, 256, 64, torch.bfloat16, "each", 13)
        x = torch.randn((S, 256), device="cuda").to(torch.bfloat16)
        g = torch.randn((S, 80), device="cuda").to(torch.bfloat16)
        codes, t, sc, off = _packed(km, lab), table.cuda(), scales.cuda(), offsets.cuda()
        ws = km.codes_workspace(S, 2, 80, 256, x.dtype, "cuda")
        want = km.kmeans_codes_product(x, codes, t, 80, sc, 64, off), km.kmeans_codes_product_grad(g, codes, t, 256, sc, 64, off)
        outs = [torch.empty_like(w) for w in want]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            km.kmeans_codes_product(x, codes, t, 80, sc, 64, off, out=outs[0], ws=ws)
            km.kmeans_codes_product_grad(g, codes, t, 256, sc, 64, off, out=outs[1], ws=ws)
        for _ in range(3):
            for o in outs:
                o.fill_(1)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_codes_refusals(km):
    x = torch.zeros((2, 128), dtype=torch.float16, device="cuda")
    codes = km.kmeans_pack_codes(torch.zeros((16, 128), dtype=torch.int32, device="cuda"))
    table = torch.zeros((16, 16), dtype=torch.float16, device="cuda")
    sc = torch.ones((16, 3), dtype=torch.float16, device="cuda")
    with pytest.raises(km.KMeansError, match="KM_EUNSUPPORTED"):
        km.kmeans_codes_product(x.float(), codes, table.float(), 16)
    with pytest.raises(km.KMeansError, match="group"):
        km.kmeans_codes_product(x, codes, table, 16, sc, 48)
    with pytest.raises(ValueError, match="scales"):
        km.kmeans_codes_product(x, codes, table, 16, sc, 64)
    with pytest.raises(ValueError, match="tiles"):
        km.kmeans_codes_product(x, codes, table, 32)
    with pytest.raises(ValueError, match="table"):
        km.kmeans_codes_product(x, codes, table[:8].contiguous(), 16)
    with pytest.raises(TypeError, match="table"):
        km.kmeans_codes_product(x, codes, table.bfloat16(), 16)
    with pytest.raises(ValueError, match="offsets"):
        km.kmeans_codes_product(x, torch.stack([codes, codes]), torch.stack([table, table]), 16)
    with pytest.raises(ValueError, match="contiguous"):
        km.kmeans_codes_product_grad(x.t(), codes, table, 128)


def test_codes_of_more_than_4_gb(km):
    # tiles, scales and codebooks whose byte offsets pass 32 bits
    M, K, group, dtype = 1 << 20, 8320, 128, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(20)
    codes = torch.randint(0, 256, (M // 16, K // 128, 1024), generator=g, device="cuda", dtype=torch.uint8)
    assert codes.numel() > 1 << 32
    table = torch.randn((M, 16), generator=g, device="cuda").to(dtype)
    scales = (0.5 + torch.rand((M, K // group), generator=g, device="cuda")).to(dtype)
    rows = torch.tensor([0, 5, M // 2 + 3, M - 17, M - 1])
    k = torch.arange(K)
    # the code of (m, k) by the documented layout
    j, q, i = k % 128 // 32, k % 32 // 8, k % 8
    label = torch.stack([(codes[m // 16, (k // 128).cuda(), (((16 * q + m % 16) * 4 + j) * 4 + i % 4).cuda()].cpu().long()
                          >> (4 * (i // 4))) & 15 for m in rows.tolist()])
    W = torch.gather(table[rows.cuda()].cpu().double(), 1, label) * scales[rows.cuda()].cpu().double().repeat_interleave(group, 1)
    for S in (1, 2):
        x = torch.randn((S, K), generator=torch.Generator().manual_seed(21)).to(dtype)
        y = km.kmeans_codes_product(x.cuda(), codes, table, M, scales, group)
        _close(y[:, rows.cuda()], x.double() @ W.t(), x.double().abs() @ W.abs().t(), K, dtype, False, "large product")
        gy = torch.zeros((S, M), dtype=dtype)
        gy[:, rows] = torch.randn((S, len(rows)), generator=torch.Generator().manual_seed(22)).to(dtype)
        gx = km.kmeans_codes_product_grad(gy.cuda(), codes, table, K, scales, group)
        v = gy[:, rows].double()
        _close(gx, v @ W, v.abs() @ W.abs(), len(rows), dtype, True, "large gradient")


def test_a_group_of_any_length(km):
    # one group holds the row: the longest length that an int64 holds is as good as the row's own
    S, E, M, K = 20, 2, 48, 300
    lab, table, scales, offsets, W = _case(S, E, M, K, 384, torch.bfloat16, "each", 40)
    g = torch.Generator().manual_seed(41)
    x, gy = torch.randn((S, K), generator=g).to(torch.bfloat16), torch.randn((S, M), generator=g).to(torch.bfloat16)
    args = (_packed(km, lab), table.cuda())
    for group in (384, (1 << 63) - 128):
        y = km.kmeans_codes_product(x.cuda(), *args, M, scales.cuda(), group, offsets.cuda())
        ref, mag = _ref(x, W, offsets, False)
        _close(y, ref, mag, K, torch.bfloat16, False, f"product, group {group}")
        gx = km.kmeans_codes_product_grad(gy.cuda(), *args, K, scales.cuda(), group, offsets.cuda())
        ref, mag = _ref(gy, W, offsets, True)
        _close(gx, ref, mag, M, torch.bfloat16, True, f"gradient, group {group}")


@pytest.mark.parametrize("E,M,K", [(3, 48, 64), (1, 33, 63), (4096, 16, 32), (4096, 5, 31)])
def test_as_many_rows_as_a_call_takes(km, E, M, K):
    S, dtype = 1 << 20, torch.bfloat16
    lab, table, scales, offsets, W = _case(S, E, M, K, 32, dtype, "each", 50, S - 100)
    g = torch.Generator().manual_seed(51)
    x, gy = torch.randn((S, K), generator=g).to(dtype), torch.randn((S, M), generator=g).to(dtype)
    args = (_packed(km, lab), table.cuda())
    y = km.kmeans_codes_product(x.cuda(), *args, M, scales.cuda(), 32, offsets.cuda())
    ref, mag = _ref(x, W, offsets, False)
    _close(y, ref, mag, K, dtype, False, "product")
    gx = km.kmeans_codes_product_grad(gy.cuda(), *args, K, scales.cuda(), 32, offsets.cuda())
    ref, mag = _ref(gy, W, offsets, True)
    _close(gx, ref, mag, M, dtype, True, "gradient")


def test_the_product_takes_no_workspace(km):
    # a shape whose gradient adds 16 MB of partial sums
    S, M, K = 256, 4096, 4096
    codes = torch.zeros((M // 16, K // 128, 1024), dtype=torch.uint8, device="cuda")
    table = torch.ones((M, 16), dtype=torch.bfloat16, device="cuda")
    x = torch.ones((S, K), dtype=torch.bfloat16, device="cuda")
    assert km.codes_workspace(S, 1, M, K, x.dtype, "cuda").numel() >= 1 << 24
    out = torch.empty((S, M), dtype=x.dtype, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    km.kmeans_codes_product(x, codes, table, M, out=out)
    assert torch.cuda.max_memory_allocated() == before
    assert (out == K).all()
    km.kmeans_codes_product(x, codes, table, M, out=out, ws=torch.empty(1, dtype=torch.uint8, device="cuda"))
