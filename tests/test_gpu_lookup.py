"""kmeans_lookup and kmeans_lookup_grad against plain float64 sums.

Bounds: the lookup is one float32 product rounded once to the row type, so it
is compared bit for bit.  The gradient sums n rows in float32: each of the n - 1
additions and the scaling adds at most u32 of the partial magnitude, so
|err| <= (n + 1) u32 |scale| sum|g| + u |ref|, u the output type's rounding.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -140, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -130}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def km():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import exact_lloyd_means_03_amd as km
    km.load()
    return km


def _rows(shape, dtype, seed, std=1.0, off=0):
    """Rows on the GPU whose storage starts `off` elements into an allocation."""
    g = torch.Generator().manual_seed(seed)
    n = int(np.prod(shape))
    flat = torch.empty(n + off, dtype=dtype, device="cuda")
    flat[off:] = (torch.randn(n, generator=g) * std).to(dtype)
    return flat[off:].view(shape)


def _labels(B, N, V, seed, kind):
    g = torch.Generator().manual_seed(seed)
    if kind == "uniform":
        lab = torch.randint(0, V, (B, N), generator=g)
    elif kind == "same":
        lab = torch.full((B, N), V // 2)
    elif kind == "none":
        lab = torch.where(torch.rand((B, N), generator=g) < 0.5, -1, V)
    elif kind == "skewed":
        lab = (torch.rand((B, N), generator=g) ** 6 * V).long().clamp(max=V - 1)
        lab[torch.rand((B, N), generator=g) < 0.1] = -7
        lab[torch.rand((B, N), generator=g) < 0.02] = V + 5
        if N > 3:
            lab[:, 1], lab[:, 2] = -2 ** 31, 2 ** 31 - 1
    return lab.to(torch.int32)


def _check_grad(got, g, lab, V, scale, what):
    B, N, d = g.shape
    dt = got.dtype
    g64 = g.cpu().double().numpy()
    for b in range(B):
        ok = ((lab[b] >= 0) & (lab[b] < V)).numpy()
        idx = lab[b].numpy()[ok].astype(np.int64)
        ref, mag = np.zeros((V, d)), np.zeros((V, d))
        np.add.at(ref, idx, g64[b][ok])
        np.add.at(mag, idx, np.abs(g64[b][ok]))
        n = np.bincount(idx, minlength=V)[:, None]
        ref *= scale
        tol = (n + 1) * U32 * abs(scale) * mag + U[dt] * np.abs(ref) * (1 + (n + 1) * U32) + TINY[dt] * (n > 0)
        err = np.abs(got[b].cpu().double().numpy() - ref)
        assert (err <= tol).all(), f"{what} b={b}: worst {np.nanmax(err - tol)}"
        assert not got[b].cpu().numpy(force=True).any() if n.sum() == 0 and dt != torch.bfloat16 else True


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,V,N,d,kind,off", [
    (1, 1, 1, 1, "uniform", 0), (1, 5, 7, 3, "skewed", 1), (1, 100, 300, 8, "skewed", 0), (2, 33, 129, 65, "skewed", 3),
    (3, 1000, 517, 1000, "uniform", 0), (1, 70000, 40, 4097, "skewed", 1), (1, 64, 50, 256, "none", 0),
    (1, 9, 0, 16, "uniform", 0), (1, 50, 2000, 31, "same", 0),
])
def test_lookup(km, dtype, B, V, N, d, kind, off):
    table = _rows((B, V, d), dtype, 1, off=off)
    lab = _labels(B, N, V, 2, kind)
    for scale in (1.0, -45.3):
        got = km.kmeans_lookup(table, lab.cuda(), scale)
        ok = (lab >= 0) & (lab < V)
        pick = table.cpu().float()[torch.arange(B)[:, None], torch.where(ok, lab, 0).long()]
        want = torch.where(ok[..., None], pick * torch.tensor(scale, dtype=torch.float32), torch.tensor(0.0)).to(dtype)
        assert torch.equal(got.cpu(), want), f"scale {scale}"


def test_lookup_passes_infinities_and_nan_but_not_to_other_rows(km):
    table = _rows((1, 4, 33), torch.bfloat16, 5)
    table[0, 1] = float("inf")
    table[0, 2] = float("nan")
    lab = torch.tensor([[0, 1, 2, 3, -1]], dtype=torch.int32)
    got = km.kmeans_lookup(table, lab.cuda(), 0.0).float().cpu()
    assert (got[0, [0, 3, 4]] == 0).all() and got[0, 1].isnan().all() and got[0, 2].isnan().all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,V,N,d,kind,off", [
    (1, 1, 1, 1, "uniform", 0), (1, 5, 7, 3, "skewed", 1), (2, 33, 129, 65, "skewed", 3), (1, 64, 50, 256, "none", 0),
    (1, 9, 0, 16, "uniform", 0), (1, 50, 3000, 33, "same", 0), (1, 300, 8192, 40, "skewed", 0),
    (3, 700, 5000, 9, "skewed", 0), (1, 5000, 9001, 24, "skewed", 1), (1, 100000, 20011, 16, "uniform", 0),
    (1, 17, 40000, 130, "skewed", 0), (2, 4095, 12345, 64, "skewed", 0), (2, 4096, 12345, 8, "uniform", 0),
])
def test_lookup_grad(km, dtype, B, V, N, d, kind, off):
    g = _rows((B, N, d), dtype, 3, 0.3, off)
    lab = _labels(B, N, V, 4, kind)
    for out_dtype in {dtype, torch.float32}:
        out = torch.full((B, V, d), float("nan"), dtype=out_dtype, device="cuda")
        got = km.kmeans_lookup_grad(g, lab.cuda(), V, 0.75, out=out)
        _check_grad(got, g, lab, V, 0.75, f"{out_dtype}")
        again = km.kmeans_lookup_grad(g, lab.cuda(), V, 0.75, out=torch.empty_like(out))
        assert torch.equal(got, again)


def test_lookup_grad_of_a_label_over_many_pieces(km):
    # one label holds almost every row, with others before and after it
    V, N, d = 40, 60000, 72
    g = _rows((1, N, d), torch.float32, 6)
    lab = torch.full((1, N), 20, dtype=torch.int32)
    lab[0, ::997] = 3
    lab[0, 5::1999] = 39
    _check_grad(km.kmeans_lookup_grad(g, lab.cuda(), V), g, lab, V, 1.0, "wide label")


def test_lookup_grad_beyond_three_digits(km):
    # labels of 25 bits: three passes of the sort
    V, N, d = 1 << 25, 9000, 4
    g = _rows((1, N, d), torch.float16, 7)
    lab = _labels(1, N, V, 8, "uniform")
    lab[0, :100] = V - 1
    got = km.kmeans_lookup_grad(g, lab.cuda(), V)
    uniq, inv = torch.unique(lab[0], return_inverse=True)
    small = torch.zeros((1, len(uniq), d), dtype=torch.float16)
    small[0] = got[0, uniq.long().cuda()].cpu()
    _check_grad(small, g, inv.to(torch.int32)[None], len(uniq), 1.0, "25 bits")
    assert int((got != 0).any(-1).sum()) <= len(uniq)


def test_lookup_grad_against_differences(km):
    # L(table) = <lookup(table), c>; the central difference along v is <grad, v>
    B, V, N, d, h = 2, 50, 400, 19, 0.5
    table, v = _rows((B, V, d), torch.float32, 9), _rows((B, V, d), torch.float32, 10)
    c = _rows((B, N, d), torch.float32, 11)
    lab = _labels(B, N, V, 12, "skewed").cuda()
    loss = lambda t: (km.kmeans_lookup(t, lab, 1.5).double() * c.double()).sum()  # noqa: E731
    diff = (loss(table + h * v) - loss(table - h * v)) / (2 * h)
    grad = km.kmeans_lookup_grad(c, lab, V, 1.5).double()
    want = (grad * v.double()).sum()
    mag = (km.kmeans_lookup(table.abs() + h * v.abs(), lab, 1.5).double() * c.double().abs()).sum()
    # table +- h v and the lookups round in float32; the gradient sums at most N rows in float32
    assert abs(diff - want) <= (4 / h + N + 1) * U32 * mag


def test_more_than_2_31_elements(km):
    # rows past element 2^31, and past 2^32 bytes
    V, d = 1000, 4096
    N = (1 << 31) // d + 1500
    table = _rows((1, V, d), torch.bfloat16, 13)
    lab = torch.arange(N, dtype=torch.int32).remainder(V)[None].cuda()
    out = km.kmeans_lookup(table, lab)
    for i in (0, N // 2, N - 1501, N - 1):
        assert torch.equal(out[0, i], table[0, i % V])
    grad = km.kmeans_lookup_grad(out, lab, V, out=torch.empty((1, V, d), dtype=torch.float32, device="cuda"))
    n = torch.bincount(lab[0].long(), minlength=V).float()[:, None].cuda()
    # every row of a label is the same: n times it, summed in float32
    assert ((grad[0] - n * table[0].float()).abs() <= (n + 1) * U32 * n * table[0].float().abs()).all()


def test_lookups_on_another_stream_and_in_a_graph(km):
    B, V, N, d = 1, 900, 9000, 136
    table, g = _rows((B, V, d), torch.float16, 14), _rows((B, N, d), torch.float16, 15)
    lab = _labels(B, N, V, 16, "skewed").cuda()
    want_o, want_g = km.kmeans_lookup(table, lab), km.kmeans_lookup_grad(g, lab, V)
    out, grad = torch.empty_like(want_o), torch.empty_like(want_g)
    ws = km.lookup_grad_workspace(B, N, d, V, g.dtype, "cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        km.kmeans_lookup(table, lab, out=out)
        km.kmeans_lookup_grad(g, lab, V, out=grad, ws=ws)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want_o) and torch.equal(grad, want_g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        km.kmeans_lookup(table, lab, out=out)
        km.kmeans_lookup_grad(g, lab, V, out=grad, ws=ws)
    for _ in range(3):
        out.fill_(1)
        grad.fill_(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want_o) and torch.equal(grad, want_g)


def test_lookup_of_a_fitted_codebook(km):
    # the labels and centroids of a fit, as they come: every point's centroid
    x = _rows((2, 500, 24), torch.float32, 17)
    cen, lab, cnt, _ = km.kmeans_fit(x, x[:, :16].clone(), 3)
    near = km.kmeans_lookup(cen, lab)
    assert torch.equal(near, torch.gather(cen, 1, lab.long()[..., None].expand(-1, -1, 24)))
    # and the sums of its points from the gradient of that lookup
    lab2, _, _ = km.kmeans_assign(x, cen)
    sums = km.kmeans_lookup_grad(x, lab2, 16)
    means, n = km.kmeans_update(x, lab2, cen)
    assert torch.allclose(sums / n.clamp(min=1)[..., None], torch.where(n[..., None] > 0, means, 0.0), rtol=1e-5, atol=1e-5)


def test_lookup_refusals(km):
    t, lab = _rows((1, 8, 4), torch.float32, 1), torch.zeros((1, 3), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match=r"\[B, V, d\]"):
        km.kmeans_lookup(t[0], lab)
    with pytest.raises(TypeError, match="int32"):
        km.kmeans_lookup(t, lab.long())
    with pytest.raises(ValueError, match="contiguous"):
        km.kmeans_lookup(t.transpose(1, 2), lab)
    with pytest.raises(ValueError, match="GPU"):
        km.kmeans_lookup(t, lab.cpu())
    with pytest.raises(ValueError, match="shape"):
        km.kmeans_lookup(t, lab, out=torch.empty((1, 2, 4), device="cuda"))
    g = _rows((1, 3, 4), torch.float16, 1)
    with pytest.raises(km.KMeansError, match="KM_EUNSUPPORTED"):
        km.kmeans_lookup_grad(g, lab, 8, out=torch.empty((1, 8, 4), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(km.KMeansError, match="KM_EWORKSPACE"):
        km.kmeans_lookup_grad(g, lab, 8, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(km.KMeansError, match="KM_EINVAL"):
        km.kmeans_lookup_grad(g, lab, 0, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
