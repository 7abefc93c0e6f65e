"""kmeans_dispatch, kmeans_combine and kmeans_combine_grad against plain
float64 references.

Bounds: the dispatched rows and the rows' gradient (one float32 product
rounded once) are compared bit for bit.  A weighted return sums `top` terms in
float32: |err| <= (top + 1) u32 sum|w r| + u |ref|.  A weight's gradient sums d
products in float32: |err| <= (d + 1) u32 sum|g r|.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -140, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -130}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]

SHAPES = [  # T, top, E, d, kind
    (1, 1, 1, 1, "uniform"), (1, 2, 8, 64, "uniform"), (5, 3, 4, 7, "dropped"), (24, 2, 8, 4096, "uniform"),
    (100, 9, 16, 33, "dropped"), (64, 1, 200, 129, "none"), (200, 20, 64, 24, "dropped"), (4096, 1, 4096, 8, "uniform"),
    (2049, 2, 5, 40, "same"), (5000, 1, 1, 16, "dropped"), (3001, 4, 61, 65, "dropped"), (1500, 6, 512, 72, "dropped"),
    (1200, 8, 4096, 10, "uniform"), (9000, 3, 300, 8, "none"), (2, 3000, 7, 5, "uniform"), (0, 2, 8, 16, "uniform"),
]


@pytest.fixture(scope="module")
def km():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import exact_lloyd_means_03_amd as km
    km.load()
    return km


def _rows(shape, dtype, seed, off=0):
    g = torch.Generator().manual_seed(seed)
    n = int(np.prod(shape))
    flat = torch.empty(n + off, dtype=dtype, device="cuda")
    flat[off:] = torch.randn(n, generator=g).to(dtype)
    return flat[off:].view(shape)


def _experts(T, top, E, kind, seed=1):
    g = torch.Generator().manual_seed(seed)
    e = torch.randint(0, E, (T, top), generator=g)
    if kind == "same":
        e[:] = E - 1
    if kind == "none":
        e = torch.where(e % 2 == 0, -1, E + 3)
    if kind == "dropped":
        e[torch.rand((T, top), generator=g) < 0.2] = -1
        e[torch.rand((T, top), generator=g) < 0.05] = E
        e[0, 0] = -2 ** 31
    return e.to(torch.int32)


def _plan(e, E):
    flat = e.numpy().reshape(-1)
    live = np.nonzero((flat >= 0) & (flat < E))[0]
    by = live[np.argsort(flat[live], kind="stable")]
    slots = np.full(flat.shape, -1, np.int32)
    slots[by] = np.arange(len(by))
    order = np.full(flat.shape, -1, np.int32)
    order[:len(by)] = by
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[live], minlength=E))]).astype(np.int32)
    return offsets, slots.reshape(e.shape), order


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,top,E,d,kind", SHAPES)
def test_dispatch(km, dtype, T, top, E, d, kind):
    x, e = _rows((T, d), dtype, 2, off=1), _experts(T, top, E, kind) if T else torch.zeros((0, top), dtype=torch.int32)
    rows = torch.full((T * top, d), 7.0, dtype=dtype, device="cuda")
    got = km.kmeans_dispatch(x, e.cuda(), E, rows=rows)
    offsets, slots, order = _plan(e, E)
    np.testing.assert_array_equal(got[1].cpu().numpy(), offsets)
    np.testing.assert_array_equal(got[2].cpu().numpy(), slots)
    np.testing.assert_array_equal(got[3].cpu().numpy(), order)
    want = torch.zeros((T * top, d), dtype=dtype)
    n = int(offsets[-1])
    want[:n] = x.cpu()[torch.from_numpy(order[:n] // top).long()]
    assert torch.equal(got[0].cpu(), want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,top,E,d,kind", SHAPES[:-1])
def test_combine_and_gradients(km, dtype, T, top, E, d, kind):
    e = _experts(T, top, E, kind)
    offsets, slots, order = _plan(e, E)
    rows, gy = _rows((T * top, d), dtype, 3, off=1), _rows((T, d), dtype, 4)
    w = torch.rand((T, top), generator=torch.Generator().manual_seed(5))
    w[slots < 0] = float("nan")  # a dropped choice's weight is never used
    sl = torch.from_numpy(slots)
    r64 = rows.cpu().double()
    picked = torch.where((sl >= 0)[..., None], r64[sl.clamp(min=0).long()], 0.0)  # [T, top, d]
    w64 = torch.where(sl >= 0, w.double(), 0.0)
    for weights in (w, None):
        got = km.kmeans_combine(rows, sl.cuda(), None if weights is None else weights.cuda())
        terms = picked if weights is None else picked * w64[..., None]
        ref, mag = terms.sum(1), terms.abs().sum(1)
        tol = (top + 1) * U32 * mag + U[dtype] * ref.abs() * (1 + top * U32) + TINY[dtype]
        assert ((got.cpu().double() - ref).abs() <= tol).all()
    grows, gw = km.kmeans_combine_grad(gy, rows, sl.cuda(), torch.from_numpy(order).cuda(), w.cuda(),
                                       grad_rows=torch.full_like(rows, 7.0))
    n = int(offsets[-1])
    want = torch.zeros((T * top, d), dtype=dtype)
    o = torch.from_numpy(order[:n]).long()
    want[:n] = (w.reshape(-1)[o][:, None] * gy.cpu().float()[o // top]).to(dtype)
    assert torch.equal(grows.cpu(), want)
    prod = picked * gy.cpu().double()[:, None]
    assert ((gw.cpu().double() - prod.sum(-1)).abs() <= (d + 1) * U32 * prod.abs().sum(-1)).all()


def test_gradients_against_differences(km):
    # L = <combine(dispatch(x), w), c>, in x and in w (float32, linear in each)
    T, top, E, d, h = 300, 3, 9, 50, 0.5
    e = _experts(T, top, E, "dropped").cuda()
    x, vx, c = (_rows((T, d), torch.float32, s) for s in (6, 7, 8))
    w, vw = (torch.rand((T, top), generator=torch.Generator().manual_seed(s)).cuda() for s in (9, 10))

    def loss(x, w):
        rows, _, slots, _ = km.kmeans_dispatch(x, e, E)
        return (km.kmeans_combine(rows, slots, w).double() * c.double()).sum()

    rows, _, slots, order = km.kmeans_dispatch(x, e, E)
    grows, gw = km.kmeans_combine_grad(c, rows, slots, order, w)
    gx = km.kmeans_combine(grows, slots, None)
    mag = float((((x.abs() + vx.abs()) * c.abs()).double().sum(1) * (w + vw).double().sum(1)).sum())
    for diff, want in (((loss(x + h * vx, w) - loss(x - h * vx, w)) / (2 * h), (gx.double() * vx.double()).sum()),
                       ((loss(x, w + h * vw) - loss(x, w - h * vw)) / (2 * h), (gw.double() * vw.double()).sum())):
        # a few float32 roundings of each loss over 2h, and the gradients' own sums
        assert abs(diff - want) <= (4 * (top + 2) / h + d + 2) * U32 * mag


def test_rows_past_2_31_elements(km):
    T, top, d = (1 << 30) // 4096 + 800, 2, 4096
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda").random_(-8, 8)
    e = torch.stack([torch.arange(T) % 5, 4 - torch.arange(T) % 5], 1).to(torch.int32).cuda()
    rows, offsets, slots, order = km.kmeans_dispatch(x, e, 5)
    for p in (0, T - 1, T, 2 * T - 1):
        assert torch.equal(rows[p], x[int(order[p]) // top])
    y = km.kmeans_combine(rows, slots, None)
    assert torch.equal(y[-3:], 2 * x[-3:]) and torch.equal(y[:3], 2 * x[:3])


def test_routing_in_a_graph(km):
    for T in (50, 5000):
        E, top, d = 12, 2, 96
        x, e = _rows((T, d), torch.bfloat16, 11), _experts(T, top, E, "dropped").cuda()
        w = torch.rand((T, top), device="cuda")
        want = km.kmeans_dispatch(x, e, E)
        want_y = km.kmeans_combine(want[0], want[2], w)
        want_g = km.kmeans_combine_grad(x, want[0], want[2], want[3], w)
        outs = [torch.empty_like(t) for t in (*want, want_y, *want_g)]
        ws = km.dispatch_workspace(T, top, E, "cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            km.kmeans_dispatch(x, e, E, rows=outs[0], plan=outs[1:4], ws=ws)
            km.kmeans_combine(outs[0], outs[2], w, out=outs[4])
            km.kmeans_combine_grad(x, outs[0], outs[2], outs[3], w, grad_rows=outs[5], grad_weights=outs[6])
        for _ in range(3):
            for t in outs:
                t.fill_(1)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, (*want, want_y, *want_g)):
                assert torch.equal(a, b)


def test_routing_refusals(km):
    x, e = _rows((4, 8), torch.float32, 1), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match=r"\[T, d\]"):
        km.kmeans_dispatch(x[None], e, 2)
    with pytest.raises(ValueError, match=r"\[T, top\]"):
        km.kmeans_dispatch(x, e[:3], 2)
    with pytest.raises(TypeError, match="int32"):
        km.kmeans_dispatch(x, e.long(), 2)
    with pytest.raises(km.KMeansError, match="KM_EUNSUPPORTED"):
        km.kmeans_dispatch(x, e, 5000)
    rows, _, slots, order = km.kmeans_dispatch(x, e, 2)
    with pytest.raises(ValueError, match="rows"):
        km.kmeans_combine(rows[:5], slots)
    with pytest.raises(TypeError, match="float32"):
        km.kmeans_combine(rows, slots, torch.ones((4, 2), dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        km.kmeans_combine_grad(x[:3], rows, slots, order, torch.ones((4, 2), device="cuda"))
