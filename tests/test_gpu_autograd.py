"""The operators on labels and codebooks under torch's autograd: a call whose
input requires a gradient is recorded, and its gradient is the one of the
explicit gradient call, bit for bit; what has no gradient is refused, never
returned without history.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def km():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import exact_lloyd_means_03_amd as km
    km.load()
    return km


def _inputs(km, T=50, top=3, V=40, d=96, M=80, E=5, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    s = dict(table=rand(1, V, d).to(dtype), ids=torch.randint(-1, V, (1, T), generator=g, device="cuda", dtype=torch.int32),
             experts=torch.randint(-1, E, (T, top), generator=g, device="cuda", dtype=torch.int32),
             weights=rand(T, top).abs(), books=rand(E, M, 16).to(dtype), scales=(rand(E, M, 2) + 2).to(dtype),
             gy=rand(T, M).to(dtype), E=E, M=M, d=d, V=V)
    s["codes"] = torch.stack([km.kmeans_pack_codes(torch.randint(0, 16, (M, d), generator=g, device="cuda", dtype=torch.int32))
                              for _ in range(E)])
    return s


def _forward(km, s, table, weights):
    x = km.kmeans_lookup(table, s["ids"], 1.5)
    rows, offsets, slots, order = km.kmeans_dispatch(x[0], s["experts"], s["E"])
    h = km.kmeans_codes_product(rows, s["codes"], s["books"], s["M"], s["scales"], 64, offsets)
    return km.kmeans_combine(h, slots, weights), h, offsets, slots, order


@pytest.mark.parametrize("weighted", [True, False])
def test_gradients_are_the_explicit_calls(km, weighted):
    s = _inputs(km)
    table = s["table"].clone().requires_grad_()
    weights = s["weights"].clone().requires_grad_() if weighted else None
    y, _, offsets, slots, order = _forward(km, s, table, weights)
    assert y.requires_grad and not any(t.requires_grad for t in (offsets, slots, order))
    y.backward(s["gy"])
    with torch.no_grad():
        w = s["weights"] if weighted else None
        y2, h, offsets, slots, order = _forward(km, s, s["table"], w)
        ones = torch.ones_like(s["weights"])
        grows, gw = km.kmeans_combine_grad(s["gy"], h, slots, order, s["weights"] if weighted else ones)
        gx = km.kmeans_codes_product_grad(grows, s["codes"], s["books"], s["d"], s["scales"], 64, offsets)
        gt = km.kmeans_lookup_grad(km.kmeans_combine(gx, slots, None)[None], s["ids"], s["V"], 1.5)
    assert torch.equal(y, y2) and torch.equal(table.grad, gt)
    if weighted:
        assert torch.equal(weights.grad, gw)


def test_gradients_of_expanded_and_partial_outputs(km):
    # sum() hands an expanded gradient back; the weights alone may be recorded
    s = _inputs(km, dtype=torch.float16)
    weights = s["weights"].clone().requires_grad_()
    y = km.kmeans_combine(s["gy"].repeat_interleave(3, 0), torch.arange(150, dtype=torch.int32, device="cuda").view(50, 3), weights)
    y.sum().backward()
    want = s["gy"].double().sum(1, keepdim=True).expand(50, 3)
    # 80 products by one, summed in float32
    assert ((weights.grad.double() - want).abs() <= 81 * 2.0 ** -24 * s["gy"].double().abs().sum(1, keepdim=True)).all()
    table = s["table"].clone().requires_grad_()
    km.kmeans_lookup(table, s["ids"]).sum().backward()
    n = torch.bincount(s["ids"][0][s["ids"][0] >= 0].long(), minlength=s["V"])
    assert torch.equal(table.grad[0], n[:, None].expand(-1, s["d"]).to(torch.float16))


def test_rows_without_a_choice_get_zeros(km):
    rows = torch.ones((8, 4), device="cuda", requires_grad=True)
    slots = torch.tensor([[0, -1], [2, 1], [-1, -1], [3, 100]], dtype=torch.int32, device="cuda")
    km.kmeans_combine(rows, slots, None).sum().backward()
    want = torch.zeros((8, 4))
    want[:4] = 1
    assert torch.equal(rows.grad.cpu(), want)


def test_nothing_is_recorded_without_need(km):
    s = _inputs(km)
    table = s["table"].clone().requires_grad_()
    with torch.no_grad():
        out = torch.empty((1, 50, 96), dtype=table.dtype, device="cuda")
        assert km.kmeans_lookup(table, s["ids"], out=out) is out and not out.requires_grad
    assert not _forward(km, s, s["table"], s["weights"])[0].requires_grad


def test_what_has_no_gradient_is_refused(km):
    s = _inputs(km)
    table = s["table"].clone().requires_grad_()
    with pytest.raises(ValueError, match="given tensors"):
        km.kmeans_lookup(table, s["ids"], out=torch.empty((1, 50, 96), dtype=table.dtype, device="cuda"))
    x = s["gy"].new_zeros((50, 96)).requires_grad_()
    with pytest.raises(ValueError, match="given tensors"):
        km.kmeans_dispatch(x, s["experts"], 5, rows=torch.empty((150, 96), dtype=x.dtype, device="cuda"))
    rows, offsets, slots, order = km.kmeans_dispatch(x.detach(), s["experts"], 5)
    with pytest.raises(ValueError, match="given tensors"):
        km.kmeans_combine(rows, slots, s["weights"].clone().requires_grad_(), out=torch.empty_like(x))
    for name in ("books", "scales"):
        t = dict(s, **{name: s[name].clone().requires_grad_()})
        for call in (lambda: km.kmeans_codes_product(rows, t["codes"], t["books"], 80, t["scales"], 64, offsets),
                     lambda: km.kmeans_codes_product_grad(torch.zeros((150, 80), dtype=rows.dtype, device="cuda"),
                                                          t["codes"], t["books"], 96, t["scales"], 64, offsets)):
            with pytest.raises(ValueError, match="no gradient of (table|scales)"):
                call()
    for call in (lambda g: km.kmeans_lookup_grad(g[None], s["ids"], 40),
                 lambda g: km.kmeans_combine_grad(g, rows, slots, order, s["weights"]),
                 lambda g: km.kmeans_codes_product_grad(g.new_zeros((150, 80)).requires_grad_(), s["codes"], s["books"],
                                                        96, s["scales"], 64, offsets)):
        with pytest.raises(ValueError, match="no gradient of grad"):
            call(x)
    y = km.kmeans_lookup(table, s["ids"])
    (gt,) = torch.autograd.grad(y, table, torch.ones_like(y).requires_grad_(), create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable|twice"):
        gt.sum().backward()


def test_gradients_against_differences(km):
    # L = <combine(dispatch(lookup(table)), w), c> is linear in the table and in w (float32)
    s = _inputs(km, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(2)
    c = torch.randn((50, 96), generator=g, device="cuda")
    vt, vw = torch.randn(s["table"].shape, generator=g, device="cuda"), torch.randn((50, 3), generator=g, device="cuda")

    def loss(table, w):
        x = km.kmeans_lookup(table, s["ids"])
        rows, _, slots, _ = km.kmeans_dispatch(x[0], s["experts"], 5)
        return (km.kmeans_combine(rows, slots, w).double() * c.double()).sum()

    table, w = s["table"].clone().requires_grad_(), s["weights"].clone().requires_grad_()
    loss(table, w).backward()
    with torch.no_grad():
        mag = (km.kmeans_lookup(table.abs() + vt.abs(), s["ids"])[0].double() * c.double().abs()).sum(1)
        mag = float((mag * (w + vw.abs()).double().sum(1)).sum())
        for diff, want in (((loss(table + vt, w) - loss(table - vt, w)) / 2, (table.grad.double() * vt.double()).sum()),
                           ((loss(table, w + vw) - loss(table, w - vw)) / 2, (w.grad.double() * vw.double()).sum())):
            # the losses round their inputs and three terms in float32, the gradients sum at
            # most 50 rows of three, or 96 products
            assert abs(diff - want) <= (12 + 160) * 2.0 ** -24 * mag
