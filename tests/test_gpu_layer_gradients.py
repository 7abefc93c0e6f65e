"""A layer of 8-bit experts trained through autograd with all its paths at once (the
rows gathered by the plan's order, the weights of the choices, the balance loss, the
residual's stream), its gradients against a float64 graph of the formulas in which
the choices and the codes are held and rounding is passed through.

Bounds.  The matrix instruction loses less than 7 * 2^-13 of sum |X W|
(test_gpu_block_product.py); that error is carried through the layer's gradients as
absolute values, next to the sums of the absolute terms themselves, of which float32
costs 2000 u32 (sums of 128 terms in four products and a norm, u32 = 2^-24).  Weights
and probabilities are off by twice the largest error of a logit, relative, which is
(128 + 74) u32 of sum |y router|: four factors of a term are such.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
LOST = 7 * 2.0 ** -13
EPS = 1e-5


@pytest.fixture(scope="module")
def km():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import exact_lloyd_means_03_amd as km
    km.load()
    return km


class Held(torch.autograd.Function):
    """rows X W^T; backward the product of the gradient's codes, whose values are given."""

    @staticmethod
    def forward(ctx, x, w, codes_values):
        ctx.save_for_backward(w, codes_values)
        return x @ w.t()

    @staticmethod
    def backward(ctx, _):
        w, g = ctx.saved_tensors
        return g @ w, None, None


def _values(codes, scales):
    return codes.float().double() * scales.double().repeat_interleave(128, 1)[:, :codes.shape[1]]


@pytest.mark.parametrize("T,top,normalized", [(50, 2, True), (50, 2, False), (33, 1, False), (70, 4, True)])
def test_gradients(km, T, top, normalized):
    d, E, c = 128, 5, 50.0 * T
    g = torch.Generator().manual_seed(T + top)
    x, residual, gy, gh = (torch.randn((T, d), generator=g).cuda() for _ in range(4))
    weight = (1.0 + 0.1 * torch.randn(d, generator=g)).cuda()
    router = (torch.randn((d, E), generator=g) / d ** 0.5).cuda()
    codes, scales = km.kmeans_quantize((torch.randn((E, d, d), generator=g) / d ** 0.5).cuda(), 128)

    # the layer
    leaves = [t.clone().requires_grad_() for t in (x, residual, weight)]
    y, h = km.kmeans_norm(leaves[0], leaves[2], EPS, residual=leaves[1])
    experts, weights, counts, _, loss = km.kmeans_gate(y @ router, top, normalized)
    offsets, slots, order = km.kmeans_plan(experts, E)
    rows = km.kmeans_block_product(y, None, codes, scales, offsets, order=order)
    seen = []
    rows.register_hook(lambda v: seen.append(v.clone()))
    out = km.kmeans_combine(rows, slots, weights)
    ((out * gy).sum() + (h * gh).sum() + c * loss).backward()

    # the formulas; what is held: choices, counts, codes of y and of the rows' gradient
    W = torch.stack([_values(codes[e], scales[e].repeat_interleave(128, 0)[:d]) for e in range(E)])
    X, G = _values(*km.kmeans_quantize(y.detach())), _values(*km.kmeans_quantize(seen[0]))
    ends, token, kth = offsets.tolist(), (order // top).long(), order.long()
    segments = [(e, slice(ends[e], ends[e + 1])) for e in range(E) if ends[e] < ends[e + 1]]
    assert ends[E] == T * top
    R, e64 = router.double(), experts.long()
    f = c * E * counts[:E].double() / (T * counts[:E].sum())

    def reference(balance=True, stream=True, rows_path=True, weights_path=True):
        """Gradients of (x, residual, weight), any of the paths left out."""
        a, b, w = (t.double().requires_grad_() for t in (x, residual, weight))
        hd = a + b
        yd = hd / (hd.square().mean(1, keepdim=True) + EPS).sqrt() * w
        logits = yd @ R
        p = torch.softmax(logits, 1)
        wd = p.gather(1, e64)
        if normalized:
            wd = wd / wd.sum(1, keepdim=True)
        Xd = (yd + (X - yd).detach())[token]
        rd = torch.cat([Held.apply(Xd[s], W[e], G[s] if rows_path else 0 * G[s]) for e, s in segments])
        wk = wd if weights_path else wd.detach()
        od = torch.zeros_like(yd).index_add(0, token, wk.reshape(-1)[kth][:, None] * rd)
        total = (od * gy.double()).sum()
        if stream:
            total = total + (hd * gh.double()).sum()
        if balance:
            total = total + (p.mean(0) * f * T).sum()
        total.backward()
        return [t.grad for t in (a, b, w)], (hd.detach(), yd.detach(), p.detach(), wd.detach(), rd.detach())

    want, (hd, yd, p, wd, rd) = reference()
    rho = 2 * 202 * U32 * (yd.abs() @ R.abs()).max().item()
    # the rows' gradient that reached the product is weights * gy
    assert ((seen[0].double() - wd.reshape(-1)[kth][:, None] * gy.double()[token]).abs() <=
            (rho + 200 * U32) * wd.reshape(-1)[kth][:, None] * gy.double()[token].abs() + 1e-30).all()

    # sums of absolute terms, and the instruction's errors, through the same steps
    agy = gy.double().abs()[token]
    size_rows = torch.cat([X[token][s].abs() @ W[e].abs().t() for e, s in segments])
    back_rows = torch.zeros_like(yd).index_add(0, token, torch.cat([G[s].abs() @ W[e].abs() for e, s in segments]))

    def carried(of_rows, of_back, of_loss, of_stream):
        gw = torch.zeros((T * top,), dtype=torch.float64, device="cuda")
        gw[kth] = (agy * of_rows).sum(1)
        gw = gw.view(T, top)
        spread = torch.zeros_like(p).scatter(1, e64, gw if not normalized else wd * (gw + (wd * gw).sum(1, keepdim=True)))
        if not normalized:
            spread = p * (spread + (p * spread).sum(1, keepdim=True))
        spread = spread + of_loss * p * (f + (p * f).sum(1, keepdim=True))
        v = spread @ R.abs().t() + of_back
        r = 1 / (hd.square().mean(1, keepdim=True) + EPS).sqrt()
        u = v * weight.double().abs()
        gx = r * u + hd.abs() * r ** 3 * (u * hd.abs()).mean(1, keepdim=True) + of_stream * gh.double().abs()
        return gx, (v * hd.abs() * r).sum(0)
    terms, errors = carried(size_rows, back_rows, 1, 1), carried(LOST * size_rows, LOST * back_rows, 0, 0)
    bounds = [lost + (4 * rho + 2000 * U32) * size for lost, size in zip(errors, terms)]
    bounds = [bounds[0], bounds[0], bounds[1]]

    def off(grads):
        return [((leaf.grad.double() - v).abs() - b).max().item() for leaf, v, b in zip(leaves, grads, bounds)]
    assert max(off(want)) <= 0, off(want)
    # each path is large enough to be missed
    for path in ("balance", "stream", "rows_path") + (("weights_path",) if top > 1 or not normalized else ()):
        assert max(off(reference(**{path: False})[0])) > 0, path
