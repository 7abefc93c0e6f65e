"""kmeans_codes_product_grad in float16 where scale * entry leaves float16's
range, against plain float64 products.

The bound is the one of the gradient's other tests (test_gpu_codes.py): every
weight is off by u relative at most, of whatever size it is, so a token that
meets only small or only large weights is as exact as one that meets ordinary
ones.
"""
import pytest
import torch
from test_gpu_codes import _close, _packed, _ref, km  # noqa: F401

pytestmark = pytest.mark.gpu

F16 = torch.float16


def _signed(shape, lo, hi, g):
    """Values of random sign, their size even over the logarithm of [lo, hi]."""
    size = torch.exp(torch.empty(shape, dtype=torch.float64).uniform_(float(torch.tensor(lo).log()),
                                                                       float(torch.tensor(hi).log()), generator=g))
    return size * (torch.randint(0, 2, shape, generator=g) * 2 - 1)


# entries, scales and the gradient's values of a row of the matrix: products
# above 65504, ordinary ones, below 2^-27, and on both sides of 4 and of 2^-27
KINDS = [((300, 400), (300, 400), (5e-5, 5e-4)), ((0.3, 3), (0.5, 1.5), (0.1, 3)),
         ((1e-5, 1e-4), (1e-5, 6e-5), (1e4, 6e4)), ((0.5, 8), (1.5, 2.5), (0.1, 1)),
         ((2e-5, 2e-4), (2e-5, 4e-4), (1e3, 6e4))]


@pytest.mark.parametrize("S,E,M,K,group,used", [
    (1, 1, 90, 128, 64, None), (7, 2, 64, 200, 32, 7), (40, 3, 203, 333, 128, 37), (70, 1, 700, 130, 64, None),
    (300, 2, 331, 257, 256, 290), (500, 1, 200, 8200, 64, None), (600, 1, 4100, 130, 32, None),
])
def test_weights_of_any_size(km, S, E, M, K, group, used):  # noqa: F811
    g = torch.Generator().manual_seed(S + M)
    n, groups = len(KINDS), -(-K // group)
    lab = torch.randint(0, 16, (E, M, K), generator=g).to(torch.int32)
    table, scales = torch.zeros((E, M, 16)), torch.zeros((E, M, groups))
    gy = torch.zeros((S, M))
    for i, (entry, scale, value) in enumerate(KINDS):
        # tokens of kind i meet the rows of kind i alone; the rest of their row is zeros
        rows = torch.arange(i, M, n)
        table[:, rows] = _signed((E, len(rows), 16), *entry, g).float()
        scales[:, rows] = _signed((E, len(rows), groups), *scale, g).float()
        tok = torch.tensor(range(i, S, n + 1), dtype=torch.long)
        gy[tok[:, None], rows] = _signed((len(tok), len(rows)), *value, g).float()
        every = torch.tensor(range(n, S, n + 1), dtype=torch.long)  # ... and these meet all rows
        gy[every[:, None], rows] = _signed((len(every), len(rows)), *value, g).float()
    table[:, :, 5] = 0.0
    table, scales, gy = table.to(F16), scales.to(F16), gy.to(F16)
    W = torch.gather(table.double(), 2, lab.long()) * scales.double().repeat_interleave(group, 2)[..., :K]
    assert W.abs().max() > 65504 and W[W != 0].abs().min() < 2.0 ** -27
    cut = torch.randint(0, (used or S) + 1, (E - 1,), generator=g).sort()[0]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), cut, torch.tensor([used or S])]).to(torch.int32)
    got = km.kmeans_codes_product_grad(gy.cuda(), _packed(km, lab), table.cuda(), K, scales.cuda(), group,
                                       None if used is None else offsets.cuda(),
                                       out=torch.full((S, K), 7.0, dtype=F16, device="cuda"))
    ref, mag = _ref(gy, W, offsets, True)
    assert ref.abs().max() < 6e4
    _close(got, ref, mag, M, F16, True, "gradient")
    again = km.kmeans_codes_product_grad(gy.cuda(), _packed(km, lab), table.cuda(), K, scales.cuda(), group,
                                         None if used is None else offsets.cuda())
    assert torch.equal(got, again)


def test_one_codebook_and_scales_of_any_size(km):  # noqa: F811
    # one codebook of a matrix; the scales of a row differ by group from 2^-23 to 2^15
    S, M, K, group = 33, 200, 384, 64
    g = torch.Generator().manual_seed(5)
    lab = torch.randint(0, 16, (1, M, K), generator=g).to(torch.int32)
    table = _signed((1, 1, 16), 0.002, 1.9, g).to(F16)
    scales = _signed((1, M, K // group), 2.0 ** -23, 2.0 ** 15, g).to(F16)
    gy = _signed((S, M), 1e-4, 0.05, g).to(F16)
    W = torch.gather(table.double().expand(1, M, 16), 2, lab.long()) * scales.double().repeat_interleave(group, 2)
    got = km.kmeans_codes_product_grad(gy.cuda(), _packed(km, lab), table.cuda(), K, scales.cuda(), group)
    ref, mag = _ref(gy, W, [0, S], True)
    _close(got, ref, mag, M, F16, True, "gradient")


def test_infinite_weights_reach_their_columns_alone(km):  # noqa: F811
    S, M, K, group = 20, 100, 256, 64
    g = torch.Generator().manual_seed(6)
    lab = torch.randint(1, 16, (1, M, K), generator=g).to(torch.int32)
    lab[0, 70, 9], lab[0, 3, 200] = 0, 0
    table = _signed((1, M, 16), 0.3, 3, g).to(F16)
    table[0, :, 0] = float("inf")
    table[0, 3, 0] = float("nan")
    scales = _signed((1, M, K // group), 0.5, 1.5, g).to(F16)
    gy = _signed((S, M), 0.1, 1, g).to(F16)
    got = km.kmeans_codes_product_grad(gy.cuda(), _packed(km, lab), table.cuda(), K, scales.cuda(), group).cpu()
    hit = torch.zeros(K, dtype=torch.bool)
    hit[9] = hit[200] = True
    assert torch.isfinite(got[:, ~hit]).all() and not torch.isfinite(got[:, hit]).any()
