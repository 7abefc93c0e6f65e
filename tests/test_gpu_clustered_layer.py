"""The operators together: examples/clustered_layer.py against the same layer
written out in float64 from its tables, labels and routing.

Bounds: every stage rounds its result to bfloat16 (u = 2^-8) and the next one
carries those errors through a product of absolute values, so forward |err| <=
3 u |w| (|x| |W|) (the product, the combine, and their sums) and backward the
same with one more stage for the scaled rows, taken over absolute values.
"""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


@pytest.mark.parametrize("T", [1, 37, 1500])
def test_layer_forward_and_backward(T):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import clustered_layer
    layer = clustered_layer.ClusteredLayer(vocabulary=300, d=192, experts=5, seed=T)
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(0, 300, (T,), generator=g).to(torch.int32)
    ids[T // 3 + 1::7] = -1
    grad = torch.randn((T, 192), generator=g).to(torch.bfloat16)
    y = layer.forward(ids.cuda()).cpu().double()
    gtable, gw = (t.cpu().double() for t in layer.backward(grad.cuda()))

    W = torch.gather(layer.books.cpu().double(), 2, layer.labels.cpu().long())
    table, w = layer.table[0].cpu().double(), layer.weights[:, 0].cpu().double()
    e = layer.experts[:, 0].cpu()
    live = ids >= 0
    assert (e[~live] == -1).all() and ((e[live] >= 0) & (e[live] < 5)).all()
    x = torch.where(live[:, None], table[ids.clamp(min=0).long()], 0.0)
    h, hm = torch.zeros(T, 192, dtype=torch.float64), torch.zeros(T, 192, dtype=torch.float64)
    gx, gm = torch.zeros_like(h), torch.zeros_like(h)
    gy = grad.double()
    for k in range(5):
        m = e == k
        h[m], hm[m] = x[m] @ W[k].t(), x[m].abs() @ W[k].abs().t()
        gx[m], gm[m] = (w[m, None] * gy[m]) @ W[k], (w[m, None] * gy[m].abs()) @ W[k].abs()
    want = torch.where(live[:, None], w[:, None] * h, 0.0)
    assert ((y - want).abs() <= 3 * U * w[:, None] * hm + 1e-30).all()
    wgrad = torch.where(live, (h * gy).sum(1), 0.0)
    assert ((gw[:, 0] - wgrad).abs() <= 3 * U * (hm * gy.abs()).sum(1) + 1e-30).all()
    tgrad = torch.zeros(300, 192, dtype=torch.float64).index_add_(0, ids[live].long(), gx[live])
    tmag = torch.zeros(300, 192, dtype=torch.float64).index_add_(0, ids[live].long(), gm[live])
    assert ((gtable - tgrad).abs() <= 4 * U * tmag + 1e-30).all()
