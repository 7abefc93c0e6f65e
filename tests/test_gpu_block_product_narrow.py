"""Products with matrices of a few columns and their input's gradient, whose rows are
shorter than the 16 codes that a copy takes (bounds: test_gpu_block_product.py; what
the copies read: test_block_copy.py)."""
import pytest
import torch

from tests.test_gpu_block_product import _check, _codes, _offsets, _reference, _scales, _wide, km  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S,E,M,K,kind", [
    (3, 1, 641, 1, "even"), (3, 1, 655, 1, "even"), (5, 2, 897, 9, "even"), (40, 1, 642, 7, "even"), (200, 1, 1154, 5, "even"),
    (700, 3, 641, 2, "tail"), (2000, 1, 769, 14, "even"), (9, 1, 2049, 7, "even"), (130, 1, 1281, 1, "even")])
def test_narrow_matrices(km, S, E, M, K, kind):  # noqa: F811
    w, ws = _codes((E, M, K), 7), _scales((E, -(-M // 128), 1), 8)
    offsets, wide = _offsets(S, E, kind, 4), _wide(w, ws, 128)
    g, gs = _codes((S, M), 5), _scales((S, -(-M // 128)), 6)
    want, size = _reference(_wide(g, gs, 1), wide, offsets, True)
    got = km.kmeans_block_product_grad(g, gs, w, ws, offsets, dtype=torch.float32)
    _check(got, want, size, -(-M // 128), torch.float32)
    x, xs = _codes((S, K), 1), _scales((S, 1), 2)
    want, size = _reference(_wide(x, xs, 1), wide, offsets, False)
    _check(km.kmeans_block_product(x, xs, w, ws, offsets, dtype=torch.float32), want, size, 1, torch.float32)
