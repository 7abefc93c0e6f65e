"""A product under autograd takes and refuses the arguments that it takes and refuses
without."""
import pytest
import torch

from tests.test_gpu_block_product import _codes, _scales, km  # noqa: F401

pytestmark = pytest.mark.gpu


def _case(S=300, M=512, K=2049):
    x = torch.randn((S, K), generator=torch.Generator().manual_seed(1)).cuda()
    return x, _codes((M, K), 2), _scales((-(-M // 128), -(-K // 128)), 3)


@pytest.mark.parametrize("recorded", [False, True])
def test_scales_beside_wide_rows(km, recorded):  # noqa: F811
    x, w, ws = _case()
    with pytest.raises(ValueError, match="scales of x go with 8-bit codes"):
        km.kmeans_block_product(x.requires_grad_(recorded), _scales((300, 17), 4), w, ws)


@pytest.mark.parametrize("recorded", [False, True])
def test_the_workspace_given_is_the_one_used(km, recorded):  # noqa: F811
    x, w, ws = _case()
    n = km.block_product_workspace(300, 1, 512, 2049, x.device)
    assert n.numel() > 256  # (the sums of splits: these shapes need one)
    n.fill_(0)
    y = km.kmeans_block_product(x.requires_grad_(recorded), None, w, ws, ws=n)
    assert n.any() and torch.equal(y.detach(), km.kmeans_block_product(x.detach(), None, w, ws))
    with pytest.raises(km.KMeansError, match="workspace"):
        km.kmeans_block_product(x, None, w, ws, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError, match="workspace"):
        km.kmeans_block_product(x, None, w, ws, ws=n.float())
