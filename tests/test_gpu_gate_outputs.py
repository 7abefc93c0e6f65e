"""What kmeans_gate returns are tensors of their own: a training loop scales the
routing weights and the balance loss in place, and keeps the loss of many steps."""
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


def _logits(T, E):
    return torch.randn((T, E), generator=torch.Generator().manual_seed(T)).cuda()


@pytest.mark.parametrize("T,E,top", [(1, 1, 1), (24, 8, 2), (3000, 64, 6)])
def test_scaled_in_place_while_training(km, T, E, top):
    l = _logits(T, E)
    gw = torch.randn((T, top), generator=torch.Generator().manual_seed(1)).cuda()
    x = l.clone().requires_grad_()
    experts, weights, counts, _, loss = km.kmeans_gate(x, top)
    weights *= 2.5  # (autograd scales its gradients by the same float32 products)
    loss *= 0.5
    ((weights * gw).sum() + loss).backward()
    want = km.kmeans_gate_grad(l, experts, counts, gw * 2.5, torch.full((), 0.5, device="cuda"))
    assert torch.equal(x.grad, want)


@pytest.mark.parametrize("recorded", [False, True])
@pytest.mark.parametrize("T,E,top", [(1, 1, 1), (24, 8, 2), (3000, 64, 6), (0, 8, 2)])
def test_an_output_keeps_its_own_memory_alone(km, T, E, top, recorded):
    for t in km.kmeans_gate(_logits(T, E).requires_grad_(recorded), top):
        assert t.untyped_storage().nbytes() == t.numel() * t.element_size() and not t._is_view()


def test_scaled_by_a_factor_that_is_trained(km):
    # a frozen gate's weights, made without recording, become part of a recorded product
    factor = torch.ones((), device="cuda", requires_grad=True)
    with torch.no_grad():
        _, weights, _, _, loss = km.kmeans_gate(_logits(24, 8), 2)
    total = weights.sum() + loss
    weights.mul_(factor)
    loss.mul_(factor)
    (weights.sum() + loss).backward()
    assert abs(factor.grad.item() - total.item()) <= 64 * 2.0 ** -24 * total.item()
