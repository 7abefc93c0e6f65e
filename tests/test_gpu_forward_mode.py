"""Forward-mode derivatives, which no operator has, are refused where they would be
lost: a dual tensor does not require a gradient, and results without a tangent would
pass for constants."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def km():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import exact_lloyd_means_03_amd as km
    km.load()
    return km


def _calls(km):
    """name -> (a call of one differentiable tensor, that tensor)."""
    half, f32 = torch.ones((4, 128), dtype=torch.bfloat16, device="cuda"), torch.ones((4, 128), device="cuda")
    e = torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    codes, scales = km.kmeans_quantize(torch.ones((128, 128), device="cuda"), 128)
    offsets, slots, order = km.kmeans_plan(e, 1)
    experts, weights, counts, _, _ = km.kmeans_gate(f32, 2)
    packed = km.kmeans_pack_codes(torch.zeros((16, 128), dtype=torch.int32, device="cuda"))
    table = torch.ones((1, 16), dtype=torch.bfloat16, device="cuda")
    ones = torch.ones(128, device="cuda")
    return {
        "quantize": (lambda x: km.kmeans_quantize(x), f32),
        "norm": (lambda x: km.kmeans_norm(x), f32),
        "norm, weight": (lambda w: km.kmeans_norm(f32, w), ones),
        "norm, residual": (lambda r: km.kmeans_norm(f32, None, residual=r), f32),
        "norm_quantize": (lambda x: km.kmeans_norm_quantize(x), f32),
        "norm_grad": (lambda g: km.kmeans_norm_grad(g, f32), f32),
        "gate": (lambda x: km.kmeans_gate(x, 2), f32),
        "gate_grad": (lambda g: km.kmeans_gate_grad(f32, experts, counts, g), weights),
        "block_product": (lambda x: km.kmeans_block_product(x, None, codes, scales), f32),
        "block_product, scales": (lambda s: km.kmeans_block_product(f32, None, codes, s), scales),
        "block_product_grad": (lambda g: km.kmeans_block_product_grad(g, None, codes, scales), f32),
        "lookup": (lambda t: km.kmeans_lookup(t, e.view(1, 4)), f32[None].contiguous()),
        "lookup_grad": (lambda g: km.kmeans_lookup_grad(g, e.view(1, 4), 4), f32[None].contiguous()),
        "dispatch": (lambda x: km.kmeans_dispatch(x, e, 1), f32),
        "combine": (lambda r: km.kmeans_combine(r, slots), f32),
        "combine, weights": (lambda w: km.kmeans_combine(f32, slots, w), torch.ones((4, 1), device="cuda")),
        "combine_grad": (lambda g: km.kmeans_combine_grad(g, f32, slots, order, torch.ones((4, 1), device="cuda")), f32),
        "codes_product": (lambda x: km.kmeans_codes_product(x, packed, table, 16), half),
        "codes_product, table": (lambda t: km.kmeans_codes_product(half, packed, t, 16), table),
        "codes_product_grad": (lambda g: km.kmeans_codes_product_grad(g, packed, table, 128), half[:, :16].contiguous()),
    }


def test_dual_tensors_are_refused(km):
    lost = []
    for name, (call, t) in _calls(km).items():
        with fwd.dual_level():
            call(t)  # (a tensor without a tangent is one as before)
            dual = fwd.make_dual(t, torch.ones_like(t))
            for recording in (True, False):
                with torch.set_grad_enabled(recording):
                    try:
                        call(dual)
                        lost.append((name, recording))
                    except ValueError as e:
                        assert "forward-mode" in str(e), (name, e)
        call(t)
    assert not lost
