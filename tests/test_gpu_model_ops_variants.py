"""Variants of the operators that their launch rules take at sizes which the
other tests do not reach.  Bounds and references as there."""
import pytest
import torch
from test_gpu_codes import _case, _close, _packed, _ref
from test_gpu_lookup import U32, _check_grad, _labels, _rows, km  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,out_dtype", [(torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16),
                                             (torch.bfloat16, torch.float32), (torch.float32, torch.float32)])
@pytest.mark.parametrize("B,V,N,d,off", [
    (3, 5003, 700, 7, 0),     # 70042 or 140084 bytes a table: two or three blocks clear it, the last one 16-byte pieces and a tail
    (2, 400, 100, 3, 1),      # less than a block, tables that start anywhere
    (4, 4097, 1024, 16, 0),   # as few labels for the rows as the rule asks for
    (2, 33, 8, 1, 0), (1, 65536, 4096, 8, 0),
])
def test_table_cleared_beside_the_ranking(km, dtype, out_dtype, B, V, N, d, off):  # noqa: F811
    assert 4 * N <= V
    g = _rows((B, N, d), dtype, 1, 0.3, off)
    lab = _labels(B, N, V, 2, "skewed")
    flat = torch.full((B * V * d + 2 + off,), float("nan"), dtype=out_dtype, device="cuda")
    out = flat[1 + off:-1].view(B, V, d)
    _check_grad(km.kmeans_lookup_grad(g, lab.cuda(), V, 0.75, out=out), g, lab, V, 0.75, "cleared")
    # nothing outside the table is touched
    assert flat[:1 + off].isnan().all() and flat[-1:].isnan().all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("S,E,M,K,group", [(500, 1, 203, 8200, 64), (600, 1, 203, 8200, 32), (1000, 2, 331, 8200, 0),
                                           (700, 1, 203, 9000, 128)])
def test_gradient_of_256_token_blocks_with_ragged_rows(km, dtype, S, E, M, K, group):  # noqa: F811
    lab, table, scales, offsets, W = _case(S, E, M, K, group, dtype, "each", 3, S - 9)
    gy = torch.randn((S, M), generator=torch.Generator().manual_seed(4)).to(dtype)
    got = km.kmeans_codes_product_grad(gy.cuda(), _packed(km, lab), table.cuda(), K,
                                       None if scales is None else scales.cuda(), group, offsets.cuda())
    ref, mag = _ref(gy, W, offsets, True)
    _close(got, ref, mag, M, dtype, group > 0, "gradient")


@pytest.mark.parametrize("what", ["grad", "table", "scales and out"])
@pytest.mark.parametrize("S,M,K", [(500, 200, 8200), (90, 640, 260), (5, 1024, 136)])
def test_gradient_of_tensors_that_start_anywhere(km, S, M, K, what):  # noqa: F811
    dtype, group = torch.float16, 64
    lab, table, scales, offsets, W = _case(S, 1, M, K, group, dtype, "each", 5)
    gy = torch.randn((S, M), generator=torch.Generator().manual_seed(6)).to(dtype)

    def odd(t):
        flat = torch.empty(t.numel() + 1, dtype=dtype, device="cuda")
        flat[1:] = t.reshape(-1).cuda()
        return flat[1:].view(t.shape)

    a = odd(gy) if what == "grad" else gy.cuda()
    t = odd(table) if what == "table" else table.cuda()
    sc = odd(scales) if what == "scales and out" else scales.cuda()
    out = odd(torch.zeros((S, K))) if what == "scales and out" else None
    got = km.kmeans_codes_product_grad(a, _packed(km, lab), t, K, sc, group, None, out=out)
    ref, mag = _ref(gy, W, [0, S], True)
    _close(got, ref, mag, M, dtype, True, "gradient")


@pytest.mark.parametrize("dtype,T,top,d", [(torch.bfloat16, 9000, 4, 2049), (torch.float32, 20011, 7, 250),
                                           (torch.float16, 70001, 1, 1000)])
def test_combine_gradients_too_large_for_the_cache(km, dtype, T, top, d):  # noqa: F811
    assert T * top * d * torch.empty((), dtype=dtype).element_size() >= 1 << 27
    g = torch.Generator(device="cuda").manual_seed(7)
    S = T * top
    rows = torch.randn((S, d), generator=g, device="cuda").to(dtype)
    gy = torch.randn((T, d), generator=g, device="cuda").to(dtype)
    w = torch.rand((T, top), generator=g, device="cuda")
    # a random plan with a tenth of the choices dropped
    perm = torch.randperm(S, generator=g, device="cuda")
    live = S - S // 10
    order = torch.cat([perm[:live], torch.full((S - live,), -1, device="cuda")]).to(torch.int32)
    slots = torch.full((S,), -1, dtype=torch.int32, device="cuda")
    slots[perm[:live]] = torch.arange(live, dtype=torch.int32, device="cuda")
    grows, gw = km.kmeans_combine_grad(gy, rows, slots.view(T, top), order, w,
                                       grad_rows=torch.full((S, d), 7.0, dtype=dtype, device="cuda"))
    o = perm[:live]
    assert torch.equal(grows[:live], (w.view(-1)[o][:, None] * gy.float()[o // top]).to(dtype))
    assert not grows[live:].any()
    for k in range(top):
        sl = slots.view(T, top)[:, k]
        prod = torch.where((sl >= 0)[:, None], gy.double() * rows[sl.clamp(min=0).long()].double(), 0.0)
        assert ((gw[:, k].double() - prod.sum(1)).abs() <= (d + 1) * U32 * prod.abs().sum(1)).all()
