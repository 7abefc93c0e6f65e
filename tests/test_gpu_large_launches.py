"""Calls of more blocks than one launch takes: they are launched in parts, and
the rows on both sides of a part's end and the last ones are right.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BLOCKS = 1 << 22  # of a launch (kLaunchBlocks in csrc/rows.h)


@pytest.fixture()
def km():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import exact_lloyd_means_03_amd as km
    km.load()
    torch.cuda.empty_cache()
    yield km
    torch.cuda.empty_cache()


def _around(*places):
    return [q for p in places for q in (p - 2, p - 1, p, p + 1) if q >= 0]


def test_lookup(km):
    # 1024 chunks of 16 bytes a block, rows of 3
    V, d, N = 1000, 24, BLOCKS * 1024 // 3 + 1000
    table = torch.randn((1, V, d), device="cuda").to(torch.bfloat16)
    lab = torch.arange(N, dtype=torch.int32, device="cuda").remainder_(V)[None]
    out = km.kmeans_lookup(table, lab)
    at = torch.tensor(_around(1, BLOCKS * 1024 // 3, N - 1)[:-1], device="cuda")
    assert torch.equal(out[0, at], table[0, at % V])


def test_dispatch_and_combine(km):
    # 256 chunks a block, rows of one
    T, d = BLOCKS * 256 + 300, 8
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda").random_(-8, 8)
    e = torch.arange(T, dtype=torch.int32, device="cuda").bitwise_and_(1)[:, None].contiguous()
    rows, offsets, slots, order = km.kmeans_dispatch(x, e, 2)
    half = (T + 1) // 2
    assert offsets.tolist() == [0, half, T]
    for t in _around(2, BLOCKS * 256, T - 2):
        p = t // 2 + (half if t % 2 else 0)
        assert int(slots[t, 0]) == p and int(order[p]) == t and torch.equal(rows[p], x[t])
    y = km.kmeans_combine(rows, slots, None)
    at = torch.tensor(_around(2, BLOCKS * 256, T - 2), device="cuda")
    assert torch.equal(y[at], x[at])


@pytest.mark.parametrize("T,d", [(BLOCKS * 4 + 5, 1), (BLOCKS + 3, 1032)])
def test_combine_gradients(km, T, d):
    # four tokens a block, or one
    gy = torch.empty((T, d), dtype=torch.bfloat16, device="cuda").random_(-4, 5)
    rows = torch.empty((T, d), dtype=torch.bfloat16, device="cuda").random_(-4, 5)
    slots = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")[:, None].contiguous()
    order = slots.view(-1).clone()
    w = torch.full((T, 1), 0.5, device="cuda")
    grows, gw = km.kmeans_combine_grad(gy, rows, slots, order, w)
    part = BLOCKS * 4 if d == 1 else BLOCKS
    at = torch.tensor(_around(2, part, T - 2), device="cuda")
    assert torch.equal(grows[T - 1 - at].float(), gy[at].float() * 0.5)
    assert torch.equal(gw[at, 0], (gy[at].float() * rows[T - 1 - at].float()).sum(1))  # (small whole numbers)


def test_pack_codes(km):
    # 2048 codes a block: tiles of 16 rows by 128 columns
    M, K = 1 << 20, 8320
    assert M * K > BLOCKS * 2048
    labels = torch.empty((M, K), dtype=torch.int32, device="cuda").random_(0, 16)
    codes = km.kmeans_pack_codes(labels)
    small = torch.cat([labels[:16], labels[M // 2:M // 2 + 16], labels[-32:]])
    want = km.kmeans_pack_codes(small)
    row = BLOCKS * 2048 // (16 * K)  # the row of tiles in which the second launch begins
    assert torch.equal(codes[[0, M // 32, M // 16 - 2, M // 16 - 1]], want)
    assert torch.equal(codes[row - 1:row + 2], km.kmeans_pack_codes(labels[16 * (row - 1):16 * (row + 2)].contiguous()))
