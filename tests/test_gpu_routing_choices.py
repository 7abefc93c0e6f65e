"""kmeans_dispatch around the numbers of choices at which it changes its way of
sorting, against the plan written out."""
import numpy as np
import pytest
import torch
from test_gpu_routing import _experts, _plan, _rows, km  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,top", [(512, 8), (513, 8), (113, 9), (114, 9), (64, 16), (65, 16), (15, 17), (16, 17),
                                   (10, 24), (11, 24), (1, 25), (1, 300), (0, 4096), (1, 4096)])
def test_dispatch_of_many_choices(km, T, top):  # noqa: F811
    E, d = 37, 24
    x = _rows((T, d), torch.bfloat16, 2)
    e = _experts(T, top, E, "dropped") if T else torch.zeros((0, top), dtype=torch.int32)
    rows, *got = km.kmeans_dispatch(x, e.cuda(), E, rows=torch.full((T * top, d), 7.0, dtype=x.dtype, device="cuda"))
    offsets, slots, order = _plan(e, E)
    for a, b in zip(got, (offsets, slots, order)):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    n = int(offsets[-1])
    want = torch.zeros((T * top, d), dtype=x.dtype)
    want[:n] = x.cpu()[torch.from_numpy(order[:n] // top).long()]
    assert torch.equal(rows.cpu(), want)
