"""Exact Lloyd k-means for AMD Instinct MI355X (gfx950).

The computation lives in libkmeans_mi355x.so (hand-written HIP kernels behind
the C ABI of include/kmeans.h); this package only marshals torch tensors into
that ABI.
"""
from .api import (  # noqa: F401
    emeans_steps, kmeans_assign, kmeans_emeans, kmeans_fit, kmeans_fit_static, kmeans_fit_stream,
    kmeans_optimal_1d, kmeans_sort_labels, kmeans_update, workspace, workspace_bytes,
)
from .api import (  # noqa: F401
    codes_workspace, dispatch_workspace, kmeans_codes_product, kmeans_codes_product_grad, kmeans_combine,
    kmeans_combine_grad, kmeans_dispatch, kmeans_lookup, kmeans_lookup_grad, kmeans_pack_codes,
    lookup_grad_workspace,
)
from ._lib import KMeansError, load  # noqa: F401

__all__ = ["emeans_steps", "kmeans_assign", "kmeans_emeans", "kmeans_fit", "kmeans_fit_static", "kmeans_fit_stream",
           "kmeans_optimal_1d", "kmeans_sort_labels", "kmeans_update", "workspace", "workspace_bytes",
           "kmeans_lookup", "kmeans_lookup_grad", "lookup_grad_workspace", "kmeans_dispatch", "kmeans_combine",
           "kmeans_combine_grad", "dispatch_workspace", "kmeans_pack_codes", "kmeans_codes_product",
           "kmeans_codes_product_grad", "codes_workspace", "KMeansError", "load"]
