"""A layer of experts built from what clustering leaves: labels and codebooks.

Token ids are looked up in a table; the tokens' clusters (kmeans_fit, then
kmeans_assign) are their experts; every expert's weight matrix is clustered row
by row to 16 values (kmeans_fit over scalar rows) and used as 4-bit labels; the
tokens are sorted by expert, multiplied, and brought back with weights; the
gradient goes the same way back to the table.

    python examples/clustered_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import exact_lloyd_means_03_amd as km  # noqa: E402


class ClusteredLayer:
    """T token ids -> T rows of width d, through E experts of 4-bit weights."""

    def __init__(self, vocabulary=1000, d=256, experts=8, dtype=torch.bfloat16, seed=0, iterations=8):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.d, self.E = d, experts
        self.table = torch.randn((1, vocabulary, d), generator=g, device="cuda").to(dtype)
        # experts: clusters of the table's rows
        centers, _, _, _ = km.kmeans_fit(self.table, self.table[:, :experts].float().contiguous(), iterations)
        self.centers = centers
        # weights: every row of every matrix clustered to 16 values, from an even grid
        w = torch.randn((experts * d, d, 1), generator=g, device="cuda") / d ** 0.5
        lo, hi = w.amin(1, keepdim=True), w.amax(1, keepdim=True)
        grid = lo + (hi - lo) * torch.linspace(0, 1, 16, device="cuda").view(1, 16, 1)
        books, _, _, _ = km.kmeans_fit(w, grid.contiguous(), iterations)
        labels, _, _ = km.kmeans_assign(w, books)
        self.labels = labels.view(experts, d, d)
        self.codes = torch.stack([km.kmeans_pack_codes(m) for m in self.labels])
        self.books = books.view(experts, d, 16).to(dtype)

    def forward(self, ids):
        """ids [T] int32 (negative: padding, whose row is zeros) -> [T, d]."""
        T = ids.shape[0]
        x = km.kmeans_lookup(self.table, ids.view(1, T))
        cluster, distance, _ = km.kmeans_assign(x, self.centers, min_dist=True)
        # padding goes to no expert
        self.experts = torch.where(ids >= 0, cluster[0], -1).view(T, 1)
        self.weights = (1.0 / (1.0 + distance[0] / self.d)).view(T, 1).contiguous()
        rows, self.offsets, self.slots, self.order = km.kmeans_dispatch(x[0], self.experts, self.E)
        self.rows = km.kmeans_codes_product(rows, self.codes, self.books, self.d, offsets=self.offsets)
        self.ids = ids
        return km.kmeans_combine(self.rows, self.slots, self.weights)

    def backward(self, grad):
        """grad [T, d] -> (gradient of the table [V, d] float32, of the weights
        [T, 1]); the clusters and the 4-bit matrices are held."""
        grows, gweights = km.kmeans_combine_grad(grad, self.rows, self.slots, self.order, self.weights)
        grows = km.kmeans_codes_product_grad(grows, self.codes, self.books, self.d, offsets=self.offsets)
        gx = km.kmeans_combine(grows, self.slots, None)
        gtable = torch.empty(self.table.shape, dtype=torch.float32, device="cuda")
        km.kmeans_lookup_grad(gx[None], self.ids.view(1, -1), self.table.shape[1], out=gtable)
        return gtable[0], gweights


def main():
    layer = ClusteredLayer()
    for T in (1, 37, 4096):
        ids = torch.randint(-1, 1000, (T,), device="cuda", dtype=torch.int32)
        y = layer.forward(ids)
        gtable, gweights = layer.backward(y)
        used = (layer.offsets[1:] > layer.offsets[:-1]).sum().item()
        print(f"{T} tokens, {used} experts used: |y| {y.float().norm().item():.4g}, "
              f"|table gradient| {gtable.norm().item():.4g}, |weight gradient| {gweights.norm().item():.4g}")


if __name__ == "__main__":
    main()
