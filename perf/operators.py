"""What is measured of the operators on labels and codebooks inside a model.

Three operators, each with its gradient:

  lookup, lookup_grad    rows of a table by label, scaled, and the table's
                         gradient by sorted labels
  route, route_grad      tokens sorted by expert and back with weights, and
                         the gradients of both ways
  product, product_grad  products with 4-bit weights (a codebook of 16 values
                         a row, scales for groups of columns) of the experts'
                         segments, and the gradient of their input

`run` computes them with elementary torch operations in float32 where `own`
is false, and with this repository's entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"


def listed():
    return [
        # the tokens of one decoding step of 32 sequences
        dict(name="lookup-decode", kind="lookup", B=1, V=65536, N=32, d=2048, dtype="bf16", zipf=1.0, pad=0.0, scale=45.25),
        # a training batch of long sequences, ragged, with padding
        dict(name="lookup-batch", kind="lookup", B=1, V=131072, N=49999, d=4096, dtype="bf16", zipf=1.1, pad=0.02, scale=1.0),
        # a small fine-tuning batch: few of the vocabulary's rows get a gradient
        dict(name="lookupgrad-small", kind="lookup_grad", B=1, V=32768, N=2000, d=1024, dtype="f16", zipf=1.0, pad=0.0, scale=32.0),
        # a pretraining batch: a few words make up much of the text
        dict(name="lookupgrad-batch", kind="lookup_grad", B=1, V=131072, N=131072, d=2048, dtype="bf16", zipf=1.1, pad=0.01, scale=1.0),
        # codebooks of a product quantiser, as kmeans_fit leaves them (float32, odd width)
        dict(name="lookupgrad-codebooks", kind="lookup_grad", B=8, V=1024, N=16411, d=65, dtype="f32", zipf=0.3, pad=0.0, scale=1.0),
        # the tokens of one decoding step among 8 experts
        dict(name="route-decode", kind="route", T=24, top=2, E=8, d=4096, dtype="bf16", drop=0.0, skew=0.5),
        # a training batch among many experts, some choices dropped over capacity
        dict(name="route-batch", kind="route", T=16421, top=6, E=64, d=2048, dtype="bf16", drop=0.02, skew=0.5),
        # its gradients
        dict(name="routegrad-batch", kind="route_grad", T=8192, top=4, E=32, d=4096, dtype="bf16", drop=0.02, skew=0.5),
        # one token through one 4-bit matrix
        dict(name="product-token", kind="product", S=1, E=1, M=4096, K=4096, G=128, dtype="f16", skew=0.0, rows="each"),
        # a decoding step's sorted tokens through 16 experts
        dict(name="product-decode", kind="product", S=64, E=16, M=4096, K=2048, G=64, dtype="bf16", skew=0.5, rows="each"),
        # a prompt through 8 experts
        dict(name="product-prompt", kind="product", S=4096, E=8, M=4096, K=4096, G=128, dtype="bf16", skew=0.5, rows="each"),
        # the input's gradient in adapter training over frozen 4-bit experts
        dict(name="productgrad-batch", kind="product_grad", S=2048, E=8, M=4096, K=2048, G=64, dtype="bf16", skew=0.5, rows="each"),
    ]


def _size(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm; two of three rounded to a multiple of 8 or more."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(max(n, lo), hi)
    if n >= 64 and rng.random() < 0.67:
        n = max(lo, n // 64 * 64 if n >= 512 else n // 8 * 8)
    return n + 1 if n == 3 * 1024 else n


def _one(rng):
    kind = rng.choice(["lookup", "lookup_grad", "route", "route_grad", "product", "product_grad"])
    if kind.startswith("lookup"):
        c = dict(kind=kind, dtype=rng.choice(["f32", "f16", "bf16", "bf16"]), zipf=rng.choice([0.0, 0.5, 1.0, 1.2]),
                 pad=rng.choice([0.0, 0.02, 0.3]), scale=rng.choice([1.0, 0.125, 45.25]))
        if rng.random() < 0.3:
            return dict(c, B=rng.randint(2, 16), V=_size(rng, 16, 4096), N=_size(rng, 1, 20000), d=_size(rng, 4, 256))
        return dict(c, B=1, V=_size(rng, 64, 262144), N=_size(rng, 1, 131072), d=_size(rng, 32, 8192))
    if kind.startswith("route"):
        E = _size(rng, 2, 256)
        return dict(kind=kind, T=_size(rng, 1, 32768), top=min(E, rng.choice([1, 2, 2, 4, 6, 8])), E=E,
                    d=_size(rng, 32, 8192), dtype=rng.choice(["f32", "f16", "bf16", "bf16"]),
                    drop=rng.choice([0.0, 0.02, 0.2]), skew=rng.choice([0.0, 0.5, 2.0]))
    return dict(kind=kind, S=_size(rng, 1, 4096), E=rng.choice([1, 1, 4, 8, 16, 32]), M=_size(rng, 64, 8192),
                K=_size(rng, 64, 8192), G=rng.choice([0, 32, 64, 128, 256]), dtype=rng.choice(["f16", "bf16"]),
                skew=rng.choice([0.0, 0.5, 2.0]), rows=rng.choice(["each", "each", "shared"]))


def draw(rng):
    most = [work(c) for c in listed()]
    top_bytes, top_flops = max(w["bytes"] for w in most), max(w["flops"] for w in most)
    while True:
        c = _one(rng)
        w = work(c)
        # the plain form decodes whole matrices to float32
        whole = c["E"] * c["M"] * c["K"] if "M" in c else 0
        if w["bytes"] <= top_bytes and w["flops"] <= top_flops and whole <= 1 << 28:
            return c


def _probs(V, s):
    p = 1.0 / np.arange(1, V + 1, dtype=np.float64) ** s
    return p / p.sum()


def work(c):
    kind = c["kind"]
    es = {"f32": 4, "f16": 2, "bf16": 2}[c["dtype"]]
    if kind.startswith("lookup"):
        B, V, N, d = c["B"], c["V"], c["N"], c["d"]
        used = N * (1.0 - c["pad"])
        if kind == "lookup":  # the distinct rows, the labels, every output row
            distinct = float((1.0 - np.exp(used * np.log1p(-np.minimum(_probs(V, c["zipf"]), 1.0 - 1e-12)))).sum())
            return {"bytes": B * (distinct * d * es + 4 * N + N * d * es), "flops": B * used * d}
        # every labelled row of the gradient, the labels, the whole table's gradient
        return {"bytes": B * (used * d * es + 4 * N + V * d * es), "flops": B * used * d}
    if kind.startswith("route"):
        T, top, d = c["T"], c["top"], c["d"]
        used = T * top * (1.0 - c["drop"])
        S = T * top
        if kind == "route":  # x, the sorted rows written and read once, the combined rows, labels, slots, order, weights
            return {"bytes": T * d * es + S * d * es + used * d * es + T * d * es + S * 16, "flops": 2 * used * d}
        # gy, the rows, their gradient written, read for x's gradient, x's gradient, weights in and out
        return {"bytes": T * d * es + used * d * es + S * d * es + used * d * es + T * d * es + S * 16,
                "flops": 4 * used * d}
    S, E, M, K, G = c["S"], c["E"], c["M"], c["K"], c["G"]
    p = np.exp(c["skew"] * np.linspace(1.0, 0.0, E))
    p /= p.sum()
    live = float((1.0 - (1.0 - p) ** S).sum()) if E > 1 else 1.0
    groups = -(-K // G) if G else 0
    tab = 32 * (M if c["rows"] == "each" else 1)
    return {"bytes": live * (M * ((K + 1) // 2) + tab + 2 * M * groups) + 2 * S * K + 2 * S * M + 4 * (E + 1),
            "flops": 2.0 * S * M * K}


def _ids(c, g, B, N, V):
    if c["zipf"] > 0:
        cum = torch.from_numpy(np.cumsum(_probs(V, c["zipf"]))).to(DEV)
        u = torch.rand((B, N), generator=g, device=DEV, dtype=torch.float64)
        ids = torch.searchsorted(cum, u).clamp_(max=V - 1)
        ids = torch.randperm(V, generator=g, device=DEV)[ids]
    else:
        ids = torch.randint(0, V, (B, N), generator=g, device=DEV)
    pad = torch.rand((B, N), generator=g, device=DEV) < c["pad"]
    return torch.where(pad, -1, ids).to(torch.int32)


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt, kind = DT[c["dtype"]], c["kind"]

    def normal(*shape, std=1.0):
        # from float32 pieces, so that the largest inputs need no float32 copy of themselves
        out = torch.empty(shape, dtype=dt, device=DEV)
        flat = out.view(-1)
        for i in range(0, flat.numel(), 1 << 26):
            n = min(1 << 26, flat.numel() - i)
            flat[i:i + n] = torch.randn(n, generator=g, device=DEV) * std
        return out

    s = dict(case=c)
    if kind.startswith("lookup"):
        B, V, N, d = c["B"], c["V"], c["N"], c["d"]
        s["ids"] = _ids(c, g, B, N, V)
        if kind == "lookup":
            s["table"] = normal(B, V, d, std=0.02)
        else:
            s["grad"] = normal(B, N, d, std=0.1)
        if own:
            import exact_lloyd_means_03_amd as km
            s["km"] = km
            if kind == "lookup":
                s["out"] = torch.empty((B, N, d), dtype=dt, device=DEV)
            else:
                s["out"] = torch.empty((B, V, d), dtype=dt, device=DEV)
                s["ws"] = km.lookup_grad_workspace(B, N, d, V, dt, DEV)
        return s
    if kind.startswith("route"):
        T, top, E, d = c["T"], c["top"], c["E"], c["d"]
        logits = torch.randn((T, E), generator=g, device=DEV) + c["skew"] * torch.linspace(1, 0, E, device=DEV)
        p, e = torch.softmax(logits, 1).topk(top, 1)
        s["w"] = (p / p.sum(1, keepdim=True)).contiguous()
        dropped = torch.rand((T, top), generator=g, device=DEV) < c["drop"]
        s["experts"] = torch.where(dropped, -1, e).to(torch.int32).contiguous()
        S = T * top
        if own:
            import exact_lloyd_means_03_amd as km
            s["km"] = km
            s["ws"] = km.dispatch_workspace(T, top, E, DEV)
            s["y"] = torch.empty((T, d), dtype=dt, device=DEV)
            s["rows_out"] = torch.empty((S, d), dtype=dt, device=DEV)
            s["plan"] = (torch.empty(E + 1, dtype=torch.int32, device=DEV),
                         torch.empty((T, top), dtype=torch.int32, device=DEV),
                         torch.empty(S, dtype=torch.int32, device=DEV))
        if kind == "route":
            s["x"] = normal(T, d)
        else:
            s["gy"], s["rows"] = normal(T, d, std=0.1), normal(S, d)
            # the forward pass's plan
            offsets, slots, order = _plan(s["experts"], E)
            s["slots"], s["order"] = slots, order
            if own:
                s["gw"] = torch.empty((T, top), dtype=torch.float32, device=DEV)
        return s
    S, E, M, K, G = c["S"], c["E"], c["M"], c["K"], c["G"]
    R = M if c["rows"] == "each" else 1
    # the codes of normal weights: the nearest of 16 sorted values, the middle ones the likeliest
    labels = torch.randn((E, M, K), generator=g, device=DEV).mul_(3.0).add_(7.5).round_().clamp_(0, 15).to(torch.int32)
    centers = torch.randn((E, R, 16), generator=g, device=DEV).sort(-1)[0] * 0.02
    s["table"] = centers.to(dt)
    s["scales"] = (0.5 + torch.rand((E, M, -(-K // G)), generator=g, device=DEV)).to(dt) if G else None
    p = torch.softmax(c["skew"] * torch.linspace(1, 0, E, device=DEV), 0)
    owner = torch.multinomial(p, S, replacement=True, generator=g).sort()[0]
    counts = torch.zeros(E, dtype=torch.int64, device=DEV).index_add_(0, owner, torch.ones_like(owner))
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["x"] = normal(S, K) if kind == "product" else normal(S, M, std=0.1)
    if own:
        import exact_lloyd_means_03_amd as km
        s["km"] = km
        s["codes"] = torch.stack([km.kmeans_pack_codes(labels[e]) for e in range(E)])
        s["out"] = torch.empty((S, M if kind == "product" else K), dtype=dt, device=DEV)
        s["ws"] = km.codes_workspace(S, E, M, K, dt, DEV)
    else:
        # two codes a byte, the even column in the low half
        if K % 2:
            labels = torch.cat([labels, labels.new_zeros((E, M, 1))], -1)
        s["codes"] = (labels[..., 0::2] | (labels[..., 1::2] << 4)).to(torch.uint8)
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    c, km = s["case"], s["km"]
    kind = c["kind"]
    if kind == "lookup":
        return km.kmeans_lookup(s["table"], s["ids"], c["scale"], out=s["out"])
    if kind == "lookup_grad":
        return km.kmeans_lookup_grad(s["grad"], s["ids"], c["V"], c["scale"], out=s["out"], ws=s["ws"])
    if kind == "route":
        rows, offsets, slots, order = km.kmeans_dispatch(s["x"], s["experts"], c["E"], rows=s["rows_out"],
                                                         plan=s["plan"], ws=s["ws"])
        y = km.kmeans_combine(rows, slots, s["w"], out=s["y"])
        return rows, offsets, slots, order, y
    if kind == "route_grad":
        grows, gw = km.kmeans_combine_grad(s["gy"], s["rows"], s["slots"], s["order"], s["w"],
                                           grad_rows=s["rows_out"], grad_weights=s["gw"])
        gx = km.kmeans_combine(grows, s["slots"], None, out=s["y"])
        return grows, gw, gx
    if kind == "product":
        return km.kmeans_codes_product(s["x"], s["codes"], s["table"], c["M"], s["scales"], c["G"], s["offsets"],
                                       out=s["out"], ws=s["ws"])
    return km.kmeans_codes_product_grad(s["x"], s["codes"], s["table"], c["K"], s["scales"], c["G"], s["offsets"],
                                        out=s["out"], ws=s["ws"])


def _plan(experts, E):
    """(offsets, slots, order) of the stable sort by expert; experts outside [0, E) have none."""
    T, top = experts.shape
    flat = experts.reshape(-1).long()
    ok = (flat >= 0) & (flat < E)
    key = torch.where(ok, flat, E)
    perm = torch.sort(key, stable=True)[1]
    counts = torch.zeros(E + 1, dtype=torch.int64, device=flat.device).index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([counts.new_zeros(1), counts[:E].cumsum(0)])
    at = torch.arange(T * top, device=flat.device)
    slots = torch.empty_like(at).index_copy_(0, perm, at)
    slots = torch.where(ok, slots, -1).view(T, top)
    order = torch.where(at < offsets[E], perm, -1)
    return offsets.to(torch.int32), slots.to(torch.int32), order.to(torch.int32)


def _gathered(rows, index, scale=None):
    """float32 rows[index], zero where the index is negative, each times its scale."""
    out = rows[index.clamp(min=0).long()].float()
    if scale is not None:
        out = out * scale.unsqueeze(-1)
    return torch.where((index >= 0).unsqueeze(-1), out, 0.0)


def _decoded(s, e):
    """float32 weights [M, K] of expert e."""
    c = s["case"]
    b = s["codes"][e]
    codes = torch.stack([b & 15, b >> 4], -1).view(c["M"], -1)[:, :c["K"]].long()
    w = s["table"][e].float().expand(c["M"], 16).gather(1, codes)
    if s["scales"] is not None:
        w = w * s["scales"][e].float().repeat_interleave(c["G"], 1)[:, :c["K"]]
    return w


def _run_plain(s):
    c = s["case"]
    kind = c["kind"]
    dt = DT[c["dtype"]]
    if kind == "lookup":
        ids = s["ids"]
        return torch.stack([(_gathered(s["table"][b], ids[b]) * c["scale"]).to(dt) for b in range(c["B"])])
    if kind == "lookup_grad":
        out = torch.empty((c["B"], c["V"], c["d"]), dtype=dt, device=DEV)
        for b in range(c["B"]):
            ids = s["ids"][b].long()
            key = torch.where((ids >= 0) & (ids < c["V"]), ids, c["V"])
            acc = torch.zeros((c["V"] + 1, c["d"]), device=DEV)
            acc.index_add_(0, key, s["grad"][b].float())
            out[b] = (acc[:c["V"]] * c["scale"]).to(dt)
        return out
    if kind == "route":
        offsets, slots, order = _plan(s["experts"], c["E"])
        rows = _gathered(s["x"], torch.where(order >= 0, order // c["top"], -1)).to(dt)
        y = 0.0
        for k in range(c["top"]):
            y = y + _gathered(rows, slots[:, k], s["w"][:, k])
        return rows, offsets, slots, order, y.to(dt)
    if kind == "route_grad":
        slots, order, w = s["slots"], s["order"], s["w"]
        token = torch.where(order >= 0, order // c["top"], -1)
        grows = _gathered(s["gy"], token, w.reshape(-1)[order.clamp(min=0).long()]).to(dt)
        gy = s["gy"].float()
        gw = torch.stack([(gy * _gathered(s["rows"], slots[:, k])).sum(1) for k in range(c["top"])], 1)
        gx = 0.0
        for k in range(c["top"]):
            gx = gx + _gathered(grows, slots[:, k])
        return grows, gw, gx.to(dt)
    ends = s["offsets"].tolist()
    out = torch.zeros((c["S"], c["M"] if kind == "product" else c["K"]), device=DEV)
    for e in range(c["E"]):
        if ends[e + 1] > ends[e]:
            x = s["x"][ends[e]:ends[e + 1]].float()
            w = _decoded(s, e)
            out[ends[e]:ends[e + 1]] = x @ (w.t() if kind == "product" else w)
    return out.to(dt)


def exact(c, seed):
    """The definitions in float64, on the plain form's inputs."""
    global own
    kept, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = kept
    kind = c["kind"]
    if kind == "lookup":
        out = torch.zeros((c["B"], c["N"], c["d"]), dtype=torch.float64, device=DEV)
        b, i = torch.nonzero(s["ids"] >= 0, as_tuple=True)
        out[b, i] = s["table"][b, s["ids"][b, i].long()].double() * c["scale"]
        return out
    if kind == "lookup_grad":
        out = torch.zeros((c["B"] * c["V"], c["d"]), dtype=torch.float64, device=DEV)
        b, i = torch.nonzero(s["ids"] >= 0, as_tuple=True)
        out.index_add_(0, b * c["V"] + s["ids"][b, i].long(), s["grad"][b, i].double() * c["scale"])
        return out.view(c["B"], c["V"], c["d"])
    if kind == "route":
        # dispatched rows are copies, so y is the weighted sum of the token itself
        keep = (s["experts"] >= 0).double()
        y = s["x"].double() * (s["w"].double() * keep).sum(1, keepdim=True)
        flat = s["experts"].reshape(-1).cpu().numpy()
        live = np.nonzero(flat >= 0)[0]
        by = live[np.lexsort((live, flat[live]))]
        rows = torch.zeros((c["T"] * c["top"], c["d"]), dtype=torch.float64, device=DEV)
        rows[:len(by)] = s["x"].double()[torch.from_numpy(by // c["top"]).to(DEV)]
        return rows, None, None, None, y
    if kind == "route_grad":
        T, top, d = c["T"], c["top"], c["d"]
        grows = torch.zeros((T * top, d), dtype=torch.float64, device=DEV)
        gw = torch.zeros((T, top), dtype=torch.float64, device=DEV)
        gx = torch.zeros((T, d), dtype=torch.float64, device=DEV)
        gy = s["gy"].double()
        for k in range(top):
            t = torch.nonzero(s["slots"][:, k] >= 0).view(-1)
            p = s["slots"][t, k].long()
            grows[p] = gy[t] * s["w"][t, k].double().unsqueeze(1)
            gw[t, k] = (gy[t] * s["rows"][p].double()).sum(1)
            # the rows' gradient is handed on in its own type
            gx[t] += grows[p].to(DT[c["dtype"]]).double()
        return grows, gw, gx
    M, K, G = c["M"], c["K"], c["G"]
    out = torch.zeros((c["S"], M if kind == "product" else K), dtype=torch.float64, device=DEV)
    ends = s["offsets"].cpu().numpy()
    column = torch.arange(K, device=DEV)
    row = torch.arange(M, device=DEV).unsqueeze(1)
    for e in range(c["E"]):
        a, z = int(ends[e]), int(ends[e + 1])
        if a == z:
            continue
        code = (s["codes"][e].long()[:, column // 2] >> (4 * (column % 2))) & 15
        w = s["table"][e].double()[row if c["rows"] == "each" else torch.zeros_like(row), code]
        if G:
            w *= s["scales"][e].double()[:, column // G]
        out[a:z] = torch.matmul(s["x"][a:z].double(), w.t().contiguous() if kind == "product" else w)
    return out
