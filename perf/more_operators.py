"""Measured cases of the experts' bf16 products with their gradients, and of the gradient norm with clipping.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges,
``prepare`` makes a program's data, ``run`` makes one pass: through plain
torch operations where ``own`` is false, through this library's entry points
where it is true.  ``exact`` gives the same values from the definitions in 64
bits, and ``work`` what a pass cannot do without.

The operators, for the R rows of a dispatch plan (rows offsets[e] to
offsets[e + 1] are expert e's, the rows from offsets[E] on are nobody's):

    product       D[r]  = act(alpha * A[r] * W_e^T), zeros in nobody's rows
    rows_grad     dA[r] = alpha * dD[r] * W_e,       zeros in nobody's rows
    weights_grad  dW_e  = alpha * sum over e's rows of dD[r]^T A[r]  (+ beta * dW_e)
    norm          sqrt(sum of the squares of all values of all tensors)
    clip          the norm, and every tensor times min(1, max_norm / norm)
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
PRODUCTS = ("product", "rows_grad", "weights_grad")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # A decode step of 16 sequences through 2 of 8 experts: the experts' matrices are read once.
        dict(name="product_decode", kind="product", T=16, k=2, E=8, N=4096, K=4096, drop=0.0, act="none", out="bf16"),
        # One prompt through 8 of 128 experts: about 512 rows for each, some experts liked more.
        dict(name="product_prompt", kind="product", T=8192, k=8, E=128, N=4096, K=2048, drop=0.0, act="silu",
             out="bf16"),
        # A ragged batch whose full experts dropped some slots, with an fp32 result.
        dict(name="product_ragged", kind="product", T=3001, k=3, E=61, N=5000, K=2000, drop=0.05, act="none",
             out="f32"),
        # The training step's way back through eight wide experts.
        dict(name="rows_grad_training", kind="rows_grad", T=8192, k=2, E=8, N=8192, K=4096, drop=0.02, out="bf16"),
        # The same for a short batch and many experts: a few rows each.
        dict(name="rows_grad_short", kind="rows_grad", T=130, k=4, E=64, N=2048, K=2000, drop=0.0, out="bf16"),
        # The eight wide experts' own gradients.
        dict(name="weights_grad_training", kind="weights_grad", T=8192, k=2, E=8, N=8192, K=4096, drop=0.02,
             beta=0.0, out="bf16"),
        # Gradients of many experts added to fp32 sums over micro-batches: as much memory traffic as product.
        dict(name="weights_grad_added", kind="weights_grad", T=4096, k=4, E=64, N=2048, K=2048, drop=0.0, beta=1.0,
             out="f32"),
        # A short batch: experts with a few rows, some with none.
        dict(name="weights_grad_short", kind="weights_grad", T=100, k=2, E=61, N=1000, K=2000, drop=0.05, beta=0.0,
             out="bf16"),
        # The gradients of a small layer: sixteen tensors, latency.
        dict(name="norm_small", kind="norm", tensors=16, values=1 << 20, dtype="f32"),
        # Those of the eight wide experts' two matrices and a few hundred small tensors.
        dict(name="norm_large", kind="norm", tensors=300, values=8 * 8192 * 4096 * 2, dtype="bf16"),
        # A small model's gradients, clipped.
        dict(name="clip_small", kind="clip", tensors=40, values=3000001, dtype="bf16", to="bf16", part=0.25),
        # fp32 sums of a layer of experts, clipped and rounded for the optimiser.
        dict(name="clip_large", kind="clip", tensors=200, values=64 * 2048 * 2048, dtype="f32", to="bf16", part=0.5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["product", "rows_grad", "weights_grad", "norm", "clip"])
    if kind in PRODUCTS:
        while True:
            c = dict(kind=kind, T=_log(rng, 1, 8192), k=rng.randint(1, 8), E=rng.choice([8, 16, 61, 64, 128]),
                     N=_log(rng, 64, 8192), K=_log(rng, 64, 8192), drop=rng.choice([0.0, 0.0, 0.02, 0.3]),
                     out=rng.choice(["bf16", "bf16", "f32"]))
            if kind == "product":
                c["act"] = rng.choice(["none", "silu"])
            if kind == "weights_grad":
                c["beta"] = rng.choice([0.0, 1.0])
            if (c["E"] * c["N"] * c["K"] <= 64 * 2048 * 2048 and c["T"] * c["k"] * c["N"] * c["K"] <= 16384 * 8192 * 4096
                    and c["T"] * c["k"] * max(c["N"], c["K"]) <= 65536 * 4096):
                return c
    c = dict(kind=kind, tensors=_log(rng, 1, 300), values=_log(rng, 1000, 64 * 2048 * 2048),
             dtype=rng.choice(["bf16", "f32"]))
    if kind == "clip":
        c.update(to=rng.choice(["bf16", "f32"]), part=rng.choice([0.1, 0.5, 2.0]))
    return c


# ------------------------------------------------------------------ inputs
def _matrix(shape, gen, scale=1.0):
    """bf16 values whose rows start on 16 bytes."""
    pad = -(-shape[-1] // 8) * 8
    buf = torch.randn(*shape[:-1], pad, generator=gen, device=gen.device, dtype=torch.float32)
    return buf.mul_(scale).bfloat16()[..., :shape[-1]]


def _plan(c, gen):
    """offsets, slot_row and row_token of a router's choice: k different experts for each token, some slots dropped."""
    dev, T, k, E = gen.device, c["T"], c["k"], c["E"]
    liked = torch.randn(E, generator=gen, device=dev) * 0.5
    ids = torch.topk(torch.randn(T, E, generator=gen, device=dev) + liked, k, dim=1).indices
    lost = torch.rand(T, k, generator=gen, device=dev) < c["drop"]
    key = torch.where(lost, torch.full_like(ids, E), ids).reshape(-1)
    by, order = torch.sort(key, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(T * k, device=dev)
    offsets = torch.searchsorted(by, torch.arange(E + 1, device=dev))
    slot_row = torch.where(key < E, row, torch.full_like(row, -1)).view(T, k)
    row_token = torch.where(by < E, order // k, torch.full_like(order, -1))
    return offsets.int(), slot_row.int(), row_token.int()


def _sizes(c):
    """Lengths of a model's gradient tensors: one matrix in four, the rest small and odd, `values` together."""
    n, total = c["tensors"], c["values"]
    weights = [1.0 if i % 4 == 0 else 0.0005 * (1 + i % 7) for i in range(n)]
    scale = total / sum(weights)
    sizes = [max(1, int(w * scale)) for w in weights]
    sizes[0] = max(1, sizes[0] + total - sum(sizes))
    return sizes


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    if own:
        import tensor_core_dense_tn_gb300 as g
    s = dict(case=c)
    if c["kind"] in PRODUCTS:
        s["plan"] = _plan(c, gen)
        if own:             # the plan that the layer's dispatch filled
            s["own_plan"] = g.ExpertPlan.of(*s["plan"], experts=c["E"])
        R, E, N, K = c["T"] * c["k"], c["E"], c["N"], c["K"]
        if c["kind"] == "product":
            s["A"], s["W"] = _matrix((R, K), gen), _matrix((E, N, K), gen, K ** -0.5)
        elif c["kind"] == "rows_grad":
            s["dD"], s["W"] = _matrix((R, N), gen, 0.01), _matrix((E, N, K), gen, K ** -0.5)
        else:
            s["dD"], s["A"] = _matrix((R, N), gen, 0.01), _matrix((R, K), gen)
            if c["beta"]:   # the sums so far, and a place for the new ones (so that a pass can be made again)
                s["sum"] = (0.01 * torch.randn(E, N, K, generator=gen, device=dev)).to(DTYPES[c["out"]])
                s["new"] = torch.empty_like(s["sum"])
        return s
    s["tensors"] = [(torch.randn(n, generator=gen, device=dev) * 10.0 ** (-2 - i % 3)).to(DTYPES[c["dtype"]])
                    for i, n in enumerate(_sizes(c))]
    if c["kind"] == "clip":
        s["max_norm"] = c["part"] * 0.01 * math.sqrt(c["values"] * 0.337)    # about `part` of the norm
        s["flat"], s["to"] = _bucket([t.numel() for t in s["tensors"]], DTYPES[c["to"]], dev)
    return s


def _bucket(sizes, dtype, dev):
    """One buffer for all tensors, as optimisers keep it, and their places in it, each on 64 elements; zeros between."""
    starts, end = [], 0
    for n in sizes:
        starts.append(end)
        end += -(-n // 64) * 64
    flat = torch.zeros(end, dtype=dtype, device=dev)
    return flat, [flat[at:at + n] for at, n in zip(starts, sizes)]


# ------------------------------------------------------------------ plain forms
def _act(x, act):
    return x / (1.0 + torch.exp(-x)) if act == "silu" else x


def _plain_products(s):
    c = s["case"]
    out, E, R = DTYPES[c["out"]], c["E"], c["T"] * c["k"]
    bounds = s["plan"][0].tolist()
    if c["kind"] == "weights_grad":
        dW = torch.zeros(E, c["N"], c["K"], dtype=out, device=s["A"].device)
        for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
            total = s["dD"][lo:hi].float().t() @ s["A"][lo:hi].float()
            if c["beta"]:
                total = total + c["beta"] * s["sum"][e].float()
            dW[e] = total.to(out)
        return dict(dW=dW)
    forward = c["kind"] == "product"
    X, W = s["A"] if forward else s["dD"], s["W"]
    D = torch.zeros(R, c["N"] if forward else c["K"], dtype=out, device=X.device)
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if hi > lo:
            M = W[e].float()
            D[lo:hi] = _act(X[lo:hi].float() @ (M.t() if forward else M), c.get("act")).to(out)
    return dict(D=D) if forward else dict(dA=D)


def _plain_norm(tensors):
    return torch.stack([t.float().square().sum(dtype=torch.float64) for t in tensors]).sum().sqrt().float()


def _plain(s):
    c = s["case"]
    if c["kind"] in PRODUCTS:
        return _plain_products(s)
    norm = _plain_norm(s["tensors"])
    if c["kind"] == "norm":
        return dict(norm=norm)
    part = torch.clamp(s["max_norm"] / norm, max=1.0)
    for t, to in zip(s["tensors"], s["to"]):
        to.copy_(t.float() * part)
    return dict(norm=norm, clipped=s["flat"])


# ------------------------------------------------------------------ one pass
def run(state):
    if not own:
        return _plain(state)
    import tensor_core_dense_tn_gb300 as g
    s, c = state, state["case"]
    kind = c["kind"]
    if kind == "product":
        act = g.ACT_SILU if c["act"] == "silu" else g.ACT_NONE
        return dict(D=g.gemm_experts(s["A"], s["W"], s["own_plan"], activation=act, out_dtype=DTYPES[c["out"]]))
    if kind == "rows_grad":
        return dict(dA=g.gemm_experts_backward_a(s["dD"], s["W"], s["own_plan"], out_dtype=DTYPES[c["out"]]))
    if kind == "weights_grad":
        if c["beta"]:
            return dict(dW=g.gemm_experts_backward_w(s["dD"], s["A"], s["own_plan"], beta=c["beta"], C=s["sum"],
                                                     out=s["new"]))
        return dict(dW=g.gemm_experts_backward_w(s["dD"], s["A"], s["own_plan"], out_dtype=DTYPES[c["out"]]))
    if kind == "norm":
        return dict(norm=g.grad_norm(s["tensors"]))
    return dict(norm=g.clip_grad_norm(s["tensors"], s["max_norm"], out=s["to"]), clipped=s["flat"])


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    c = case
    s = prepare(case, seed)
    f64 = torch.float64
    if c["kind"] in PRODUCTS:
        # every row's expert from the plan's definition: the number of experts that end at or before it
        ends = s["plan"][0][1:].long()
        row = torch.arange(c["T"] * c["k"], device=ends.device)
        expert = (ends[None, :] <= row[:, None]).sum(1)
        if c["kind"] == "weights_grad":
            dW = torch.empty(c["E"], c["N"], c["K"], dtype=f64, device=row.device)
            for e in range(c["E"]):
                mine = torch.nonzero(expert == e)[:, 0]
                torch.mm(s["dD"].to(f64)[mine].mT, s["A"].to(f64)[mine], out=dW[e])
            return dict(dW=dW.add_(s["sum"].to(f64), alpha=c["beta"]) if c["beta"] else dW)
        forward = c["kind"] == "product"
        X = s["A"] if forward else s["dD"]
        D = torch.zeros(X.shape[0], c["N"] if forward else c["K"], dtype=f64, device=X.device)
        for e in range(c["E"]):
            mine = torch.nonzero(expert == e)[:, 0]
            W = s["W"][e].to(f64)
            y = torch.einsum("rk,nk->rn" if forward else "rn,nk->rk", X[mine].to(f64), W)
            D[mine] = y * torch.sigmoid(y) if c.get("act") == "silu" else y
        return dict(D=D) if forward else dict(dA=D)
    norm = math.sqrt(math.fsum(float(torch.dot(w, w)) for w in (t.to(f64) for t in s["tensors"])))
    total = torch.tensor(norm, dtype=f64, device=s["tensors"][0].device)
    if c["kind"] == "norm":
        return dict(norm=total)
    flat, to = _bucket([t.numel() for t in s["tensors"]], f64, total.device)
    for t, at in zip(s["tensors"], to):
        at.copy_(t.to(f64) * min(1.0, s["max_norm"] / norm))
    return dict(norm=total, clipped=flat)


# ------------------------------------------------------------------ floors
def work(case):
    c = case
    if c["kind"] in PRODUCTS:
        R, E, N, K = c["T"] * c["k"], c["E"], c["N"], c["K"]
        kept = R * (1.0 - c["drop"])
        out = 2 if c["out"] == "bf16" else 4
        flops = 2 * kept * N * K
        if c["kind"] == "weights_grad":
            return dict(bytes=2 * kept * (N + K) + E * N * K * out * (2 if c["beta"] else 1) + 4 * (E + 1), flops=flops)
        active = E * (1.0 - (1.0 - c["k"] / E) ** c["T"])        # expected, of a router without favourites
        inner, outer = (K, N) if c["kind"] == "product" else (N, K)
        return dict(bytes=active * N * K * 2 + kept * inner * 2 + R * outer * out + 4 * (E + 1), flops=flops)
    n, size = c["values"], 2 if c["dtype"] == "bf16" else 4
    if c["kind"] == "norm":
        return dict(bytes=n * size, flops=2 * n)
    return dict(bytes=n * (size + (2 if c["to"] == "bf16" else 4)), flops=3 * n)
