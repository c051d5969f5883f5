"""Measured cases of the expert and 4-bit-weight operators.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges,
``prepare`` makes a program's data, ``run`` makes one pass: through plain
torch operations where ``own`` is false, through this library's entry points
where it is true.  ``exact`` gives the same values from the definitions in 64
bits, and ``work`` what a pass cannot do without.

The operators, for T tokens with k expert slots each (ids outside [0, E) are
dropped slots), rows sorted by expert and stable within it:

    dispatch            offsets, slot_row, row_token and Xs[r] = X[row_token[r]]
    dispatch_backward   dX[t]  = sum_j dXs[slot_row[t, j]]
    combine             out[t] = sum_j w[t, j] * Y[slot_row[t, j]]
    combine_backward    dY[slot_row[t, j]] = w[t, j] * dout[t],
                        dw[t, j] = <dout[t], Y[slot_row[t, j]]>
    w4                  D = act(alpha * A * W^T), W[n, k] = s[n, k/g] * (q[n, k] - z[n, k/g])
    w4_experts          the same for rows in expert order, one W per expert
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # A decode step of 16 sequences: latency of the sort and the copy.
        dict(name="dispatch_decode", kind="dispatch", T=16, k=2, E=8, H=4096, dtype="bf16", wide_ids=True, drop=0.0),
        # A prompt's tokens to eight of 128 experts.
        dict(name="dispatch_prompt", kind="dispatch", T=8192, k=8, E=128, H=2048, dtype="bf16", wide_ids=True,
             drop=0.0),
        # A ragged fp32 batch whose full experts dropped some slots.
        dict(name="dispatch_ragged", kind="dispatch", T=3001, k=3, E=61, H=2001, dtype="f32", wide_ids=False,
             drop=0.05),
        # The training step's way back to the tokens.
        dict(name="dispatch_backward", kind="dispatch_backward", T=8192, k=2, E=8, H=4096, dtype="bf16",
             wide_ids=True, drop=0.02),
        # A decode step's results.
        dict(name="combine_decode", kind="combine", T=16, k=2, E=8, H=4096, dtype="bf16", wdtype="f32", drop=0.0),
        # A prompt's results.
        dict(name="combine_prompt", kind="combine", T=8192, k=8, E=128, H=2048, dtype="bf16", wdtype="f32", drop=0.0),
        # A training step: gradients of the rows and of the router's weights.
        dict(name="combine_backward", kind="combine_backward", T=16384, k=4, E=64, H=4096, dtype="bf16",
             wdtype="f32", drop=0.02),
        # One token through the decode workload's matrix.
        dict(name="w4_one_token", kind="w4", M=1, N=8192, K=8192, g=128, zeros=False, act="none", out="bf16"),
        # 16 tokens through the MLP up-projection.
        dict(name="w4_batch", kind="w4", M=16, N=28672, K=4096, g=128, zeros=True, act="silu", out="bf16"),
        # The ragged workload's matrix with small groups and an fp32 result.
        dict(name="w4_ragged", kind="w4", M=5, N=5000, K=2000, g=32, zeros=True, act="none", out="f32"),
        # One token through its 8 of 64 experts.
        dict(name="w4_experts_one_token", kind="w4_experts", T=1, k=8, E=64, N=4096, K=2048, g=128, zeros=False,
             act="silu", out="bf16"),
        # 32 sequences through all of 16 experts.
        dict(name="w4_experts_batch", kind="w4_experts", T=32, k=2, E=16, N=8192, K=4096, g=64, zeros=True,
             act="silu", out="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["dispatch", "dispatch_backward", "combine", "combine_backward", "w4", "w4_experts"])
    if kind == "w4":
        while True:
            c = dict(kind=kind, M=_log(rng, 1, 16), N=_log(rng, 256, 28672), K=_log(rng, 256, 16384),
                     g=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5, act=rng.choice(["none", "silu"]),
                     out=rng.choice(["bf16", "f32"]))
            if c["N"] * c["K"] <= 28672 * 4096:
                return c
    if kind == "w4_experts":
        while True:
            c = dict(kind=kind, T=_log(rng, 1, 32), k=rng.randint(1, 8), E=rng.choice([8, 16, 24, 64, 100]),
                     N=_log(rng, 256, 8192), K=_log(rng, 256, 8192), g=rng.choice([32, 64, 128]),
                     zeros=rng.random() < 0.5, act=rng.choice(["none", "silu"]), out=rng.choice(["bf16", "f32"]))
            if c["E"] * c["N"] * c["K"] <= 16 * 8192 * 4096:
                return c
    while True:
        c = dict(kind=kind, T=_log(rng, 1, 16384), k=rng.randint(1, 8), E=rng.choice([8, 16, 61, 64, 128, 256]),
                 H=_log(rng, 64, 8192), dtype=rng.choice(["bf16", "bf16", "f32"]),
                 drop=rng.choice([0.0, 0.0, 0.02, 0.3]))
        if kind.startswith("dispatch"):
            c["wide_ids"] = rng.random() < 0.5
        else:
            c["wdtype"] = rng.choice(["f32", "bf16"])
        if c["T"] * c["k"] * c["H"] * (2 if c["dtype"] == "bf16" else 4) <= 8192 * 8 * 2048 * 2:
            return c


# ------------------------------------------------------------------ inputs
def _route(c, gen, dev):
    """A router's choice: k different experts for each token, some of the slots dropped."""
    liked = torch.randn(c["E"], generator=gen, device=dev) * (0.0 if c["kind"] == "w4_experts" else 0.5)
    logits = torch.randn(c["T"], c["E"], generator=gen, device=dev) + liked
    top, ids = torch.topk(logits, c["k"], dim=1)
    weights = torch.softmax(top, dim=1)
    if c.get("drop", 0.0) > 0.0:
        ids = torch.where(torch.rand(ids.shape, generator=gen, device=dev) < c["drop"], torch.full_like(ids, -1), ids)
    return ids if c.get("wide_ids", True) else ids.int(), weights


def _sorted(ids, E):
    """offsets, slot_row and row_token of the stable order by expert."""
    T, k = ids.shape
    n = T * k
    key = ids.reshape(-1).long()
    key = torch.where((key >= 0) & (key < E), key, torch.full_like(key, E))
    by, order = torch.sort(key, stable=True)
    place = torch.arange(n, device=ids.device)
    row = torch.empty_like(place)
    row[order] = place
    bounds = (by[None, :] < torch.arange(E + 1, device=ids.device)[:, None]).sum(1)
    slot_row = torch.where(key < E, row, torch.full_like(row, -1)).view(T, k)
    row_token = torch.where(by < E, order // k, torch.full_like(order, -1))
    return bounds.int(), slot_row.int(), row_token.int()


def _w4(c, gen, dev, count):
    """Codes (two to a byte, the even k in the low half, rows padded to 16 bytes), group scales and zero points."""
    N, K, g = c["N"], c["K"], c["g"]
    groups = -(-K // g)
    pitch = -(-K // 32) * 16
    codes = torch.randint(0, 256, (count, N, pitch), generator=gen, device=dev, dtype=torch.uint8)
    scales = (torch.rand(count, N, groups, generator=gen, device=dev) + 0.5) * (0.22 / math.sqrt(K))
    zeros = torch.randint(4, 12, (count, N, groups), generator=gen, device=dev, dtype=torch.uint8) if c["zeros"] else None
    return codes, scales.bfloat16(), zeros


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    if own:
        import tensor_core_dense_tn_gb300 as g
    s = dict(case=c)
    if c["kind"].startswith("w4"):
        if c["kind"] == "w4":
            s["A"] = torch.randn(c["M"], c["K"], generator=gen, device=dev)
            codes, scales, zeros = (None if t is None else t[0] for t in _w4(c, gen, dev, 1))
        else:
            ids, _ = _route(c, gen, dev)
            s["plan"] = _sorted(ids, c["E"])
            s["A"] = torch.randn(c["T"], c["K"], generator=gen, device=dev)
            codes, scales, zeros = _w4(c, gen, dev, c["E"])
        if c["K"] % 8:      # rows start on 16 bytes
            pad = torch.zeros(s["A"].shape[0], -(-c["K"] // 8) * 8, device=dev)
            pad[:, :c["K"]] = s["A"]
            s["A"] = pad.bfloat16()[:, :c["K"]]
        else:
            s["A"] = s["A"].bfloat16()
        s["codes"], s["scales"], s["zeros"] = codes, scales, zeros
        if own:             # the weights' handle and the plan, which a serving program keeps
            s["W"] = g.W4Matrix(codes, scales, zeros, K=c["K"], group=c["g"])
            if c["kind"] == "w4_experts":
                s["own_plan"] = g.ExpertPlan.of(*s["plan"], experts=c["E"])
        return s
    dt = DTYPES[c["dtype"]]
    s["ids"], weights = _route(c, gen, dev)
    if c["kind"] == "dispatch":
        s["X"] = torch.randn(c["T"], c["H"], generator=gen, device=dev).to(dt)
        if own:             # the plan's arrays, which a program keeps from step to step
            s["own_plan"] = g.ExpertPlan(c["T"], c["k"], c["E"], dev)
        return s
    s["plan"] = _sorted(s["ids"], c["E"])
    if own:
        s["own_plan"] = g.ExpertPlan.of(*s["plan"], experts=c["E"])
    n = c["T"] * c["k"]
    if c["kind"] == "dispatch_backward":
        s["dXs"] = torch.randn(n, c["H"], generator=gen, device=dev).to(dt)
        return s
    s["weights"] = weights.to(DTYPES[c["wdtype"]])
    s["Y"] = torch.randn(n, c["H"], generator=gen, device=dev).to(dt)
    if c["kind"] == "combine_backward":
        s["dout"] = torch.randn(c["T"], c["H"], generator=gen, device=dev).to(dt)
    return s


# ------------------------------------------------------------------ plain forms
def _rows(x, slot_row):
    """x[slot_row] in fp32, zeros for dropped slots."""
    got = x[slot_row.clamp(min=0).long()].float()
    return torch.where((slot_row >= 0)[..., None], got, torch.zeros((), device=x.device))


def _dequant(codes, scales, zeros, K, g):
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)[..., :K].float()
    z = 8.0 if zeros is None else zeros.float().repeat_interleave(g, dim=-1)[..., :K]
    return (q - z) * scales.float().repeat_interleave(g, dim=-1)[..., :K]


def _act(x, act):
    return x / (1.0 + torch.exp(-x)) if act == "silu" else x


def _plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "dispatch":
        offsets, slot_row, row_token = _sorted(s["ids"], c["E"])
        got = s["X"][row_token.clamp(min=0).long()]
        Xs = torch.where((row_token >= 0)[:, None], got, torch.zeros((), dtype=got.dtype, device=got.device))
        return dict(offsets=offsets, slot_row=slot_row, row_token=row_token, Xs=Xs)
    if kind == "dispatch_backward":
        return dict(dX=_rows(s["dXs"], s["plan"][1]).sum(1).to(s["dXs"].dtype))
    if kind == "combine":
        y = _rows(s["Y"], s["plan"][1])
        return dict(out=(s["weights"].float()[..., None] * y).sum(1).to(s["Y"].dtype))
    if kind == "combine_backward":
        slot_row = s["plan"][1]
        n, H = s["Y"].shape
        dout = s["dout"].float()[:, None, :]
        dw = (dout * _rows(s["Y"], slot_row)).sum(-1).to(s["weights"].dtype)
        dY = torch.zeros(n + 1, H, dtype=s["Y"].dtype, device=s["Y"].device)     # one row more for the dropped
        at = torch.where(slot_row >= 0, slot_row, torch.full_like(slot_row, n)).reshape(-1).long()
        dY[at] = (s["weights"].float()[..., None] * dout).reshape(-1, H).to(dY.dtype)
        return dict(dY=dY[:n], dweights=dw)
    dt = DTYPES[c["out"]]
    if kind == "w4":
        W = _dequant(s["codes"], s["scales"], s["zeros"], c["K"], c["g"])
        return dict(D=_act(s["A"].float() @ W.t(), c["act"]).to(dt))
    offsets, _, row_token = s["plan"]
    A = s["A"][row_token.long()].float()
    row = torch.arange(A.shape[0], device=A.device)
    expert = (offsets[None, 1:] <= row[:, None]).sum(1)
    codes, scales, zeros = s["codes"], s["scales"], s["zeros"]
    if A.shape[0] <= c["E"]:        # each row with a matrix of its own
        W = _dequant(codes[expert], scales[expert], None if zeros is None else zeros[expert], c["K"], c["g"])
        D = torch.matmul(W, A[:, :, None])[:, :, 0]
    else:                           # every expert's matrix once, and each row's own result of them
        W = _dequant(codes, scales, zeros, c["K"], c["g"])
        D = torch.matmul(A[None], W.transpose(1, 2))[expert, row]
    return dict(D=_act(D, c["act"]).to(dt))


# ------------------------------------------------------------------ one pass
def run(state):
    if not own:
        return _plain(state)
    import tensor_core_dense_tn_gb300 as g
    s, c = state, state["case"]
    kind = c["kind"]
    if kind == "dispatch":
        plan = s["own_plan"]
        Xs = g.expert_dispatch(s["ids"], plan, s["X"])
        return dict(offsets=plan.offsets, slot_row=plan.slot_row, row_token=plan.row_token, Xs=Xs)
    if kind == "dispatch_backward":
        return dict(dX=g.expert_dispatch_backward(s["own_plan"], s["dXs"]))
    if kind == "combine":
        return dict(out=g.expert_combine(s["own_plan"], s["Y"], s["weights"]))
    if kind == "combine_backward":
        dY, dw = g.expert_combine_backward(s["own_plan"], s["Y"], s["weights"], s["dout"])
        return dict(dY=dY, dweights=dw)
    act = g.ACT_SILU if c["act"] == "silu" else g.ACT_NONE
    if kind == "w4":
        return dict(D=g.gemm_w4(s["A"], s["W"], activation=act, out_dtype=DTYPES[c["out"]]))
    return dict(D=g.gemm_w4_experts(s["A"], s["W"], s["own_plan"], gather=True, activation=act,
                                    out_dtype=DTYPES[c["out"]]))


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    c = case
    s = prepare(case, seed)
    f64 = torch.float64
    if c["kind"] == "w4":
        return dict(D=_exact_product(s["A"].to(f64), s["codes"], s["scales"], s["zeros"], c))
    if c["kind"] == "w4_experts":
        bounds = s["plan"][0].tolist()
        token = s["plan"][2].tolist()
        D = torch.zeros(len(token), c["N"], dtype=f64, device=s["A"].device)
        for e in range(c["E"]):
            lo, hi = bounds[e], bounds[e + 1]
            if hi > lo:
                D[lo:hi] = _exact_product(s["A"][token[lo:hi]].to(f64), s["codes"][e], s["scales"][e],
                                          None if s["zeros"] is None else s["zeros"][e], c)
        return dict(D=D)
    ids = s["ids"].tolist()
    T, k = c["T"], c["k"]
    # the order by expert, straight from the definition
    buckets = [[] for _ in range(c["E"])]
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t][j] < c["E"]:
                buckets[ids[t][j]].append((t, j))
    order = [tj for b in buckets for tj in b]
    dev = s["ids"].device
    tok = torch.tensor([t for t, _ in order], dtype=torch.long, device=dev)
    slot = torch.tensor([j for _, j in order], dtype=torch.long, device=dev)
    V, n = len(order), T * k
    if c["kind"] == "dispatch":
        Xs = torch.zeros(n, c["H"], dtype=f64, device=dev)
        Xs[:V] = s["X"].to(f64)[tok]
        return dict(offsets=None, slot_row=None, row_token=None, Xs=Xs)
    if c["kind"] == "dispatch_backward":
        dX = torch.zeros(T, c["H"], dtype=f64, device=dev)
        return dict(dX=dX.index_add_(0, tok, s["dXs"][:V].to(f64)))
    w = s["weights"].to(f64)[tok, slot]
    if c["kind"] == "combine":
        out = torch.zeros(T, c["H"], dtype=f64, device=dev)
        return dict(out=out.index_add_(0, tok, s["Y"][:V].to(f64) * w[:, None]))
    grad = s["dout"].to(f64)[tok]
    dw = torch.zeros(T, k, dtype=f64, device=dev)
    dw[tok, slot] = torch.einsum("rh,rh->r", grad, s["Y"][:V].to(f64))
    dY = torch.zeros(n, c["H"], dtype=f64, device=dev)
    dY[:V] = grad * w[:, None]
    return dict(dY=dY, dweights=dw)


def _exact_product(A, codes, scales, zeros, c):
    """Group by group: sum_g scale_g * (A_g q_g^T - zero_g * sum A_g)."""
    K, g = c["K"], c["g"]
    total = torch.zeros(A.shape[0], c["N"], dtype=torch.float64, device=A.device)
    for i, k0 in enumerate(range(0, K, g)):
        k1 = min(K, k0 + g)
        q = torch.zeros(c["N"], k1 - k0, dtype=torch.float64, device=A.device)
        part = codes[:, k0 // 2:(k1 + 1) // 2]          # a group starts on an even k
        q[:, 0::2] = (part % 16).to(torch.float64)
        q[:, 1::2] = (part // 16).to(torch.float64)[:, :(k1 - k0) // 2]
        z = 8.0 if zeros is None else zeros[:, i].to(torch.float64)
        a = A[:, k0:k1]
        total += scales[:, i].to(torch.float64) * (torch.matmul(a, q.T) - a.sum(1, keepdim=True) * z)
    return total * torch.sigmoid(total) if c["act"] == "silu" else total


# ------------------------------------------------------------------ floors
def work(case):
    c = case
    if c["kind"].startswith("w4"):
        N, K = c["N"], c["K"]
        esize = 2 if c["out"] == "bf16" else 4
        groups = -(-K // c["g"])
        matrix = N * (-(-K // 2)) + N * groups * (3 if c["zeros"] else 2)
        if c["kind"] == "w4":
            return dict(bytes=matrix + c["M"] * (2 * K + N * esize), flops=2 * c["M"] * N * K)
        n = c["T"] * c["k"]
        active = c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"])      # expected, of a router without favourites
        return dict(bytes=active * matrix + c["T"] * 2 * K + n * (N * esize + 4) + 4 * (c["E"] + 1), flops=2 * n * N * K)
    e = 2 if c["dtype"] == "bf16" else 4
    T, H, n = c["T"], c["H"], c["T"] * c["k"]
    kept = n * (1.0 - c["drop"])
    if c["kind"] == "dispatch":
        return dict(bytes=n * (8 if c["wide_ids"] else 4) + (T + n) * H * e + 4 * (2 * n + c["E"] + 1), flops=0)
    if c["kind"] == "dispatch_backward":
        return dict(bytes=(kept + T) * H * e + 4 * n, flops=kept * H)
    w = 2 if c["wdtype"] == "bf16" else 4
    if c["kind"] == "combine":
        return dict(bytes=(kept + T) * H * e + (4 + w) * n, flops=2 * kept * H)
    return dict(bytes=(kept + n + T) * H * e + (4 + 2 * w) * n, flops=3 * kept * H)
