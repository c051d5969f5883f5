"""GPU parity of the expert calls: dispatch and combine with their gradients.

The expected values are loops over the definitions in 64 bits.  Copies and
plans have to be equal.  Sums are held to bounds that follow from the
arithmetic: fp32 sums of n terms in any order are within n 2^-23 of the sum
of the magnitudes, and rounding to bf16 (fp32) adds 2^-8 (2^-24) of the value.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

g = pytest.importorskip("tensor_core_dense_tn_gb300")

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
OUT_EPS = {"bf16": 2.0 ** -8 * 1.01, "f32": 2.0 ** -24}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make_ids(T, k, E, seed, how):
    r = np.random.default_rng(seed)
    ids = r.integers(0, E, (T, k))
    if how == "dropped":
        ids[r.random((T, k)) < 0.3] = -1
        ids[r.random((T, k)) < 0.1] = E + 5
    elif how == "one expert":
        ids[:] = E - 1
    elif how == "none":
        ids[:] = -7
    return ids


def expected_plan(ids, E):
    T, k = ids.shape
    order = [(t, j) for e in range(E) for t, j in zip(*np.nonzero(ids == e))]
    offsets = np.array([np.count_nonzero((ids >= 0) & (ids < e)) for e in range(E + 1)])
    slot_row = np.full((T, k), -1)
    row_token = np.full(T * k, -1)
    for r, (t, j) in enumerate(order):
        slot_row[t, j] = r
        row_token[r] = t
    return offsets, slot_row, row_token


def on_gpu(ids, wide=True):
    return torch.from_numpy(ids.astype(np.int64 if wide else np.int32)).cuda()


def rows_like(n, H, dtype, seed, pad=0, shift=0):
    """An n x H matrix inside a larger allocation: row pitch H + pad, starting `shift` elements in."""
    buf = torch.randn(shift + n * (H + pad) + 8, generator=gen(seed), device="cuda").to(DT[dtype])
    return buf[shift:shift + n * (H + pad)].view(n, H + pad)[:, :H]


def status():
    assert g.gemm_get_status(torch.cuda.current_stream().cuda_stream) == 0


SIZES = [  # T, k, E, H
    (1, 1, 1, 8), (1, 8, 64, 4096), (16, 2, 8, 4096), (5, 3, 7, 1), (7, 64, 16, 40), (1024, 2, 8, 64),
    (700, 3, 61, 257), (1025, 2, 8, 72), (683, 3, 1024, 33), (3001, 5, 128, 136), (9000, 1, 3, 16),
]


@pytest.mark.parametrize("T,k,E,H", SIZES)
@pytest.mark.parametrize("how", ["all", "dropped", "one expert", "none"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dispatch(T, k, E, H, how, dtype):
    ids = make_ids(T, k, E, 11 * T + k, how)
    plan = g.ExpertPlan(T, k, E, "cuda")
    for t in (plan.offsets, plan.slot_row, plan.row_token):
        t.fill_(-99)
    X = rows_like(T, H, dtype, 1)
    out = torch.full((T * k, H), float("nan"), device="cuda", dtype=DT[dtype])
    Xs = g.expert_dispatch(on_gpu(ids, wide=how != "dropped"), plan, X, out=out)
    status()
    offsets, slot_row, row_token = expected_plan(ids, E)
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets)
    assert np.array_equal(plan.slot_row.cpu().numpy(), slot_row)
    assert np.array_equal(plan.row_token.cpu().numpy(), row_token)
    tok = torch.from_numpy(row_token).cuda()
    want = torch.where((tok >= 0)[:, None], X[tok.clamp(min=0)], torch.zeros((), device="cuda", dtype=X.dtype))
    assert torch.equal(Xs, want)


@pytest.mark.parametrize("T,k,E", [(0, 2, 8), (1, 1, 1), (300, 4, 16), (5000, 4, 1024), (140000, 2, 61)])
def test_plan_alone(T, k, E):
    ids = make_ids(T, k, E, 3, "dropped")
    plan = g.ExpertPlan(T, k, E, "cuda")
    assert g.expert_dispatch(on_gpu(ids), plan) is None
    status()
    key = np.where((ids >= 0) & (ids < E), ids, E).reshape(-1)
    order = np.argsort(key, kind="stable")
    V = np.count_nonzero(key < E)
    slot_row = np.full(T * k, -1)
    slot_row[order[:V]] = np.arange(V)
    assert np.array_equal(plan.offsets.cpu().numpy(), np.searchsorted(np.sort(key), np.arange(E + 1)))
    assert np.array_equal(plan.slot_row.cpu().numpy().reshape(-1), slot_row)
    assert np.array_equal(plan.row_token.cpu().numpy(), np.where(np.arange(T * k) < V, order // k, -1))


def make_plan(T, k, E, seed, how):
    ids = make_ids(T, k, E, seed, how)
    offsets, slot_row, row_token = expected_plan(ids, E)
    i32 = lambda a: torch.from_numpy(a.astype(np.int32)).cuda()  # noqa: E731
    return g.ExpertPlan.of(i32(offsets), i32(slot_row), i32(row_token)), torch.from_numpy(slot_row).cuda()


def slot_rows64(Y, slot_row):
    """(T, k, H) rows of the slots in 64 bits, zero where dropped."""
    got = Y.double()[slot_row.clamp(min=0)]
    return torch.where((slot_row >= 0)[..., None], got, torch.zeros((), device="cuda", dtype=torch.float64))


LAYOUTS = [(0, 0), (3, 0), (8, 0), (0, 1), (24, 8)]   # pad, shift in elements


@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 8), (16, 2, 8, 4096), (5, 3, 7, 1), (9, 20, 16, 100), (333, 8, 61, 257),
                                     (200, 4, 16, 2056), (130, 1, 8, 72)])
@pytest.mark.parametrize("how", ["all", "dropped", "none"])
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
def test_combine(T, k, E, H, how, dtype, wdtype):
    plan, slot_row = make_plan(T, k, E, 5 * T + H, how)
    pad, shift = LAYOUTS[(T + H) % len(LAYOUTS)]
    Y = rows_like(T * k, H, dtype, 2, pad, shift)
    w = torch.randn(T, k, generator=gen(3), device="cuda").to(DT[wdtype])
    out = g.expert_combine(plan, Y, w)
    status()
    terms = slot_rows64(Y, slot_row) * w.double()[..., None]
    ref, mag = terms.sum(1), terms.abs().sum(1)
    bound = k * 2.0 ** -23 * mag + OUT_EPS[dtype] * ref.abs()
    assert torch.all((out.double() - ref).abs() <= bound)
    dX = g.expert_dispatch_backward(plan, Y)
    status()
    terms = slot_rows64(Y, slot_row)
    ref, mag = terms.sum(1), terms.abs().sum(1)
    assert torch.all((dX.double() - ref).abs() <= k * 2.0 ** -23 * mag + OUT_EPS[dtype] * ref.abs())


@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 8), (16, 2, 8, 4096), (5, 3, 7, 1), (9, 20, 16, 100), (333, 8, 61, 257),
                                     (200, 4, 16, 2056), (130, 1, 8, 72), (3, 2, 4, 8200)])
@pytest.mark.parametrize("how", ["all", "dropped", "none"])
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
def test_combine_backward(T, k, E, H, how, dtype, wdtype):
    plan, slot_row = make_plan(T, k, E, 7 * T + H, how)
    pad, shift = LAYOUTS[(T + k) % len(LAYOUTS)]
    Y = rows_like(T * k, H, dtype, 4, pad, shift)
    dout = rows_like(T, H, dtype, 5)
    w = torch.randn(T, k, generator=gen(6), device="cuda").to(DT[wdtype])
    nan = lambda *s, dt: torch.full(s, float("nan"), device="cuda", dtype=dt)  # noqa: E731
    dY, dw = g.expert_combine_backward(plan, Y, w, dout, dY=nan(T * k, H, dt=DT[dtype]), dweights=nan(T, k, dt=DT[wdtype]))
    status()
    # dY: one fp32 product and one rounding; zeros where no slot is
    want = torch.zeros(T * k, H, device="cuda", dtype=torch.float64)
    keep = slot_row >= 0
    want[slot_row[keep]] = (w.double()[..., None] * dout.double()[:, None, :])[keep]
    assert torch.all((dY.double() - want).abs() <= (2.0 ** -24 + OUT_EPS[dtype]) * want.abs())
    # dweights: each of at least 32 lanes adds H / 32 products, then 5 + 8 joins
    terms = slot_rows64(Y, slot_row) * dout.double()[:, None, :]
    ref, mag = terms.sum(-1), terms.abs().sum(-1)
    assert torch.all((dw.double() - ref).abs() <= (H / 32 + 32) * 2.0 ** -23 * mag + OUT_EPS[wdtype] * ref.abs())
    assert torch.all(dw[~keep] == 0)


def test_one_gradient_at_a_time():
    plan, slot_row = make_plan(40, 3, 8, 1, "dropped")
    Y, dout = rows_like(120, 136, "bf16", 1), rows_like(40, 136, "bf16", 2)
    w = torch.rand(40, 3, device="cuda")
    dY, dw = g.expert_combine_backward(plan, Y, w, dout)
    s = torch.cuda.current_stream().cuda_stream
    dY2, dw2 = torch.empty_like(dY), torch.empty_like(dw)
    a = (plan.info, 136, 0, 136, dout.data_ptr(), 136, 0, w.data_ptr(), 3, 1)
    assert g.gemm_expert_combine_backward(*a, dY2.data_ptr(), 136, 0, 0, s) == 0
    a = (plan.info, 136, Y.data_ptr(), 136, dout.data_ptr(), 136, 0, w.data_ptr(), 3, 1)
    assert g.gemm_expert_combine_backward(*a, 0, 0, dw2.data_ptr(), 3, s) == 0
    status()
    assert torch.equal(dY, dY2) and torch.equal(dw, dw2)


def test_gradients_against_differences():
    """combine is linear in Y and in the weights: differences of the loss <dout, combine> along a direction equal
    the gradient's product with it, up to the rounding of the two sums (k terms each) and of the outputs."""
    T, k, E, H = 50, 3, 8, 40
    plan, slot_row = make_plan(T, k, E, 9, "dropped")
    Y, dout = rows_like(T * k, H, "f32", 1), rows_like(T, H, "f32", 2)
    w = torch.rand(T, k, generator=gen(3), device="cuda")
    dY, dw = g.expert_combine_backward(plan, Y, w, dout)
    dirY = torch.randn(T * k, H, generator=gen(4), device="cuda")
    dirw = torch.randn(T, k, generator=gen(5), device="cuda")
    loss = lambda Y, w: (dout.double() * g.expert_combine(plan, Y, w).double()).sum()  # noqa: E731
    for Y1, w1, want in ((Y + dirY, w, (dY.double() * ((Y + dirY).double() - Y.double())).sum()),
                         (Y, w + dirw, (dw.double() * ((w + dirw).double() - w.double())).sum())):
        mags = [((slot_rows64(a, slot_row) * b.double()[..., None]).abs().sum(1) * dout.double().abs()).sum()
                for a, b in ((Y, w), (Y1, w1))]
        slack = (k + H) * 2.0 ** -23 * (mags[0] + mags[1])
        assert (loss(Y1, w1) - loss(Y, w) - want).abs() <= slack
    # the copy's gradient: <dXs, dispatch(X)> = <dispatch_backward(dXs), X>, both sums of the same products
    X = rows_like(T, H, "f32", 6)
    ids = on_gpu(make_ids(T, k, E, 9, "dropped"))
    Xs = g.expert_dispatch(ids, plan, X)
    dXs = rows_like(T * k, H, "f32", 7)
    dX = g.expert_dispatch_backward(plan, dXs)
    left, right = (dXs.double() * Xs.double()).sum(), (dX.double() * X.double()).sum()
    assert (left - right).abs() <= k * 2.0 ** -23 * (dXs.double() * Xs.double()).abs().sum()


def test_non_finite_rows_stay_where_they_are():
    """A dropped slot's row and the rows of other tokens do not reach a token; its own do."""
    T, k, E, H = 64, 2, 4, 64
    plan, slot_row = make_plan(T, k, E, 2, "dropped")
    Y = rows_like(T * k, H, "f32", 1).clone()
    w = torch.rand(T, k, generator=gen(3), device="cuda") + 0.5
    clean = g.expert_combine(plan, Y, w)
    V = int(plan.offsets[-1])
    Y[V:] = float("nan")                       # rows of no slot
    w[slot_row < 0] = float("nan")             # weights of dropped slots
    assert torch.equal(g.expert_combine(plan, Y, w), clean)
    dY, dw = g.expert_combine_backward(plan, Y, w, clean)
    assert torch.isfinite(dY).all() and torch.isfinite(dw).all() and torch.all(dY[V:] == 0)
    Y[0] = float("inf")
    out = g.expert_combine(plan, Y, w)
    t = int(plan.row_token[0])
    assert torch.isinf(out[t]).all()
    others = torch.arange(T, device="cuda") != t
    assert torch.equal(out[others], clean[others])


def test_rows_of_a_foreign_plan_are_checked():
    """Rows outside [0, T k) in a plan count as dropped."""
    plan, slot_row = make_plan(20, 2, 4, 2, "all")
    Y, w = rows_like(40, 32, "f32", 1), torch.rand(20, 2, device="cuda")
    plan.slot_row[3, 0], plan.slot_row[4, 1] = 40, -(1 << 31)
    slot_row[3, 0] = slot_row[4, 1] = -1
    out = g.expert_combine(plan, Y, w)
    ref = (slot_rows64(Y, slot_row) * w.double()[..., None]).sum(1)
    assert torch.allclose(out.double(), ref, rtol=1e-5, atol=1e-5)
    dY, dw = g.expert_combine_backward(plan, Y, w, out)
    assert dw[3, 0] == 0 and dw[4, 1] == 0


def test_side_stream_and_repeats():
    """The same bits on another stream, run after run, and under graph replay."""
    T, k, E, H = 2000, 4, 32, 264
    ids = on_gpu(make_ids(T, k, E, 2, "dropped"))
    X, w = rows_like(T, H, "bf16", 1), torch.rand(T, k, device="cuda")

    def step(plan):
        Xs = g.expert_dispatch(ids, plan, X)
        out = g.expert_combine(plan, Xs, w)
        dY, dw = g.expert_combine_backward(plan, Xs, w, X)
        return [plan.offsets.clone(), plan.slot_row.clone(), plan.row_token.clone(), Xs, out, dY, dw]

    first = step(g.ExpertPlan(T, k, E, "cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan = g.ExpertPlan(T, k, E, "cuda")
        second = step(plan)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            third = step(plan)
        for t in third:
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_offsets_past_32_bits():
    """Rows whose byte offsets need more than 32 bits: 70000 rows of a pitch of 65536 bytes."""
    T, k, E, H = 35000, 2, 8, 40
    buf = torch.empty(T * k * 32768, dtype=torch.bfloat16, device="cuda")
    Xs = buf.view(T * k, 32768)[:, :H]
    ids = on_gpu(make_ids(T, k, E, 2, "all"))
    plan = g.ExpertPlan(T, k, E, "cuda")
    X = rows_like(T, H, "bf16", 1)
    g.expert_dispatch(ids, plan, X, out=Xs)
    status()
    assert torch.equal(Xs, X[plan.row_token.long()])
    dX = g.expert_dispatch_backward(plan, Xs)
    assert torch.equal(dX, 2 * X)


@pytest.mark.parametrize("T,k,E", [(512, 1, 7), (513, 1, 7), (256, 2, 200), (171, 3, 61), (1024, 4, 128), (4097, 1, 128),
                                   (2049, 2, 33), (600001, 1, 61), (70000, 9, 1024)])
def test_plans_of_every_kernel(T, k, E):
    test_plan_alone(T, k, E)


@pytest.mark.parametrize("H,pad,shift", [(34, 0, 0), (33, 1, 0), (262, 2, 2), (1002, 0, 0), (1, 1, 0), (3, 1, 4)])
@pytest.mark.parametrize("k", [1, 2, 3, 4, 8, 12])
def test_bf16_rows_at_4_byte_addresses(H, pad, shift, k):
    T, E = 77, 9
    plan, slot_row = make_plan(T, k, E, H + k, "dropped")
    X, Y, dout = (rows_like(n, H, "bf16", 20 + i, pad, shift) for i, n in enumerate((T, T * k, T)))
    assert X.stride(0) % 2 == 0 or H == 1
    w = torch.randn(T, k, generator=gen(3), device="cuda")
    ids = on_gpu(make_ids(T, k, E, H + k, "dropped"))
    got = rows_like(T * k, H, "bf16", 30, pad, shift)
    g.expert_dispatch(ids, plan, X, out=got)
    tok = plan.row_token.long()
    want = torch.where((tok >= 0)[:, None], X[tok.clamp(min=0)], torch.zeros((), device="cuda", dtype=X.dtype))
    assert torch.equal(got, want)
    out = rows_like(T, H, "bf16", 31, pad, shift)
    g.expert_combine(plan, Y, w, out=out)
    terms = slot_rows64(Y, slot_row) * w.double()[..., None]
    ref, mag = terms.sum(1), terms.abs().sum(1)
    assert torch.all((out.double() - ref).abs() <= k * 2.0 ** -23 * mag + OUT_EPS["bf16"] * ref.abs())
    dY = rows_like(T * k, H, "bf16", 32, pad, shift)
    _, dw = g.expert_combine_backward(plan, Y, w, dout, dY=dY)
    status()
    want = torch.zeros(T * k, H, device="cuda", dtype=torch.float64)
    keep = slot_row >= 0
    want[slot_row[keep]] = (w.double()[..., None] * dout.double()[:, None, :])[keep]
    assert torch.all((dY.double() - want).abs() <= (2.0 ** -24 + OUT_EPS["bf16"]) * want.abs())
    terms = slot_rows64(Y, slot_row) * dout.double()[:, None, :]
    ref, mag = terms.sum(-1), terms.abs().sum(-1)
    assert torch.all((dw.double() - ref).abs() <= (H / 32 + 32) * 2.0 ** -23 * mag + OUT_EPS["f32"] * ref.abs())
