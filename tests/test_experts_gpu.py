"""GPU parity of the bf16 products by expert and their gradients.

The expected values are loops over the experts in 64 bits.  Whole numbers
whose sums stay below 2^24 have to come out exactly (rounded once to bf16
where the result is bf16).  Other values are held to bounds that follow from
the arithmetic: an fp32 sum of n products in any order, each addition rounded
or cut off, is within n 2^-23 of the sum of the magnitudes; the factors and
beta * C add 2^-23 of theirs each; the result's rounding is half a step,
2^-8 of the value for bf16 and 2^-24 for fp32.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

g = pytest.importorskip("tensor_core_dense_tn_gb300")

BF16, F32 = torch.bfloat16, torch.float32
EPS = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def plan_of(counts, lost):
    """A plan with counts[e] rows of expert e and `lost` rows of nobody behind them."""
    i32 = dict(dtype=torch.int32, device="cuda")
    offsets = torch.tensor([sum(counts[:e]) for e in range(len(counts) + 1)], **i32)
    rows = sum(counts) + lost
    return g.ExpertPlan.of(offsets, torch.zeros(rows, 1, **i32), torch.zeros(rows, **i32))


def values(shape, seed, whole, pad=None):
    """bf16 values; whole numbers in [-3, 3], or normal ones.  Rows start on 16 bytes, `pad` elements apart from
    their end (by default as few as that takes), and the padding holds NaN."""
    wide = -(-shape[-1] // 8) * 8 + (pad or 0)
    buf = torch.full((*shape[:-1], wide), float("nan"), device="cuda", dtype=BF16)
    t = torch.randint(-3, 4, shape, generator=gen(seed), device="cuda").float() if whole else \
        torch.randn(shape, generator=gen(seed), device="cuda")
    buf[..., :shape[-1]] = t
    return buf[..., :shape[-1]]


def bounds_of(plan):
    return plan.offsets.tolist()


def forward64(A, W, plan):
    """The product and the sum of its terms' magnitudes."""
    ref = torch.zeros(A.shape[0], W.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    b = bounds_of(plan)
    for e, (lo, hi) in enumerate(zip(b, b[1:])):
        a, w = A[lo:hi].double(), W[e].double()
        ref[lo:hi], mag[lo:hi] = a @ w.T, a.abs() @ w.abs().T
    return ref, mag


def weights64(dD, A, plan):
    b = bounds_of(plan)
    pairs = [(dD[lo:hi].double(), A[lo:hi].double()) for lo, hi in zip(b, b[1:])]
    return torch.stack([d.T @ a for d, a in pairs]), torch.stack([d.abs().T @ a.abs() for d, a in pairs])


def status():
    assert g.gemm_get_status(torch.cuda.current_stream().cuda_stream) == 0


def check(got, ref, mag, terms, whole):
    assert not torch.isnan(got).any()
    if whole:
        assert torch.equal(got, ref.to(F32).to(got.dtype))
    else:
        bound = (terms + 2) * 2.0 ** -23 * mag + EPS[got.dtype] * 1.01 * ref.abs()
        assert torch.all((got.double() - ref).abs() <= bound)


def canvas(shape, dtype, pad):
    """An output of `shape` inside a larger buffer of sevens, `pad` elements behind each row."""
    buf = torch.full((*shape[:-1], shape[-1] + pad), 7.0, device="cuda", dtype=dtype)
    return buf, buf[..., :shape[-1]]


CASES = [  # rows of each expert, rows of nobody, N, K
    ([1], 0, 8, 8), ([0, 1, 0, 0], 0, 256, 64), ([2], 3, 1, 1), ([5, 0, 130, 64, 1], 17, 72, 136),
    ([256, 255, 257, 1, 0, 128], 0, 264, 200), ([700], 1, 520, 1000), ([3] * 61, 5, 1000, 2000),
    ([300, 513, 90], 300, 768, 512), ([33, 16, 15, 17], 0, 33, 77), ([0, 0, 0], 40, 64, 64),
    ([16] * 7 + [128] * 3, 0, 512, 320), ([129, 127, 640], 2, 2048, 72), ([1] * 1024, 8, 64, 128),
]


@pytest.mark.parametrize("counts,lost,N,K", CASES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("whole", [True, False])
def test_rows(counts, lost, N, K, dtype, whole):
    plan = plan_of(counts, lost)
    W = values((len(counts), N, K), 1, whole)
    for call, S, width, right in ((g.gemm_experts, K, N, W), (g.gemm_experts_backward_a, N, K, W.transpose(1, 2))):
        X = values((plan.rows, S), 2, whole)
        X[sum(counts):] = float("nan")          # nobody's rows are not used
        ref, mag = forward64(X, right, plan)
        check(call(X, W, plan, out_dtype=dtype), ref, mag, S, whole)
        buf, out = canvas((plan.rows, width), dtype, 3 if N % 16 else 8)
        assert call(X, W, plan, alpha=0.5, out=out) is out
        status()
        check(out, 0.5 * ref, mag, S, whole and dtype == F32)
        assert torch.all(buf[:, width:] == 7)


@pytest.mark.parametrize("counts,lost,N,K", CASES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("whole", [True, False])
def test_weights(counts, lost, N, K, dtype, whole):
    plan = plan_of(counts, lost)
    dD, A = values((plan.rows, N), 3, whole), values((plan.rows, K), 4, whole, pad=8)
    dD[sum(counts):] = float("nan")
    A[sum(counts):] = float("nan")
    ref, mag = weights64(dD, A, plan)
    check(g.gemm_experts_backward_w(dD, A, plan, out_dtype=dtype), ref, mag, max(counts), whole)
    status()
    # added to what is there, in place, in a padded buffer
    buf, out = canvas((len(counts), N, K), dtype, 3 if K % 16 else 8)
    start = torch.randint(-8, 9, out.shape, generator=gen(5), device="cuda").to(dtype)
    out.copy_(start)
    g.gemm_experts_backward_w(dD, A, plan, beta=2.0, C=out, out=out)
    status()
    check(out, ref + 2 * start.double(), mag + 2 * start.double().abs(), max(counts), whole)
    assert torch.all(buf[..., K:] == 7)
    # and from another buffer, with a factor
    C = start.clone()
    got = g.gemm_experts_backward_w(dD, A, plan, alpha=0.5, beta=-1.0, C=C)
    assert got.dtype == dtype and torch.equal(C, start)
    check(got, 0.5 * ref - start.double(), mag + start.double().abs(), max(counts), whole and dtype == F32)


@pytest.mark.parametrize("act", [g.ACT_RELU, g.ACT_GELU, g.ACT_GELU_TANH, g.ACT_SILU])
@pytest.mark.parametrize("counts", [[5, 0, 40], [300, 200, 77]])
def test_activation(act, counts):
    """The activations' slopes lie in [-0.13, 1.13]; their own error is a few fp32 steps of the value (2^-20)."""
    plan = plan_of(counts, 9)
    A, W = values((plan.rows, 200), 1, False), values((3, 136, 200), 2, False) * 200 ** -0.5
    ref, mag = forward64(A, W, plan)
    fn = {g.ACT_RELU: torch.relu, g.ACT_GELU: torch.nn.functional.gelu, g.ACT_SILU: torch.nn.functional.silu,
          g.ACT_GELU_TANH: lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[act]
    for dtype in (BF16, F32):
        got = g.gemm_experts(A, W, plan, activation=act, out_dtype=dtype)
        status()
        bound = 1.2 * 202 * 2.0 ** -23 * mag + 2.0 ** -20 * ref.abs() + EPS[dtype] * 1.01 * fn(ref).abs()
        assert torch.all((got.double() - fn(ref)).abs() <= bound)
        assert torch.all(got[sum(counts):] == 0)


@pytest.mark.parametrize("counts", [[5, 7, 3, 11], [200, 130, 61, 300]])
def test_what_is_not_finite_stays_in_its_expert(counts):
    plan = plan_of(counts, 0)
    b = bounds_of(plan)
    for bad in (float("nan"), float("inf")):
        A, dD, W = values((plan.rows, 96), 1, True), values((plan.rows, 80), 2, True), values((4, 80, 96), 3, True)
        clean = g.gemm_experts(A, W, plan), g.gemm_experts_backward_a(dD, W, plan), g.gemm_experts_backward_w(dD, A, plan)
        A[b[1]:b[2]] = bad
        dD[b[2]:b[3], 5] = bad
        D, dA, dW = g.gemm_experts(A, W, plan), g.gemm_experts_backward_a(dD, W, plan), g.gemm_experts_backward_w(dD, A, plan)
        status()
        keep = torch.ones(plan.rows, dtype=torch.bool, device="cuda")
        keep[b[1]:b[2]] = False
        assert torch.equal(D[keep], clean[0][keep]) and not torch.isfinite(D[~keep]).any()
        keep[:] = True
        keep[b[2]:b[3]] = False
        assert torch.equal(dA[keep], clean[1][keep])
        assert torch.equal(dW[0], clean[2][0]) and torch.equal(dW[3], clean[2][3])
        assert torch.equal(dW[2, :5], clean[2][2, :5]) and torch.equal(dW[2, 6:], clean[2][2, 6:])


def test_gradients_against_differences():
    """d<out, D>/dA and /dW against differences of the product with fp32 results, on whole numbers: the product is
    linear in each, so the difference of one step is the gradient, and all sums are exact."""
    plan = plan_of([6, 0, 19], 2)
    A, W, out = values((plan.rows, 40), 1, True), values((3, 24, 40), 2, True), values((plan.rows, 24), 3, True)
    dA = g.gemm_experts_backward_a(out, W, plan, out_dtype=F32)
    dW = g.gemm_experts_backward_w(out, A, plan, out_dtype=F32)
    at = lambda: (out[:25].double() * g.gemm_experts(A, W, plan, out_dtype=F32)[:25].double()).sum()  # noqa: E731
    base = at()
    for t, grad, places in ((A, dA, [(0, 0), (5, 39), (6, 1), (24, 7)]), (W, dW, [(0, 0, 0), (2, 23, 39), (2, 4, 5), (1, 3, 3)])):
        for where in places:
            t[where] += 1
            assert at() - base == grad[where].double()
            t[where] -= 1
    assert torch.all(dA[25:] == 0)


@pytest.mark.parametrize("N,K", [(512, 256), (40, 72)])
def test_a_captured_step_follows_the_offsets(N, K):
    """One graph of all three calls, replayed after the plan, the rows and the matrices changed, beside eager calls."""
    T, k, E = 300, 2, 8
    plan = g.ExpertPlan(T, k, E, "cuda")
    ids = torch.zeros(T, k, dtype=torch.int64, device="cuda")
    X, W, dD = values((T, K), 1, True), values((E, N, K), 2, True), values((T * k, N), 3, True)

    def step():
        rows = g.expert_dispatch(ids, plan, X)
        return (g.gemm_experts(rows, W, plan, out_dtype=F32), g.gemm_experts_backward_a(dD, W, plan, out_dtype=F32),
                g.gemm_experts_backward_w(dD, rows, plan, out_dtype=F32))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = step()
    torch.cuda.current_stream().wait_stream(side)
    for seed in range(3):
        ids.copy_(torch.randint(-1, E if seed else 2, (T, k), generator=gen(seed), device="cuda"))
        X.copy_(values((T, K), 10 + seed, True))
        W.copy_(values((E, N, K), 20 + seed, True))
        graph.replay()
        got = [t.clone() for t in held]
        rows = g.expert_dispatch(ids, plan, X)
        status()
        for a, b in zip(got, (forward64(rows, W, plan)[0], forward64(dD, W.transpose(1, 2), plan)[0],
                              weights64(dD, rows, plan)[0])):
            assert torch.equal(a.double(), b)


@pytest.mark.parametrize("offsets", [[5, 3, 9, 1], [-7, 40, 90, 10 ** 9], [2 ** 31 - 1] * 4, [-2 ** 31] * 4, [0, 0, 0, 0]])
def test_plans_that_no_dispatch_filled(offsets):
    """Nothing outside the outputs is written; for offsets out of order the experts' rows are those up to the largest
    offset so far."""
    rows = 64
    i32 = dict(dtype=torch.int32, device="cuda")
    plan = g.ExpertPlan.of(torch.tensor(offsets, **i32), torch.zeros(rows, 1, **i32), torch.zeros(rows, **i32))
    A, dD, W = values((rows, 72), 1, True), values((rows, 40), 2, True), values((3, 40, 72), 3, True)
    big = torch.full((rows + 64, 40), 7.0, device="cuda")
    g.gemm_experts(A, W, plan, out=big[32:32 + rows])
    g.gemm_experts_backward_a(dD, W, plan)
    g.gemm_experts_backward_w(dD, A, plan)
    status()
    assert torch.all(big[:32] == 7) and torch.all(big[32 + rows:] == 7)
    top = 0
    row = [top := max(top, min(max(o, 0), rows)) for o in offsets]
    want = torch.zeros(rows, 40, dtype=torch.float64, device="cuda")
    for e in range(3):
        want[row[e]:row[e + 1]] = A[row[e]:row[e + 1]].double() @ W[e].double().T
    assert torch.equal(big[32 + row[0]:32 + rows].double(), want[row[0]:])


def test_another_stream():
    plan = plan_of([100, 40], 3)
    A, W = values((plan.rows, 512), 1, True), values((2, 264, 512), 2, True)
    ref = g.gemm_experts(A, W, plan)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = g.gemm_experts(A, W, plan, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, ref)


def test_empty_calls():
    plan = plan_of([0, 0], 0)
    A, dD, W = values((0, 64), 1, True), values((0, 32), 2, True), values((2, 32, 64), 3, True)
    assert g.gemm_experts(A, W, plan).shape == (0, 32)
    assert g.gemm_experts_backward_a(dD, W, plan).shape == (0, 64)
    out = torch.full((2, 32, 64), 3.0, device="cuda")
    assert torch.all(g.gemm_experts_backward_w(dD, A, plan, beta=2.0, C=out.clone(), out=out) == 6)
    assert torch.all(g.gemm_experts_backward_w(dD, A, plan, out=out) == 0)
    plan = plan_of([4, 5], 1)
    none = torch.empty(10, 0, device="cuda", dtype=BF16)
    assert torch.all(g.gemm_experts(none, torch.empty(2, 32, 0, device="cuda", dtype=BF16), plan) == 0)
    assert torch.all(g.gemm_experts_backward_a(none, torch.empty(2, 0, 32, device="cuda", dtype=BF16), plan) == 0)
    assert g.gemm_experts_backward_w(none, none, plan).shape == (2, 0, 0)
    status()


def test_tiles_without_a_sum_between_others_many_times():
    """CTA pairs that store zeros for rows of nobody, or for experts without rows, before, between and after tiles with
    long sums, one launch close behind another: the two CTAs of a pair must stay in step whichever is ahead."""
    plan = plan_of([900, 0, 0, 1800, 0, 333, 0], 700)
    A, dD, W = values((plan.rows, 1024), 1, True), values((plan.rows, 2048), 2, True), values((7, 2048, 1024), 3, True)
    first = None
    for _ in range(60):
        got = [(g.gemm_experts(A, W, plan), g.gemm_experts_backward_a(dD, W, plan),
                g.gemm_experts_backward_w(dD, A, plan)) for _ in range(3)]
        status()
        first = first or got[0]
        for three in got:
            assert all(torch.equal(a, b) for a, b in zip(three, first))
    check(first[0], *forward64(A, W, plan), 1024, True)
    check(first[1], *forward64(dD, W.transpose(1, 2), plan), 2048, True)
    check(first[2], *weights64(dD, A, plan), 1800, True)


def test_a_training_step_without_the_host():
    """Dispatch, two products, combine, the gradients of all, added up over two micro-batches, and the clip, captured in
    one graph and replayed on other tokens and routes, against the formulas in 64 bits.  Every stage rounds to bf16
    once (2^-9 of a value); norms of errors are compared with 2^-6 of the norms, eight times that."""
    T, k, E, H, F = 96, 2, 5, 64, 136
    x, dout = values((T, H), 1, False), values((T, H), 2, False)
    ids = torch.zeros(T, k, dtype=torch.int64, device="cuda")
    w = torch.rand(T, k, generator=gen(3), device="cuda")
    up, down = values((E, F, H), 4, False) * H ** -0.5, values((E, H, F), 5, False) * F ** -0.5
    plan = g.ExpertPlan(T, k, E, "cuda")
    sums = [torch.zeros(E, F, H, device="cuda"), torch.zeros(E, H, F, device="cuda")]
    clipped = [torch.empty_like(t, dtype=BF16) for t in sums]
    limit = 5.0

    def step():
        for i in range(2):
            rows = g.expert_dispatch(ids, plan, x)
            hidden = g.gemm_experts(rows, up, plan, activation=g.ACT_RELU)
            Y = g.gemm_experts(hidden, down, plan)
            out = g.expert_combine(plan, Y, w)
            dY, dw = g.expert_combine_backward(plan, Y, w, dout)
            dhidden = g.gemm_experts_backward_a(dY, down, plan) * (hidden > 0)
            for total, a, b in ((sums[1], dY, hidden), (sums[0], dhidden, rows)):
                g.gemm_experts_backward_w(a, b, plan, beta=float(i), C=total, out=total)
            dx = g.expert_dispatch_backward(plan, g.gemm_experts_backward_a(dhidden, up, plan))
        return out, dx, dw, g.clip_grad_norm(sums, limit, out=clipped)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = step()
    torch.cuda.current_stream().wait_stream(side)
    near = lambda a, b: ((a.double() - b).norm() <= 2.0 ** -6 * b.norm()).item()  # noqa: E731
    for seed in range(3):
        ids.copy_(torch.randint(-1, E, (T, k), generator=gen(70 + seed), device="cuda"))
        x.copy_(values((T, H), 80 + seed, False))
        graph.replay()
        status()
        wide = [t.double().requires_grad_() for t in (x, w, up, down)]
        y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            e = ids[:, j].clamp(min=0)
            h = torch.relu(torch.einsum("th,tfh->tf", wide[0], wide[2][e]))
            y = y + ((ids[:, j] >= 0) * wide[1][:, j])[:, None] * torch.einsum("tf,thf->th", h, wide[3][e])
        y.backward(dout.double())
        out, dx, dw, norm = held
        gx, gw, gup, gdown = [t.grad for t in wide]
        assert near(out, y.detach()) and near(dx, gx) and near(dw, gw * (ids >= 0))
        assert near(sums[0], 2 * gup) and near(sums[1], 2 * gdown)
        want = 2 * torch.sqrt(gup.square().sum() + gdown.square().sum())
        assert abs(norm.item() - want.item()) <= 2.0 ** -6 * want.item()
        for c, t in zip(clipped, sums):
            assert torch.all((c.double() - t.double() * min(1.0, limit / norm.item())).abs() <= 2.0 ** -8 * 1.01 * t.double().abs())


@pytest.mark.parametrize("what", ["rows", "columns"])
def test_places_beyond_2_31(what):
    """Outputs and operands of more than 2^31 elements, a few of whose values are looked at."""
    if torch.cuda.get_device_properties(0).total_memory < 60 << 30:
        pytest.skip("needs 60 GB")
    R, N, K, E = (70000, 40000, 64, 3) if what == "rows" else (64, 1 << 15, 1 << 15, 3)
    counts = [R - 30, 0, 29]
    plan = plan_of(counts, 1)
    A, W = values((R, K), 1, True), values((E, N, K), 2, True)
    D = g.gemm_experts(A, W, plan)
    status()
    rows = torch.tensor([0, R // 2, R - 31, R - 30, R - 2, R - 1], device="cuda")
    cols = torch.tensor([0, 1, N // 2, N - 1], device="cuda")
    for r in rows.tolist():
        e = 0 if r < counts[0] else 2 if r < R - 1 else None
        want = torch.zeros(len(cols), dtype=torch.float64, device="cuda") if e is None else W[e][cols].double() @ A[r].double()
        assert torch.equal(D[r, cols], want.to(F32).to(BF16))
    dD = D.clamp_(-3, 3)
    dD[R - 1] = 1.0
    dA = g.gemm_experts_backward_a(dD, W, plan, out_dtype=F32)
    for r in (0, R - 30, R - 2):
        e = 0 if r < counts[0] else 2
        assert torch.equal(dA[r].double(), dD[r].double() @ W[e].double())
    assert torch.all(dA[R - 1] == 0)
    del D, dA
    dW = g.gemm_experts_backward_w(dD, A, plan)
    status()
    for e, lo, hi in ((0, 0, counts[0]), (2, counts[0], R - 1)):
        want = dD[lo:hi, cols].double().T @ A[lo:hi].double()
        assert torch.equal(dW[e, cols], want.to(F32).to(BF16))
    assert torch.all(dW[1] == 0)


SEGMENT = 768      # terms that an fp32 result's sum takes between two rounded additions


@pytest.mark.parametrize("terms", [769, 832, 1536, 1537, 2304, 2305, 4096, 5000])
@pytest.mark.parametrize("counts", [[5, 0, 40], [300, 1, 128, 0, 257]])
def test_long_sums_of_products_in_fp32(terms, counts):
    """Whole numbers come out exactly at lengths around whole segments, few rows and many."""
    plan, N = plan_of(counts, 3), 200
    A, W = values((sum(counts) + 3, terms), 41, True), values((len(counts), N, terms), 42, True)
    buf, D = canvas((A.shape[0], N), F32, 5)
    g.gemm_experts(A, W, plan, out=D)
    check(D, forward64(A, W, plan)[0], None, terms, True)
    assert torch.all(buf[:, N:] == 7)
    dD, W = values((sum(counts) + 3, terms), 43, True), values((len(counts), terms, N), 44, True)
    dA = g.gemm_experts_backward_a(dD, W, plan, out_dtype=F32)
    check(dA, forward64(dD, W.transpose(1, 2), plan)[0], None, terms, True)
    status()


@pytest.mark.parametrize("counts", [[0, 1, 767, 768, 769, 1536, 1537, 2305, 5000], [9000, 0, 16], [3001, 2999]])
@pytest.mark.parametrize("with_c", [True, False])
def test_long_sums_of_weights_in_fp32(counts, with_c):
    """Experts of few rows and of many in one call, in place and with pitches of no alignment."""
    plan, N, K = plan_of(counts, 2), 300, 270
    dD, A = values((sum(counts) + 2, N), 45, True), values((sum(counts) + 2, K), 46, True)
    buf, dW = canvas((len(counts), N, K), F32, 3)
    C = torch.randint(-99, 100, dW.shape, generator=gen(47), device="cuda").float()
    dW.copy_(C)
    g.gemm_experts_backward_w(dD, A, plan, out=dW, beta=1.0 if with_c else 0.0, C=dW if with_c else None)
    check(dW, weights64(dD, A, plan)[0] + (C.double() if with_c else 0), None, 0, True)
    assert torch.all(buf[..., K:] == 7)
    status()


def test_fp32_results_keep_their_bits_over_long_sums():
    """Terms of one sign, where what the tensor core cuts off adds up.  Within a segment of 48 MMAs each one loses
    less than two units of 2^-23 of the sum (its terms' alignment, its result); the segments are added rounded."""
    terms, rows, N = 32768, 40, 136
    bound = (2 * SEGMENT // 16 + -(-terms // SEGMENT) + 2) * 2.0 ** -23

    def positive(shape, seed):
        return (torch.rand(shape, generator=gen(seed), device="cuda") / 2 + 0.5).to(BF16)

    def near(got, ref):
        assert torch.all((got.double() - ref).abs() <= bound * ref)

    plan = plan_of([rows], 0)
    A, W = positive((rows, terms), 51), positive((1, N, terms), 52)
    near(g.gemm_experts(A, W, plan, out_dtype=F32), forward64(A, W, plan)[0])
    Wt = W.transpose(1, 2).contiguous()
    near(g.gemm_experts_backward_a(A, Wt, plan, out_dtype=F32), forward64(A, W, plan)[0])
    plan = plan_of([terms], 0)
    dD, A = positive((terms, N), 53), positive((terms, rows), 54)
    near(g.gemm_experts_backward_w(dD, A, plan, out_dtype=F32), weights64(dD, A, plan)[0])
    status()


@pytest.mark.parametrize("act", [g.ACT_RELU, g.ACT_GELU, g.ACT_GELU_TANH, g.ACT_SILU])
def test_activation_of_long_sums_in_fp32(act):
    plan, terms = plan_of([300, 0, 77], 9), 1000
    A, W = values((plan.rows, terms), 61, False), values((3, 136, terms), 62, False) * terms ** -0.5
    ref, mag = forward64(A, W, plan)
    fn = {g.ACT_RELU: torch.relu, g.ACT_GELU: torch.nn.functional.gelu, g.ACT_SILU: torch.nn.functional.silu,
          g.ACT_GELU_TANH: lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[act]
    got = g.gemm_experts(A, W, plan, alpha=2.0, activation=act, out_dtype=F32)
    bound = 1.2 * (terms + 2) * 2.0 ** -23 * 2 * mag + 2.0 ** -20 * 2 * ref.abs() + EPS[F32] * 1.01 * fn(2 * ref).abs()
    assert torch.all((got.double() - fn(2 * ref)).abs() <= bound)
    assert torch.all(got[sum(plan.offsets.diff().tolist()):] == 0)
    status()


def test_what_is_not_finite_stays_in_its_expert_over_long_sums():
    plan, N, K = plan_of([1601, 770, 903], 0), 800, 840
    b = bounds_of(plan)
    A, dD, W = values((plan.rows, K), 63, True), values((plan.rows, N), 64, True), values((3, N, K), 65, True)
    C = torch.randint(-99, 100, (3, N, K), generator=gen(66), device="cuda").float()

    def run():
        return (g.gemm_experts(A, W, plan, out_dtype=F32), g.gemm_experts_backward_a(dD, W, plan, out_dtype=F32),
                g.gemm_experts_backward_w(dD, A, plan, beta=1.0, C=C))

    clean = run()
    A[b[1]:b[2]] = float("nan")
    dD[b[1]:b[2], 5] = float("inf")
    C[2, 7, 9] = float("nan")
    got = run()
    status()
    keep = torch.ones(plan.rows, dtype=torch.bool, device="cuda")
    keep[b[1]:b[2]] = False
    for x, y in zip(got[:2], clean[:2]):
        assert torch.equal(x[keep], y[keep]) and not torch.isfinite(x[~keep]).any()
    other = torch.ones((N, K), dtype=torch.bool, device="cuda")
    other[7, 9] = False
    assert torch.equal(got[2][0], clean[2][0]) and torch.isnan(got[2][1]).all()
    assert torch.equal(got[2][2][other], clean[2][2][other]) and torch.isnan(got[2][2][7, 9])


def test_a_captured_long_sum_follows_the_offsets():
    """One graph, replayed with other row counts: few, none, and more than a segment, on tiles of both accumulators."""
    E, N, K, rows = 4, 136, 832, 4000
    plan = plan_of([1000] * 4, 0)
    A, dD, W = values((rows, K), 71, True), values((rows, N), 72, True), values((E, N, K), 73, True)
    D, dW = torch.empty(rows, N, device="cuda"), torch.empty(E, N, K, device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.gemm_experts(A, W, plan, out=D)
        g.gemm_experts_backward_w(dD, A, plan, out=dW)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            g.gemm_experts(A, W, plan, out=D)
            g.gemm_experts_backward_w(dD, A, plan, out=dW)
    torch.cuda.current_stream().wait_stream(side)
    for counts in ([4000, 0, 0, 0], [1, 0, 3998, 1], [0, 0, 0, 0], [769, 1537, 15, 1600], [5, 6, 7, 8]):
        plan.offsets.copy_(plan_of(counts, 0).offsets)
        for _ in range(3):
            graph.replay()
        status()
        check(D, forward64(A, W, plan)[0], None, K, True)
        check(dW, weights64(dD, A, plan)[0], None, 0, True)
