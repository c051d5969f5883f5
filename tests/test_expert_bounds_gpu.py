"""Expert calls at the edges of what they accept: plans that no dispatch filled, sizes near 2^31, padding.

Everything a call may not touch lies inside a larger allocation of the test's
own, filled with a value that is looked for afterwards.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

g = pytest.importorskip("tensor_core_dense_tn_gb300")


def status():
    assert g.gemm_get_status(torch.cuda.current_stream().cuda_stream) == 0


def guarded(n, H, dtype, rows_around):
    """An n x H matrix of NaN with rows_around more of them before and behind, and the whole."""
    whole = torch.full((n + 2 * rows_around, H), float("nan"), device="cuda", dtype=dtype)
    return whole[rows_around:rows_around + n], whole


def untouched(whole, rows_around):
    return bool(whole[:rows_around].isnan().all() and whole[-rows_around:].isnan().all())


@pytest.mark.parametrize("filled", [-1, -5, -(1 << 31), 41, (1 << 31) - 1])
@pytest.mark.parametrize("H", [32, 33])
def test_number_of_rows_of_a_foreign_plan_is_checked(filled, H):
    """The combine's gradient zeroes dY from row offsets[E] on: a value outside [0, T k] counts as the nearer end."""
    T, k, E = 20, 2, 4
    plan = g.ExpertPlan(T, k, E, "cuda")
    g.expert_dispatch(torch.randint(0, E, (T, k), device="cuda"), plan)
    plan.offsets[E] = filled
    slot_row = plan.slot_row.long()
    Y, dout, w = torch.randn(T * k, H, device="cuda"), torch.randn(T, H, device="cuda"), torch.rand(T, k, device="cuda")
    dY, whole = guarded(T * k, H, torch.float32, 64)
    _, dw = g.expert_combine_backward(plan, Y, w, dout, dY=dY)
    status()
    assert untouched(whole, 64)
    terms = Y.double()[slot_row] * dout.double()[:, None]
    ref, mag = terms.sum(-1), terms.abs().sum(-1)      # a lane adds H / 32 products, then 5 + 8 joins
    assert torch.all((dw.double() - ref).abs() <= (H / 32 + 32) * 2.0 ** -23 * mag + 2.0 ** -24 * ref.abs())
    if filled > 0:
        assert torch.equal(dY[slot_row], w[..., None] * dout[:, None])


def free_gigabytes():
    torch.cuda.empty_cache()
    return torch.cuda.mem_get_info()[0] / 2 ** 30


def ramp(n, dtype, period=251):
    """0 1 .. period - 1 0 1 .. over n elements, made in pieces."""
    out = torch.empty(n, dtype=dtype, device="cuda")
    step = period << 20
    piece = (torch.arange(min(n, step), device="cuda") % period).to(dtype)
    for lo in range(0, n, step):
        out[lo:lo + step] = piece[:min(step, n - lo)]
    return out


def equal_in_pieces(a, b, step=1 << 28):
    return all(torch.equal(a[lo:lo + step], b[lo:lo + step]) for lo in range(0, a.shape[0], step))


def test_rows_past_the_last_with_half_of_2_to_the_31_tokens():
    """offsets[E] + t passes 2^31 here: no row is set to zero, not one in front of the matrix either."""
    if free_gigabytes() < 60:
        pytest.skip("needs 60 GB")
    T = (1 << 30) + 9
    plan = g.ExpertPlan(T, 1, 1, "cuda")
    X = ramp(T, torch.bfloat16).view(T, 1)
    front = 1 << 31
    whole = torch.full((front + T, 1), float("nan"), device="cuda", dtype=torch.bfloat16)
    g.expert_dispatch(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), plan, X, out=whole[front:])
    status()
    assert plan.offsets.tolist() == [0, T]
    assert equal_in_pieces(whole[front:], X)
    assert all(bool(part.isnan().all()) for part in whole[:front].split(1 << 28))
    whole[front:].fill_(float("nan"))
    w = torch.ones(T, 1, device="cuda", dtype=torch.bfloat16)
    _, dw = g.expert_combine_backward(plan, X, w, X, dY=whole[front:])
    status()
    assert equal_in_pieces(whole[front:], X)
    assert all(bool(part.isnan().all()) for part in whole[:front].split(1 << 28))
    assert equal_in_pieces(dw, X * X)       # one product each, rounded once
    del plan, X, whole, w, dw
    torch.cuda.empty_cache()


def test_plan_of_the_most_slots():
    """The last slots that a plan may have, nearly all of them dropped."""
    if free_gigabytes() < 60:
        pytest.skip("needs 60 GB")
    n, E = (1 << 31) - 4097, 2
    ids = torch.full((n, 1), -1, dtype=torch.int32, device="cuda")
    ids[0], ids[n // 2], ids[n - 1] = 1, 1, 0
    plan = g.ExpertPlan(n, 1, E, "cuda")
    plan.row_token.fill_(-99)
    g.expert_dispatch(ids, plan)
    status()
    assert plan.offsets.tolist() == [0, 1, 3]
    assert plan.row_token[:3].tolist() == [n - 1, 0, n // 2]
    assert [plan.slot_row[t].item() for t in (n - 1, 0, n // 2)] == [0, 1, 2]
    assert all(bool((part == -1).all()) for part in plan.row_token[3:].split(1 << 28))
    assert sum(int((part != -1).sum()) for part in plan.slot_row.split(1 << 28)) == 3
    del plan, ids
    torch.cuda.empty_cache()


@pytest.mark.parametrize("H,weighted", [(1, False), (1, True), (8, False), (8, True)])
def test_combine_of_the_most_tokens(H, weighted):
    """The blocks that walk over the tokens (of rows in 16-byte chunks) stop at the last one, also where the next step
    passes 2^31."""
    if free_gigabytes() < 50 + 10 * H:
        pytest.skip("needs 60 or 130 GB")
    T = (1 << 31) - 4097
    slot_row = torch.arange(T, dtype=torch.int32, device="cuda").view(T, 1)
    plan = g.ExpertPlan.of(torch.tensor([0, T], dtype=torch.int32, device="cuda"), slot_row, slot_row.view(-1))
    Y = ramp(T * H, torch.bfloat16).view(T, H)
    if weighted:
        out = g.expert_combine(plan, Y, torch.ones(T, 1, dtype=torch.bfloat16, device="cuda"))
    else:
        out = g.expert_dispatch_backward(plan, Y)
    status()
    assert equal_in_pieces(out, Y, 1 << 26)
    del plan, slot_row, Y, out
    torch.cuda.empty_cache()


def test_the_longest_rows():
    """One row of nearly 2^31 elements, moved one at a time (an odd pitch) and in 16-byte chunks with a tail."""
    if free_gigabytes() < 60:
        pytest.skip("needs 60 GB")
    H = (1 << 31) - 5
    ids = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    w = torch.ones(1, 1, device="cuda")
    X = ramp(H, torch.bfloat16, 2)                # 0 1 0 1 ..: sums of fewer than 2^24 products are exact
    for pitch in (H, H + 5):
        plan = g.ExpertPlan(1, 1, 1, "cuda")
        matrix = lambda t: t.as_strided((1, H), (pitch, 1))  # noqa: E731
        row = torch.empty(pitch, dtype=torch.bfloat16, device="cuda")
        row[:H] = X
        out = torch.full((pitch,), float("nan"), dtype=torch.bfloat16, device="cuda")
        g.expert_dispatch(ids, plan, matrix(row), out=matrix(out))
        status()
        assert equal_in_pieces(out[:H], X) and bool(out[H:].isnan().all())
        out.fill_(float("nan"))
        g.expert_combine(plan, matrix(row), w, out=matrix(out))
        status()
        assert equal_in_pieces(out[:H], X) and bool(out[H:].isnan().all())
        out.fill_(float("nan"))
        _, dw = g.expert_combine_backward(plan, matrix(row), w, matrix(row), dY=matrix(out))
        status()
        assert equal_in_pieces(out[:H], X) and bool(out[H:].isnan().all())
        # 256 lanes add fewer than 2^23 ones each, which is exact, then 8 + 8 rounded joins
        ones = H // 2
        assert abs(dw.item() - ones) <= 16 * 2.0 ** -24 * ones
        del row, out
    del X
    torch.cuda.empty_cache()


@pytest.mark.parametrize("K,parts", [(256, 1), (2048, 8)])
@pytest.mark.parametrize("offsets,used", [([0, 40, 8, 8, 60], [(0, 8, 0), (8, 60, 3)]),
                                          ([30, 20, 20, 44, 60], [(20, 44, 2), (44, 60, 3)]),
                                          ([0, 20, 60, 8, 60], [(0, 8, 0), (20, 60, 3)]),
                                          ([0, 8, 8, 50, 44], [(0, 8, 0), (8, 44, 2), (44, 60, None)])])
def test_products_of_decreasing_offsets(K, parts, offsets, used):
    """Offsets that no dispatch makes: every part of a split product takes the same rows, an expert's up to the next
    one's first, and nothing outside the result is written."""
    rows, N, E = 60, 100, 4
    i32 = dict(dtype=torch.int32, device="cuda")
    plan = g.ExpertPlan.of(torch.tensor(offsets, **i32), torch.zeros(rows, 1, **i32), torch.arange(rows, **i32))
    codes = torch.randint(0, 256, (E, N, K // 2), device="cuda", dtype=torch.uint8)
    A = torch.randint(-2, 3, (rows, K), device="cuda").bfloat16()
    W = g.W4Matrix(codes, torch.ones(E, N, K // 128, device="cuda"), K=K, group=128)
    D, whole = guarded(rows, N, torch.float32, 64)
    g.gemm_w4_experts(A, W, plan, out=D)
    assert g.last_launch_info()["k_parts"] == parts
    status()
    assert untouched(whole, 64)
    q = torch.stack([codes & 15, codes >> 4], dim=-1).view(E, N, K).double() - 8      # whole numbers: exact sums
    for lo, hi, e in used:       # rows of one expert alone, or past the last (which are zero)
        want = torch.zeros(1, 1, device="cuda") if e is None else A[lo:hi].double() @ q[e].T
        assert torch.equal(D[lo:hi].double(), want.double().expand(hi - lo, N))


def sorted_plan(ids, E):
    key = ids.reshape(-1).long()
    order = torch.sort(key, stable=True).indices
    slot_row = torch.empty_like(order)
    slot_row[order] = torch.arange(key.numel(), device="cuda")
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device="cuda"))
    return offsets.int(), slot_row.int().view(ids.shape), (order // ids.shape[1]).int()


def holds(plan, want):
    return all(torch.equal(a, b) for a, b in zip((plan.offsets, plan.slot_row, plan.row_token), want))


@pytest.mark.parametrize("with_rows", [False, True])
def test_a_captured_sort_owns_its_memory(with_rows):
    """A dispatch of many slots captured on a stream that has seen none, replayed on another stream while larger ones
    run on the first: every plan comes out right, so the two share nothing."""
    T, k, E, H = 40000, 2, 61, 24
    ids = torch.randint(0, E, (T, k), device="cuda")
    X = torch.randn(T, H, device="cuda") if with_rows else None
    more = torch.randint(0, 1024, (500000, 4), device="cuda", dtype=torch.int32)
    plan, larger = g.ExpertPlan(T, k, E, "cuda"), g.ExpertPlan(500000, 4, 1024, "cuda")
    out = torch.empty(T * k, H, device="cuda") if with_rows else None
    want, want_larger = sorted_plan(ids, E), sorted_plan(more, 1024)
    torch.cuda.synchronize()
    captured, replayed = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=captured):
        g.expert_dispatch(ids, plan, X, out=out)
    for _ in range(5):
        for t in (plan.offsets, plan.slot_row, plan.row_token, larger.offsets, larger.slot_row, larger.row_token):
            t.fill_(-99)
        torch.cuda.synchronize()
        with torch.cuda.stream(captured):
            for _ in range(4):
                g.expert_dispatch(more, larger)
        with torch.cuda.stream(replayed):
            for _ in range(8):
                graph.replay()
        torch.cuda.synchronize()
        assert holds(plan, want) and holds(larger, want_larger)
        if with_rows:
            assert torch.equal(out, X[want[2].long()])
    status()


@pytest.mark.parametrize("T,k,E", [(4097, 1, 1024), (5000, 1, 1024), (1366, 3, 1000), (70000, 9, 1024), (66000, 1, 7)])
@pytest.mark.parametrize("H", [0, 8])
def test_histograms_fit_the_plan(T, k, E, H):
    """Sorts whose histograms are nearly as large as the plan's arrays, with and without rows; dropped slots."""
    ids = torch.randint(-E // 4, E, (T, k), device="cuda")
    whole = torch.full((E + 1 + 2 * T * k + 128,), -99, dtype=torch.int32, device="cuda")
    n = T * k
    parts = whole[32:32 + n].view(T, k), whole[64 + n:64 + 2 * n], whole[96 + 2 * n:97 + 2 * n + E]
    plan = g.ExpertPlan.of(parts[2], parts[0], parts[1])
    X = torch.randn(T, H, device="cuda")
    Xs = g.expert_dispatch(ids, plan, X if H else None)
    status()
    key = torch.where(ids < 0, torch.full_like(ids, E), ids).reshape(-1)
    by, order = torch.sort(key, stable=True)
    V = int((by < E).sum())
    assert torch.equal(plan.offsets.long(), torch.searchsorted(by, torch.arange(E + 1, device="cuda")))
    assert torch.equal(plan.row_token[:V].long(), order[:V] // k) and bool((plan.row_token[V:] == -1).all())
    rows = torch.full((n,), -1, device="cuda")
    rows[order[:V]] = torch.arange(V, device="cuda")
    assert torch.equal(plan.slot_row.view(-1).long(), rows)
    for lo, hi in ((0, 32), (32 + n, 64 + n), (64 + 2 * n, 96 + 2 * n), (97 + 2 * n + E, len(whole))):
        assert bool((whole[lo:hi] == -99).all())
    if H:
        assert torch.equal(Xs[:V], X[order[:V] // k]) and bool((Xs[V:] == 0).all())


def test_gradients_of_a_plan_filled_again_raise():
    """Two layers with one plan, forward twice before backward: the first layer's gradients would be wrong."""
    from test_expert_example import example, setup
    ex = example()
    T, k, E, H = 20, 2, 4, 64
    _, _, _, x, dout = setup(T, k, E, H, 32)
    x.requires_grad_()
    plan, w = g.ExpertPlan(T, k, E, "cuda"), torch.rand(T, k, device="cuda", requires_grad=True)
    ids = [torch.randint(0, E, (T, k), device="cuda") for _ in range(2)]
    rows = ex.Dispatch.apply(x, ids[0], plan)
    y = ex.Combine.apply(rows, w, plan)
    y.backward(dout, retain_graph=True)
    want = 0.5 * x.grad
    g.expert_dispatch(ids[1], plan)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward(dout)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        rows.backward(torch.ones_like(rows))
    assert torch.equal(0.5 * x.grad, want)
