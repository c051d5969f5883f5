"""Expert rows in the shapes that reach every loop of the copying and adding kernels, and their outputs' padding.

Bounds as in test_expert_gpu: fp32 sums of n terms are within n 2^-23 of the
sum of the magnitudes, plus the rounding of the output.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

g = pytest.importorskip("tensor_core_dense_tn_gb300")

from test_expert_gpu import DT, OUT_EPS, gen, make_plan, rows_like, slot_rows64, status  # noqa: E402


def padded(n, H, dtype, pad, shift):
    """An n x H matrix of NaN with `pad` elements after each row, `shift` before the first, and the whole buffer."""
    whole = torch.full((shift + n * (H + pad) + 8,), float("nan"), device="cuda", dtype=DT[dtype])
    return whole[shift:shift + n * (H + pad)].view(n, H + pad)[:, :H], whole


def padding_untouched(whole, n, H, pad, shift):
    at = torch.arange(whole.numel(), device="cuda") - shift
    inside = (at >= 0) & (at < n * (H + pad)) & (at % (H + pad) < H)
    return bool(whole[~inside].isnan().all())


def random_plan(T, k, E, seed, dropped=0.1):
    """A plan filled by the library, whose sort has tests of its own."""
    r = gen(seed)
    ids = torch.randint(0, E, (T, k), generator=r, device="cuda")
    ids[torch.rand(T, k, generator=r, device="cuda") < dropped] = -1
    plan = g.ExpertPlan(T, k, E, "cuda")
    g.expert_dispatch(ids, plan)
    return ids, plan, plan.slot_row.long()


def check_sum(out, terms, k, dtype):
    ref, mag = terms.sum(1), terms.abs().sum(1)
    assert torch.all((out.double() - ref).abs() <= k * 2.0 ** -23 * mag + OUT_EPS[dtype] * ref.abs())


# more blocks than the GPU holds at once, so that each block takes several tokens, on wide and on narrow rows
@pytest.mark.parametrize("T,H,dtype", [(9001, 4096, "bf16"), (9001, 4097, "bf16"), (9001, 4098, "bf16"), (9001, 2050, "f32"),
                                       (7003, 2048, "f32"), (400001, 8, "bf16"), (400001, 7, "f32")])
@pytest.mark.parametrize("k", [1, 2, 3])
def test_sums_of_many_tokens(T, H, dtype, k):
    _, plan, slot_row = random_plan(T, k, 61, T + H)
    Y = rows_like(T * k, H, dtype, 2)
    w = torch.randn(T, k, generator=gen(3), device="cuda")
    out = torch.full((T, H), float("nan"), device="cuda", dtype=DT[dtype])
    g.expert_combine(plan, Y, w, out=out)
    rows = slot_rows64(Y, slot_row)
    check_sum(out, rows * w.double()[..., None], k, dtype)
    out.fill_(float("nan"))
    g.expert_dispatch_backward(plan, Y, out=out)
    check_sum(out, rows, k, dtype)
    status()


# rows longer than a block copies at once, with enough tokens that one block has the whole row
@pytest.mark.parametrize("T,k", [(700, 2), (5000, 1)])
@pytest.mark.parametrize("H,dtype", [(8192, "f32"), (8201, "f32"), (8192, "bf16"), (8201, "bf16"), (12290, "bf16")])
def test_copies_of_long_rows(T, k, H, dtype):
    X = rows_like(T, H, dtype, 1)
    ids, plan, _ = random_plan(T, k, 16, H)
    out = torch.full((T * k, H), float("nan"), device="cuda", dtype=DT[dtype])
    g.expert_dispatch(ids, plan, X, out=out)
    status()
    tok = plan.row_token.long()
    assert torch.equal(out, torch.where((tok >= 0)[:, None], X[tok.clamp(min=0)], torch.zeros((), device="cuda", dtype=X.dtype)))
    assert int((tok < 0).sum()) > 0


@pytest.mark.parametrize("H,pad,shift", [(40, 24, 8), (40, 3, 0), (33, 1, 0), (34, 2, 2), (257, 6, 1), (1, 2, 3), (4100, 4, 0)])
@pytest.mark.parametrize("T,k", [(5, 1), (77, 2), (300, 4), (90, 12), (5003, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_is_written_beside_the_rows(H, pad, shift, T, k, dtype):
    E = 9
    ids, plan, slot_row = random_plan(T, k, E, H + k, 0.3)
    n = T * k
    X, Y, dout = (rows_like(m, H, dtype, 20 + i) for i, m in enumerate((T, n, T)))
    w = torch.randn(T, k, generator=gen(3), device="cuda")
    for rows, call in ((n, lambda o: g.expert_dispatch(ids, plan, X, out=o)),
                       (T, lambda o: g.expert_dispatch_backward(plan, Y, out=o)),
                       (T, lambda o: g.expert_combine(plan, Y, w, out=o)),
                       (n, lambda o: g.expert_combine_backward(plan, Y, w, dout, dY=o))):
        out, whole = padded(rows, H, dtype, pad, shift)
        call(out)
        assert not bool(out.isnan().any())
        assert padding_untouched(whole, rows, H, pad, shift)
    dw, whole = padded(T, k, "f32", 5, 1)
    g.expert_combine_backward(plan, Y, w, dout, dweights=dw)
    assert not bool(dw.isnan().any()) and padding_untouched(whole, T, k, 5, 1)
    status()


def test_make_plan_and_the_sort_agree():
    """The plans of these tests and those built by the definition are the same."""
    plan, slot_row = make_plan(333, 3, 61, 4, "dropped")
    ids = torch.full((333, 3), -1, device="cuda")
    ends = torch.searchsorted(plan.offsets[1:].contiguous(), slot_row.clamp(min=0).int(), right=True)
    ids[slot_row >= 0] = ends[slot_row >= 0]
    again = g.ExpertPlan(333, 3, 61, "cuda")
    g.expert_dispatch(ids, again)
    assert torch.equal(again.offsets, plan.offsets) and torch.equal(again.slot_row, plan.slot_row)
    assert torch.equal(again.row_token, plan.row_token)
