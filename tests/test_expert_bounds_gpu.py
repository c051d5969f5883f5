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
    assert torch.allclose(dw, (Y[slot_row] * dout[:, None]).sum(-1), rtol=1e-4, atol=1e-4)
    if filled > 0:
        assert torch.equal(dY[slot_row], w[..., None] * dout[:, None])
