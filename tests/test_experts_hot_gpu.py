"""fp32 weights' gradients of experts whose rows are far from the average of their call.

Bound.  The tensor core adds 16 products at a step and cuts the sum S_j after
step j off at its last place, an error of U units, U spread over [0, 1).  The
root of its mean square is sqrt(1 / 3) units, and a unit is at most 2^-23 of a
normal sum, sqrt(0.52) 2^-23 of it in the root of the mean square over a binary
order (the mean of 1 / m^2 over 1 <= m < 2, m equally likely in the logarithm,
is 0.54; in itself 0.5).  So a step leaves below 0.43 2^-23 of |S_j|, and |S_j|
is sqrt(j / J) of what it is after all J steps of a segment.  Added up as if all
were in one direction: 0.43 2^-23 (2 J / 3 + 1 / 2).  J is at most 52 (twelve
blocks of 64 terms and what is left of one): 1.81e-6.  Segments are independent,
so their errors grow as their sum does.  Joining n of them rounds n times,
below 2^-25 sqrt(n / 2) of the result: 0.13e-6 for n = 40.  Together below 2e-6
of the norm, at any length and whatever the other experts have.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

g = pytest.importorskip("tensor_core_dense_tn_gb300")
from test_experts_gpu import gen, plan_of, status, values  # noqa: E402

NORM_EPS = 2e-6


@pytest.mark.parametrize("counts", [[16000] + [100] * 63, [30, 8192] + [40] * 60, [1] * 100 + [30000],
                                    [0] * 7 + [9001, 0, 831, 833], [500] * 20 + [20000, 0, 17], [1000, 24000, 64]],
                         ids=lambda c: f"{max(c)} of {sum(c)} by {len(c)}")
@pytest.mark.parametrize("with_c", [False, True])
@pytest.mark.parametrize("N,K", [(136, 200), (512, 264)])
def test_an_experts_accuracy_is_its_own(counts, with_c, N, K):
    plan = plan_of(counts, 5)
    dD, A = values((plan.rows, N), 81, False), values((plan.rows, K), 82, False)
    C = torch.randn(len(counts), N, K, generator=gen(83), device="cuda") if with_c else None
    got = g.gemm_experts_backward_w(dD, A, plan, beta=1.0 if with_c else 0.0, C=C, out_dtype=torch.float32)
    status()
    at = 0
    for e, n in enumerate(counts):
        ref = dD[at:at + n].double().T @ A[at:at + n].double()
        if with_c:
            ref += C[e].double()
        at += n
        assert (got[e].double() - ref).norm() <= NORM_EPS * ref.norm()


@pytest.mark.parametrize("rows", [700, 769, 832, 5000])
def test_an_experts_bits_do_not_depend_on_the_others(rows):
    """Alone, among many of few rows, and beside one of many: the same terms in the same order."""
    N, K = 264, 136
    dD, A = values((rows, N), 84, False), values((rows, K), 85, False)
    alone = g.gemm_experts_backward_w(dD, A, plan_of([rows], 0), out_dtype=torch.float32)[0]
    for others in ([3] * 90, [20000], [900] * 4):
        n = sum(others)
        plan = plan_of(others + [rows], 0)
        more = [torch.cat([values((n, w), 86, False), t]) for w, t in ((N, dD), (K, A))]
        got = g.gemm_experts_backward_w(*more, plan, out_dtype=torch.float32)[-1]
        status()
        assert torch.equal(got, alone)


def test_products_keep_their_accuracy_beside_a_hot_expert():
    """Products segment by the sum's length, which all experts share."""
    counts, N, K = [4000] + [9] * 31, 200, 5000
    plan = plan_of(counts, 0)
    A, W = values((plan.rows, K), 87, False), values((32, N, K), 88, False)
    got = g.gemm_experts(A, W, plan, out_dtype=torch.float32)
    status()
    at = 0
    for e, n in enumerate(counts):
        ref = A[at:at + n].double() @ W[e].double().T
        assert (got[at:at + n].double() - ref).norm() <= NORM_EPS * ref.norm()
        at += n
