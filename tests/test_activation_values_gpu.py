"""Activations of values that a working model does not make: not finite, and far from zero.

Each row of the product is one value v (v times one), so that the activation's
argument is known exactly.  The expected values are the formulas in 64 bits;
what they make of a NaN or of -infinity times zero is NaN, and a NaN that came
out as a number would hide a model that has diverged.

Bounds.  ReLU is exact.  The logistic forms' argument t is rounded a few times
(below 4 2^-24 of itself), which moves e^t by as much times |t|; the exponential
adds 2 units, or 2^-22 of the value per unit of t where the result is bf16, the
add and the divide 3 units: below (6 |t| + 16) 2^-23 of the value, 2^-13.9 for the largest
|t| whose exponential is finite (89), 2^-13 with what that leaves out.  Where the
divisor passes 2^126 the result is zero, |v| 2^-126 from the value; |v| is below
89 there, or the value itself is smaller than that.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

g = pytest.importorskip("tensor_core_dense_tn_gb300")

BF16, F32 = torch.bfloat16, torch.float32
NAN, INF = math.nan, math.inf
FORMULAS = {
    g.ACT_RELU: lambda v: torch.where(v.isnan(), v, v.clamp(min=0)),
    g.ACT_GELU: lambda v: v * (0.5 * (1 + torch.erf(v / 2 ** 0.5))),
    g.ACT_GELU_TANH: lambda v: v * (0.5 * (1 + torch.tanh((2 / math.pi) ** 0.5 * (v + 0.044715 * v ** 3)))),
    g.ACT_SILU: lambda v: v / (1 + torch.exp(-v)),
}
ACTS = list(FORMULAS)
# the erf form loses its bits below -2 by its own formula in fp32: no values between there and -6
VALUES = [NAN, INF, -INF, 0.0, -0.0, 1.0, -1.0, 5.5, 40.0, -40.0, -75.0, -79.5, -80.5, -85.0, -87.5, -88.5, -89.0, -100.0,
          -104.0, -1000.0, -1e10, -1e30, -3e38, 100.0, 1e4, 1e30, 3e38]


def column(rows, width, dtype=BF16):
    """Row r is VALUES[r] and zeros."""
    A = torch.zeros(rows, width, device="cuda", dtype=dtype)
    A[:, 0] = torch.tensor([VALUES[r % len(VALUES)] for r in range(rows)], device="cuda").to(dtype)
    return A


def ones(shape):
    W = torch.zeros(shape, device="cuda", dtype=BF16)
    W[..., 0] = 1
    return W


def near(D, v, act):
    v = v.double()[:, None].expand(D.shape)
    want, got = FORMULAS[act](v), D.double()
    nan, inf = want.isnan(), want.isinf()
    assert torch.equal(got.isnan(), nan), f"{v[got.isnan() != nan].unique().tolist()}"
    assert torch.equal(got[inf], want[inf])
    rest = ~(nan | inf)
    rel = (2.0 ** -8 if D.dtype == BF16 else 2.0 ** -24) * 1.01 + (0 if act == g.ACT_RELU else 2.0 ** -13)
    wrong = rest & ((got - want).abs() > rel * want.abs() + 2.0 ** -119)
    assert not wrong.any(), f"{v[wrong].unique().tolist()} -> {got[wrong].unique().tolist()}"


def status():
    assert g.gemm_get_status(torch.cuda.current_stream().cuda_stream) == 0


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,K", [(40, 64), (40, 72), (700, 64), (40, 1024), (700, 1024)])
def test_products_by_expert(act, dtype, rows, K):
    """Short sums and long ones (in segments for fp32), few rows and many."""
    i32 = dict(dtype=torch.int32, device="cuda")
    plan = g.ExpertPlan.of(torch.tensor([0, rows // 3, rows], **i32), torch.zeros(rows, 1, **i32), torch.zeros(rows, **i32))
    A = column(rows, K)
    D = g.gemm_experts(A, ones((2, 136, K)), plan, activation=act, out_dtype=dtype)
    status()
    near(D, A[:, 0], act)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,path", [(27, 520, 3), (100, 520, 1), (2200, 1040, 2)])
def test_dense_products(act, dtype, M, N, path):
    A, B = column(M, 128), ones((N, 128))
    D = torch.empty(M, N, device="cuda", dtype=dtype)
    s = torch.cuda.current_stream().cuda_stream
    assert g.gemm_bf16_tn_bias_act(M, N, 128, A.data_ptr(), 128, B.data_ptr(), 128, 0, 0, D.data_ptr(), N, 1.0, 0.0,
                                   g.OUT_BF16 if dtype == BF16 else g.OUT_F32, 0, 0, act, s) == 0
    assert g.last_launch_info()["path"] == path
    status()
    near(D, A[:, 0], act)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_4_bit_products(act, dtype):
    """Codes 9 and 8 with the zero point 8: one and zeros."""
    N, K = 64, 128
    codes = torch.full((N, K // 2), 0x88, device="cuda", dtype=torch.uint8)
    codes[:, 0] = 0x89
    W = g.W4Matrix(codes, torch.ones(N, 1, device="cuda"), None, K=K, group=128)
    for M in (9, 27):
        A = column(M, K)
        D = g.gemm_w4(A, W, activation=act, out_dtype=dtype)
        status()
        near(D, A[:, 0], act)
