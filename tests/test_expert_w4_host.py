"""Argument rules of the expert and 4-bit-weight calls, checked on the host
before any device call, and the ctypes structs against the header."""
import ctypes

import pytest

import tensor_core_dense_tn_gb300 as g
from tensor_core_dense_tn_gb300 import build as gbuild
from test_host_api import _struct_fields


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    return g.load()


@pytest.mark.parametrize("name,cls", [("gemm_expert_plan", g.ExpertPlanInfo), ("gemm_w4_matrix", g.W4MatrixInfo)])
def test_ctypes_structs_follow_the_header(name, cls):
    assert _struct_fields(name) == [f for f, _ in cls._fields_]


def plan(**kw):
    a = dict(tokens=4, slots=2, experts=8, offsets=0x1000, slot_row=0x2000, row_token=0x3000)
    a.update(kw)
    return g.ExpertPlanInfo(*a.values())


BAD_PLANS = [
    (dict(tokens=-1), g.GEMM_ERR_INVALID_VALUE),
    (dict(slots=0), g.GEMM_ERR_INVALID_VALUE),
    (dict(slots=65), g.GEMM_ERR_INVALID_VALUE),
    (dict(experts=0), g.GEMM_ERR_INVALID_VALUE),
    (dict(experts=1025), g.GEMM_ERR_INVALID_VALUE),
    (dict(tokens=1 << 30, slots=2), g.GEMM_ERR_INVALID_VALUE),      # 2^31 slots
    (dict(offsets=0), g.GEMM_ERR_INVALID_VALUE),
    (dict(slot_row=0), g.GEMM_ERR_INVALID_VALUE),
    (dict(row_token=0), g.GEMM_ERR_INVALID_VALUE),
    (dict(slot_row=0x2002), g.GEMM_ERR_MISALIGNED),
]


def refused(rc, code):
    assert rc == code
    assert g.last_error() != ""


def dispatch(p, **kw):
    a = dict(ids=0x4000, ld_ids=2, ids_64bit=1, H=16, X=0x5000, ldx=16, dtype=0, Xs=0x6000, ldxs=16, stream=0)
    a.update(kw)
    return g.gemm_expert_dispatch(p, *a.values())


def back(p, **kw):
    a = dict(H=16, dXs=0x5000, lddxs=16, dtype=0, dX=0x6000, lddx=16, stream=0)
    a.update(kw)
    return g.gemm_expert_dispatch_backward(p, *a.values())


def combine(p, **kw):
    a = dict(H=16, Y=0x5000, ldy=16, dtype=0, weights=0x7000, ldw=2, weights_dtype=1, out=0x6000, ldo=16, stream=0)
    a.update(kw)
    return g.gemm_expert_combine(p, *a.values())


def combine_back(p, **kw):
    a = dict(H=16, Y=0x5000, ldy=16, dout=0x6000, lddo=16, dtype=0, weights=0x7000, ldw=2, weights_dtype=1,
             dY=0x8000, lddy=16, dweights=0x9000, lddw=2, stream=0)
    a.update(kw)
    return g.gemm_expert_combine_backward(p, *a.values())


@pytest.mark.parametrize("call", [dispatch, back, combine, combine_back])
@pytest.mark.parametrize("kw,code", BAD_PLANS)
def test_bad_plans(call, kw, code):
    refused(call(plan(**kw)), code)


@pytest.mark.parametrize("call", [dispatch, back, combine, combine_back])
def test_missing_plan(call):
    refused(call(None), g.GEMM_ERR_INVALID_VALUE)


INV, MIS = g.GEMM_ERR_INVALID_VALUE, g.GEMM_ERR_MISALIGNED


@pytest.mark.parametrize("call,kw,code", [
    (dispatch, dict(ids=0), INV), (dispatch, dict(ld_ids=1), INV), (dispatch, dict(ids_64bit=2), INV),
    (dispatch, dict(ids=0x4004), MIS), (dispatch, dict(H=-1), INV), (dispatch, dict(dtype=2), INV),
    (dispatch, dict(ldx=15), INV), (dispatch, dict(Xs=0), INV), (dispatch, dict(ldxs=8), INV),
    (dispatch, dict(X=0x5001), MIS), (dispatch, dict(dtype=1, Xs=0x6002), MIS),
    (back, dict(dXs=0), INV), (back, dict(dX=0), INV), (back, dict(lddxs=15), INV), (back, dict(dtype=-1), INV),
    (back, dict(dX=0x6001), MIS), (back, dict(H=1 << 31), INV),
    (combine, dict(weights=0), INV), (combine, dict(ldw=1), INV), (combine, dict(weights_dtype=2), INV),
    (combine, dict(weights=0x7002), MIS), (combine, dict(Y=0), INV), (combine, dict(out=0), INV),
    (combine, dict(ldo=3), INV),
    (combine_back, dict(dout=0), INV), (combine_back, dict(Y=0), INV), (combine_back, dict(weights=0), INV),
    (combine_back, dict(lddw=1), INV), (combine_back, dict(lddy=15), INV), (combine_back, dict(dweights=0x9002), MIS),
    (combine_back, dict(dtype=3), INV), (combine_back, dict(weights_dtype=3), INV),
])
def test_bad_rows(call, kw, code):
    refused(call(plan(), **kw), code)


def test_calls_without_work():
    none = plan(tokens=0, slot_row=0, row_token=0)
    assert back(none) == combine(none) == combine_back(none) == g.GEMM_OK
    assert back(plan(), H=0) == combine(plan(), H=0) == g.GEMM_OK
    assert combine_back(plan(), dY=0, dweights=0) == g.GEMM_OK


def matrix(**kw):
    a = dict(N=64, K=128, count=1, group=64, scales_dtype=0, codes=0x10000, ldc=128, stride_codes=0, scales=0x20000,
             lds=2, stride_scales=0, zeros=0, ldz=0, stride_zeros=0)
    a.update(kw)
    return g.W4MatrixInfo(*a.values())


def w4(W, **kw):
    a = dict(M=3, A=0x30000, lda=128, W=W, D=0x40000, ldd=64, alpha=1.0, out_dtype=0, activation=0, stream=0)
    a.update(kw)
    return g.gemm_w4_tn(*a.values())


def w4_experts(W, p=None, **kw):
    a = dict(A=0x30000, lda=128, gather=0, W=W, D=0x40000, ldd=64, alpha=1.0, out_dtype=0, activation=0, stream=0)
    a.update(kw)
    return g.gemm_w4_tn_experts(plan() if p is None else p, *a.values())


BAD_MATRICES = [
    (dict(N=-1), INV), (dict(K=-1), INV), (dict(group=0), INV), (dict(group=16), INV), (dict(group=96), INV),
    (dict(group=384), INV), (dict(scales_dtype=2), INV), (dict(codes=0), INV), (dict(ldc=96), INV),
    (dict(codes=0x10008), MIS), (dict(K=100, ldc=120), MIS), (dict(scales=0), INV), (dict(lds=1), INV),
    (dict(scales=0x20001), MIS), (dict(scales_dtype=1, scales=0x20002), MIS), (dict(zeros=0x50000, ldz=1), INV),
]


@pytest.mark.parametrize("kw,code", BAD_MATRICES)
def test_bad_matrices(kw, code):
    refused(w4(matrix(**kw)), code)
    many = dict(count=8, stride_codes=64 * 128, stride_scales=128)
    refused(w4_experts(matrix(**{**many, **kw})), code)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INV), (dict(A=0), INV), (dict(lda=120), INV), (dict(A=0x30008), MIS), (dict(lda=132), MIS),
    (dict(D=0), INV), (dict(ldd=63), INV), (dict(D=0x40001), MIS), (dict(out_dtype=1, D=0x40002), MIS),
    (dict(out_dtype=2), INV), (dict(activation=5), INV), (dict(activation=-1), INV),
    (dict(M=0), g.GEMM_OK),
])
def test_bad_operands(kw, code):
    rc = w4(matrix(), **kw)
    assert rc == code
    assert code == g.GEMM_OK or g.last_error() != ""


def test_matrices_and_experts_have_to_agree():
    refused(w4(None), INV)
    refused(w4(matrix(count=8)), INV)
    refused(w4_experts(matrix(count=4, stride_codes=8192)), INV)
    refused(w4_experts(matrix(count=8, stride_codes=64 * 128 - 32)), INV)     # the matrices would overlap
    refused(w4_experts(matrix(count=8, stride_codes=64 * 128 + 16)), MIS)
    refused(w4_experts(matrix(count=8, stride_codes=64 * 128, stride_scales=-1)), INV)
    refused(w4_experts(matrix(count=8, stride_codes=64 * 128), gather=2), INV)
    refused(g.gemm_w4_tn_experts(None, 0x30000, 128, 0, matrix(), 0x40000, 64, 1.0, 0, 0, 0), INV)
    assert w4_experts(matrix(count=8, stride_codes=64 * 128), plan(tokens=0)) == g.GEMM_OK
    assert w4(matrix(N=0)) == g.GEMM_OK


def test_tensor_wrappers_check_types():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        g.W4Matrix(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1))        # not on a GPU
    with pytest.raises(ValueError):
        g.W4Matrix(torch.zeros(4, 16, dtype=torch.int8), torch.zeros(4, 1))
    p = g.ExpertPlan(4, 2, 8, "cpu")
    assert p.offsets.shape == (9,) and p.slot_row.shape == (4, 2) and p.row_token.shape == (8,)
    assert ctypes.cast(p.info.offsets, ctypes.c_void_p).value == p.offsets.data_ptr()
    with pytest.raises(ValueError):
        g.ExpertPlan.of(p.offsets.long(), p.slot_row, p.row_token)
    with pytest.raises(ValueError):
        g.ExpertPlan.of(p.offsets, p.slot_row, p.row_token[:-1])
    ids = torch.zeros(4, 2, dtype=torch.int64)
    with pytest.raises(ValueError):
        g.expert_dispatch(ids.float(), p)
    with pytest.raises(ValueError):
        g.expert_dispatch(ids, p)                                                   # not on a GPU
    with pytest.raises(ValueError):
        g.expert_combine(p, torch.zeros(8, 16, dtype=torch.float16), torch.zeros(4, 2))
    with pytest.raises(ValueError):
        g.gemm_w4(torch.zeros(1, 32), None)
