"""Refusals of the bf16 products by expert and what their wrappers hand to the C ABI, without a GPU: the C calls fail
before any device call, and the wrappers get host tensors that say they are on a GPU and a library that records."""
import pytest

torch = pytest.importorskip("torch")

import tensor_core_dense_tn_gb300 as g
from tensor_core_dense_tn_gb300 import build as gbuild
from test_expert_tensors_host import Recorder, elsewhere, gpu, in_host_memory, zeros
from test_expert_w4_host import BAD_PLANS, plan, refused

INV, MIS = g.GEMM_ERR_INVALID_VALUE, g.GEMM_ERR_MISALIGNED
BF16, F32 = torch.bfloat16, torch.float32
T, K2, E, N, K = 4, 2, 8, 32, 64        # tokens, slots, experts, matrix
R = T * K2


# ------------------------------------------------------------------ the C ABI
def forward(p, **kw):
    a = dict(N=N, K=K, A=0x10000, lda=K, W=0x20000, ldw=K, stride_w=N * K, D=0x30000, ldd=N, alpha=1.0, out_dtype=0,
             activation=0, stream=0)
    a.update(kw)
    return g.gemm_bf16_tn_experts(p, *a.values())


def back_a(p, **kw):
    a = dict(N=N, K=K, dD=0x10000, lddd=N, W=0x20000, ldw=K, stride_w=N * K, dA=0x30000, ldda=K, alpha=1.0, out_dtype=0,
             stream=0)
    a.update(kw)
    return g.gemm_bf16_tn_experts_backward_a(p, *a.values())


def back_w(p, **kw):
    a = dict(N=N, K=K, dD=0x10000, lddd=N, A=0x20000, lda=K, C=0, ldc=0, stride_c=0, dW=0x30000, lddw=K, stride_dw=N * K,
             alpha=1.0, beta=0.0, out_dtype=0, stream=0)
    a.update(kw)
    return g.gemm_bf16_tn_experts_backward_w(p, *a.values())


@pytest.fixture(scope="module")
def built():
    gbuild.build()
    return g.load()


@pytest.mark.parametrize("call", [forward, back_a, back_w])
@pytest.mark.parametrize("kw,code", BAD_PLANS)
def test_bad_plans(built, call, kw, code):
    refused(call(plan(**kw)), code)


@pytest.mark.parametrize("call,kw,code", [
    (forward, dict(N=-1), INV), (forward, dict(K=1 << 31), INV), (forward, dict(out_dtype=2), INV),
    (forward, dict(activation=5), INV), (forward, dict(A=0), INV), (forward, dict(lda=K - 8), INV),
    (forward, dict(A=0x10008), MIS), (forward, dict(lda=K + 4), MIS), (forward, dict(W=0), INV),
    (forward, dict(W=0x20002), MIS), (forward, dict(ldw=K - 8), INV), (forward, dict(ldw=K + 2), MIS),
    (forward, dict(stride_w=N * K - 8), INV), (forward, dict(stride_w=0), INV), (forward, dict(stride_w=N * K + 4), MIS),
    (forward, dict(D=0), INV), (forward, dict(ldd=N - 1), INV), (forward, dict(D=0x30001), MIS),
    (forward, dict(D=0x30002, out_dtype=1), MIS), (forward, dict(N=(1 << 31) - 8192, ldd=1 << 31, stride_w=1 << 40), INV),
    (back_a, dict(N=-1), INV), (back_a, dict(K=-1), INV), (back_a, dict(out_dtype=-1), INV), (back_a, dict(dD=0), INV),
    (back_a, dict(lddd=N - 8), INV), (back_a, dict(dD=0x10002), MIS), (back_a, dict(lddd=N + 1), MIS),
    (back_a, dict(W=0), INV), (back_a, dict(stride_w=N * K - 8), INV), (back_a, dict(dA=0), INV),
    (back_a, dict(ldda=K - 1), INV),
    (back_w, dict(N=-1), INV), (back_w, dict(dD=0), INV), (back_w, dict(lddd=N - 8), INV), (back_w, dict(dD=0x10002), MIS),
    (back_w, dict(A=0), INV), (back_w, dict(lda=K + 4), MIS), (back_w, dict(dW=0), INV), (back_w, dict(lddw=K - 1), INV),
    (back_w, dict(stride_dw=N * K - 1), INV), (back_w, dict(out_dtype=3), INV),
    (back_w, dict(beta=1.0), INV),                                                          # C is NULL
    (back_w, dict(beta=1.0, C=0x40000, ldc=K - 1, stride_c=N * K), INV),
    (back_w, dict(beta=1.0, C=0x40000, ldc=K, stride_c=N * K - 1), INV),
    (back_w, dict(beta=1.0, C=0x40001, ldc=K, stride_c=N * K), MIS),
])
def test_bad_arguments(built, call, kw, code):
    if kw.get("N", 0) > 1 << 30:
        kw = dict(kw, K=8, lda=8, ldw=8)
        if torch.cuda.is_available() is False:      # the number of tiles is known behind the device's check
            code = None
    rc = call(plan(), **kw)
    if code is None:
        assert rc != g.GEMM_OK
    else:
        refused(rc, code)


@pytest.mark.parametrize("call,kw", [
    (forward, dict(N=0)), (back_a, dict(K=0)), (back_w, dict(N=0)), (back_w, dict(K=0)),
])
def test_empty_outputs_launch_nothing(built, call, kw):
    assert call(plan(), **kw) == g.GEMM_OK


def test_no_rows_launch_nothing(built):
    p = plan(tokens=0, slot_row=0, row_token=0)
    assert forward(p) == g.GEMM_OK and back_a(p) == g.GEMM_OK


# ------------------------------------------------------------------ the tensor wrappers
@pytest.fixture
def lib(monkeypatch):
    recorder = Recorder()
    monkeypatch.setattr(g, "_lib", recorder)
    g._t()
    monkeypatch.setattr(g, "_several_gpus", True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return recorder


def make_plan(how=lambda t: t):
    i32 = torch.int32
    return g.ExpertPlan.of(how(zeros(E + 1, dtype=i32)), how(zeros(T, K2, dtype=i32)), how(zeros(R, dtype=i32)))


CALLS = {
    "forward": (lambda p, o: g.gemm_experts(o["A"], o["W"], p, out=o["out"], stream=1),
                dict(A=(R, K), W=(E, N, K), out=(R, N))),
    "backward_a": (lambda p, o: g.gemm_experts_backward_a(o["dD"], o["W"], p, out=o["out"], stream=1),
                   dict(dD=(R, N), W=(E, N, K), out=(R, K))),
    "backward_w": (lambda p, o: g.gemm_experts_backward_w(o["dD"], o["A"], p, beta=1.0, C=o["C"], out=o["out"], stream=1),
                   dict(dD=(R, N), A=(R, K), C=(E, N, K), out=(E, N, K))),
}
OPERANDS = [(name, what) for name, (_, shapes) in CALLS.items() for what in shapes]


def operands(name, **other):
    return {what: other.get(what, zeros(*shape, dtype=BF16)) for what, shape in CALLS[name][1].items()}


@pytest.mark.parametrize("name", CALLS)
def test_dense_operands_reach_the_library(lib, name):
    CALLS[name][0](make_plan(), operands(name))
    assert len(lib.calls) == 1


def test_strides_reach_the_library(lib):
    W, A = zeros(E, N + 3, K + 8, dtype=BF16)[:, :N, :K], zeros(R, K + 16, dtype=BF16)[:, :K]
    g.gemm_experts(A, W, make_plan(), out=zeros(R, N), activation=g.ACT_SILU, alpha=0.5, stream=7)
    (name, args), = lib.calls
    assert name == "gemm_bf16_tn_experts"
    assert args[1:] == (N, K, A.data_ptr(), K + 16, W.data_ptr(), K + 8, (N + 3) * (K + 8), args[8], N, 0.5, g.OUT_F32,
                        g.ACT_SILU, 7)


@pytest.mark.parametrize("name,what", OPERANDS)
def test_wrong_shapes_and_strides_are_refused(lib, name, what):
    shape = CALLS[name][1][what]
    dense = zeros(*shape, dtype=BF16)
    bad = [zeros(*shape[:-1], shape[-1] + 1, dtype=BF16), zeros(*shape[:-2], shape[-2] + 1, shape[-1], dtype=BF16),
           zeros(*shape[:-2], shape[-1], shape[-2], dtype=BF16).transpose(-1, -2),
           zeros(shape[-1], dtype=BF16).expand(shape), zeros(*shape, 2, dtype=BF16)[..., 0], dense[0]]
    if len(shape) == 3:         # one matrix for all experts
        bad.append(zeros(*shape[1:], dtype=BF16).expand(shape))
    if name == "backward_w" and what in ("dD", "A"):
        bad = bad[1:]           # its width is the result's
    for t in bad:
        with pytest.raises(ValueError):
            CALLS[name][0](make_plan(), operands(name, **{what: t}))
    assert lib.calls == []


@pytest.mark.parametrize("name,what", OPERANDS)
def test_wrong_types_are_refused(lib, name, what):
    shape = CALLS[name][1][what]
    bad = [torch.float16, torch.float64] + ([F32] if what in ("A", "dD", "W", "C") else [])
    for dtype in bad:
        with pytest.raises(ValueError):
            CALLS[name][0](make_plan(), operands(name, **{what: zeros(*shape, dtype=dtype)}))
    assert lib.calls == []


@pytest.mark.parametrize("name,what", OPERANDS)
@pytest.mark.parametrize("how", [in_host_memory, elsewhere])
def test_operands_elsewhere_are_refused(lib, name, what, how):
    with pytest.raises(ValueError):
        CALLS[name][0](make_plan(), operands(name, **{what: how(zeros(*CALLS[name][1][what], dtype=BF16))}))
    with pytest.raises(ValueError):
        CALLS[name][0](make_plan(how), operands(name))
    assert lib.calls == []


@pytest.mark.parametrize("name", CALLS)
def test_operands_of_another_gpu_than_the_current_one_are_refused(lib, name, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        CALLS[name][0](make_plan(), operands(name))
    assert lib.calls == []


def test_c_is_needed_only_for_beta(lib):
    o = operands("backward_w")
    g.gemm_experts_backward_w(o["dD"], o["A"], make_plan(), out=o["out"], stream=1)
    with pytest.raises(ValueError):
        g.gemm_experts_backward_w(o["dD"], o["A"], make_plan(), beta=1.0, out=o["out"], stream=1)
    assert len(lib.calls) == 1


def test_out_dtype_of_another_out_is_refused(lib):
    o = operands("forward")
    with pytest.raises(ValueError):
        g.gemm_experts(o["A"], o["W"], make_plan(), out=o["out"], out_dtype=F32, stream=1)
    assert lib.calls == []
