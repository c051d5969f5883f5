"""Bounded waits of the products by expert: a dropped load ends in GEMM_ERR_TIMEOUT on every kernel, not in a hang.

CTA 0 arms a block's transaction count without issuing its loads, so that the
wait for them can never be met.  Within the limit set by the host all roles of
the CTA, and of the pair's other one, whose loads have all arrived, give up, free
Tensor Memory and return; the status word says so, and the next call is right.
"""
import time

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

g = pytest.importorskip("tensor_core_dense_tn_gb300")
from test_experts_gpu import forward64, plan_of, values, weights64  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
LIMIT = 20_000_000


@pytest.fixture
def config():
    yield lambda **kw: g.gemm_experts_config(g.GemmConfig(**kw))
    g.gemm_experts_config(None)


def calls(plan, dtype, N, K):
    """The three calls with their exact results, rounded to dtype."""
    A, dD, W = values((plan.rows, K), 1, True), values((plan.rows, N), 2, True), values((plan.experts, N, K), 3, True)
    right = lambda t: t.to(F32).to(dtype)  # noqa: E731
    return {"forward": (lambda: g.gemm_experts(A, W, plan, out_dtype=dtype), right(forward64(A, W, plan)[0])),
            "rows": (lambda: g.gemm_experts_backward_a(dD, W, plan, out_dtype=dtype),
                     right(forward64(dD, W.transpose(1, 2), plan)[0])),
            "weights": (lambda: g.gemm_experts_backward_w(dD, A, plan, out_dtype=dtype), right(weights64(dD, A, plan)[0]))}


# Every kernel: products of few rows (boxes of several blocks) and of many, rows' gradients, weights' gradients on
# single CTAs and on pairs; with short sums in bf16 and with long ones in fp32.  One tile, whose loads fit the ring,
# and more; last blocks that are whole, of 16 rows, and ragged.
CASES = [(which, dtype, counts, N, K)
         for dtype, size in ((BF16, 512), (F32, 1088))
         for which, counts, N, K in (("forward", [9, 5], 200, size), ("forward", [300, 200], 200, size),
                                     ("forward", [300, 20], 1000, size), ("rows", [9, 5], size, 200),
                                     ("rows", [300, 200], size, 1000), ("weights", [size, 16] * 2 + [1] * 30, 200, 200),
                                     ("weights", [size + 16] + [3] * 60, 520, 500), ("weights", [size + 7, 500, 0, 48], 520, 500),
                                     ("weights", [size, 2900], 1000, 1000), ("weights", [7, 1024, 1024], 300, 300))]


@pytest.mark.parametrize("which,dtype,counts,N,K", CASES)
@pytest.mark.parametrize("fault", [1, 2])
def test_a_dropped_load_ends_in_a_timeout(config, which, dtype, counts, N, K, fault):
    call, right = calls(plan_of(counts, 7), dtype, N, K)[which]
    s = torch.cuda.current_stream().cuda_stream
    assert torch.equal(call(), right) and g.gemm_get_status(s) == 0
    assert config(wait_timeout_ns=LIMIT, test_fault=fault) == 0
    began = time.monotonic()
    call()
    assert g.gemm_get_status(s) == g.GEMM_ERR_TIMEOUT
    assert time.monotonic() - began < 1.0       # the limit, what settles behind it, and the host
    assert (g.gemm_get_status_detail() >> 24) in (1, 2, 3)
    assert g.gemm_get_status(s) == 0            # cleared by the read
    config()
    for _ in range(3):
        assert torch.equal(call(), right) and g.gemm_get_status(s) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts,N,K", [([8192] * 40 + [17], 4096, 4096), ([1 << 22], 64, 64)])
def test_a_limit_shorter_than_the_call(config, dtype, counts, N, K):
    """The limit is on standing still: a call of many times its length is right, also where a role waits all that time
    (for the one ragged block, behind all others; for the sum of a single tile)."""
    limit = 500_000
    plan = plan_of(counts, 0)
    A, dD, W = values((plan.rows, K), 1, False), values((plan.rows, N), 2, False), values((len(counts), N, K), 3, False)
    s = torch.cuda.current_stream().cuda_stream
    for call, takes_long in ((lambda: g.gemm_experts_backward_w(dD, A, plan, out_dtype=dtype), True),
                             (lambda: g.gemm_experts(A, W, plan, out_dtype=dtype), K > 64),
                             (lambda: g.gemm_experts_backward_a(dD, W, plan, out_dtype=dtype), K > 64)):
        config()
        call()
        began, ended = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        began.record()
        want = call()
        ended.record()
        assert g.gemm_get_status(s) == 0
        took = began.elapsed_time(ended) * 1e6
        assert config(wait_timeout_ns=limit) == 0
        for _ in range(3):
            assert torch.equal(call(), want) and g.gemm_get_status(s) == 0
        assert took > 4 * limit or not takes_long, took


def test_the_settings_are_the_threads_own(config):
    import threading
    assert config(wait_timeout_ns=LIMIT, test_fault=1) == 0
    call, right = calls(plan_of([300, 200], 7), BF16, 200, 512)["forward"]
    out, s = [], torch.cuda.current_stream().cuda_stream

    def elsewhere():
        torch.cuda.synchronize()
        out.append((call(), g.gemm_get_status(s)))

    other = threading.Thread(target=elsewhere)
    other.start()
    other.join()
    assert out[0][1] == 0 and torch.equal(out[0][0], right)


def test_settings_that_are_refused(config):
    for fault in (-1, 3):
        assert config(test_fault=fault) == g.GEMM_ERR_INVALID_VALUE
