"""Calls from threads that have made no CUDA call before: nothing but this library's call has to bind the device."""
import os
import subprocess
import sys
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

g = pytest.importorskip("tensor_core_dense_tn_gb300")
from test_experts_gpu import gen, plan_of, status, values  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def make_calls():
    """Every kind of call, with its output given: name -> (call without arguments, output)."""
    A, B, small = values((300, 512), 1, True), values((1040, 512), 2, True), values((16, 512), 3, True)
    plan = plan_of([40, 0, 200], 3)
    Xs, dD, W = values((243, 512), 4, True), values((243, 264), 5, True), values((3, 264, 512), 6, True)
    codes = torch.randint(0, 256, (264, 256), generator=gen(7), device="cuda", dtype=torch.uint8)
    w4 = g.W4Matrix(codes, torch.ones(264, 4, device="cuda"), None, K=512, group=128)
    a8, b8 = (torch.randint(0, 0x60, (n, 512), generator=gen(8), device="cuda", dtype=torch.uint8) for n in (300, 1040))
    new = lambda *shape, dtype=F32: torch.zeros(*shape, device="cuda", dtype=dtype)  # noqa: E731
    route = g.ExpertPlan(100, 2, 5, "cuda")
    ids, X = torch.randint(0, 5, (100, 2), generator=gen(9), device="cuda"), values((100, 64), 10, True)
    s = torch.cuda.current_stream().cuda_stream
    f32, D8, Dn = g.OUT_F32, new(300, 1040), new(16, 1040)

    def checked(rc):
        assert rc == 0, (rc, g.last_error())

    calls = {
        "tiled": (lambda o: g.gemm(A, B, out=o, stream=s), new(300, 1040)),
        "skinny": (lambda o: g.gemm(small, B, out=o, stream=s), new(16, 1040)),
        "fp8": (lambda o: checked(g.gemm_fp8_tn(300, 1040, 512, a8.data_ptr(), 512, b8.data_ptr(), 512, g.FP8_E4M3, 1.0, 1.0,
                                                0, 0, o.data_ptr(), 1040, 1.0, 0.0, f32, s)), D8),
        "no allocation": (lambda o: checked(g.gemm_bf16_tn_skinny_noalloc(
            16, 1040, 512, small.data_ptr(), small.stride(0), B.data_ptr(), B.stride(0), 0, 0, o.data_ptr(), 1040, 1.0, 0.0, f32,
            s)), Dn),
        "experts": (lambda o: g.gemm_experts(Xs, W, plan, out=o, stream=s), new(243, 264)),
        "rows' gradient": (lambda o: g.gemm_experts_backward_a(dD, W, plan, out=o, stream=s), new(243, 512)),
        "weights' gradient": (lambda o: g.gemm_experts_backward_w(dD, Xs, plan, out=o, stream=s), new(3, 264, 512)),
        "4 bits": (lambda o: g.gemm_w4(small, w4, out=o, stream=s), new(16, 264)),
        "dispatch": (lambda o: g.expert_dispatch(ids, route, X, out=o, stream=s), new(200, 64, dtype=BF16)),
        "norm": (lambda o: g.grad_norm([A], norm=o), new(1)),
    }
    return {name: (lambda f=f, o=o: f(o), o) for name, (f, o) in calls.items()}


def in_a_thread(*calls):
    """Runs the calls in new threads at once and raises what they raise."""
    errors, start = [], threading.Barrier(len(calls))

    def run(call):
        try:
            start.wait()
            call()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


CALLS = ["tiled", "skinny", "fp8", "no allocation", "experts", "rows' gradient", "weights' gradient", "4 bits", "dispatch",
         "norm"]


@pytest.mark.parametrize("name", CALLS)
def test_the_first_cuda_call_of_a_thread(name):
    call, out = make_calls()[name]
    call()
    status()
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    in_a_thread(call)
    status()
    assert torch.equal(out, want)


def first_calls_at_once():
    calls = make_calls()
    torch.cuda.synchronize()
    in_a_thread(*(call for call, _ in calls.values()))
    status()
    for name, (call, out) in calls.items():
        got = out.clone()
        out.zero_()
        call()
        status()
        assert torch.equal(out, got), name


def test_a_process_whose_first_calls_come_at_once():
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here), os.environ.get("PYTHONPATH", "")]))
    done = subprocess.run([sys.executable, "-c", "import test_threads_gpu as t; t.first_calls_at_once()"], env=env, cwd=here,
                          capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr
