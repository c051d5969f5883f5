"""Refusals of the gradient norm's calls, and what the wrappers hand to the C ABI, without a GPU."""
import contextlib
import ctypes

import pytest

torch = pytest.importorskip("torch")

import tensor_core_dense_tn_gb300 as g
from tensor_core_dense_tn_gb300 import build as gbuild
from test_expert_tensors_host import Recorder, elsewhere, gpu, in_host_memory, zeros
from test_expert_w4_host import refused
from test_host_api import _struct_fields

INV, MIS = g.GEMM_ERR_INVALID_VALUE, g.GEMM_ERR_MISALIGNED
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def built():
    gbuild.build()
    return g.load()


def test_struct_follows_the_header():
    assert _struct_fields("gemm_tensor") == [f for f, _ in g.TensorInfo._fields_]
    assert ctypes.sizeof(g.TensorInfo) == 24        # three words, which the wrappers fill


def array(*rows):
    return (g.TensorInfo * max(1, len(rows)))(*[g.TensorInfo(*r) for r in rows])


GOOD = (0x10000, 100, 1)


@pytest.mark.parametrize("clip", [False, True])
@pytest.mark.parametrize("num,rows,norm,work,code", [
    (-1, [GOOD], 0x1000, 0x2000, INV), (1, None, 0x1000, 0x2000, INV), (1, [GOOD], 0, 0x2000, INV),
    (1, [GOOD], 0x1002, 0x2000, MIS), (1, [GOOD], 0x1000, 0, INV), (1, [GOOD], 0x1000, 0x2004, MIS),
    (1, [(0x10000, -1, 1)], 0x1000, 0x2000, INV), (1, [(0x10000, 1 << 44, 1)], 0x1000, 0x2000, INV),
    (1, [(0x10000, 5, 2)], 0x1000, 0x2000, INV), (1, [(0x10000, 5, -1)], 0x1000, 0x2000, INV),
    (1, [(0, 5, 0)], 0x1000, 0x2000, INV), (1, [(0x10001, 5, 0)], 0x1000, 0x2000, MIS),
    (1, [(0x10002, 5, 1)], 0x1000, 0x2000, MIS), (2, [GOOD, (0, 1, 1)], 0x1000, 0x2000, INV),
])
def test_bad_arguments(built, clip, num, rows, norm, work, code):
    a = None if rows is None else array(*rows)
    refused(g.gemm_clip_grad_norm(num, a, 1.0, None, norm, work, 0) if clip else g.gemm_grad_norm(num, a, norm, work, 0), code)


@pytest.mark.parametrize("max_norm,out,code", [
    (-1.0, None, INV), (float("nan"), None, INV), (1.0, [(0x20000, 99, 1)], INV), (1.0, [(0x20000, 100, 7)], INV),
    (1.0, [(0, 100, 1)], INV), (1.0, [(0x20001, 100, 0)], MIS), (1.0, [(0x20002, 100, 1)], MIS),
])
def test_bad_clips(built, max_norm, out, code):
    refused(g.gemm_clip_grad_norm(1, array(GOOD), max_norm, None if out is None else array(*out), 0x1000, 0x2000, 0), code)


@pytest.mark.parametrize("rows,out", [
    ([(0x10000, 100, 1), (0x10000, 100, 1)], None), ([(0x10000, 100, 1), (0x10000 + 396, 100, 1)], None),
    ([(0x10000, 100, 0), (0x10000 - 198, 100, 0)], None), ([(0x10000, 9, 1)], [(0x10000, 9, 0)]),
    ([(0x10000, 100, 1)], [(0x10004, 100, 1)]), ([(0x10000, 8, 1), (0x20000, 8, 1)], [(0x20000, 8, 1), (0x10000, 8, 1)]),
    ([(0x10000, 8, 1), (0x20000, 8, 1)], [(0x30000, 8, 1), (0x3001C, 8, 1)]),
    ([(0x10000, 1000, 1), (0x40000, 8, 1)], [(0x50000, 1000, 1), (0x10100, 8, 1)]),
])
def test_outputs_that_overlap_are_refused(built, rows, out):
    """They would be scaled twice, or before they are read."""
    refused(g.gemm_clip_grad_norm(len(rows), array(*rows), 1.0, None if out is None else array(*out), 0x1000, 0x2000, 0), INV)
    assert "overlap" in g.last_error()


@pytest.mark.parametrize("clip", [True, False])
@pytest.mark.parametrize("norm,work", [
    (0x10000, 0x2000), (0x1018C, 0x2000), (0x1000, 0x10000), (0x1000, 0x10188), (0x1000, 0x10000 - 8),
])
def test_a_norm_or_workspace_in_a_tensor_is_refused(built, clip, norm, work):
    """It would be written before the values there are read, or are scaled."""
    a = array((0x40000, 8, 0), (0x10000, 100, 1))
    refused(g.gemm_clip_grad_norm(2, a, 1.0, None, norm, work, 0) if clip else g.gemm_grad_norm(2, a, norm, work, 0), INV)
    assert "overlap" in g.last_error()


def test_a_norm_in_an_output_is_refused(built):
    refused(g.gemm_clip_grad_norm(1, array(GOOD), 1.0, array((0x30000, 100, 1)), 0x30010, 0x2000, 0), INV)
    assert "overlap" in g.last_error()


def test_neighbours_do_not_overlap(built):
    """Without a GPU the call gets as far as asking for the device."""
    rows = [(0x10000, 100, 1), (0x10000 + 400, 100, 0), (0x10000 + 600, 3, 0)]
    for out in (None, rows, [(r[0] + 0x100000, *r[1:]) for r in rows]):
        g.gemm_clip_grad_norm(3, array(*rows), 1.0, None if out is None else array(*out), 0x1000, 0x2000, 0) \
            if not torch.cuda.is_available() else None
        assert "overlap" not in g.last_error()


def test_workspace(built):
    assert g.gemm_grad_workspace(-1) == 0
    sizes = [g.gemm_grad_workspace(n) for n in (0, 1, 960, 961, 5000)]
    assert sizes == sorted(sizes) and sizes[0] == sizes[2] and sizes[2] < sizes[3] and all(s % 8 == 0 for s in sizes)


# ------------------------------------------------------------------ the tensor wrappers
class Answering(Recorder):
    def gemm_grad_workspace(self, num):
        return 4096


@pytest.fixture
def lib(monkeypatch):
    recorder = Answering()
    monkeypatch.setattr(g, "_lib", recorder)
    g._t()
    monkeypatch.setattr(g, "_several_gpus", True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(g, "_GRAD_WORKSPACE", {})
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "default_stream", lambda gpu: None)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: gpu(empty(*a, **{n: v for n, v in k.items() if n != "device"})))
    return recorder


def test_lists_reach_the_library(lib):
    ts = [zeros(5, 7), zeros(3, dtype=BF16), zeros(0), zeros(4, 6, dtype=BF16).t()]
    out = [zeros(5, 7, dtype=BF16), zeros(3), zeros(0), zeros(4, 6).t()]
    norm = zeros(1)
    assert g.clip_grad_norm(ts, 2.0, out=out, norm=norm, stream=0) is norm
    (name, args), = lib.calls
    assert name == "gemm_clip_grad_norm" and args[0] == 4 and args[2] == 2.0 and args[4] == norm.data_ptr()
    row = lambda t: [t.data_ptr(), t.numel(), int(t.dtype == F32)]  # noqa: E731
    assert args[1] == bytes(array(*map(row, ts))) and args[3] == bytes(array(*map(row, out)))


BAD = {
    "type": lambda: zeros(4, dtype=torch.float16), "whole numbers": lambda: zeros(4, dtype=torch.int32),
    "gaps": lambda: zeros(4, 8)[:, :6], "one row for all": lambda: zeros(6).expand(4, 6), "every other": lambda: zeros(9)[::2],
    "host": lambda: in_host_memory(zeros(4)), "another GPU": lambda: elsewhere(zeros(4)),
}


@pytest.mark.parametrize("bad", BAD)
def test_bad_tensors_are_refused(lib, bad):
    for ts in ([BAD[bad]()], [zeros(3), BAD[bad]()], [BAD[bad](), zeros(3, dtype=BF16)]):
        with pytest.raises(ValueError):
            g.grad_norm(ts, stream=0)
        with pytest.raises(ValueError):
            g.clip_grad_norm(ts, 1.0, stream=0)
        with pytest.raises(ValueError):
            g.clip_grad_norm([zeros(*t.shape) for t in ts], 1.0, out=ts, stream=0)
    assert lib.calls == []


@pytest.mark.parametrize("out", [[], [zeros(4)], [zeros(5), zeros(3)], [zeros(4), zeros(3), zeros(1)]])
def test_outputs_of_other_shapes_are_refused(lib, out):
    with pytest.raises(ValueError):
        g.clip_grad_norm([zeros(4), zeros(3)], 1.0, out=out, stream=0)
    assert lib.calls == []


def test_outputs_in_another_order_are_refused(lib):
    with pytest.raises(ValueError):
        g.clip_grad_norm([zeros(4, 6)], 1.0, out=[zeros(6, 4).t()], stream=0)
    assert lib.calls == []


@pytest.mark.parametrize("norm", [zeros(2), zeros(1, dtype=BF16), in_host_memory(zeros(1)), elsewhere(zeros(1))])
def test_bad_norms_are_refused(lib, norm):
    with pytest.raises(ValueError):
        g.grad_norm([zeros(4)], norm=norm, stream=0)
    assert lib.calls == []


def test_tensors_of_another_gpu_than_the_current_one_are_refused(lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        g.grad_norm([zeros(4)], stream=0)
    assert lib.calls == []
