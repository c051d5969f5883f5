"""Tensors of the caller's that a call writes count as changed in place, so that autograd raises where one that it has
saved was written; what a call only reads does not.  No GPU: the library is a recorder."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import tensor_core_dense_tn_gb300 as g
import test_expert_tensors_host as rows
import test_experts_host as products
from test_expert_tensors_host import OnGpu, gpu, zeros
from test_grad_norm_host import Answering

WRITTEN = ("out", "dY", "dweights")


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


CALLS = [(m, name) for m in (rows, products) for name in m.CALLS]


@pytest.mark.parametrize("module,name", CALLS, ids=[name for _, name in CALLS])
def test_given_outputs_count_as_changed(lib, module, name):
    ops = module.operands(name)
    before = {what: t._version for what, t in ops.items()}
    module.CALLS[name][0](module.make_plan(), ops)
    assert len(lib.calls) == 1
    for what, t in ops.items():
        assert (t._version > before[what]) == (what in WRITTEN), what


def test_norms_and_clips(lib):
    ts, out, norm = [zeros(5), zeros(3, 4)], [zeros(5), zeros(3, 4)], zeros(1)
    g.grad_norm(ts, norm=norm, stream=0)
    assert [t._version for t in (*ts, *out, norm)] == [0, 0, 0, 0, 1]
    g.clip_grad_norm(ts, 1.0, out=out, norm=norm, stream=0)
    assert [t._version for t in (*ts, *out, norm)] == [0, 0, 1, 1, 2]
    g.clip_grad_norm(ts, 1.0, stream=0)
    assert [t._version for t in (*ts, *out, norm)] == [1, 1, 1, 1, 2]


def test_the_dense_product(lib, monkeypatch):
    monkeypatch.setattr(g, "load", lambda: lib)
    A, B, out = zeros(4, 8, dtype=torch.bfloat16), zeros(16, 8, dtype=torch.bfloat16), zeros(4, 16)
    assert g.gemm(A, B, out=out, stream=1) is out
    assert [t._version for t in (A, B, out)] == [0, 0, 1]


def test_autograd_raises_for_a_saved_output(lib):
    """A saved factor that a later product overwrites."""
    x = torch.ones(products.R, products.N, requires_grad=True)
    kept = zeros(products.R, products.N)
    y = (x * kept.as_subclass(torch.Tensor)).sum()
    ops = products.operands("forward", out=kept)
    products.CALLS["forward"][0](products.make_plan(), ops)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_inference_tensors_have_no_version(lib):
    with torch.inference_mode():
        ops = products.operands("forward")
        ops["out"] = torch.zeros(products.R, products.N, dtype=torch.bfloat16).as_subclass(OnGpu)
        assert ops["out"].is_inference()
        products.CALLS["forward"][0](products.make_plan(), ops)
    products.CALLS["forward"][0](products.make_plan(), ops)
    assert len(lib.calls) == 2
