"""The example layer against plain PyTorch in 64 bits: its result, its gradients and its 4-bit form.

Every value of the layer is rounded to bf16 (2^-9 of it) a few times on its
way, with independent signs: hidden before and after silu, the expert rows and
the result forward, and as many backward.  Norms of errors are therefore
compared with 2^-6 of the norms (eight times one rounding).
"""
import importlib.util
import pathlib

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

g = pytest.importorskip("tensor_core_dense_tn_gb300")


def example():
    path = pathlib.Path(__file__).resolve().parent.parent / "examples" / "expert_mlp.py"
    spec = importlib.util.spec_from_file_location("expert_mlp", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def layer64(x, ids, weights, up, down):
    y = torch.zeros_like(x)
    for j in range(ids.shape[1]):
        h = torch.nn.functional.silu(torch.einsum("th,tfh->tf", x, up[ids[:, j]]))
        y = y + weights[:, j:j + 1] * torch.einsum("tf,thf->th", h, down[ids[:, j]])
    return y


def setup(T, k, E, H, F):
    r = torch.Generator(device="cuda").manual_seed(T + E)
    randn = lambda *s: torch.randn(*s, generator=r, device="cuda")  # noqa: E731
    gate = randn(E, H).bfloat16()
    up, down = (randn(E, F, H) / H ** 0.5).bfloat16(), (randn(E, H, F) / F ** 0.5).bfloat16()
    return gate, up, down, randn(T, H).bfloat16(), randn(T, H).bfloat16()


def near(a, b, part=2.0 ** -6):
    return ((a.double() - b.double()).norm() <= part * b.double().norm()).item()


@pytest.mark.parametrize("T,k,E,H,F", [(48, 2, 4, 64, 96), (5, 3, 8, 128, 64), (200, 1, 3, 72, 136)])
def test_training_step(T, k, E, H, F):
    ex = example()
    gate, up, down, x, dout = setup(T, k, E, H, F)
    mine = [t.clone().requires_grad_() for t in (x, up, down)]
    y = ex.train_forward(mine[0], gate, mine[1], mine[2], k)
    y.backward(dout)
    wide = [t.double().requires_grad_() for t in (x, up, down)]
    logits = wide[0] @ gate.double().T
    ids, _ = ex.route(x, gate, k)
    weights = torch.softmax(logits.gather(1, ids), dim=1)
    ref = layer64(wide[0], ids, weights, wide[1], wide[2])
    ref.backward(dout.double())
    assert near(y, ref)
    for a, b in zip(mine, wide):
        assert near(a.grad, b.grad)


@pytest.mark.parametrize("T", [1, 7])
def test_decode_step_equals_the_layer_on_the_4_bit_values(T):
    ex = example()
    k, E, H, F = 2, 8, 256, 512
    gate, up, down, x, _ = setup(T, k, E, H, F)
    decoder = ex.Decoder(T, k, gate, up, down)

    def values(W):
        q = torch.stack([W.codes & 15, W.codes >> 4], dim=-1).view(E, W.N, W.K).double()
        wide = lambda t: t.double().repeat_interleave(W.group, dim=-1)  # noqa: E731
        return wide(W.scales) * (q - wide(W.zeros))

    for step in range(3):
        at = (x.float() + step).bfloat16()
        ids, weights = ex.route(at, gate, k)
        ref = layer64(at.double(), ids, weights.double(), values(decoder.up), values(decoder.down))
        assert near(decoder.step(at), ref)
    assert near(values(decoder.up), up, 0.2)
