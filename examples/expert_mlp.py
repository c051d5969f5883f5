"""A mixture-of-experts MLP on the expert and 4-bit-weight calls.

    y[t] = sum_j w[t, j] * down_e( silu( up_e( x[t] ) ) ),   e = the token's j-th expert

Training: dispatch, two grouped bf16 products, combine, and the gradients of
all of them.  Decoding: the experts' matrices held in 4 bits, the plan of a
step and its products on few tokens, captured in a CUDA graph.

    python examples/expert_mlp.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import tensor_core_dense_tn_gb300 as g  # noqa: E402


def route(x, gate, k):
    """The k experts of each token and their weights (which sum to one)."""
    logits = x.float() @ gate.float().T
    top, ids = torch.topk(logits, k, dim=1)
    return ids, torch.softmax(top, dim=1)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def grouped(A, bounds, B):
    """Rows bounds[e] .. bounds[e + 1] of A times B[e].T, one launch for all experts."""
    D = torch.zeros(A.shape[0], B.shape[1], dtype=A.dtype, device=A.device)
    problems = [dict(M=hi - lo, N=B.shape[1], K=B.shape[2], A=A[lo:].data_ptr(), lda=A.stride(0), B=B[e].data_ptr(),
                     ldb=B.stride(1), C=None, ldc=0, D=D[lo:].data_ptr(), ldd=D.stride(0))
                for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])) if hi > lo]
    if problems:
        rc = g.gemm_bf16_tn_grouped(problems, 1.0, 0.0, g.OUT_BF16, _stream())
        if rc:
            raise RuntimeError(f"grouped GEMM failed: {rc}")
    return D


class Dispatch(torch.autograd.Function):
    """The tokens' rows in expert order; fills the plan.  Its arrays are saved, so that autograd raises where the
    plan was filled again before the gradients were taken."""

    @staticmethod
    def forward(ctx, X, ids, plan):
        rows = g.expert_dispatch(ids, plan, X)
        ctx.save_for_backward(plan.offsets, plan.slot_row, plan.row_token)
        return rows

    @staticmethod
    def backward(ctx, dXs):
        return g.expert_dispatch_backward(g.ExpertPlan.of(*ctx.saved_tensors), dXs.contiguous()), None, None


class Combine(torch.autograd.Function):
    """The weighted sum of each token's expert rows."""

    @staticmethod
    def forward(ctx, Y, weights, plan):
        ctx.save_for_backward(Y, weights, plan.offsets, plan.slot_row, plan.row_token)
        return g.expert_combine(plan, Y, weights)

    @staticmethod
    def backward(ctx, dout):
        Y, weights, *arrays = ctx.saved_tensors
        dY, dweights = g.expert_combine_backward(g.ExpertPlan.of(*arrays), Y, weights, dout.contiguous())
        return dY, dweights, None


class ExpertLinear(torch.autograd.Function):
    """Each expert's rows times its matrix."""

    @staticmethod
    def forward(ctx, A, W, bounds):
        ctx.bounds = bounds
        ctx.save_for_backward(A, W)
        return grouped(A, bounds, W)

    @staticmethod
    def backward(ctx, dD):
        A, W = ctx.saved_tensors
        dD = dD.contiguous()
        dA = grouped(dD, ctx.bounds, W.transpose(1, 2).contiguous())
        dW = torch.stack([dD[lo:hi].T @ A[lo:hi] for lo, hi in zip(ctx.bounds, ctx.bounds[1:])])
        return dA, dW, None


def train_forward(x, gate, up, down, k):
    """The layer on x (T, H) with gate (E, H), up (E, F, H) and down (E, H, F), all bf16, with gradients."""
    ids, weights = route(x, gate, k)
    plan = g.ExpertPlan(x.shape[0], k, gate.shape[0], x.device)
    rows = Dispatch.apply(x, ids, plan)
    bounds = plan.offsets.tolist()          # the grouped call's row counts live on the host
    hidden = torch.nn.functional.silu(ExpertLinear.apply(rows, up, bounds))
    return Combine.apply(ExpertLinear.apply(hidden, down, bounds), weights, plan)


def to_4_bits(W, group):
    """(E, N, K) to 4-bit codes with a scale and a zero point per `group` values along K (a multiple of group)."""
    E, N, K = W.shape
    w = W.float().view(E, N, K // group, group)
    lo, hi = w.amin(-1, keepdim=True).clamp(max=0), w.amax(-1, keepdim=True).clamp(min=0)
    scale = ((hi - lo) / 15).clamp(min=1e-8).bfloat16()
    zero = torch.round(-lo / scale.float()).clamp(0, 15)
    q = torch.round(w / scale.float() + zero).clamp(0, 15).to(torch.uint8).view(E, N, K)
    codes = (q[..., 0::2] | q[..., 1::2] << 4).contiguous()
    return g.W4Matrix(codes, scale.squeeze(-1).contiguous(), zero.squeeze(-1).to(torch.uint8), K=K, group=group)


class Decoder:
    """The same layer for a fixed small number of tokens on 4-bit matrices, one CUDA graph per step."""

    def __init__(self, tokens, k, gate, up, down, group=128):
        self.gate, self.k = gate, k
        self.up, self.down = to_4_bits(up, group), to_4_bits(down, group)
        self.x = torch.zeros(tokens, gate.shape[1], dtype=torch.bfloat16, device=gate.device)
        self.plan = g.ExpertPlan(tokens, k, gate.shape[0], gate.device)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self._run()
            side.synchronize()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph, stream=side):
                self.y = self._run()

    def _run(self):
        ids, weights = route(self.x, self.gate, self.k)
        g.expert_dispatch(ids, self.plan)
        hidden = g.gemm_w4_experts(self.x, self.up, self.plan, gather=True, activation=g.ACT_SILU)
        return g.expert_combine(self.plan, g.gemm_w4_experts(hidden, self.down, self.plan), weights)

    def step(self, x):
        self.x.copy_(x)
        self.graph.replay()
        return self.y


def main():
    torch.manual_seed(0)
    T, k, E, H, F = 4096, 4, 16, 2048, 4096
    dev = "cuda"
    gate = torch.randn(E, H, device=dev).bfloat16()
    up = (torch.randn(E, F, H, device=dev) / H ** 0.5).bfloat16().requires_grad_()
    down = (torch.randn(E, H, F, device=dev) / F ** 0.5).bfloat16().requires_grad_()
    x = torch.randn(T, H, device=dev).bfloat16().requires_grad_()
    y = train_forward(x, gate, up, down, k)
    loss = y.float().square().mean()
    loss.backward()
    print(f"training: {T} tokens through {k} of {E} experts, loss {loss.item():.5f}, |dx| {x.grad.float().norm():.3f}")
    with torch.no_grad():
        decoder = Decoder(8, k, gate, up, down)
        full = train_forward(x[:8], gate, up, down, k)
        few = decoder.step(x[:8])
        error = (few - full).float().norm() / full.float().norm()
    print(f"decoding: 8 tokens on 4-bit matrices, {error:.3f} from bf16")


if __name__ == "__main__":
    main()
