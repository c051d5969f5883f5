"""GPU parity of the 4-bit-weight products, dense and by expert.

The expected values are the definition in 64 bits.  Products of bf16 values
and whole numbers below 256 are exact in fp32, so the error is that of the
sums: inside a group at most group / 16 tensor-core steps (each within a few
units of the last place of its largest term), then one fp32 sum per group and
the parts' joins.  With S = sum |s a (q - z)| the bound is
(group / 4 + groups + 8) 2^-23 S, plus the rounding of the output (2^-8 of the
value in bf16, 2^-23 in fp32).  An activation's slope is at most 1.13 and its
own error below 2^-19 of the value.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

g = pytest.importorskip("tensor_core_dense_tn_gb300")

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make(count, N, K, group, zeros, sdtype, seed, pad_groups=0, pad_bytes=0):
    r = gen(seed)
    pitch = -(-K // 32) * 16 + pad_bytes
    groups = -(-K // group)
    codes = torch.randint(0, 256, (count, N, pitch), generator=r, device="cuda", dtype=torch.uint8)
    scales = (torch.randn(count, N, groups + pad_groups, generator=r, device="cuda") / K ** 0.5).to(DT[sdtype])
    z = torch.randint(0, 16, (count, N, groups + pad_groups), generator=r, device="cuda", dtype=torch.uint8)
    return codes, scales[..., :groups], z[..., :groups] if zeros else None


def weights64(codes, scales, zeros, K, group):
    """(s, q - z) of one matrix, both (N, K) in 64 bits, k by k from the bytes."""
    k = torch.arange(K, device="cuda")
    byte = codes[:, k // 2].long()
    q = torch.where(k % 2 == 0, byte % 16, byte // 16)
    z = torch.full_like(q, 8) if zeros is None else zeros[:, k // group].long()
    return scales[:, k // group].double(), (q - z).double()


def act64(x, act):
    if act == g.ACT_RELU:
        return x.clamp(min=0)
    if act == g.ACT_SILU:
        return x * torch.sigmoid(x)
    if act == g.ACT_GELU:
        return 0.5 * x * (1 + torch.erf(x / 2 ** 0.5))
    if act == g.ACT_GELU_TANH:
        return 0.5 * x * (1 + torch.tanh((2 / np.pi) ** 0.5 * (x + 0.044715 * x ** 3)))
    return x


def check(D, A, mat, K, group, alpha=1.0, act=0):
    s, d = weights64(*mat, K, group)
    a = A.double()
    ref = act64(alpha * a @ (s * d).T, act)
    S = abs(alpha) * a.abs() @ (s * d).abs().T
    eps = 2.0 ** -8 * 1.01 if D.dtype == torch.bfloat16 else 2.0 ** -23
    bound = 1.13 * (group / 4 + -(-K // group) + 8) * 2.0 ** -23 * S + (eps + 2.0 ** -19 * (act != 0)) * ref.abs()
    worst = ((D.double() - ref).abs() - bound).max().item() if D.numel() else 0.0
    assert worst <= 0.0, worst


def status():
    assert g.gemm_get_status(torch.cuda.current_stream().cuda_stream) == 0


def acts(M, K, seed):
    ld = -(-max(K, 1) // 8) * 8
    return torch.randn(M, ld, generator=gen(seed), device="cuda").bfloat16()[:, :K]


CASES = [  # M, N, K, group
    (1, 1, 1, 32), (1, 128, 256, 128), (1, 8192, 8192, 128), (3, 129, 255, 32), (5, 5000, 2000, 32), (8, 127, 257, 64),
    (9, 300, 4096, 64), (16, 1000, 1111, 128), (17, 200, 520, 32), (33, 130, 96, 32), (100, 140, 640, 128),
    (2, 40, 16384, 256), (4, 264, 1000, 1024), (1, 16, 31, 32), (16, 64, 2048, 32), (7, 28672, 288, 32),
]


@pytest.mark.parametrize("M,N,K,group", CASES)
@pytest.mark.parametrize("zeros,sdtype,out", [(False, "bf16", "bf16"), (True, "bf16", "f32"), (True, "f32", "bf16")])
def test_dense(M, N, K, group, zeros, sdtype, out):
    mat = make(1, N, K, group, zeros, sdtype, M + N + K, pad_groups=M % 3, pad_bytes=16 * (M % 2))
    one = tuple(None if t is None else t[0] for t in mat)
    A = acts(M, K, 5)
    W = g.W4Matrix(*one, K=K, group=group)
    pitch = N + M % 4          # rows of D on their element size only
    D = torch.full((M, pitch), float("nan"), device="cuda", dtype=DT[out])
    g.gemm_w4(A, W, out=D[:, :N])
    status()
    check(D[:, :N], A, one, K, group)
    assert torch.isnan(D[:, N:]).all()


@pytest.mark.parametrize("M,N,K,group", [(3, 200, 1030, 32), (11, 130, 2000, 768), (2, 257, 700, 128), (16, 64, 900, 64)])
@pytest.mark.parametrize("sdtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,skip", [(0, 0), (1, 1), (2, 3)])
def test_every_zero_point_and_scales_at_odd_addresses(M, N, K, group, sdtype, pad, skip):
    codes, scales, _ = (None if t is None else t[0] for t in make(1, N, K, group, False, sdtype, 7 + K))
    groups = scales.shape[1]
    flat_s = torch.full((skip + N * (groups + pad),), float("nan"), device="cuda", dtype=DT[sdtype])
    flat_z = torch.full((skip + N * (groups + pad),), 255, device="cuda", dtype=torch.uint8)
    odd_s = flat_s[skip:].view(N, groups + pad)[:, :groups]
    odd_z = flat_z[skip:].view(N, groups + pad)[:, :groups]
    odd_s.copy_(scales)
    odd_z.copy_(torch.randint(0, 256, (N, groups), generator=gen(K), device="cuda", dtype=torch.uint8))
    A = acts(M, K, 6)
    D = g.gemm_w4(A, g.W4Matrix(codes, odd_s, odd_z, K=K, group=group), out_dtype=torch.float32)
    status()
    check(D, A, (codes, odd_s, odd_z), K, group)


@pytest.mark.parametrize("act", [g.ACT_RELU, g.ACT_GELU, g.ACT_GELU_TANH, g.ACT_SILU])
def test_activation_and_alpha(act):
    mat = make(1, 300, 512, 128, True, "bf16", 1)
    one = tuple(t[0] for t in mat)
    A = acts(6, 512, 2)
    for out in ("bf16", "f32"):
        D = g.gemm_w4(A, g.W4Matrix(*one, K=512), alpha=-0.75, activation=act, out_dtype=DT[out])
        status()
        check(D, A, one, 512, 128, -0.75, act)


def test_whole_numbers_are_exact():
    """Small whole activations and scales that are powers of two: every sum is exact in fp32."""
    M, N, K, group = 11, 260, 1184, 32
    codes, scales, zeros = (t[0] for t in make(1, N, K, group, True, "f32", 3))
    scales = 2.0 ** torch.randint(-2, 3, scales.shape, generator=gen(4), device="cuda").float()
    A = torch.randint(-4, 5, (M, K), generator=gen(5), device="cuda").bfloat16()
    D = g.gemm_w4(A, g.W4Matrix(codes, scales, zeros, K=K, group=group), out_dtype=torch.float32)
    s, d = weights64(codes, scales, zeros, K, group)
    assert torch.equal(D.double(), A.double() @ (s * d).T)


def test_no_k():
    W = g.W4Matrix(torch.zeros(5, 16, dtype=torch.uint8, device="cuda"), torch.zeros(5, 0, device="cuda"), K=0)
    A = torch.empty(3, 0, dtype=torch.bfloat16, device="cuda")
    D = g.gemm_w4(A, W, out=torch.full((3, 5), float("nan"), device="cuda"))
    status()
    assert torch.all(D == 0)


def test_non_finite_activations_stay_in_their_token():
    mat = tuple(t[0] for t in make(1, 200, 700, 64, True, "bf16", 1))
    W = g.W4Matrix(*mat, K=700, group=64)
    A = acts(12, 700, 2)
    clean = g.gemm_w4(A, W)
    A[3, 5], A[7, 699] = float("nan"), float("inf")
    D = g.gemm_w4(A, W)
    rows = [m for m in range(12) if m not in (3, 7)]
    assert torch.equal(D[rows], clean[rows])
    assert torch.isnan(D[3]).all() and not torch.isfinite(D[7]).any()


def test_padding_of_codes_and_scales_is_not_read_into_results():
    """Bytes past K (also the odd K's high nibble) and NaN scales past the groups do not matter."""
    N, K, group = 130, 333, 32
    codes, scales, zeros = (t[0] for t in make(1, N, K, group, True, "f32", 1, pad_groups=2, pad_bytes=16))
    scales.as_strided((N, 2), (scales.stride(0), 1), scales.storage_offset() + scales.shape[1]).fill_(float("nan"))
    A = acts(4, K, 2)
    D = g.gemm_w4(A, g.W4Matrix(codes, scales, zeros, K=K, group=group))
    codes[:, (K + 1) // 2:] = 0xFF
    codes[:, K // 2] |= 0xF0
    again = g.gemm_w4(A, g.W4Matrix(codes, scales, zeros, K=K, group=group))
    status()
    assert torch.equal(D, again) and torch.isfinite(D).all()


def make_plan(T, k, E, seed, how):
    r = np.random.default_rng(seed)
    ids = np.stack([r.permutation(E)[:k] for _ in range(T)]) if k <= E else r.integers(0, E, (T, k))
    if how == "dropped":
        ids[r.random((T, k)) < 0.4] = -1
    elif how == "one expert":
        ids[:] = E // 2
    elif how == "none":
        ids[:] = -1
    plan = g.ExpertPlan(T, k, E, "cuda")
    g.expert_dispatch(torch.from_numpy(ids).cuda(), plan)
    return plan


EXPERT_CASES = [  # T, k, E, N, K, group
    (1, 8, 64, 512, 768, 128), (1, 1, 1, 5, 33, 32), (32, 2, 16, 300, 520, 64), (7, 3, 5, 129, 1000, 32),
    (40, 4, 300, 140, 256, 256), (130, 2, 3, 260, 300, 128), (3, 2, 1024, 130, 96, 32),
]


@pytest.mark.parametrize("T,k,E,N,K,group", EXPERT_CASES)
@pytest.mark.parametrize("how", ["all", "dropped", "one expert", "none"])
@pytest.mark.parametrize("gather", [False, True])
def test_experts(T, k, E, N, K, group, how, gather):
    plan = make_plan(T, k, E, T + E, how)
    codes, scales, zeros = make(E, N, K, group, gather, "bf16", E + N)
    A = acts(T if gather else T * k, K, 5)
    out = torch.full((T * k, N), float("nan"), device="cuda", dtype=torch.float32)
    D = g.gemm_w4_experts(A, g.W4Matrix(codes, scales, zeros, K=K, group=group), plan, gather=gather,
                          activation=g.ACT_SILU, out=out)
    status()
    bounds = plan.offsets.tolist()
    for e in range(E):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            rows = plan.row_token[lo:hi].long() if gather else slice(lo, hi)
            check(D[lo:hi], A[rows], (codes[e], scales[e], None if zeros is None else zeros[e]), K, group,
                  act=g.ACT_SILU)
    assert torch.all(D[bounds[-1]:] == 0)


def test_matrices_apart_and_scales_shared():
    """Matrices with space between them, and one set of scales for all (a stride of zero)."""
    E, N, K, group = 4, 200, 384, 128
    plan = make_plan(10, 2, E, 1, "all")
    codes, scales, _ = make(2 * E, N, K, group, False, "f32", 1)
    shared = scales[:1].expand(E, N, K // group)
    A = acts(20, K, 2)
    D = g.gemm_w4_experts(A, g.W4Matrix(codes[::2], shared, K=K, group=group), plan)
    status()
    bounds = plan.offsets.tolist()
    for e in range(E):
        check(D[bounds[e]:bounds[e + 1]], A[bounds[e]:bounds[e + 1]], (codes[2 * e], scales[0], None), K, group)


def test_rows_of_a_foreign_plan_are_checked():
    """Offsets and tokens out of range are clamped or read as zero rows, not followed."""
    plan = make_plan(6, 2, 4, 1, "all")
    codes, scales, _ = make(4, 64, 64, 32, False, "bf16", 1)
    W, A = g.W4Matrix(codes, scales, K=64, group=32), acts(6, 64, 2)
    good = g.gemm_w4_experts(A, W, plan, gather=True)
    plan.row_token[5] = 1 << 30
    plan.offsets[4] = 1 << 30
    D = g.gemm_w4_experts(A, W, plan, gather=True)
    status()
    assert torch.all(D[5] == 0)
    assert torch.equal(D[:5], good[:5]) and torch.equal(D[6:], good[6:])


@pytest.mark.parametrize("T,k,E,N,K,group", [(32, 2, 16, 8192, 4096, 64), (24, 4, 12, 4096, 4096, 128), (40, 8, 10, 4100, 2048, 32)])
def test_many_tiles_per_block_are_exact_every_time(T, k, E, N, K, group):
    """Whole numbers, so every sum is exact: a stage that is overwritten before it is read shows at once."""
    r = gen(N + K)
    q = torch.randint(0, 16, (E, N, K // 32), generator=r, device="cuda")          # one code per 32 k
    codes = (q * 17).to(torch.uint8).repeat_interleave(16, dim=2)
    zeros = torch.randint(0, 16, (E, N, K // group), generator=r, device="cuda")
    scales = torch.randint(1, 3, (E, N, K // group), generator=r, device="cuda")
    W = g.W4Matrix(codes, scales.bfloat16(), zeros.to(torch.uint8), K=K, group=group)
    a = torch.randint(-2, 3, (T, K // 32), generator=r, device="cuda")
    A = a.bfloat16().repeat_interleave(32, dim=1)
    ids = torch.rand(T, E, generator=r, device="cuda").topk(k, dim=1).indices
    plan = g.ExpertPlan(T, k, E, "cuda")
    g.expert_dispatch(ids, plan)
    offsets, token = plan.offsets.tolist(), plan.row_token.long()
    per = group // 32
    ref = torch.empty(T * k, N, device="cuda", dtype=torch.float64)
    for e in range(E):
        w = (32 * scales[e].repeat_interleave(per, dim=1) * (q[e] - zeros[e].repeat_interleave(per, dim=1))).double()
        ref[offsets[e]:offsets[e + 1]] = a.double()[token[offsets[e]:offsets[e + 1]]] @ w.T
    for _ in range(30):
        D = g.gemm_w4_experts(A, W, plan, gather=True, out_dtype=torch.float32)
        assert torch.equal(D.double(), ref)
    status()


@pytest.mark.parametrize("parts", range(1, 9))
@pytest.mark.parametrize("M,group", [(3, 64), (13, 128)])
def test_every_number_of_parts(parts, M, group):
    """One tile of `parts` stages, dense, and by expert with several blocks of rows per expert."""
    N, K = 120, 256 * parts
    mat = make(3, N, K, group, True, "bf16", parts)
    A = acts(M, K, 8)
    D = g.gemm_w4(A, g.W4Matrix(*(t[0] for t in mat), K=K, group=group), out_dtype=torch.float32)
    assert g.last_launch_info()["k_parts"] == parts
    check(D, A, tuple(t[0] for t in mat), K, group)
    T = 17 * M
    ids = torch.randint(0, 3, (T, 1), generator=gen(parts), device="cuda")
    plan = g.ExpertPlan(T, 1, 3, "cuda")
    A = acts(T, K, 9)
    rows = g.expert_dispatch(ids, plan, A)
    D = g.gemm_w4_experts(rows, g.W4Matrix(*mat, K=K, group=group), plan)
    status()
    offsets = plan.offsets.tolist()
    for e in range(3):
        lo, hi = offsets[e], offsets[e + 1]
        check(D[lo:hi], rows[lo:hi], tuple(t[e] for t in mat), K, group)


def test_side_stream_and_repeats():
    mat = tuple(t[0] for t in make(1, 1000, 4096, 128, True, "bf16", 1))
    W, A = g.W4Matrix(*mat, K=4096), acts(16, 4096, 2)
    first = g.gemm_w4(A, W)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = g.gemm_w4(A, W)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            third = g.gemm_w4(A, W)
        third.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, second) and torch.equal(first, third)


def test_last_launch_info_names_the_kernel():
    mat = tuple(t[0] for t in make(1, 1000, 4096, 128, True, "bf16", 1))
    g.gemm_w4(acts(1, 4096, 2), g.W4Matrix(*mat, K=4096))
    info = g.last_launch_info()
    assert info["kernel"].startswith("gemm_w4") and info["path"] == 0 and info["k_parts"] == info["cluster"]


def test_codes_past_32_bits():
    """A code offset above 2^32 bytes: the last of 40 matrices of 128 MiB."""
    E, N, K, group = 40, 4096, 65536, 256
    codes = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    codes[-1] = torch.randint(0, 256, (N, K // 2), generator=gen(1), device="cuda", dtype=torch.uint8)
    scales = torch.full((E, N, K // group), 1 / 256, device="cuda")
    plan = make_plan(1, 1, E, 1, "none")
    g.expert_dispatch(torch.full((1, 1), E - 1, device="cuda"), plan)
    A = acts(1, K, 2)
    D = g.gemm_w4_experts(A, g.W4Matrix(codes, scales, K=K, group=group), plan, out_dtype=torch.float32)
    status()
    rows = torch.arange(0, N, 97, device="cuda")
    check(D[:, rows], A, (codes[-1][rows], scales[-1][rows], None), K, group)
