"""GPU parity of the gradient norm and of clipping by it, against sums in 64 bits.

Bounds: an fp32 sum of 32 squares is within 36 steps of 2^-24 of it (32
products and additions, each rounded by half a step at most, in four chains
that are then added), the fp64 additions do not count beside that, and a root
halves a relative error; the norm's own rounding adds 2^-24.  Together below
20 * 2^-24.  A clipped value is x * c with c = max_norm / norm rounded once (the
norm's error and 2^-24), rounded again to fp32 and, for a bf16 result, by 2^-9.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

g = pytest.importorskip("tensor_core_dense_tn_gb300")

BF16, F32 = torch.bfloat16, torch.float32
NORM_EPS = 20 * 2.0 ** -24
VALUE_EPS = {BF16: 2.0 ** -8 + 2.0 ** -18, F32: 24 * 2.0 ** -24}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def status():
    assert g.gemm_get_status(torch.cuda.current_stream().cuda_stream) == 0


def norm64(tensors):
    return math.sqrt(math.fsum(t.double().square().sum().item() for t in tensors))


def tensors_of(sizes, seed, scale=1.0, shift=0):
    """Alternating types; `shift` elements behind an aligned address."""
    out = []
    for i, n in enumerate(sizes):
        t = torch.randn(n + shift, generator=gen(seed + i), device="cuda") * scale
        out.append(t.to(BF16 if i % 2 else F32)[shift:])
    return out


SIZES = [[1], [7], [8], [15, 17], [16384], [16385, 16383], [3, 0, 100000, 1, 65536 * 3 + 5], [11] * 70, [5] * 2000,
         [40000000, 3, 123457]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_norm(sizes, shift):
    ts = tensors_of(sizes, 3, 0.01, shift)
    got = g.grad_norm(ts)
    assert got.shape == () and got.dtype == F32
    status()
    assert abs(got.item() - norm64(ts)) <= NORM_EPS * norm64(ts)
    assert torch.equal(g.grad_norm(ts), got)        # the same from run to run


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("part", [0.3, 1.5])
def test_clip_in_place(sizes, shift, part):
    ts = tensors_of(sizes, 5, 1.0, shift)
    before = [t.clone() for t in ts]
    want = norm64(ts)
    max_norm = part * want
    norm = g.clip_grad_norm(ts, max_norm)
    status()
    assert abs(norm.item() - want) <= NORM_EPS * want
    for t, b in zip(ts, before):
        if part > 1:
            assert torch.equal(t, b)
        else:
            ref = b.double() * part
            assert torch.all((t.double() - ref).abs() <= VALUE_EPS[t.dtype] * ref.abs())


@pytest.mark.parametrize("sizes", SIZES[:8], ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("to", [BF16, F32])
@pytest.mark.parametrize("shifts", [(0, 0), (1, 1), (2, 1), (0, 5)])
@pytest.mark.parametrize("part", [0.3, 1.5])
def test_clip_into_other_tensors(sizes, to, shifts, part):
    ts = tensors_of(sizes, 7, 1.0, shifts[0])
    before = [t.clone() for t in ts]
    bufs = [torch.full((n + shifts[1] + 9,), 7.0, device="cuda", dtype=to) for n in sizes]
    out = [b[shifts[1]:shifts[1] + n] for b, n in zip(bufs, sizes)]
    want = norm64(ts)
    norm = torch.zeros(1, device="cuda")
    assert g.clip_grad_norm(ts, part * want, out=out, norm=norm) is norm
    status()
    assert abs(norm.item() - want) <= NORM_EPS * want
    for t, b, o, buf in zip(ts, before, out, bufs):
        assert torch.equal(t, b)
        ref = b.double() * min(1.0, part)
        assert torch.all((o.double() - ref).abs() <= VALUE_EPS[to] * ref.abs())
        assert torch.all(buf[:shifts[1]] == 7) and torch.all(buf[shifts[1] + o.numel():] == 7)


@pytest.mark.parametrize("scale", [1e-44, 1e-40, 1e-30, 1e-23, 1e-19, 1e18, 1e19, 1e30, 3e38])
@pytest.mark.parametrize("n", [1, 9, 100000])
def test_any_size_of_values(scale, n):
    t = torch.full((n,), scale, device="cuda")
    for ts in ([t], [t, torch.zeros(50000, device="cuda")], [t.to(BF16), torch.zeros(3, device="cuda")]):
        got = g.grad_norm(ts)
        status()
        want = norm64(ts)
        if want > torch.finfo(F32).max:
            assert got.item() == math.inf
        else:       # below 2^-126 the norm's own step is 2^-149
            assert abs(got.item() - want) <= NORM_EPS * want + 2.0 ** -149
    small = torch.full((40000,), scale, device="cuda")
    small[7] = 1.0          # sizes far apart within one sum
    assert abs(g.grad_norm([small]).item() - norm64([small])) <= NORM_EPS * norm64([small]) or scale > 1e38


@pytest.mark.parametrize("bits", [1, 1 << 15, 1 << 22, 1 << 23, 0x7FFF])
def test_the_smallest_values(bits):
    for sign in (0, -2 ** 31):
        t = torch.zeros(70000, dtype=torch.int32, device="cuda")
        t[5], t[69990] = bits + sign, bits + sign
        t = t.view(F32)
        want = norm64([t])
        assert want > 0 and abs(g.grad_norm([t]).item() - want) <= NORM_EPS * want + 2.0 ** -149


def test_a_norm_that_no_fp32_holds_still_clips():
    """The norm is stored as infinity, but the values are finite and so is what scales them."""
    t = torch.full((100,), 3e38, device="cuda")
    norm = g.clip_grad_norm([t], 1.0)
    assert norm.item() == math.inf
    assert torch.all((t - 0.1).abs() <= 0.1 * VALUE_EPS[F32])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("place", [0, 17, 49999])
def test_what_is_not_finite_changes_nothing(bad, place):
    ts = [torch.randn(50000, device="cuda"), torch.randn(1000, device="cuda").to(BF16)]
    ts[0][place] = bad
    before = [t.clone() for t in ts]
    norm = g.clip_grad_norm(ts, 0.5)
    status()
    assert math.isnan(norm.item()) if math.isnan(bad) else norm.item() == math.inf
    out = [torch.zeros_like(t) for t in ts]
    g.clip_grad_norm(ts, 0.5, out=out)
    for t, b, o in zip(ts, before, out):
        assert torch.equal(t.nan_to_num(5.0), b.nan_to_num(5.0)) and torch.equal(o.nan_to_num(5.0), b.nan_to_num(5.0))


def test_limits_of_zero_and_infinity():
    t = torch.randn(1000, device="cuda")
    b = t.clone()
    g.clip_grad_norm([t], math.inf)
    assert torch.equal(t, b)
    g.clip_grad_norm([t], 0.0)
    assert torch.all(t == 0)
    assert g.clip_grad_norm([t], 0.0).item() == 0 and torch.all(t == 0)


def test_no_tensors_and_empty_ones():
    for ts in ([], [torch.empty(0, device="cuda")], [torch.empty(3, 0, device="cuda", dtype=BF16)] * 2):
        norm = torch.full((), 5.0, device="cuda")
        assert g.grad_norm(ts, norm=norm).item() == 0
        norm.fill_(5.0)
        assert g.clip_grad_norm(ts, 1.0, norm=norm).item() == 0
    status()


def test_dense_in_any_order():
    a = torch.randn(64, 33, 5, device="cuda").permute(2, 0, 1)
    b = torch.randn(40, 30, device="cuda").to(BF16).t()
    c = torch.randn(6, 1, 4, 4, device="cuda").to(memory_format=torch.channels_last)
    before = [t.clone() for t in (a, b, c)]
    want = norm64([a, b, c])
    assert abs(g.grad_norm([a, b, c]).item() - want) <= NORM_EPS * want
    g.clip_grad_norm([a, b, c], want / 2)
    for t, o in zip((a, b, c), before):
        assert torch.all((t.double() - o.double() / 2).abs() <= VALUE_EPS[t.dtype] * o.double().abs() / 2)


def test_captured_and_replayed_beside_eager_calls():
    ts = tensors_of([50000, 77, 123456], 9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.clip_grad_norm(ts, 1e9)
        side.synchronize()
        graphs = []
        for limit in (10.0, 3.0):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                norm = g.clip_grad_norm(ts, limit)
            graphs.append((limit, graph, norm))
    torch.cuda.current_stream().wait_stream(side)
    for seed in range(3):
        for t, new in zip(ts, tensors_of([50000, 77, 123456], 20 + seed)):
            t.copy_(new)
        for limit, graph, norm in graphs:
            want = norm64(ts)
            graph.replay()
            eager = g.grad_norm(ts)
            assert abs(norm.item() - want) <= NORM_EPS * want
            assert abs(eager.item() - min(limit, want)) <= 2.0 ** -8 * limit
    status()


def test_two_calls_at_once():
    sets = [tensors_of([3000000 + i, 5, 70001], 30 + i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    norms = [torch.zeros((), device="cuda") for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for ts, s, n in zip(sets, streams, norms):
            g.grad_norm(ts, norm=n, stream=s.cuda_stream)
            torch.empty(4096, device="cuda").fill_(1e30)        # what takes a freed workspace's place
    torch.cuda.synchronize()
    for ts, n in zip(sets, norms):
        assert abs(n.item() - norm64(ts)) <= NORM_EPS * norm64(ts)


def test_a_workspace_from_another_streams_memory():
    """The workspace of a call on another stream is not memory that the current stream has given back but still uses."""
    ts = tensors_of([200000, 31], 41)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        a = torch.full((2560 // 4,), 3.0, device="cuda")        # of a workspace's size
        for _ in range(50):
            a = a * 1.0
        g.grad_norm(ts, stream=side.cuda_stream)
        assert torch.all(a == 3.0)
    g.grad_norm(ts, stream=0)
    torch.cuda.synchronize()


def test_the_same_tensor_twice():
    t = torch.randn(1000, device="cuda")
    b = t.clone()
    assert abs(g.grad_norm([t, t]).item() - norm64([t, t])) <= NORM_EPS * norm64([t, t])
    with pytest.raises(g.GemmError):
        g.clip_grad_norm([t, t], 1.0)
    assert torch.equal(t, b)


def test_versions():
    """In place counts as a change of the tensors; into others does not."""
    t, o = torch.randn(100, device="cuda"), torch.empty(100, device="cuda")
    v = t._version
    g.grad_norm([t])
    g.clip_grad_norm([t], 1.0, out=[o])
    assert t._version == v
    g.clip_grad_norm([t], 1.0)
    assert t._version > v
