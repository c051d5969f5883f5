"""What the tensor wrappers of the expert and 4-bit calls hand to the C ABI, and what they refuse.

No GPU: the tensors are host tensors that say they are on one, and the library
is a recorder, so a call that gets through shows its arguments instead of
running.
"""
import pytest

torch = pytest.importorskip("torch")

import tensor_core_dense_tn_gb300 as g

T, K, E, H = 4, 2, 8, 64        # tokens, slots, experts, row length
N, KW = 32, 128                 # a weight matrix


class OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU."""
    is_cuda = True
    index = 0

    def get_device(self):
        return self.index


def gpu(t, index=0):
    t = t.detach().as_subclass(OnGpu)
    t.index = index
    return t


def zeros(*shape, dtype=torch.float32):
    return gpu(torch.zeros(*shape, dtype=dtype))


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture(autouse=True)
def lib(monkeypatch):
    recorder = Recorder()
    monkeypatch.setattr(g, "_lib", recorder)
    g._t()
    monkeypatch.setattr(g, "_several_gpus", True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return recorder


def make_plan(tokens=T):
    i32 = torch.int32
    return g.ExpertPlan.of(zeros(E + 1, dtype=i32), zeros(tokens, K, dtype=i32), zeros(tokens * K, dtype=i32))


def make_matrix(count=1):
    lead = (count,) if count > 1 else ()
    return g.W4Matrix(zeros(*lead, N, KW // 2, dtype=torch.uint8), zeros(*lead, N, KW // 64), None, K=KW, group=64)


BF16 = torch.bfloat16
# call: (wrapper, its operands as (name, rows, width, type)); rows of A for the dense product are its own
CALLS = {
    "dispatch": (lambda p, o: g.expert_dispatch(o["ids"], p, o["X"], out=o["out"], stream=1),
                 [("ids", T, K, torch.int64), ("X", T, H, BF16), ("out", T * K, H, BF16)]),
    "dispatch_backward": (lambda p, o: g.expert_dispatch_backward(p, o["dXs"], out=o["out"], stream=1),
                          [("dXs", T * K, H, BF16), ("out", T, H, BF16)]),
    "combine": (lambda p, o: g.expert_combine(p, o["Y"], o["weights"], out=o["out"], stream=1),
                [("Y", T * K, H, BF16), ("weights", T, K, torch.float32), ("out", T, H, BF16)]),
    "combine_backward": (lambda p, o: g.expert_combine_backward(p, o["Y"], o["weights"], o["dout"], o["dY"], o["dweights"],
                                                                stream=1),
                         [("Y", T * K, H, BF16), ("weights", T, K, torch.float32), ("dout", T, H, BF16),
                          ("dY", T * K, H, BF16), ("dweights", T, K, torch.float32)]),
    "w4": (lambda p, o: g.gemm_w4(o["A"], make_matrix(), out=o["out"], stream=1),
           [("A", T, KW, BF16), ("out", T, N, BF16)]),
    "w4_experts": (lambda p, o: g.gemm_w4_experts(o["A"], make_matrix(E), p, out=o["out"], stream=1),
                   [("A", T * K, KW, BF16), ("out", T * K, N, BF16)]),
    "w4_experts_gathered": (lambda p, o: g.gemm_w4_experts(o["A"], make_matrix(E), p, gather=True, out=o["out"], stream=1),
                            [("A", T, KW, BF16), ("out", T * K, N, BF16)]),
}
OPERANDS = [(name, what) for name, (_, ops) in CALLS.items() for what, *_ in ops]


def operands(name, **other):
    return {what: other.get(what, zeros(rows, width, dtype=dtype)) for what, rows, width, dtype in CALLS[name][1]}


def shape_of(name, what):
    return next((rows, width, dtype) for w, rows, width, dtype in CALLS[name][1] if w == what)


@pytest.mark.parametrize("name", CALLS)
def test_dense_operands_reach_the_library(lib, name):
    CALLS[name][0](make_plan(), operands(name))
    assert len(lib.calls) == 1


@pytest.mark.parametrize("name,what", OPERANDS)
def test_rows_that_overlap_are_refused(lib, name, what):
    """A row stride of zero (a broadcast row) or below the row length is no pitch of a matrix: taken as the row length
    it would be read, or written, past its storage."""
    rows, width, dtype = shape_of(name, what)
    broadcast = zeros(width, dtype=dtype).expand(rows, width)
    overlapping = zeros(rows * width, dtype=dtype).as_strided((rows, width), (width - 1, 1))
    for t in (broadcast, overlapping):
        with pytest.raises(ValueError):
            CALLS[name][0](make_plan(), operands(name, **{what: t}))
    assert lib.calls == []


@pytest.mark.parametrize("name,what", OPERANDS)
def test_rows_apart_keep_their_pitch(lib, name, what):
    rows, width, dtype = shape_of(name, what)
    CALLS[name][0](make_plan(), operands(name, **{what: zeros(rows, width + 8, dtype=dtype)[:, :width]}))
    assert width + 8 in lib.calls[0][1]


def test_the_stride_of_a_single_row_does_not_matter(lib):
    plan = make_plan(1)
    X, ids = zeros(H, dtype=BF16).expand(1, H).as_strided((1, H), (0, 1)), zeros(K, dtype=torch.int64).as_strided((1, K), (0, 1))
    g.expert_dispatch(ids, plan, X, stream=1)
    (_, args), = lib.calls
    assert args[2] == K and args[6] == H


PLANNED = [name for name in CALLS if name != "w4"]


def elsewhere(t):
    return gpu(t, 1)


def in_host_memory(t):
    return t.as_subclass(torch.Tensor)


def moved_plan(how):
    p = make_plan()
    return g.ExpertPlan.of(how(p.offsets), how(p.slot_row), how(p.row_token))


@pytest.mark.parametrize("name", PLANNED)
@pytest.mark.parametrize("how", [in_host_memory, elsewhere])
def test_a_plan_elsewhere_is_refused(lib, name, how):
    """The kernels read and write the plan's arrays: host memory or another GPU's would fault."""
    with pytest.raises(ValueError):
        CALLS[name][0](moved_plan(how), operands(name))
    assert lib.calls == []


@pytest.mark.parametrize("name,what", OPERANDS)
@pytest.mark.parametrize("how", [in_host_memory, elsewhere])
def test_an_operand_elsewhere_is_refused(lib, name, what, how):
    rows, width, dtype = shape_of(name, what)
    with pytest.raises(ValueError):
        CALLS[name][0](make_plan(), operands(name, **{what: how(zeros(rows, width, dtype=dtype))}))
    assert lib.calls == []


def test_host_memory_is_refused_where_there_is_one_gpu(lib, monkeypatch):
    monkeypatch.setattr(g, "_several_gpus", False)
    for name in PLANNED:
        with pytest.raises(ValueError):
            CALLS[name][0](moved_plan(in_host_memory), operands(name))
    for name, what in OPERANDS:
        rows, width, dtype = shape_of(name, what)
        with pytest.raises(ValueError):
            CALLS[name][0](make_plan(), operands(name, **{what: in_host_memory(zeros(rows, width, dtype=dtype))}))
    assert lib.calls == []
    CALLS["combine"][0](make_plan(), operands("combine"))
    assert len(lib.calls) == 1


def test_a_matrix_elsewhere_is_refused(lib):
    codes, scales = zeros(N, KW // 2, dtype=torch.uint8), zeros(N, KW // 64)
    W = g.W4Matrix(elsewhere(codes), elsewhere(scales), None, K=KW, group=64)
    with pytest.raises(ValueError):
        g.gemm_w4(zeros(T, KW, dtype=BF16), W, stream=1)
    assert lib.calls == []


@pytest.mark.parametrize("name", CALLS)
def test_operands_of_another_gpu_than_the_current_one_are_refused(lib, name, monkeypatch):
    """The library launches on the current GPU, whatever the tensors' GPU is."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        CALLS[name][0](make_plan(), operands(name))
    assert lib.calls == []


def test_parts_of_a_plan_or_a_matrix_on_different_gpus_are_refused():
    p = make_plan()
    for arrays in ((elsewhere(p.offsets), p.slot_row, p.row_token), (p.offsets, elsewhere(p.slot_row), p.row_token),
                   (p.offsets, p.slot_row, elsewhere(p.row_token))):
        with pytest.raises(ValueError):
            g.ExpertPlan.of(*arrays)
    codes, scales, points = zeros(N, KW // 2, dtype=torch.uint8), zeros(N, KW // 64), zeros(N, KW // 64, dtype=torch.uint8)
    for parts in ((elsewhere(codes), scales, points), (codes, elsewhere(scales), points), (codes, scales, elsewhere(points))):
        with pytest.raises(ValueError):
            g.W4Matrix(*parts, K=KW, group=64)


@pytest.mark.parametrize("apart", [True, False])
def test_filling_a_plan_counts_as_changing_its_arrays(lib, apart):
    """The library writes them through their addresses, which autograd does not see."""
    p = make_plan()
    if not apart:
        p = g.ExpertPlan(T, K, E, "cpu")
        p.gpu = 0
    before = [t._version for t in (p.offsets, p.slot_row, p.row_token)]
    CALLS["dispatch"][0](p, operands("dispatch"))
    assert all(t._version > v for t, v in zip((p.offsets, p.slot_row, p.row_token), before))
    after = [t._version for t in (p.offsets, p.slot_row, p.row_token)]
    for name in PLANNED[1:]:
        CALLS[name][0](p, operands(name))
    assert [t._version for t in (p.offsets, p.slot_row, p.row_token)] == after


def test_plans_of_inference_mode_can_be_filled_outside_it(lib):
    with torch.inference_mode():
        p = make_plan()
        CALLS["dispatch"][0](p, operands("dispatch"))
    CALLS["dispatch"][0](p, operands("dispatch"))
    assert len(lib.calls) == 2
