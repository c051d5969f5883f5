"""The split workspace under stream capture: a graph's buffers stay its own."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

g = pytest.importorskip("tensor_core_dense_tn_gb300")


def whole(M, K, seed):
    r = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-4, 5, (M, K), generator=r, device="cuda").bfloat16()


@pytest.mark.parametrize("config", [g.GemmConfig(path=g.PATH_SKINNY), g.GemmConfig(path=g.PATH_2SM, tiled_k_parts=2)])
def test_a_captured_call_keeps_its_workspace_when_the_stream_gets_a_larger_one(config):
    """A call captured with the stream's workspace, then a larger one on that stream: the replay neither writes into
    memory that was given back nor reads what others wrote there."""
    torch.cuda.synchronize()
    g.shutdown()                                  # so that the second call has to replace the workspace
    few, many = (16, 256) if config.path == g.PATH_SKINNY else (300, 600)
    A, larger, B = whole(few, 4096, 1), whole(many, 4096, 2), whole(2112, 4096, 3)
    stream, other = torch.cuda.Stream(), torch.cuda.Stream()
    out = torch.empty(few, 2112, device="cuda", dtype=torch.float32)
    want, want_larger = (a.double() @ B.double().T for a in (A, larger))
    torch.cuda.synchronize()
    call = lambda a, **kw: g.gemm(a, B, out_dtype=torch.float32, config=config, stream=stream.cuda_stream, **kw)  # noqa: E731
    with torch.cuda.stream(stream):
        call(A, out=out)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call(A, out=out)
        free = torch.cuda.mem_get_info()[0]
        D = call(larger)
        stream.synchronize()
        assert torch.cuda.mem_get_info()[0] < free
    # memory that was given back would be handed out again here
    taken = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.double(), want)
    assert all(bool((t == 7.0).all()) for t in taken)
    assert torch.equal(D.double(), want_larger)
    again = call(larger)
    stream.synchronize()
    assert torch.equal(again.double(), want_larger)
    assert g.gemm_get_status(stream.cuda_stream) == 0
