"""More rows of one expert than 2^30: the tiles keep their height, and places are right."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

g = pytest.importorskip("tensor_core_dense_tn_gb300")
from test_experts_gpu import gen, plan_of, status  # noqa: E402


def test_more_than_2_30_rows():
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GB")
    R, lost, N, K = (1 << 30) + 77, 5, 8, 8
    plan = plan_of([R], lost)
    draw = lambda *shape: torch.randint(-3, 4, shape, generator=gen(1), device="cuda", dtype=torch.int8).bfloat16()  # noqa: E731
    A, W = draw(R + lost, K), draw(1, N, K)
    D = g.gemm_experts(A, W, plan)
    assert g.last_launch_info()["tile_m"] == 256
    status()
    for lo in (0, 1000, (1 << 29) - 3, (1 << 30) - 100, R - 300):
        rows = slice(lo, min(lo + 300, R))
        assert torch.equal(D[rows].double(), A[rows].double() @ W[0].double().T)
    assert torch.all(D[R:] == 0)
