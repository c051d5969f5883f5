"""norm and workspace apart: a clip stores the norm while other blocks still read the sums in the workspace."""
import pytest

torch = pytest.importorskip("torch")

import tensor_core_dense_tn_gb300 as g
from test_expert_w4_host import refused
from test_grad_norm_host import GOOD, array, built  # noqa: F401

WORK = 0x2000


@pytest.mark.parametrize("clip", [True, False])
@pytest.mark.parametrize("num", [1, 961])
def test_a_norm_in_the_workspace_is_refused(built, clip, num):  # noqa: F811
    size = g.gemm_grad_workspace(num)
    rows = array(*[(0x1000000 + 0x1000 * i, 100, 1) for i in range(num)])
    for norm in (WORK, WORK + 4, WORK + size // 2, WORK + size - 4):
        rc = g.gemm_clip_grad_norm(num, rows, 1.0, None, norm, WORK, 0) if clip else g.gemm_grad_norm(num, rows, norm, WORK, 0)
        refused(rc, g.GEMM_ERR_INVALID_VALUE)
        assert "overlap" in g.last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")
def test_a_norm_beside_the_workspace_is_not_refused(built):  # noqa: F811
    """Without a GPU the call gets as far as asking for the device."""
    size = g.gemm_grad_workspace(1)
    for norm in (WORK - 4, WORK + size):
        g.gemm_clip_grad_norm(1, array(GOOD), 1.0, None, norm, WORK, 0)
        assert "overlap" not in g.last_error()
        g.gemm_grad_norm(0, None, norm, WORK, 0)
        assert "overlap" not in g.last_error()
