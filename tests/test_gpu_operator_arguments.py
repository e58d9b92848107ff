"""Tensors that the operators around the blocks refuse before anything is
launched (nothing invalid reaches the GPU)."""
import pytest

from tests.test_gpu_joint import torch  # noqa: F401

pytestmark = pytest.mark.gpu


def test_workspace_is_its_own_memory(torch):  # noqa: F811
    from orthogonal_reparameterized_poet_b200 import poet

    x = torch.zeros(4, 64, device="cuda")
    n = poet.joint_workspace_bytes(4, 64, poet.F32)
    one = torch.empty(1, dtype=torch.uint8, device="cuda")
    for ws in (one.expand(n), torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2],
               torch.empty(64, n, dtype=torch.uint8, device="cuda").t()):
        with pytest.raises(ValueError, match="ws"):
            poet.joint_backward(x, x, None, x, x, ws=ws)
    with pytest.raises(ValueError, match="ws"):
        poet.joint_backward(x, x, None, x, x, ws=torch.empty(n, dtype=torch.uint8))
    poet.joint_backward(x, x, None, x, x, ws=torch.empty(n, dtype=torch.uint8, device="cuda"))
    poet.poet_sync_status()
