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


def test_negated_views_are_refused(torch):  # noqa: F811
    """A view whose sign is only noted (of a conjugate's imaginary part, say) holds the other sign's values."""
    from orthogonal_reparameterized_poet_b200 import poet

    x = torch.randn(4, 64, device="cuda")
    neg = torch._neg_view(x)
    tk = torch.zeros(4, dtype=torch.int32, device="cuda")
    tt, tv = tk[:, None].contiguous(), torch.zeros(4, 1, device="cuda")
    saved = poet.token_logprobs(x, tk)[4]
    for call in (lambda: poet.joint_forward(neg, x), lambda: poet.joint_forward(x, neg),
                 lambda: poet.joint_forward(x, x, h_out=neg), lambda: poet.joint_backward(x, x, None, neg, x),
                 lambda: poet.token_logprobs(neg, tk), lambda: poet.distill_topk(neg, tt, tv),
                 lambda: poet.distill_topk(x, tt, torch._neg_view(tv)),
                 lambda: poet.token_logprobs_grad(x, tk, torch._neg_view(saved), tv[:, 0].contiguous())):
        with pytest.raises(ValueError, match="negated"):
            call()
    h, n = poet.joint_forward(neg.resolve_neg(), x)
    assert torch.equal(h, x + poet.joint_forward(neg.resolve_neg(), torch.zeros_like(x))[0])
    poet.poet_sync_status()
