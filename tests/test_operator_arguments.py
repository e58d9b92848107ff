"""Arguments of the operators around the blocks that Python would pass on to
the C ABI changed: refused before a tensor is looked at (no GPU needed)."""
import pytest
import torch

from orthogonal_reparameterized_poet_b200 import poet

X = torch.zeros(2, 8)


@pytest.mark.parametrize("kw", [dict(gate_rows=2**64 + 1), dict(gate_rows=2**63), dict(gate_rows=-2**63 - 1),
                                dict(gate_act=2**32), dict(gate_act=-2**31 - 1)])
def test_joint_integers_are_not_cut(kw):
    name = next(iter(kw))
    # an output or a stream of the caller's own goes past the compiled binding
    with pytest.raises(ValueError, match=name):
        poet.joint_forward(X, X, X, h_out=X, **kw)
    with pytest.raises(ValueError, match=name):
        poet.joint_backward(X, X, X, X, X, dh=X, **kw)


@pytest.mark.parametrize("topk", [2**31, 2**32 + 5, -2**32])
def test_topk_is_not_cut(topk):
    with pytest.raises(ValueError, match="topk"):
        poet.token_logprobs(X, topk=topk, saved=X)


@pytest.mark.parametrize("kw", [dict(T=2**64 + 4), dict(d=2**32 + 64), dict(dtype=2**32), dict(gate=2**32),
                                dict(gate_rows=2**64 + 1)])
def test_workspace_integers_are_not_cut(kw):
    with pytest.raises(ValueError, match=next(iter(kw))):
        poet.joint_workspace_bytes(**{**dict(T=4, d=64, dtype=poet.BF16), **kw})
