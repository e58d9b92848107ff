"""The compiled binding of the operators around the blocks: built and loaded for
this torch, and not needed (no GPU needed)."""
import types

import pytest
import torch

from orthogonal_reparameterized_poet_b200 import build, poet

X = torch.zeros(2, 8)
CALLS = [lambda: poet.joint_forward(X, X), lambda: poet.joint_backward(X, X, None, X, X), lambda: poet.token_logprobs(X),
         lambda: poet.token_logprobs_grad(X, None, X[:, :4], None, X[:, 0]), lambda: poet.distill_topk(X, X.int(), X),
         lambda: poet.distill_topk_grad(X, X.int(), X, X[:, :4])]


def test_it_is_built_for_this_torch():
    build._binding(False)
    assert isinstance(poet._native(), types.ModuleType)
    assert torch.__version__ in poet._native().__file__


def test_one_of_another_torch_is_not_loaded(monkeypatch):
    monkeypatch.setattr(poet, "_binding", None)
    monkeypatch.setattr(torch, "__version__", "0.1")
    with pytest.warns(UserWarning, match="ctypes"):
        assert poet._native() is poet._NoBinding


def test_calls_do_without_it(monkeypatch):
    monkeypatch.setattr(poet, "_binding", None)
    monkeypatch.setattr(poet, "binding_path", lambda: "/nowhere/_binding.so")
    with pytest.warns(UserWarning, match="ctypes"):
        poet._native()
    for call in CALLS:
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_the_build_does_without_it(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "binding_path", lambda: str(tmp_path / "_binding.so"))
    monkeypatch.setenv("CXX", "/nowhere/c++")
    with pytest.warns(UserWarning, match="ctypes"):
        build._binding_if_possible(False)
