"""The compiled binding of the operators around the blocks."""
import pytest

from tests.test_gpu_joint import torch  # noqa: F401

pytestmark = pytest.mark.gpu


def test_calls_without_it_give_the_same(torch, monkeypatch):  # noqa: F811
    from orthogonal_reparameterized_poet_b200 import poet

    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    o, h = (torch.randn(37, 96, generator=g, device="cuda").bfloat16() for _ in range(2))
    gate = torch.randn(5, 96, generator=g, device="cuda").bfloat16()
    w = torch.rand(96, generator=g, device="cuda")
    x = torch.randn(9, 3001, generator=g, device="cuda")
    tk = torch.randint(0, 3001, (9,), generator=g, device="cuda", dtype=torch.int32)
    tt, tv = tk[:, None].contiguous(), torch.zeros(9, 1, device="cuda")
    kw = dict(w_post=w, w_pre=w, gate_act=poet.GATE_SIGMOID, gate_rows=8, alpha=0.9, beta=0.4)

    def calls():
        a = poet.joint_forward(o, h, gate, **kw)
        b = poet.joint_backward(o, a[0], gate, h, o, **kw)
        c = poet.token_logprobs(x, tk, topk=6, scale=0.7)
        d = poet.token_logprobs_grad(x, tk, c[4], tv[:, 0] + 1, tv[:, 0] - 1, scale=0.7)
        e = poet.distill_topk(x, tt, tv, grad=True)
        return [*a, *b, *c, d, *e, poet.distill_topk_grad(x, tt, tv, e[2])]

    want = calls()
    monkeypatch.setattr(poet, "_binding", poet._NoBinding)
    got = calls()
    poet.poet_sync_status()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
