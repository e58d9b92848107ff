"""Operators on logits at the edges of what they accept, against the float64
oracle (oracle/logits.py), with the bounds of tests/test_gpu_logits.py."""
import pytest

from tests.test_gpu_logits import INF, _make, _teacher_case, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [float("nan"), INF])
@pytest.mark.parametrize("V", [300, 40000])
@pytest.mark.parametrize("tail", [False, True])
def test_a_masked_teacher_token_in_a_row_of_nan(torch, value, V, tail):  # noqa: F811
    from orthogonal_reparameterized_poet_b200 import poet

    x, r = _make(torch, 3, V, torch.float32)
    tokens, values = _teacher_case(r, 3, V, 4, tail)
    for t in range(3):
        x[t, int(tokens[t, 1])] = -INF
    x[1, (int(tokens[1].max()) + 1) % V] = value
    tt, tv = torch.from_numpy(tokens).cuda(), torch.from_numpy(values).cuda()
    loss, d, saved = poet.distill_topk(x, tt, tv, tail=tail, grad=True)
    again = poet.distill_topk_grad(x, tt, tv, saved, tail=tail)
    poet.poet_sync_status()
    for g in (d, again):
        assert torch.isnan(g[1]).all() and torch.isfinite(g[[0, 2]]).all()
    assert torch.isnan(loss[1])


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_masked_targets(torch, dtype):  # noqa: F811
    """A masked token that is given or that the teacher lists: log probability -inf, an infinite loss, and the
    formulas' gradients with p = 0 there."""
    from orthogonal_reparameterized_poet_b200 import poet

    x, r = _make(torch, 3, 700, getattr(torch, dtype))
    x[:, 100:400] = -INF
    tk = torch.tensor([150, 20, 399], dtype=torch.int32, device="cuda")
    logp, _, _, _, saved = poet.token_logprobs(x, tk, scale=0.5)
    assert logp[0] == -INF and logp[2] == -INF and torch.isfinite(logp[1])
    w = torch.tensor([0.75, -1.5, 2.0], device="cuda")
    d = poet.token_logprobs_grad(x, tk, saved, w, scale=0.5)
    assert d[0, 150] == 0.375 and d[2, 399] == 1.0
    masked = torch.isneginf(x)
    masked[0, 150] = masked[2, 399] = False
    assert (d[masked] == 0).all()
    tokens = torch.stack([tk, torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")], 1).contiguous()
    values = torch.zeros(3, 2, device="cuda")
    loss, d, saved = poet.distill_topk(x, tokens, values, dloss=w, scale=0.5, grad=True)
    again = poet.distill_topk_grad(x, tokens, values, saved, w, scale=0.5)
    poet.poet_sync_status()
    assert loss[0] == INF and loss[2] == INF and torch.isfinite(loss[1])
    for g in (d, again):  # q = 1/2
        assert g[0, 150] == -0.5 * 0.75 * 0.5 and g[2, 399] == -0.5 * 2.0 * 0.5 and (g[masked] == 0).all()
