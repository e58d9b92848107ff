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
