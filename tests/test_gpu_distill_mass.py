"""The distillation with the tail where the teacher's outcomes do not sum to 1,
against the float64 oracle (oracle/logits.py), with the bounds of tests/test_gpu_logits.py."""
import numpy as np
import pytest

from tests.test_gpu_logits import INF, U, _check_distill, _make, _np, _steps, _teacher_case, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def _masses(r, T, V, K, kind):
    """Teachers with the tail whose outcomes do not sum to 1: (tokens, values, value_scale)."""
    if kind == "all listed":  # V = K: less than the whole mass, and nothing outside
        tokens, values = _teacher_case(r, T, V, K, True)
        return tokens, values - np.float32(0.4), 1.0
    tokens, values = _teacher_case(r, T, V, K, True, twice=kind == "twice")
    if kind == "twice":  # the token that is listed twice has 0.6 each time, beside the others
        values -= 0.1
        values[:, 0] = values[:, K // 2] = np.log(np.float32(0.6))
        return tokens, values, 1.0
    return tokens, values, 0.5  # true log probabilities, scaled down


# The mass itself is off by (K + 16 + 4 |value|) half steps of float of its size, which the bound on each gradient
# already counts on p times the mass.
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,V,K,kind", [(1, 1, 1, "all listed"), (6, 12, 12, "all listed"), (3, 128, 128, "all listed"),
                                        (7, 33, 3, "twice"), (500, 777, 9, "twice"), (2, 32000, 64, "twice"),
                                        (1, 128000, 20, "twice"), (7, 33, 4, "scaled"), (300, 1111, 16, "scaled"),
                                        (2, 50257, 20, "scaled"), (1, 128000, 128, "scaled")])
def test_distill_gradient_of_any_mass(torch, T, V, K, kind, dtype):  # noqa: F811
    x, r = _make(torch, T, V, getattr(torch, dtype), seed=K)
    tokens, values, value_scale = _masses(r, T, V, K, kind)
    loss, d = _check_distill(torch, x, tokens, values, r, True, 1.25, value_scale)
    if V == 1:  # the only token there is: no logit changes the loss
        assert torch.equal(d, torch.zeros_like(d))


@pytest.mark.parametrize("kind", ["twice", "scaled"])
def test_distill_gradient_of_any_mass_of_many_rows(torch, kind):  # noqa: F811
    """More rows than the GPU works on at once, the gradient written over the logits."""
    from orthogonal_reparameterized_poet_b200 import poet

    few, T, V, K = 16, 1500, 20000, 12
    base, r = _make(torch, few, V, torch.float32)
    tokens, values, value_scale = _masses(r, few, V, K, kind)
    loss, d = _check_distill(torch, base, tokens, values, r, True, 1.0, value_scale, weights=False)
    order = torch.from_numpy(r.integers(0, few, T)).cuda()
    x, tt, tv = base[order].contiguous(), torch.from_numpy(tokens).cuda()[order], torch.from_numpy(values).cuda()[order]
    got, same, _ = poet.distill_topk(x, tt, tv, value_scale=value_scale, tail=True, dlogits=x)
    poet.poet_sync_status()
    # the sums may be split otherwise with more rows
    bound = 4 * _steps(V) * U
    assert ((got - loss[order]).abs() <= bound * (1 + loss[order].abs())).all()
    assert ((x - d[order]).abs() <= 2 * bound * (d[order].abs() + torch.softmax(base.double(), 1)[order] * 2) + 1e-9).all()
