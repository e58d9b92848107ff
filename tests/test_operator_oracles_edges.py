"""The oracles of the operators on logits where the teacher's outcomes do not
sum to 1, pinned against central differences of the documented loss, written
out here."""
import numpy as np
import pytest

from oracle import logits as G
from tests.test_operator_oracles import _differences


def _loss(x, tokens, values, value_scale, scale):
    """sum_k q_k (ln q_k - ln p_k) + q_r (ln q_r - ln p_r) of one row, q_r = max(0, 1 - sum q)."""
    z = x * scale
    lp = z - np.log(np.exp(z).sum())
    keep = tokens >= 0
    q = np.exp(values[keep] * value_scale)
    loss = np.sum(q * (np.log(q) - lp[tokens[keep]]))
    outside = np.ones(x.size, bool)
    outside[tokens[keep]] = False
    rest = max(0.0, 1.0 - q.sum())
    if rest > 0 and outside.any():
        loss += rest * (np.log(rest) - np.log(np.exp(lp[outside]).sum()))
    return loss


@pytest.mark.parametrize("V,tokens,q,value_scale", [
    (7, [2, 2, 5], [0.6, 0.6, 0.1], 1.0),            # a token listed twice: 1.3
    (7, [2, 4, 5], [0.6, 0.2, 0.1], 0.5),            # log probabilities scaled down: 1.5
    (5, [3, 0, 1, 4, 2], [0.2, 0.1, 0.1, 0.2, 0.1], 1.0),  # every token listed, with less than the whole mass
    (1, [0], [0.5], 1.0),                            # the only token there is: a loss that no logit changes
    (7, [2, -1, 5], [0.5, 0.9, 0.3], 2.0),           # less than 1, the rest outside: as before
])
def test_distill_gradient_of_any_mass(V, tokens, q, value_scale):
    r = np.random.default_rng(V)
    x = r.standard_normal((1, V))
    tokens, values = np.array([tokens]), np.log(np.array([q]))
    scale = 0.8
    loss, d, mag = G.distill(x, tokens, values, None, value_scale, True, scale)
    assert np.allclose(loss[0], _loss(x[0], tokens[0], values[0], value_scale, scale), rtol=1e-12)
    # central differences: truncation STEP^2 f''' / 6 and rounding 2^-52 |f| / STEP, both below 1e-9 here
    want = _differences(lambda: _loss(x[0], tokens[0], values[0], value_scale, scale), x)
    assert np.allclose(d, want, rtol=1e-6, atol=1e-8)
    assert (np.abs(d) <= mag * (1 + 1e-12)).all()
    if V == 1:
        assert abs(d[0, 0]) < 1e-12
