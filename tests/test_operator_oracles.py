"""The float64 oracles of the joint and of the operators on logits, pinned
without the CUDA library: their gradients against central differences of their
forwards, closed forms, and the cases with nothing to sum."""
import numpy as np
import pytest

from oracle import joint as J
from oracle import logits as G

STEP = 1e-5


def _differences(f, x):
    """Central differences of the scalar f at every element of x (x is changed in place and put back)."""
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        v = x[i]
        x[i] = v + STEP
        up = f()
        x[i] = v - STEP
        down = f()
        x[i] = v
        out[i] = (up - down) / (2 * STEP)
    return out


@pytest.mark.parametrize("gate,rows,sigmoid,post", [(None, 1, False, True), ("channel", 1, True, True),
                                                    ("channel", 2, False, True), ("channel", 5, True, False),
                                                    ("row", 1, False, True), ("row", 3, True, True)])
def test_joint_gradients_match_differences(gate, rows, sigmoid, post):
    r = np.random.default_rng(3)
    T, d = 5, 6
    o, h, dh_out, dn = (r.standard_normal((T, d)) for _ in range(4))
    G_ = -(-T // rows)
    g = None if gate is None else r.standard_normal((G_, d) if gate == "channel" else (G_,))
    wq = 1 + 0.3 * r.standard_normal(d) if post else None
    wn = 1 + 0.3 * r.standard_normal(d)
    kw = dict(post_norm=post, sigmoid=sigmoid, rows=rows, alpha=0.8, beta=0.6)

    def loss():
        a, n, _, _ = J.forward(o, h, g, wq, wn, **kw)
        return np.sum(a * dh_out) + np.sum(n * dn)

    after = J.forward(o, h, g, wq, wn, **kw)[0]
    got = J.backward(o, after, g, dh_out, dn, wq, wn, **kw)
    for name, x in (("do", o), ("dh", h), ("dgate", g), ("dw_post", wq), ("dw_pre", wn)):
        if x is not None:
            # central differences: truncation STEP^2 f'''/6 and rounding 2^-52 |f| / STEP, both < 1e-8 here
            assert np.allclose(got[name][0], _differences(loss, x), rtol=1e-6, atol=1e-7), name


@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_logprob_gradients_match_differences(scale):
    r = np.random.default_rng(4)
    x = r.standard_normal((3, 7))
    tokens = np.array([2, -1, 6])
    dl, de = r.standard_normal(3), r.standard_normal(3)

    def loss():
        logp, H, _, _ = G.token_logprobs(x, tokens, 0, scale)
        return np.sum(dl * logp) + np.sum(de * H)

    d, _ = G.token_logprobs_grad(x, tokens, dl, de, scale)
    assert np.allclose(d, _differences(loss, x), rtol=1e-6, atol=1e-7)
    assert np.all(d[1] == 0)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("twice", [False, True])
def test_distill_gradients_match_differences(tail, twice):
    r = np.random.default_rng(5)
    x = r.standard_normal((4, 9))
    tokens = np.array([[1, 4, 7], [0, 8, -1], [-1, -1, -1], [3, 3 if twice else 5, 2]])
    values = np.log(r.dirichlet(np.ones(4), 4)[:, :3])
    w = r.standard_normal(4)

    def loss():
        return np.sum(w * G.distill(x, tokens, values, None, 1.0, tail, 0.8)[0])

    d = G.distill(x, tokens, values, w, 1.0, tail, 0.8)[1]
    assert np.allclose(d, _differences(loss, x), rtol=1e-6, atol=1e-7)
    assert np.all(d[2] == 0)


def test_closed_forms():
    # a uniform row: -ln V, entropy ln V, alternatives in order of index
    logp, H, top, topl = G.token_logprobs(np.zeros((1, 8)), np.array([3]), 3, 2.0)
    assert np.allclose([logp[0], H[0]], [-np.log(8), np.log(8)]) and list(top[0]) == [0, 1, 2]
    # one entry: cross-entropy
    x = np.random.default_rng(0).standard_normal((2, 5))
    loss, d, _ = G.distill(x, np.array([[1], [4]]), np.zeros((2, 1)))
    logp = G.token_logprobs(x, np.array([1, 4]), 0, 1.0)[0]
    assert np.allclose(loss, -logp)
    assert np.allclose(d, -G.token_logprobs_grad(x, np.array([1, 4]), np.ones(2), None, 1.0)[0])
    # the student is the teacher: loss and gradient 0, with and without the tail
    lp = G.row_log_softmax(x, 1.0)
    tokens = np.array([[0, 2], [3, 1]])
    loss, d, _ = G.distill(x, tokens, np.take_along_axis(lp, tokens, 1), tail=True)
    assert np.allclose(loss, 0) and np.allclose(d, 0)


def test_rows_with_nothing():
    x = np.full((2, 4), -np.inf)
    x[1, 2] = 0.5
    logp, H, top, topl = G.token_logprobs(x, np.array([1, 2]), 2, 1.0)
    assert np.isneginf(logp[0]) and logp[1] == 0 and np.all(H == 0)
    assert list(top[0]) == [-1, -1] and list(top[1]) == [2, -1]
    assert np.all(G.token_logprobs_grad(x, np.array([1, 2]), np.ones(2), np.ones(2), 1.0)[0][0] == 0)
    loss, d, _ = G.distill(x, np.array([[0], [2]]), np.zeros((2, 1)))
    assert np.isposinf(loss[0]) and loss[1] == 0 and np.all(d == 0)
