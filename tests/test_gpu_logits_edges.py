"""Operators on logits at the edges of what they accept, against the float64
oracle (oracle/logits.py), with the bounds of tests/test_gpu_logits.py."""
import numpy as np
import pytest

from oracle import logits as G
from tests.test_gpu_logits import (INF, U, _check_distill, _check_logprobs, _gap, _make, _np, _steps, _teacher_case,
                                   _within, torch)  # noqa: F401

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


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V", [5, 3000, 40000])
@pytest.mark.parametrize("scale", [1e-37, 1e30, 2e38, 3.4e38])
def test_extreme_scales(torch, V, scale, dtype):  # noqa: F811
    """Up to the largest float: all the mass on the largest logits."""
    from orthogonal_reparameterized_poet_b200 import poet

    x, r = _make(torch, 4, V, getattr(torch, dtype))
    x[:, 2] = 30.0
    x[1, 4] = 30.0  # two of them
    if V > 5:
        x[2, 7] = -INF
    tokens = np.array([2, 4, 3, 0])
    tk, saved = _check_logprobs(torch, x, tokens, 3, scale)
    dl, de = (r.standard_normal(4).astype(np.float32) * np.float32(0.5 / scale) for _ in range(2))
    got = poet.token_logprobs_grad(x, tk, saved, torch.from_numpy(dl).cuda(), torch.from_numpy(de).cuda(), scale=scale)
    s = float(np.float32(scale))
    want, mag = G.token_logprobs_grad(_np(x), tokens, dl.astype(float), de.astype(float), s)
    near = np.minimum(_gap(_np(x), s), 200)  # beyond, a probability is 0 in float
    half = torch.finfo(x.dtype).eps / 2
    _within("dlogits", _np(got), want, half * np.abs(want) * 1.01 + (2 * _steps(V) + 6 * (near + np.log(V)) + 16) * U * mag
            + 1e-36)
    tokens, values = _teacher_case(r, 4, V, 3, False)
    tokens[:, 0] = 2
    if V > 5:
        tokens[2][tokens[2] == 7] = 9
    _check_distill(torch, x, tokens, values, r, False, scale, weights=False)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("weight", [1.0, 1e9, 1e30])
def test_large_weights_of_the_entropy(torch, weight, dtype):  # noqa: F811
    """Probabilities of 0 (masked logits, far ones) have a gradient of 0, whatever the entropy's weight."""
    from orthogonal_reparameterized_poet_b200 import poet

    V = 2000
    x, r = _make(torch, 5, V, getattr(torch, dtype), masked=0.3)
    x[0, ::2] = torch.finfo(x.dtype).min
    x[:, 11] = -500.0
    tk = torch.from_numpy(r.integers(0, V, 5).astype(np.int32)).cuda()
    saved = poet.token_logprobs(x, tk)[4]
    de = (r.standard_normal(5) * weight).astype(np.float32)
    got = poet.token_logprobs_grad(x, tk, saved, None, torch.from_numpy(de).cuda())
    want, mag = G.token_logprobs_grad(_np(x), tk.cpu().numpy(), None, de.astype(float), 1.0)
    half = torch.finfo(x.dtype).eps / 2
    near = np.minimum(_gap(_np(x), 1.0), 200)
    _within("dlogits", _np(got), want, half * np.abs(want) * 1.01 + (2 * _steps(V) + 6 * (near + np.log(V)) + 16) * U * mag
            + 1e-36 * weight)
    assert (got[torch.isneginf(x)] == 0).all()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,V,K", [(3, 7, 0), (5, 1000, 0), (400, 3001, 0), (2, 50257, 0), (1, 300000, 0), (300, 16000, 0),
                                   (3, 40, 5), (5, 1000, 20), (4, 32000, 20), (400, 3000, 128), (300, 20000, 40), (1, 128000, 9)])
@pytest.mark.parametrize("kind", ["plain", "masked", "far"])
def test_without_entropy(torch, T, V, K, kind, dtype):  # noqa: F811
    """Through the C ABI with neither the entropy nor what the backward reads: a sum of its own."""
    from orthogonal_reparameterized_poet_b200 import poet

    t = getattr(torch, dtype)
    x, r = _make(torch, T, V, t, masked=0.4 if kind == "masked" else 0.0, seed=K)
    if kind == "masked":
        x[0] = -INF
        if T > 1:
            x[1, ::3] = torch.finfo(t).min
    elif kind == "far":  # sums against a base that a fused operation would not do for
        x += torch.tensor(3.0e6 if t == torch.float32 else 2.0 ** 30, device="cuda").to(t)
    tokens = r.integers(0, V, T)
    tk = torch.from_numpy(tokens.astype(np.int32)).cuda()
    logp = torch.empty(T, device="cuda")
    top = torch.empty(T, K, dtype=torch.int32, device="cuda")
    topl = torch.empty(T, K, device="cuda")
    at = lambda v: v.data_ptr() if K else None  # noqa: E731
    st = torch.cuda.current_stream().cuda_stream
    status = poet.lib().poet_token_logprobs(x.data_ptr(), V, poet.BF16 if t == torch.bfloat16 else poet.F32, T, V, 0.9,
                                            tk.data_ptr(), K, logp.data_ptr(), None, at(top), at(topl), None, st)
    assert status == poet.OK
    poet.poet_sync_status()
    X, s = _np(x), float(np.float32(0.9))
    want, _, want_top, want_topl = G.token_logprobs(X, tokens, K, s)
    gap, N, lse = _gap(X, s), _steps(V), np.log(V) + 1
    _within("logp", _np(logp), want, (N + 3 * gap[np.arange(T), tokens] + 2 * np.abs(want) + 2 * lse) * U)
    if K:
        assert np.array_equal(top.cpu().numpy(), want_top)
        finite = np.isfinite(want_topl)
        g = np.take_along_axis(gap, np.maximum(want_top, 0).astype(np.int64), 1)
        with np.errstate(invalid="ignore"):
            _within("top_logp", _np(topl), want_topl, (N + 3 * g + 2 * np.where(finite, np.abs(want_topl), 0) + 2 * lse) * U)


@pytest.mark.parametrize("K", [1, 5, 64])
@pytest.mark.parametrize("value_scale", [1e-37, 1e20, 3.4e38])
def test_extreme_scales_of_the_teacher(torch, K, value_scale):  # noqa: F811
    """Up to the largest float: all the mass on the teacher's largest values, also where their products overflow."""
    x, r = _make(torch, 6, 900, torch.float32)
    tokens, values = _teacher_case(r, 6, 900, K, False)
    values[0] = 2.0  # all equal
    values[1] = -3.0
    if K > 1:
        values[2, 0] = values[2, 1] = 9.0  # two of them
        values[3, 1] = -INF
        tokens[4, 0] = -1
    loss, d = _check_distill(torch, x, tokens, values, r, False, 1.0, value_scale, weights=False)
    # q is 0 or a whole number's inverse, off by K half steps; ln p and p as ever
    want, dwant, mag = G.distill(_np(x), tokens, values.astype(float), None, float(np.float32(value_scale)))
    bound = (2 * _steps(900) + 6 * (_gap(_np(x), 1.0).max() + np.log(900)) + 64 + K) * U
    _within("loss", _np(loss), want, bound * (1 + np.abs(want)))
    _within("dlogits", _np(d), dwant, bound * mag + 1e-36)
