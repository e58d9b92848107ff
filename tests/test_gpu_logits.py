"""Log probabilities with entropy and alternatives, distillation from a
teacher's top logits, and their gradients, against the float64 oracle
(oracle/logits.py) on the same inputs.

Tolerances, derived before the first run (u = 2^-24, half a step of float):
  * a row's sum: a thread adds V / 256 terms in sequence (at most as many
    rescalings as it has vectors, each an exponential of 4u), 13 levels join the
    threads and CTAs, each with a rescaling, and every term is an exponential
    (4u) of an argument off by 2u of itself, which the exponential damps to
    below 2u: N = V / 256 * 2 + 128 half steps bound the sum's relative error;
  * a log probability: N u for the logarithm of the sum, plus 3u of the
    difference to the maximum and 2u of the logarithm and the result;
  * an entropy: the sums' N u on each of its terms;
  * a probability: N u + 3u |ln p| of itself, and a gradient that of the
    magnitudes of its terms, plus half a step of its type;
  * q: 16u + 4u |value| of itself; q_r = 1 - sum q: (K + 16) u of 1.
Whole numbers are equal.
"""
import numpy as np
import pytest

from oracle import logits as G

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF = float("inf")


@pytest.fixture(scope="module")
def torch():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from orthogonal_reparameterized_poet_b200 import poet

    poet.lib()
    poet.poet_sync_status()
    return torch


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _steps(V):
    return V / 256 * 2 + 128


def _assert(ok, name, got, want, bound):
    bad = ~ok
    with np.errstate(invalid="ignore"):
        assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                               f"{got[bad][0]} for {want[bad][0]}, bound {np.broadcast_to(bound, got.shape)[bad][0]}")


def _within(name, got, want, bound):
    # a value beyond float's range (a mask of the lowest value, times a scale) rounds to infinity
    want = np.where(np.abs(want) >= 2.0 ** 128 * (1 - 2.0 ** -25), np.copysign(np.inf, want), want)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        _assert(same | (np.abs(got - want) <= bound), name, got, want, bound)


def _make(torch, T, V, dtype, ld=None, offset=0, seed=0, masked=0.0, sd=2.0):
    r = np.random.default_rng(seed + 31 * T + V)
    ld = V if ld is None else ld
    buf = torch.full((offset + T * ld + 16,), float("nan"), dtype=dtype, device="cuda")
    x = buf[offset:offset + T * ld].view(T, ld)[:, :V]
    v = r.standard_normal((T, V)) * sd
    if masked:
        v[r.random((T, V)) < masked] = -np.inf
    x.copy_(torch.from_numpy(v).to(dtype))
    return x, r


def _gap(x, scale):
    """(M - x) scale per element, 0 for masked ones."""
    m = np.max(x, axis=1, keepdims=True)
    g = (np.where(np.isneginf(m), 0.0, m) - x) * scale
    return np.where(np.isfinite(g), g, 0.0)


def _check_logprobs(torch, x, tokens, K, scale=1.0):
    from orthogonal_reparameterized_poet_b200 import poet

    tk = None if tokens is None else torch.from_numpy(tokens.astype(np.int32)).cuda()
    logp, H, top, topl, saved = poet.token_logprobs(x, tk, topk=K, scale=scale)
    poet.poet_sync_status()
    s = float(np.float32(scale))
    X = _np(x)
    T, V = X.shape
    want_logp, want_H, want_top, want_topl = G.token_logprobs(X, tokens, K, s)
    gap, N = _gap(X, s), _steps(V)
    lse = np.log(V) + 1
    if tokens is not None:
        at = gap[np.arange(T), np.maximum(tokens, 0)]
        _within("logp", _np(logp), want_logp, (N + 3 * at + 2 * np.abs(want_logp) + 2 * lse) * U)
    lp = G.row_log_softmax(X, s)
    mean_gap = (np.exp(lp) * gap).sum(1)
    _within("entropy", _np(H), want_H, (2 * N * (1 + mean_gap) + 4 * lse) * U)
    if K:
        assert np.array_equal(top.cpu().numpy(), want_top)
        finite = np.isfinite(want_topl)
        g = np.take_along_axis(gap, np.maximum(want_top, 0).astype(np.int64), 1)
        with np.errstate(invalid="ignore"):
            bound = (N + 3 * g + 2 * np.where(finite, np.abs(want_topl), 0) + 2 * lse) * U
        _within("top_logp", _np(topl), want_topl, bound)
    return tk, saved


def _check_logprobs_grad(torch, x, tokens, tk, saved, r, scale=1.0, which="both", out=None):
    from orthogonal_reparameterized_poet_b200 import poet

    T, V = x.shape
    dl = r.standard_normal(T).astype(np.float32) if which != "entropy" else None
    de = r.standard_normal(T).astype(np.float32) if which != "logp" else None
    X = _np(x)
    s = float(np.float32(scale))
    got = poet.token_logprobs_grad(x, tk, saved, None if dl is None else torch.from_numpy(dl).cuda(),
                                   None if de is None else torch.from_numpy(de).cuda(), scale=scale, dlogits=out)
    poet.poet_sync_status()
    want, mag = G.token_logprobs_grad(X, tokens, None if dl is None else dl.astype(float),
                                      None if de is None else de.astype(float), s)
    half = torch.finfo(x.dtype).eps / 2
    bound = half * np.abs(want) * 1.01 + (2 * _steps(V) + 6 * (_gap(X, s) + np.log(V)) + 16) * U * mag + 1e-36
    _within("dlogits", _np(got), want, bound)
    return got


SHAPES = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 33), (300, 257), (7, 1000), (1, 4099), (700, 512), (2, 9001), (3, 32000),
          (1, 50257), (1, 128000)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,V", SHAPES)
@pytest.mark.parametrize("K", [0, 1, 20, 128])
def test_logprobs_shapes(torch, T, V, K, dtype):
    x, r = _make(torch, T, V, getattr(torch, dtype), seed=K)
    tokens = r.integers(0, V, T)
    tk, saved = _check_logprobs(torch, x, tokens, K)
    _check_logprobs_grad(torch, x, tokens, tk, saved, r)


@pytest.mark.parametrize("scale", [0.3, 1.7])
@pytest.mark.parametrize("which", ["logp", "entropy", "both"])
def test_logprobs_scale_and_parts(torch, scale, which):
    x, r = _make(torch, 9, 3001, torch.bfloat16)
    tokens = r.integers(0, 3001, 9)
    tk, saved = _check_logprobs(torch, x, tokens, 5, scale)
    _check_logprobs_grad(torch, x, tokens, tk, saved, r, scale, which)


def test_entropy_and_alternatives_without_tokens(torch):
    from orthogonal_reparameterized_poet_b200 import poet

    x, r = _make(torch, 6, 777, torch.float32)
    _check_logprobs(torch, x, None, 10)
    logp, H, top, topl, saved = poet.token_logprobs(x, None, topk=3)
    assert logp is None and top.shape == (6, 3)
    _check_logprobs_grad(torch, x, None, None, saved, r, which="entropy")
    assert poet.token_logprobs(x, None, entropy=False)[1] is None


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("ld,offset", [(1003, 0), (1008, 0), (1001, 1), (1024, 8), (1005, 5)])
def test_strides_and_addresses(torch, dtype, ld, offset):
    t = getattr(torch, dtype)
    x, r = _make(torch, 11, 1001, t, ld, offset)
    tokens = r.integers(0, 1001, 11)
    tk, saved = _check_logprobs(torch, x, tokens, 7)
    # into rows of another stride and alignment; what lies behind a row's V columns stays as it was
    out, _ = _make(torch, 11, 1001, t, 1017, 2)
    whole = out.as_strided((10, 1017), (1017, 1))[:, 1001:]
    before = whole.clone().view(torch.int16 if dtype == "bfloat16" else torch.int32)
    _check_logprobs_grad(torch, x, tokens, tk, saved, r, out=out)
    assert torch.equal(whole.contiguous().view(before.dtype), before)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,V", [(3, 40), (4, 1003), (2, 20000), (400, 3000)])
@pytest.mark.parametrize("kind", ["constant", "two values", "zeros of both signs", "falling", "rising", "one chunk",
                                  "last", "first"])
@pytest.mark.parametrize("K", [1, 20, 128])
def test_ties_and_orders(torch, T, V, kind, K, dtype):
    x, r = _make(torch, T, V, getattr(torch, dtype))
    v = np.zeros((T, V))
    if kind == "two values":
        v = (r.random((T, V)) < 0.5).astype(float)
    elif kind == "zeros of both signs":
        v = np.where(r.random((T, V)) < 0.5, 0.0, -0.0)
    elif kind in ("falling", "rising"):
        v = np.tile(np.linspace(4, -4, V), (T, 1))
        v = v[:, ::-1].copy() if kind == "rising" else v
    elif kind == "one chunk":  # the largest side by side, in the middle
        v = r.standard_normal((T, V))
        v[:, V // 2:V // 2 + 150] += 20
    elif kind == "last":
        v[:, -1] = 1
    elif kind == "first":
        v[:, 0] = 1
    x.copy_(torch.from_numpy(v).to(x.dtype))
    _check_logprobs(torch, x, r.integers(0, V, T), K)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,V,K", [(4000, 2000, 20), (4000, 1500, 32), (3000, 3001, 50), (1500, 9000, 128), (700, 40000, 20)])
def test_alternatives_of_many_rows(torch, T, V, K, dtype):
    """More rows than the GPU works on at once, rows of every kind of order side by side: ties, few and many distinct
    values, masks, and ordinary rows."""
    x, r = _make(torch, T, V, getattr(torch, dtype))
    kind = torch.arange(T, device="cuda") % 7
    x[kind == 0] = 0.0
    x[kind == 1] = (x[kind == 1] > 0).to(x.dtype)
    x[kind == 2] = torch.linspace(-4, 4, V, device="cuda").to(x.dtype)
    x[kind == 3] = torch.where(x[kind == 3] < 4.0, -INF, x[kind == 3].float()).to(x.dtype)
    x[kind == 4] = torch.round(x[kind == 4].float()).to(x.dtype)
    _check_logprobs(torch, x, r.integers(0, V, T), K)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,V", [(3, 50), (5, 2000), (1, 33000)])
def test_masks(torch, T, V, dtype):
    t = getattr(torch, dtype)
    x, r = _make(torch, T, V, t, masked=0.5)
    tokens = r.integers(0, V, T)
    tk, saved = _check_logprobs(torch, x, tokens, 9, 1.3)
    _check_logprobs_grad(torch, x, tokens, tk, saved, r, 1.3)
    # fewer tokens left than alternatives asked for; one; none
    x.fill_(-INF)
    if T > 1:
        x[1, V // 2] = 1.5
        x[1, 3] = 2.5
        x[2, V - 1] = -3.0
    tk, saved = _check_logprobs(torch, x, tokens, 9)
    _check_logprobs_grad(torch, x, tokens, tk, saved, r)
    # masks of the type's lowest value: a probability of 0 beside others, of 1 / V among themselves
    low = torch.finfo(t).min
    x.fill_(low)
    x[0, 5] = 0.0
    tk, saved = _check_logprobs(torch, x, tokens, 3, 2.0)
    _check_logprobs_grad(torch, x, tokens, tk, saved, r, 2.0)


def test_rows_left_out(torch):
    from orthogonal_reparameterized_poet_b200 import poet

    for T, V in ((6, 500), (2, 40000)):
        x, r = _make(torch, T, V, torch.bfloat16)
        tokens = r.integers(0, V, T)
        tokens[1] = -1
        x[1] = float("nan")  # what a padded row holds does not matter
        x[1, 3] = INF
        tk = torch.from_numpy(tokens.astype(np.int32)).cuda()
        logp, H, top, topl, saved = poet.token_logprobs(x, tk, topk=4)
        d = poet.token_logprobs_grad(x, tk, saved, torch.ones(T, device="cuda"), torch.ones(T, device="cuda"))
        assert logp[1] == 0 and H[1] == 0 and (top[1] == -1).all() and (topl[1] == -INF).all() and (d[1] == 0).all()
        assert torch.isfinite(logp).all() and torch.isfinite(d).all()
        teacher = torch.full((T, 3), -1, dtype=torch.int32, device="cuda")
        teacher[0, 1] = 7
        loss, d, saved = poet.distill_topk(x, teacher, torch.zeros(T, 3, device="cuda"), grad=True)
        assert loss[1] == 0 and (d[1] == 0).all() and loss[0] > 0
        d2 = poet.distill_topk_grad(x, teacher, torch.zeros(T, 3, device="cuda"), saved)
        assert (d2[1] == 0).all()
        poet.poet_sync_status()


@pytest.mark.parametrize("value", [float("nan"), INF])
def test_a_row_of_nan_or_infinity_stays_alone(torch, value):
    from orthogonal_reparameterized_poet_b200 import poet

    for T, V in ((5, 700), (2, 30000)):
        x, r = _make(torch, T, V, torch.float32)
        tk = torch.from_numpy(r.integers(0, V, T).astype(np.int32)).cuda()
        one = torch.ones(T, device="cuda")
        teacher, values = tk[:, None].contiguous(), torch.zeros(T, 1, device="cuda")

        def everything():
            logp, H, top, topl, saved = poet.token_logprobs(x, tk, topk=4)
            d = poet.token_logprobs_grad(x, tk, saved, one, one)
            loss, dd, sv = poet.distill_topk(x, teacher, values, grad=True)
            lt, dt, st = poet.distill_topk(x, teacher, values - 0.5, grad=True, tail=True)
            return [logp, H, topl, d, loss, dd, lt, dt, poet.distill_topk_grad(x, teacher, values, sv)], top

        before, _ = everything()
        x[1, V // 3] = value
        after, top = everything()
        for a, b in zip(before, after):
            assert torch.equal(a[0], b[0])
            assert torch.isnan(b[1]).all()
        assert (top[1] == -1).all()
        poet.poet_sync_status()


def test_tokens_out_of_range_are_reported(torch):
    from orthogonal_reparameterized_poet_b200 import poet

    x, r = _make(torch, 4, 100, torch.bfloat16)
    tk = torch.tensor([1, 100, 5, 2**31 - 1], dtype=torch.int32, device="cuda")
    logp, H, top, topl, saved = poet.token_logprobs(x, tk, topk=2)
    with pytest.raises(poet.PoetError) as e:
        poet.poet_sync_status()
    assert e.value.status == poet.EBOUNDS
    assert logp[1] == 0 and logp[3] == 0 and logp[0] < 0 and (top[1] == -1).all()
    d = poet.token_logprobs_grad(x, tk, saved, torch.ones(4, device="cuda"))
    with pytest.raises(poet.PoetError):
        poet.poet_sync_status()
    assert (d[1] == 0).all() and (d[0] != 0).any()
    # a teacher's entry out of range is left out, the others of its row count
    teacher = torch.tensor([[3, 100], [4, -1], [100, 100], [5, 6]], dtype=torch.int32, device="cuda")
    val = torch.zeros(4, 2, device="cuda")
    loss, d, sv = poet.distill_topk(x, teacher, val, grad=True)
    with pytest.raises(poet.PoetError):
        poet.poet_sync_status()
    fixed = torch.where(teacher >= 100, -1, teacher)
    loss2, d2, _ = poet.distill_topk(x, fixed, val, grad=True)
    poet.poet_sync_status()
    assert torch.equal(loss, loss2) and torch.equal(d, d2)
    poet.distill_topk_grad(x, teacher, val, sv)
    with pytest.raises(poet.PoetError):
        poet.poet_sync_status()


# ------------------------------------------------------------------ distillation

def _teacher_case(r, T, V, K, tail, ragged=False, twice=False):
    tokens = np.stack([r.permutation(V)[:K] for _ in range(T)]).astype(np.int32)
    if tail:
        values = np.log(r.dirichlet(np.ones(K + 1) * 0.7, T)[:, :K] + 1e-6)
        values -= np.log(np.exp(values).sum(1, keepdims=True)) + r.uniform(0.02, 1.0, (T, 1))
    else:
        values = r.standard_normal((T, K)) * 2
    values = values.astype(np.float32)
    if ragged:
        tokens[r.random((T, K)) < 0.4] = -1
        tokens[0, :] = -1
    if twice and K > 1:
        tokens[:, K // 2] = tokens[:, 0]
    return tokens, values


def _check_distill(torch, x, tokens, values, r, tail, scale=1.0, value_scale=1.0, weights=True, out=None):
    from orthogonal_reparameterized_poet_b200 import poet

    T, V = x.shape
    K = tokens.shape[1]
    X = _np(x)
    s, vs = float(np.float32(scale)), float(np.float32(value_scale))
    w = r.standard_normal(T).astype(np.float32) if weights else None
    tw = None if w is None else torch.from_numpy(w).cuda()
    tt, tv = torch.from_numpy(tokens).cuda(), torch.from_numpy(values).cuda()
    kw = dict(tail=tail, scale=scale, value_scale=value_scale)
    plain, none, saved0 = poet.distill_topk(x, tt, tv, **kw)
    assert none is None
    loss, d, saved = poet.distill_topk(x, tt, tv, dloss=tw, grad=True, dlogits=out, **kw)
    d = d.clone()
    again = poet.distill_topk_grad(x, tt, tv, saved, tw, dlogits=out, **kw)
    poet.poet_sync_status()
    assert torch.equal(plain, loss) and torch.equal(saved0, saved)
    want, dwant, mag = G.distill(X, tokens, values.astype(float), None if w is None else w.astype(float), vs, tail, s)
    N = _steps(V)
    gap = _gap(X, s)
    av = np.abs(np.where(np.isfinite(values), values * vs, 0.0))  # a value of -inf has q = 0, exactly
    # the loss's terms: q (|ln q| + |ln p|), q off by 16u + 4u|value|, ln p by N u + 3u gap; the rest by (K + 16)u / q_r
    lp = G.row_log_softmax(X, s)
    bound = np.zeros(T)
    for t in range(T):
        teacher = G._teacher(tokens[t], values[t].astype(float), vs, tail)
        if teacher is None:
            continue
        q, lq, rest = teacher
        use = q > 0
        lpt = lp[t][tokens[t][use]]
        with np.errstate(invalid="ignore"):
            m = q[use] * ((16 + 4 * av[t][use] + K) * (np.abs(lq[use]) + np.abs(lpt) + 1) + N +
                          3 * gap[t][tokens[t][use]] + np.log(V) * 2)
            bound[t] = m.sum() * U
        if tail and rest > 0:
            ins = np.zeros(V, bool)
            ins[tokens[t][tokens[t] >= 0]] = True
            pr = np.exp(lp[t][~ins]).sum()
            if pr > 0:
                err = (K + 16 + 4 * av[t].max()) * U
                bound[t] += err * (np.abs(np.log(rest)) + np.abs(np.log(pr)) + 2) + rest * 2 * N * U * (
                    1 + np.abs(np.log(pr)))
    _within("loss", _np(loss), want, bound + K * U * np.where(np.isfinite(want), np.abs(want), 0))
    half = torch.finfo(x.dtype).eps / 2
    live = np.exp(lp)
    extra = np.zeros((T, V))
    if tail:  # q_r's absolute error, on every token outside
        for t in range(T):
            ins = np.zeros(V, bool)
            ins[tokens[t][tokens[t] >= 0]] = True
            pr = live[t][~ins].sum()
            if pr > 0 and not ins.all():
                extra[t] = np.where(ins, 0, live[t] / pr) * (K + 16 + 4 * av[t].max())
    gw = np.ones(T) if w is None else np.abs(w)
    vmax = 4 * av.max(1, keepdims=True)
    gb = half * np.abs(dwant) * 1.01 + U * ((2 * N + 6 * (gap + np.log(V)) + K + 32 + vmax) * mag +
                                             extra * s * gw[:, None]) + 1e-36
    _within("dlogits", _np(d), dwant, gb)
    _within("dlogits of the backward", _np(again), dwant, gb)
    return loss, d


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (3, 2, 1), (2, 7, 7), (5, 33, 4), (300, 257, 16), (9, 1000, 128),
                                   (1, 4099, 64), (500, 777, 3), (2, 9001, 20), (3, 32000, 64), (1, 128000, 33)])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_shapes(torch, T, V, K, tail, dtype):
    x, r = _make(torch, T, V, getattr(torch, dtype), seed=K)
    tokens, values = _teacher_case(r, T, V, K, tail)
    _check_distill(torch, x, tokens, values, r, tail)


@pytest.mark.parametrize("V,K", [(3000, 20), (32000, 64), (50257, 20), (70000, 33)])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_of_many_rows(torch, V, K, tail):
    """More rows than the GPU works on at once, of every kind of width, twice: some rows left out.  Distinct rows repeat,
    so that the oracle need not see each."""
    from orthogonal_reparameterized_poet_b200 import poet

    few, T = 24, 1800
    base, r = _make(torch, few, V, torch.bfloat16)
    tokens, values = _teacher_case(r, few, V, K, tail)
    tokens[5] = -1
    order = torch.from_numpy(r.integers(0, few, T)).cuda()
    x, tt, tv = base[order].contiguous(), torch.from_numpy(tokens).cuda()[order], torch.from_numpy(values).cuda()[order]
    want, dwant = _check_distill(torch, base, tokens, values, r, tail, weights=False)
    plain, none, _ = poet.distill_topk(base, torch.from_numpy(tokens).cuda(), torch.from_numpy(values).cuda(), tail=tail)
    for _ in range(4):
        loss, d, saved = poet.distill_topk(x, tt, tv, tail=tail, grad=True)
        alone = poet.distill_topk(x, tt, tv, tail=tail)[0]
        tk = torch.where(tt[:, 0] < 0, 0, tt[:, 0]).contiguous()
        logp, H, top, topl, sv = poet.token_logprobs(x, tk, topk=5)
        poet.poet_sync_status()
        # the sums may be split otherwise with more rows: compared within the derived bound of the sums
        bound = 4 * _steps(V) * U * (1 + want.abs()[order].double())
        assert ((loss - want[order]).double().abs() <= bound).all() and ((alone - want[order]).double().abs() <= bound).all()
        half = torch.finfo(x.dtype).eps / 2
        scale = dwant[order].double().abs()
        assert ((d.double() - dwant[order].double()).abs() <= 2 * half * scale + 8 * _steps(V) * U * scale + 1e-9).all()
        mean = torch.log_softmax(x.double(), 1)
        at = mean.gather(1, tk.long()[:, None])[:, 0]
        assert ((logp.double() - at).abs() <= (_steps(V) + 64) * U * (1 + at.abs())).all()
        assert torch.equal(top.long(), x.sort(dim=1, descending=True, stable=True)[1][:, :5])


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("ragged,twice", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("scale,value_scale", [(1.0, 1.0), (0.5, 1.3)])
def test_distill_ragged_and_listed_twice(torch, tail, ragged, twice, scale, value_scale):
    x, r = _make(torch, 13, 1111, torch.float32)
    tokens, values = _teacher_case(r, 13, 1111, 9, tail, ragged, twice)
    if tail and twice:
        values -= 0.7  # room for the mass that is counted twice
    _check_distill(torch, x, tokens, values, r, tail, scale, value_scale, weights=False)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_masks(torch, tail, dtype):
    t = getattr(torch, dtype)
    for T, V in ((6, 900), (2, 20001)):
        x, r = _make(torch, T, V, t, masked=0.4)
        tokens, values = _teacher_case(r, T, V, 5, tail)
        for i in range(T):  # the teacher's own tokens are not masked
            x[i, torch.from_numpy(tokens[i].astype(np.int64)).cuda()] = 0.5
        values[0, 2] = -np.inf  # a value of -inf: q = 0
        _check_distill(torch, x, tokens, values, r, tail)
        x[1, int(tokens[1, 0])] = -INF  # a teacher's token that the student masks: an infinite loss, finite gradients
        loss, d = _check_distill(torch, x, tokens, values, r, tail)
        assert loss[1] == INF and torch.isfinite(d).all()
        x[0] = -INF
        loss, d = _check_distill(torch, x, tokens, values, r, tail)
        assert loss[0] == INF and (d[0] == 0).all()


def test_distill_far_tail(torch):
    """The student has almost nothing outside the teacher's tokens (below what a float holds beside 1)."""
    x, r = _make(torch, 4, 600, torch.float32, sd=1.0)
    tokens, values = _teacher_case(r, 4, 600, 6, True)
    for i, up in enumerate((15.0, 40.0, 120.0, 400.0)):
        x[i, torch.from_numpy(tokens[i].astype(np.int64)).cuda()] += up
    _check_distill(torch, x, tokens, values, r, True)


def test_distill_all_tokens_listed(torch):
    x, r = _make(torch, 5, 12, torch.float32)
    tokens = np.stack([r.permutation(12) for _ in range(5)]).astype(np.int32)
    values = np.log(r.dirichlet(np.ones(12), 5)).astype(np.float32)
    _check_distill(torch, x, tokens, values, r, True)
    _check_distill(torch, x, tokens, values, r, False)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("ld,offset", [(1003, 0), (1001, 1), (1024, 8)])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_strides(torch, dtype, ld, offset, tail):
    t = getattr(torch, dtype)
    x, r = _make(torch, 6, 1001, t, ld, offset)
    tokens, values = _teacher_case(r, 6, 1001, 8, tail)
    out, _ = _make(torch, 6, 1001, t, 1017, 2)
    whole = out.as_strided((5, 1017), (1017, 1))[:, 1001:]
    before = whole.clone().view(torch.int16 if dtype == "bfloat16" else torch.int32)
    _check_distill(torch, x, tokens, values, r, tail, out=out)
    assert torch.equal(whole.contiguous().view(before.dtype), before)


@pytest.mark.parametrize("T,V", [(300, 2000), (2, 50000), (1, 128000)])
def test_in_place(torch, T, V):
    from orthogonal_reparameterized_poet_b200 import poet

    x, r = _make(torch, T, V, torch.bfloat16)
    tk = torch.from_numpy(r.integers(0, V, T).astype(np.int32)).cuda()
    dl, de = torch.randn(T, device="cuda"), torch.randn(T, device="cuda")
    saved = poet.token_logprobs(x, tk)[4]
    want = poet.token_logprobs_grad(x, tk, saved, dl, de)
    y = x.clone()
    assert torch.equal(poet.token_logprobs_grad(y, tk, saved, dl, de, dlogits=y), want)
    for tail in (False, True):
        tokens, values = _teacher_case(r, T, V, 10, tail)
        tt, tv = torch.from_numpy(tokens).cuda(), torch.from_numpy(values).cuda()
        loss, want, saved = poet.distill_topk(x, tt, tv, tail=tail, dloss=dl, grad=True)
        y = x.clone()
        got = poet.distill_topk(y, tt, tv, tail=tail, dloss=dl, dlogits=y)
        assert torch.equal(got[0], loss) and torch.equal(y, want)
        y = x.clone()
        poet.distill_topk_grad(y, tt, tv, saved, dl, tail=tail, dlogits=y)
        want2 = poet.distill_topk_grad(x, tt, tv, saved, dl, tail=tail)
        assert torch.equal(y, want2)


def test_same_bits_streams_and_graph(torch):
    from orthogonal_reparameterized_poet_b200 import poet

    x, r = _make(torch, 3, 30011, torch.bfloat16)
    tk = torch.from_numpy(r.integers(0, 30011, 3).astype(np.int32)).cuda()
    tokens, values = _teacher_case(r, 3, 30011, 12, True)
    tt, tv = torch.from_numpy(tokens).cuda(), torch.from_numpy(values).cuda()
    one = torch.ones(3, device="cuda")

    def calls(stream=None):
        a = poet.token_logprobs(x, tk, topk=6, stream=stream)
        b = poet.token_logprobs_grad(x, tk, a[4], one, one, stream=stream)
        c = poet.distill_topk(x, tt, tv, tail=True, grad=True, stream=stream)
        return list(a) + [b] + list(c) + [poet.distill_topk_grad(x, tt, tv, c[2], tail=True, stream=stream)]

    want = calls()
    torch.cuda.synchronize()
    for a, b in zip(want, calls()):
        assert torch.equal(a, b)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = calls()
    s.synchronize()
    for a, b in zip(want, other):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = calls()
    for t in held:
        t.zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, held):
        assert torch.equal(a, b)


def test_large_offsets(torch):
    """Rows beyond 2^31 elements from the first one."""
    from orthogonal_reparameterized_poet_b200 import poet

    ld = (1 << 30) + 8
    buf = torch.empty(3 * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.view(3, ld)[:, :4100]
    r = np.random.default_rng(2)
    x.copy_(torch.from_numpy(r.standard_normal((3, 4100))).to(torch.bfloat16))
    tokens = r.integers(0, 4100, 3)
    tk, saved = _check_logprobs(torch, x, tokens, 5)
    _check_logprobs_grad(torch, x, tokens, tk, saved, r, out=x.as_strided(x.shape, x.stride()).clone())
    tt, tv = _teacher_case(r, 3, 4100, 6, True)
    _check_distill(torch, x, tt, tv, r, True)


def test_largest_vocabulary(torch):
    from orthogonal_reparameterized_poet_b200 import poet

    V = 2097152
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randn(2, V, device="cuda").to(dtype)
        tk = torch.tensor([V - 1, 0], dtype=torch.int32, device="cuda")
        logp, H, top, topl, saved = poet.token_logprobs(x, tk, topk=128)
        lp = torch.log_softmax(x.double(), 1)
        assert torch.allclose(logp.double(), lp.gather(1, tk.long()[:, None])[:, 0], rtol=0, atol=_steps(V) * U)
        order = x.sort(dim=1, descending=True, stable=True)[1][:, :128]
        assert torch.equal(top.long(), order)
        loss, d, _ = poet.distill_topk(x, top, topl, tail=True, grad=True)  # the student is the teacher
        poet.poet_sync_status()
        assert loss.abs().max() < 1e-3 and d.abs().max() < 1e-4


def test_tensors_are_checked(torch):
    from orthogonal_reparameterized_poet_b200 import poet

    x = torch.zeros(4, 100, device="cuda")
    tk = torch.zeros(4, dtype=torch.int32, device="cuda")
    sv = torch.zeros(4, 4, device="cuda")
    one = torch.ones(4, device="cuda")
    val = torch.zeros(4, 2, device="cuda")
    tt = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for call in (lambda: poet.token_logprobs(x, tk.long()), lambda: poet.token_logprobs(x, tk[:3]),
                 lambda: poet.token_logprobs(x.half(), tk), lambda: poet.token_logprobs(x.t(), tk),
                 lambda: poet.token_logprobs(x[0], tk), lambda: poet.token_logprobs(x, tk.cpu()),
                 lambda: poet.token_logprobs(x, tk, saved=sv[:, :3]),
                 lambda: poet.token_logprobs_grad(x, tk, sv, one.double()),
                 lambda: poet.token_logprobs_grad(x, tk, sv, one, dlogits=x.bfloat16()),
                 lambda: poet.distill_topk(x, tt.long(), val), lambda: poet.distill_topk(x, tt, val.double()),
                 lambda: poet.distill_topk(x, tt, val[:, :1]), lambda: poet.distill_topk(x, tt[:, ::2], val),
                 lambda: poet.distill_topk(x, tt[:3], val), lambda: poet.distill_topk(x, tt, val, dloss=one[:2]),
                 lambda: poet.distill_topk_grad(x, tt, val, sv.double())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: poet.token_logprobs(x, tk, topk=129), lambda: poet.token_logprobs(x, tk, scale=0.0),
                 lambda: poet.token_logprobs_grad(x, tk, sv), lambda: poet.token_logprobs(x[:1].expand(4, 100), tk),
                 lambda: poet.distill_topk(x, tt, val, value_scale=-1.0)):
        with pytest.raises(poet.PoetError):
            call()
