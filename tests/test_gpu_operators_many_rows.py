"""The operators around the blocks with more rows than the GPU works on at
once: rows of every alignment one after the other, in place, all of them left
out, two calls at a time, against plain float64 arithmetic on the GPU.

Tolerances, derived before the first run (u = 2^-24): as in the tests of each
operator, N = V / 256 * 2 + 128 half steps of a row's sums, plus a few of each
operation, and half a step of the outputs' type."""
import pytest

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


def _steps(V):
    return V / 256 * 2 + 128


def _logits(torch, T, V, dtype, ld=None, offset=0, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + T + V)
    ld = V if ld is None else ld
    buf = torch.full((offset + T * ld + 16,), float("nan"), dtype=dtype, device="cuda")
    x = buf[offset:offset + T * ld].view(T, ld)[:, :V]
    x.copy_(torch.randn(T, V, generator=g, device="cuda") * 2)
    return x, g


def _teacher(torch, T, V, K, g, tail):
    part = V // K
    tokens = torch.arange(K, device="cuda") * part + torch.randint(0, part, (T, K), generator=g, device="cuda")
    tokens = tokens.gather(1, torch.rand(T, K, generator=g, device="cuda").argsort(1)).to(torch.int32)
    tokens[::9, 0] = -1
    tokens[4::11] = -1
    values = torch.randn(T, K, generator=g, device="cuda") * 1.5
    if tail:
        values = torch.log_softmax(values.double(), 1).float() - 0.3
    return tokens.contiguous(), values.contiguous()


def _distill(torch, x, tokens, values, tail, weight):
    """(loss, dlogits, bounds) in float64."""
    X = x.double()
    T, V = X.shape
    lp = torch.log_softmax(X, 1)
    p = lp.exp()
    live = tokens >= 0
    at = tokens.long().clamp(min=0)
    v = torch.where(live, values.double(), -INF)
    q = v.exp() if tail else torch.nan_to_num(torch.softmax(v, 1), nan=0.0)
    lq = v if tail else torch.log_softmax(v, 1)
    term = torch.where(live, q * (lq - lp.gather(1, at)), 0.0)
    loss = term.sum(1)
    dense = torch.zeros_like(p).scatter_add_(1, at, torch.where(live, q, 0.0))
    d = p - dense
    if tail:
        inside = torch.zeros_like(p).scatter_add_(1, at, live.double()) > 0
        pr = torch.where(inside, 0.0, p).sum(1, keepdim=True)
        rest = 1 - torch.where(live, q, 0.0).sum(1, keepdim=True)
        loss = loss + (rest * (rest / pr).log())[:, 0]
        d = torch.where(inside, d, p * (1 - rest / pr))
    row = live.any(1)
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    loss, d = torch.where(row, loss, zero), torch.where(row[:, None], d, zero)
    mag = (p + dense + (p / pr if tail else 0)) * weight.double()[:, None].abs()
    return loss, d * weight.double()[:, None], mag


def _check_distill(torch, got, d, want, dwant, mag, V, K, dtype):
    bound = (2 * _steps(V) + 8 * K + 256) * U
    assert ((got.double() - want).abs() <= bound * (4 + want.abs())).all()
    half = torch.finfo(dtype).eps / 2
    assert ((d.double() - dwant).abs() <= 1.01 * half * dwant.abs() + 2 * bound * mag + 1e-36).all()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,V,ld,offset", [(2000, 4099, 4103, 3), (1200, 9001, 9005, 1), (1200, 33001, 33001, 5),
                                           (500, 66003, 66007, 1)])
@pytest.mark.parametrize("tail", [False, True])
def test_rows_of_every_alignment(torch, T, V, ld, offset, tail, dtype):
    from orthogonal_reparameterized_poet_b200 import poet

    t = getattr(torch, dtype)
    x, g = _logits(torch, T, V, t, ld, offset)
    K = 17
    tokens, values = _teacher(torch, T, V, K, g, tail)
    weight = torch.randn(T, generator=g, device="cuda")
    want, dwant, mag = _distill(torch, x, tokens, values, tail, weight)
    out, _ = _logits(torch, T, V, t, ld + 2, 2)
    loss, d, saved = poet.distill_topk(x, tokens, values, tail=tail, dloss=weight, dlogits=out)
    poet.poet_sync_status()
    _check_distill(torch, loss, d, want, dwant, mag, V, K, t)
    again = poet.distill_topk_grad(x, tokens, values, saved, weight, tail=tail)
    _check_distill(torch, loss, again, want, dwant, mag, V, K, t)
    # the gradient over the logits
    before = x.clone()
    loss2, same, _ = poet.distill_topk(x, tokens, values, tail=tail, dloss=weight, dlogits=x)
    poet.poet_sync_status()
    assert same is x and torch.equal(loss, loss2) and torch.equal(x, d)
    tk = torch.where(tokens[:, 1] < 0, -1, tokens[:, 1]).contiguous()
    x.copy_(before)
    logp, H, top, topl, saved = poet.token_logprobs(x, tk, topk=9)
    lp = torch.log_softmax(before.double(), 1)
    row = tk >= 0
    at = lp.gather(1, tk.long().clamp(min=0)[:, None])[:, 0]
    bound = (_steps(V) + 64) * U
    assert ((logp.double() - torch.where(row, at, 0.0)).abs() <= bound * (1 + at.abs())).all()
    ent = -(lp.exp() * lp).sum(1)
    assert ((H.double() - torch.where(row, ent, 0.0)).abs() <= 4 * bound * (1 + ent)).all()
    order = before.sort(dim=1, descending=True, stable=True)[1][:, :9].to(torch.int32)
    assert torch.equal(top, torch.where(row[:, None], order, -1))


@pytest.mark.parametrize("T,V", [(3000, 500), (1500, 20000), (400, 70000)])
def test_every_row_left_out(torch, T, V):
    from orthogonal_reparameterized_poet_b200 import poet

    x = torch.full((T, V), float("nan"), dtype=torch.bfloat16, device="cuda")
    none = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    logp, H, top, topl, saved = poet.token_logprobs(x, none, topk=3)
    assert (logp == 0).all() and (H == 0).all() and (top == -1).all() and (topl == -INF).all()
    one = torch.ones(T, device="cuda")
    assert (poet.token_logprobs_grad(x, none, saved, one, one) == 0).all()
    for tail in (False, True):
        loss, d, _ = poet.distill_topk(x, none[:, None].contiguous(), torch.zeros(T, 1, device="cuda"), tail=tail,
                                       grad=True)
        assert (loss == 0).all() and (d == 0).all()
    poet.poet_sync_status()


def test_very_many_short_rows(torch):
    from orthogonal_reparameterized_poet_b200 import poet

    T, V = 300001, 9
    x, g = _logits(torch, T, V, torch.float32)
    tk = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    logp, H, top, topl, _ = poet.token_logprobs(x, tk, topk=4)
    lp = torch.log_softmax(x.double(), 1)
    assert ((logp.double() - lp.gather(1, tk.long()[:, None])[:, 0]).abs() <= 200 * U * (1 + lp.abs().amax(1))).all()
    assert torch.equal(top.long(), x.sort(dim=1, descending=True, stable=True)[1][:, :4])
    poet.poet_sync_status()


def test_calls_side_by_side(torch):
    """Calls on two streams at once, each with results of its own."""
    from orthogonal_reparameterized_poet_b200 import poet

    x, g = _logits(torch, 1500, 32000, torch.bfloat16)
    tokens, values = _teacher(torch, 1500, 32000, 64, g, True)
    tk = tokens[:, 1].clamp(min=0).contiguous()
    o, h = (torch.randn(5000, 1024, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.rand(1024, generator=g, device="cuda")

    def logits(stream=None):
        a = poet.token_logprobs(x, tk, topk=12, stream=stream)
        return list(a) + list(poet.distill_topk(x, tokens, values, tail=True, grad=True, stream=stream))

    def joint(stream=None):
        return list(poet.joint_forward(o, h, w_post=w, w_pre=w, stream=stream)) + \
            [t for t in poet.joint_backward(o, h, None, o, h, w_post=w, w_pre=w, stream=stream) if t is not None]

    want = logits(), joint(), logits()
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        got = logits(s[0]), joint(s[1]), logits(s[2])
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    poet.poet_sync_status()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,d", [(3000, 512), (2000, 2560), (1000, 4608), (700, 8192), (400, 16384), (900, 5001)])
@pytest.mark.parametrize("gate", ["none", "each", "shared", "row"])
def test_joint_of_many_rows(torch, T, d, gate, dtype):
    from orthogonal_reparameterized_poet_b200 import poet

    t = getattr(torch, dtype)
    g = torch.Generator(device="cuda")
    g.manual_seed(T + d)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
    o, h, dh, dn = r(T, d), r(T, d), r(T, d), r(T, d)
    w = [1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]
    rows = {"none": 1, "each": 1, "shared": 130, "row": 1}[gate]
    G = -(-T // rows)
    ga = None if gate == "none" else r(G) if gate == "row" else r(G, d)
    kw = dict(w_post=w[0], w_pre=w[1], gate_act=poet.GATE_SIGMOID, gate_rows=rows, alpha=0.8, beta=0.5)
    h1, n = poet.joint_forward(o, h, ga, **kw)
    got = poet.joint_backward(o, h1, ga, dh, dn, **kw)
    leaf = [v.double().requires_grad_() for v in (o, h1) + ((ga,) if ga is not None else ()) + tuple(w)]
    O, A, wq, wn = leaf[0], leaf[1], leaf[-2], leaf[-1]
    norm = lambda v, k: v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * k  # noqa: E731

    def branch():
        b = norm(O, wq)
        if ga is None:
            return b
        v = torch.sigmoid(leaf[2]).reshape(G, -1)
        return b * v.repeat_interleave(rows, 0)[:T]

    after = 0.8 * h.double() + 0.5 * branch()
    eps = torch.finfo(t).eps / 2
    close = lambda a, b, k: ((a.double() - b).norm() <= k * b.norm())  # noqa: E731
    assert close(h1, after.detach(), 1.1 * eps + 64 * U) and close(n, norm(after, wn).detach(), 1.1 * eps + 64 * U)
    through, dwn = torch.autograd.grad(norm(A, wn), (A, wn), dn.double())
    total = dh.double() + through
    rest = torch.autograd.grad(branch(), [leaf[0]] + ([leaf[2]] if ga is not None else []) + [wq], 0.5 * total)
    # sums over T rows cancel: bounded against sqrt(T) terms of their size, which the norm of a sum of random terms is
    for a, b, k in ((got[0], 0.8 * total, 1.1 * eps + 64 * U), (got[1], rest[0], 1.1 * eps + 64 * U),
                    (got[4], dwn, (64 + T) * U), (got[3], rest[-1], (64 + T) * U)):
        assert close(a, b, k)
    if ga is not None:
        assert close(got[2], rest[1], 1.1 * eps + (64 + rows + d) * U)
