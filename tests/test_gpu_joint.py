"""The joint between two blocks (poet_joint_forward / _backward) against the
float64 oracle (oracle/joint.py) on the same inputs.

Tolerances, element by element, derived before the first run:
  * an output of type t is rounded once: half a step, finfo(t).eps / 2 of its value;
  * the float computation before it is off by a number of half steps of float,
    2^-24, of the sum of the magnitudes of the terms that the element is made of
    (the oracle gives that sum).  A row's sums add at most 16 elements in
    sequence in a thread and 10 levels across threads, the element itself
    passes about 20 operations and a division, a root or an exponential of a
    few half steps: 64 covers them.  A column's sum adds at most the T rows of
    the test, fewer than 1100: 64 + T bounds it.
"""
import numpy as np
import pytest

from oracle import joint as J

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from orthogonal_reparameterized_poet_b200 import poet

    poet.lib()
    return torch


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _close(torch, got, want, mag, steps, name):
    half = torch.finfo(got.dtype).eps / 2
    g = _np(got)
    assert g.shape == want.shape, name
    bound = half * np.abs(want) * (1 + 2.0 ** -7) + steps * U * mag + 1e-38
    bad = ~(np.abs(g - want) <= bound)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off; worst {np.max(np.abs(g - want) / bound):.2f} bounds"


def _rows(torch, r, T, d, dtype, ld=None, offset=0, scale=1.0):
    """T x d normal values with row stride ld, starting `offset` elements into an allocation."""
    ld = d if ld is None else ld
    buf = torch.full((offset + max(T, 1) * ld + 16,), float("nan"), dtype=dtype, device="cuda")
    v = buf[offset:offset + T * ld].view(T, ld)[:, :d]
    v.copy_(torch.from_numpy((r.standard_normal((T, d)) * scale)).to(dtype))
    return v


def _case(torch, T, d, dtype, gate="none", sigmoid=False, rows=1, post=True, gains=True, alpha=0.9, beta=0.7, ld=None,
          offset=0, seed=0):
    r = np.random.default_rng(seed + 7 * T + d)
    c = dict(T=T, d=d)
    for k, s in (("o", 0.8), ("h", 1.5), ("dh_out", 1.0), ("dn", 1.0)):
        c[k] = _rows(torch, r, T, d, dtype, ld, offset, s)
    G = -(-T // rows)
    c["gate"] = None
    if gate == "channel":
        c["gate"] = _rows(torch, r, G, d, dtype, ld, offset, 0.7)
    elif gate == "row":
        c["gate"] = _rows(torch, r, G, 1, dtype).reshape(G).contiguous()
    wq = torch.from_numpy(1 + 0.2 * r.standard_normal(d)).float().cuda() if gains and post else None
    wn = torch.from_numpy(1 + 0.2 * r.standard_normal(d)).float().cuda() if gains else None
    c["kw"] = dict(w_post=wq, w_pre=wn, post_norm=post, gate_act=1 if sigmoid else 0, gate_rows=rows, alpha=alpha,
                   beta=beta)
    c["ref"] = dict(w_post=_np(wq), w_pre=_np(wn), post_norm=post, sigmoid=sigmoid, rows=rows,
                    alpha=float(np.float32(alpha)), beta=float(np.float32(beta)), eps=float(np.float32(1e-6)))
    return c


def _check_forward(torch, c, **more):
    from orthogonal_reparameterized_poet_b200 import poet

    want_h, want_n, mh, mn = J.forward(_np(c["o"]), _np(c["h"]), _np(c["gate"]), **c["ref"])
    h, n = poet.joint_forward(c["o"], c["h"], c["gate"], **c["kw"], **more)
    poet.poet_sync_status()
    _close(torch, h, want_h, mh, 64, "h'")
    _close(torch, n, want_n, mn, 64, "n")
    return h, n


def _check_backward(torch, c, after, dh_out=True, dn=True, **more):
    from orthogonal_reparameterized_poet_b200 import poet

    kw = dict(c["kw"])
    if not dn:
        kw["w_pre"] = None
    a, b = (c["dh_out"] if dh_out else None), (c["dn"] if dn else None)
    want = J.backward(_np(c["o"]), _np(after), _np(c["gate"]), _np(a), _np(b), **{**c["ref"], "w_pre": _np(kw["w_pre"])})
    got = poet.joint_backward(c["o"], after, c["gate"], a, b, **kw, **more)
    poet.poet_sync_status()
    for name, t in zip(("dh", "do", "dgate", "dw_post", "dw_pre"), got):
        if name in want and t is not None:
            steps = 64 + (c["T"] if name.startswith("dw") or name == "dgate" else 0)
            if name == "dgate" and c["gate"].dim() == 1:
                steps += 64
            _close(torch, t, want[name][0], want[name][1], steps, name)
    if c["gate"] is None:
        assert got[2] is None
    return got


SHAPES = [(1, 1), (1, 2048), (2, 7), (3, 8), (5, 33), (67, 64), (40, 96), (33, 512), (1031, 136), (9, 1376), (7, 1377),
          (19, 2048), (5, 2560), (3, 5461), (4, 8200), (2, 16384), (3, 16383)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_shapes(torch, T, d, dtype):
    c = _case(torch, T, d, getattr(torch, dtype))
    h, _ = _check_forward(torch, c)
    _check_backward(torch, c, h)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,d", [(1, 64), (37, 64), (1000, 64), (130, 100), (50, 1032)])
@pytest.mark.parametrize("gate,sigmoid", [("channel", False), ("channel", True), ("row", False), ("row", True)])
@pytest.mark.parametrize("rows", [1, 2, 9, 100, 1 << 40])
def test_gates(torch, T, d, dtype, gate, sigmoid, rows):
    c = _case(torch, T, d, getattr(torch, dtype), gate, sigmoid, rows, post=rows != 2)
    h, _ = _check_forward(torch, c)
    _check_backward(torch, c, h)


@pytest.mark.parametrize("rows", [3, 5000])
def test_many_short_and_few_long_gate_segments(torch, rows):
    # more segments than row groups, and segments that many groups share
    c = _case(torch, 20000, 32, torch.bfloat16, "channel", False, rows)
    h, _ = _check_forward(torch, c)
    _check_backward(torch, c, h)
    c = _case(torch, 20000, 32, torch.float32, "row", True, rows)
    h, _ = _check_forward(torch, c)
    _check_backward(torch, c, h)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("ld,offset", [(80, 0), (65, 0), (64, 1), (72, 3), (200, 8)])
def test_strides_and_addresses(torch, dtype, ld, offset):
    c = _case(torch, 21, 64, getattr(torch, dtype), "channel", True, 4, ld=ld, offset=offset)
    out = _rows(torch, np.random.default_rng(1), 21, 64, getattr(torch, dtype), ld, offset)
    whole = out.as_strided((21, ld), (ld, 1))
    before = whole[:-1, 64:].clone()
    h, _ = _check_forward(torch, c, h_out=out)
    assert h.data_ptr() == out.data_ptr()
    # what lies between the rows is left as it was
    assert torch.equal(whole[:-1, 64:].view(torch.int16 if dtype == "bfloat16" else torch.int32),
                       before.view(torch.int16 if dtype == "bfloat16" else torch.int32))
    _check_backward(torch, c, h, dh=out.clone(memory_format=torch.preserve_format))


@pytest.mark.parametrize("post,gains", [(False, False), (False, True), (True, False)])
def test_without_post_norm_or_gains(torch, post, gains):
    c = _case(torch, 23, 256, torch.float32, post=post, gains=gains)
    h, _ = _check_forward(torch, c)
    _check_backward(torch, c, h)


@pytest.mark.parametrize("dh_out,dn", [(True, False), (False, True)])
def test_one_incoming_gradient(torch, dh_out, dn):
    c = _case(torch, 23, 256, torch.bfloat16, "channel", True, 23)
    h, _ = _check_forward(torch, c)
    _check_backward(torch, c, h, dh_out, dn)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,d", [(1, 1), (300, 96), (5, 5461)])
def test_norm_before_the_first_block(torch, T, d, dtype):
    from orthogonal_reparameterized_poet_b200 import poet

    c = _case(torch, T, d, getattr(torch, dtype))
    w = c["kw"]["w_pre"]
    eps = float(np.float32(1e-6))
    _, want, _, mag = J.forward(None, _np(c["h"]), w_pre=_np(w), eps=eps)
    none, n = poet.joint_forward(None, c["h"], w_pre=w)
    assert none is None
    _close(torch, n, want, mag, 64, "n")
    want = J.backward(None, _np(c["h"]), None, _np(c["dh_out"]), _np(c["dn"]), w_pre=_np(w), eps=eps)
    dh, d_o, dg, dq, dw = poet.joint_backward(None, c["h"], None, c["dh_out"], c["dn"], w_pre=w)
    assert d_o is None and dg is None and dq is None
    _close(torch, dh, *want["dh"], 64, "dh")
    _close(torch, dw, *want["dw_pre"], 64 + T, "dw_pre")
    poet.poet_sync_status()


def test_residual_alone(torch):
    from orthogonal_reparameterized_poet_b200 import poet

    c = _case(torch, 11, 128, torch.float32)
    kw = {**c["kw"], "w_pre": None}
    want, _, mag, _ = J.forward(_np(c["o"]), _np(c["h"]), None, **{**c["ref"], "w_pre": None})
    h, n = poet.joint_forward(c["o"], c["h"], **kw, pre_norm=False)
    assert n is None
    _close(torch, h, want, mag, 64, "h'")


def test_in_place(torch):
    from orthogonal_reparameterized_poet_b200 import poet

    c = _case(torch, 600, 96, torch.bfloat16, "channel", False, 600)
    h, n = poet.joint_forward(c["o"], c["h"], c["gate"], **c["kw"])
    want = poet.joint_backward(c["o"], h, c["gate"], c["dh_out"], c["dn"], **c["kw"])
    o2, h2, d2 = c["o"].clone(), c["h"].clone(), c["dh_out"].clone()
    poet.joint_forward(o2, h2, c["gate"], **c["kw"], h_out=h2, n=o2)
    assert torch.equal(h2, h) and torch.equal(o2, n)
    o3 = c["o"].clone()
    got = poet.joint_backward(o3, h, c["gate"], d2, c["dn"], **c["kw"], dh=d2, d_o=o3)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert got[0].data_ptr() == d2.data_ptr() and got[1].data_ptr() == o3.data_ptr()


def test_zero_rows_and_zero_tokens(torch):
    from orthogonal_reparameterized_poet_b200 import poet

    c = _case(torch, 4, 64, torch.float32)
    c["o"][1] = 0.0
    c["h"][1] = 0.0  # a row of zeros: eps keeps its norm finite
    h, n = _check_forward(torch, c)
    assert torch.all(n[1] == 0)
    _check_backward(torch, c, h)
    e = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    h, n = poet.joint_forward(e, e, w_post=w, w_pre=w)
    assert h.shape == n.shape == (0, 64)
    got = poet.joint_backward(e, e, None, e, e, w_post=w, w_pre=w, dw_post=w.clone(), dw_pre=w.clone())
    assert torch.all(got[3] == 0) and torch.all(got[4] == 0)


def test_a_row_of_nan_or_infinity_stays_alone(torch):
    from orthogonal_reparameterized_poet_b200 import poet

    c = _case(torch, 30, 136, torch.bfloat16, "channel", False, 1)
    h0, n0 = poet.joint_forward(c["o"], c["h"], c["gate"], **c["kw"])
    c["o"][4] = float("nan")
    c["h"][9] = float("inf")
    h, n = poet.joint_forward(c["o"], c["h"], c["gate"], **c["kw"])
    keep = [i for i in range(30) if i not in (4, 9)]
    assert torch.equal(h[keep], h0[keep]) and torch.equal(n[keep], n0[keep])
    assert torch.isnan(h[4]).all() and torch.isnan(n[4]).all()


def test_same_bits_streams_and_graph(torch):
    from orthogonal_reparameterized_poet_b200 import poet

    c = _case(torch, 700, 264, torch.bfloat16, "channel", True, 90)
    h, n = poet.joint_forward(c["o"], c["h"], c["gate"], **c["kw"])
    want = poet.joint_backward(c["o"], h, c["gate"], c["dh_out"], c["dn"], **c["kw"])
    again = poet.joint_backward(c["o"], h, c["gate"], c["dh_out"], c["dn"], **c["kw"])
    for a, b in zip(want, again):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    h2, n2 = torch.empty_like(h), torch.empty_like(n)
    out = [torch.empty_like(t) for t in want]
    nbytes = poet.joint_workspace_bytes(700, 264, poet.BF16, poet.GATE_CHANNEL, 90)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    def calls(stream=None):
        poet.joint_forward(c["o"], c["h"], c["gate"], **c["kw"], h_out=h2, n=n2, stream=stream)
        poet.joint_backward(c["o"], h2, c["gate"], c["dh_out"], c["dn"], **c["kw"], dh=out[0], d_o=out[1], dgate=out[2],
                            dw_post=out[3], dw_pre=out[4], ws=ws, stream=stream)

    calls(s)
    s.synchronize()
    for a, b in zip([h, n] + list(want), [h2, n2] + out):
        assert torch.equal(a, b)
        b.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for _ in range(2):
        c["o"].mul_(1.0)
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip([h, n] + list(want), [h2, n2] + out):
        assert torch.equal(a, b)


def test_tensors_are_checked(torch):
    from orthogonal_reparameterized_poet_b200 import poet

    x = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    for kw in (dict(o=x[:3]), dict(o=x.bfloat16()), dict(h=x.t()), dict(w_post=w.bfloat16()), dict(w_pre=w[:63]),
               dict(gate=x[:3]), dict(gate=x, gate_rows=2), dict(gate=x[:, :32]), dict(gate=x, gate_rows=0),
               dict(h_out=x[:, :32]), dict(n=x.bfloat16()), dict(pre_norm=False, w_pre=w), dict(h=x.half(), o=x.half())):
        a = {"o": x, "h": x, **kw}
        with pytest.raises(ValueError):
            poet.joint_forward(a.pop("o"), a.pop("h"), a.pop("gate", None), **a)
    with pytest.raises(poet.PoetError):  # every token the same row: a stride of 0
        poet.joint_forward(x, x[:1].expand(4, 64))
    with pytest.raises(poet.PoetError):
        poet.joint_backward(x, x, None, x, x, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        poet.joint_backward(x, x, None, x, x, dgate=x)
