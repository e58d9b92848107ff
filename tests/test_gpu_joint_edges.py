"""The joint at the edges of what it accepts, against the float64 oracle
(oracle/joint.py), with the bounds of tests/test_gpu_joint.py."""
import ctypes

import pytest

from oracle import joint as J
from tests.test_gpu_joint import _case, _close, _np, torch  # noqa: F401

pytestmark = pytest.mark.gpu


# Beside the operators' 64 half steps, those of the sigmoid: of its exponent of at most 20 log2(e) = 28.9, 12 for its
# rounding, 10 for the constant's and 4 for the exponential; of the sum, the reciprocal and the products 9 more.
SIGMOID = 40


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,d", [(41, 64), (300, 136), (5, 2560), (3, 4600), (7, 1377), (2, 16384)])
@pytest.mark.parametrize("gate,rows", [("channel", 1), ("channel", 3), ("channel", 1 << 40), ("row", 1), ("row", 4)])
def test_gates_wide_open_and_closed(torch, T, d, gate, rows, dtype):  # noqa: F811
    from orthogonal_reparameterized_poet_b200 import poet

    c = _case(torch, T, d, getattr(torch, dtype), gate, True, rows)
    g = c["gate"]
    g.copy_(torch.linspace(-20, 20, g.numel(), device="cuda").reshape(g.shape))
    want_h, want_n, mh, mn = J.forward(_np(c["o"]), _np(c["h"]), _np(g), **c["ref"])
    h, n = poet.joint_forward(c["o"], c["h"], g, **c["kw"])
    _close(torch, h, want_h, mh, 64 + SIGMOID, "h'")
    _close(torch, n, want_n, mn, 64 + SIGMOID, "n")
    want = J.backward(_np(c["o"]), _np(h), _np(g), _np(c["dh_out"]), _np(c["dn"]), **c["ref"])
    got = poet.joint_backward(c["o"], h, g, c["dh_out"], c["dn"], **c["kw"])
    poet.poet_sync_status()
    for name, t in zip(("dh", "do", "dgate", "dw_post", "dw_pre"), got):
        steps = 64 + SIGMOID + (T if name.startswith("dw") or name == "dgate" else 0)
        if name == "dgate" and g.dim() == 1:
            steps += 64
        _close(torch, t, want[name][0], want[name][1], steps, name)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_gates_beyond_the_exponential(torch, dtype):  # noqa: F811
    """Gates whose exponentials leave a float's range: open is 1 and closed is 0, both with slope 0; a NaN stays."""
    from orthogonal_reparameterized_poet_b200 import poet

    c = _case(torch, 6, 64, getattr(torch, dtype), "channel", True, 1, alpha=0.0)
    g = c["gate"]
    for i, v in enumerate((float("-inf"), -3e38, -150.0, 150.0, 3e38, float("inf"))):
        g[i] = v
    h, n = poet.joint_forward(c["o"], c["h"], g, **c["kw"])
    assert torch.equal(h[:3], torch.zeros_like(h[:3])) and (h[3:] != 0).all() and torch.isfinite(h).all()
    got = poet.joint_backward(c["o"], c["h"], g, c["dh_out"], c["dn"], **c["kw"])
    # the slopes beyond 88 are below 2^-126 and the other factors below 2^20
    assert (got[2].abs() <= 2.0 ** -100).all() and all(torch.isfinite(t).all() for t in got)
    g[2, 5] = float("nan")
    got = poet.joint_backward(c["o"], c["h"], g, c["dh_out"], c["dn"], **c["kw"])
    assert torch.isnan(got[2][2, 5]) and torch.isfinite(got[2][:2]).all()


@pytest.mark.parametrize("gate", ["channel", "row"])
def test_one_gate_for_any_number_of_tokens(torch, gate):  # noqa: F811
    """gate_rows up to the largest integer: the same bits as with the number of tokens, and the same bytes recorded."""
    from orthogonal_reparameterized_poet_b200 import poet

    got = []
    for rows in (37, 2**63 - 1):
        c = _case(torch, 37, 128, torch.float32, gate, True, 37)
        c["kw"]["gate_rows"] = rows
        poet.poet_trace_enable(True)
        try:
            h, n = poet.joint_forward(c["o"], c["h"], c["gate"], **c["kw"])
            out = [h, n, *poet.joint_backward(c["o"], h, c["gate"], c["dh_out"], c["dn"], **c["kw"])]
            rec = {k: (v["launches"], v["bytes"]) for k, v in poet.poet_trace_read().items()}
        finally:
            poet.poet_trace_enable(False)
        got.append((out, rec))
    assert all(torch.equal(a, b) for a, b in zip(got[0][0], got[1][0]))
    assert got[0][1] == got[1][1] and got[0][1]["joint"][0] == 1


def test_large_offsets(torch):  # noqa: F811
    """Rows beyond 2^31 elements from the first one."""
    from orthogonal_reparameterized_poet_b200 import poet

    d, far = 264, (1 << 30) + 8
    near = _case(torch, 3, d, torch.bfloat16, "channel", True, 1)
    buf = torch.empty(4, 3, far, dtype=torch.bfloat16, device="cuda")  # 26 GB
    o, h, dh, n = (b[:, :d] for b in buf)
    for v, name in ((o, "o"), (h, "h"), (dh, "dh_out"), (n, "dn")):
        v.copy_(near[name])
    h0, n0 = poet.joint_forward(near["o"], near["h"], near["gate"], **near["kw"])
    want = poet.joint_backward(near["o"], h0, near["gate"], near["dh_out"], near["dn"], **near["kw"])
    h1, n1 = poet.joint_forward(o, h, near["gate"], **near["kw"], h_out=h)
    assert h1 is h and torch.equal(h, h0) and torch.equal(n1, n0)
    got = poet.joint_backward(o, h, near["gate"], dh, n, **near["kw"], dh=dh, d_o=o)
    poet.poet_sync_status()
    assert got[0] is dh and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows", [1, 4, 50])
def test_row_gates_of_any_stride(torch, rows):  # noqa: F811
    """Through the C ABI: the gate's values a column of a matrix, its gradient a column of another."""
    from orthogonal_reparameterized_poet_b200 import poet

    T, d = 50, 96
    c = _case(torch, T, d, torch.float32, "row", True, rows)
    G = c["gate"].numel()
    h0, n0 = poet.joint_forward(c["o"], c["h"], c["gate"], **c["kw"])
    want = poet.joint_backward(c["o"], h0, c["gate"], c["dh_out"], c["dn"], **c["kw"])
    wide, dwide = torch.full((G, 3), 7.0, device="cuda"), torch.full((G, 5), 7.0, device="cuda")
    wide[:, 1] = c["gate"]
    J_ = poet.poet_joint(d, poet.F32, 1, poet.GATE_ROW, poet.GATE_SIGMOID, 0, rows, c["kw"]["alpha"], c["kw"]["beta"], 1e-6,
                         c["kw"]["w_post"].data_ptr(), c["kw"]["w_pre"].data_ptr())
    h, n, dh, d_o = (torch.empty_like(h0) for _ in range(4))
    dwq, dwn = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(poet.joint_workspace_bytes(T, d, poet.F32, poet.GATE_ROW, rows), dtype=torch.uint8, device="cuda")
    at = lambda t: t.data_ptr()  # noqa: E731
    st = torch.cuda.current_stream().cuda_stream
    L, ref = poet.lib(), ctypes.byref(J_)
    assert L.poet_joint_forward(ref, at(c["o"]), d, at(c["h"]), d, at(wide) + 4, 3, T, at(h), d, at(n), d, st) == poet.OK
    assert L.poet_joint_backward(ref, at(c["o"]), d, at(h), d, at(wide) + 4, 3, at(c["dh_out"]), d, at(c["dn"]), d, T,
                                 at(dh), d, at(d_o), d, at(dwide) + 8, 5, at(dwq), at(dwn), at(ws), ws.nbytes, st) == poet.OK
    poet.poet_sync_status()
    assert torch.equal(h, h0) and torch.equal(n, n0)
    for a, b in zip((dh, d_o, dwide[:, 2], dwq, dwn), want):
        assert torch.equal(a, b)
    dwide[:, 2] = 7.0
    assert (dwide == 7.0).all()  # what lies between its values is left as it was
