"""Host-side validation of the joint and of the operators on logits: a bad
argument is refused before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from orthogonal_reparameterized_poet_b200 import poet

ST = ctypes.c_void_p(0)
P = 1 << 20  # a 256-byte aligned address that is never dereferenced: validation fails first


def _joint(**kw):
    J = poet.poet_joint(64, poet.BF16, 1, poet.GATE_CHANNEL, poet.GATE_LINEAR, 0, 1, 1.0, 1.0, 1e-6, None, None)
    for k, v in kw.items():
        setattr(J, k, v)
    return J


def _fwd(J, o=P, ldo=64, h=P, ldh=64, gate=P, ldg=64, T=4, ho=P, ldho=64, n=P, ldn=64):
    return poet.lib().poet_joint_forward(ctypes.byref(J) if J is not None else None, o, ldo, h, ldh, gate, ldg, T, ho,
                                         ldho, n, ldn, ST)


def _bwd(J, o=P, hp=P, gate=P, dho=P, dn=P, T=4, dh=P, d_o=P, dg=P, wq=P, wn=P, ws=P, ws_bytes=1 << 30, ld=64):
    return poet.lib().poet_joint_backward(ctypes.byref(J), o, ld, hp, ld, gate, ld, dho, ld, dn, ld, T, dh, ld, d_o, ld,
                                          dg, ld, wq, wn, ws, ws_bytes, ST)


@pytest.mark.parametrize("kw", [dict(d=0), dict(d=16385), dict(dtype=2), dict(post_norm=2), dict(gate=3), dict(gate=-1),
                                dict(gate_act=2), dict(gate_rows=0), dict(alpha=float("nan")), dict(beta=float("inf")),
                                dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(w_post=P + 2),
                                dict(post_norm=0, w_post=P)])
def test_joint_struct_is_checked(kw):
    J = _joint(**kw)
    assert _fwd(J) == poet.EINVAL
    assert _bwd(J) == poet.EINVAL
    assert poet.lib().poet_joint_workspace_bytes(ctypes.byref(J), 4) == 0


@pytest.mark.parametrize("kw", [dict(h=None), dict(h=P + 1), dict(ldh=63), dict(ldo=63), dict(ho=None), dict(ldho=8),
                                dict(gate=None), dict(ldg=63), dict(T=-1), dict(n=P + 1), dict(ldn=0),
                                dict(o=None), dict(o=None, ho=None), dict(o=None, ho=None, gate=None, n=None)])
def test_joint_forward_arguments(kw):
    assert _fwd(_joint(), **kw) == poet.EINVAL
    assert poet.lib().poet_last_error().decode()


def test_joint_forward_needs_no_rows():
    assert _fwd(_joint(), o=None, h=None, gate=None, ho=None, n=None, T=0) == poet.OK
    assert _fwd(None) == poet.EINVAL
    assert _fwd(_joint(gate=poet.GATE_NONE)) == poet.EINVAL  # a gate for a joint without one


@pytest.mark.parametrize("kw", [dict(dho=None, dn=None), dict(dn=None), dict(hp=None), dict(dh=None), dict(d_o=None),
                                dict(gate=None), dict(ld=63), dict(wq=P + 1), dict(dh=P + 1), dict(o=None),
                                dict(o=None, d_o=None, gate=None, dg=None), dict(T=-1)])
def test_joint_backward_arguments(kw):
    assert _bwd(_joint(), **kw) == poet.EINVAL


@pytest.mark.parametrize("kw", [dict(ws=None), dict(ws=P + 16), dict(ws_bytes=255)])
def test_joint_backward_workspace(kw):
    J = _joint()
    assert _bwd(J, **kw) == poet.ENOMEM_WS
    need = poet.lib().poet_joint_workspace_bytes(ctypes.byref(J), 4)
    assert need > 0 and _bwd(J, ws_bytes=need - 1) == poet.ENOMEM_WS


def test_joint_workspace_is_bounded():
    # the partial sums stay far below the activations, whatever the rows
    for d in (1, 64, 2048, 16384):
        for rows in (1, 7, 256, 1 << 20):
            J = _joint(d=d, gate_rows=rows)
            sizes = [poet.lib().poet_joint_workspace_bytes(ctypes.byref(J), T) for T in (0, 1, 100, 1 << 15, 1 << 20)]
            assert all(s > 0 for s in sizes) and sizes == sorted(sizes)
            assert sizes[-1] <= 3 * 148 * 48 * 1024 * 4 * 16


def _logp(x=P, ld=100, dt=poet.BF16, T=4, V=100, scale=1.0, tok=P, K=2, logp=P, H=P, top=P, topl=P, saved=P):
    return poet.lib().poet_token_logprobs(x, ld, dt, T, V, scale, tok, K, logp, H, top, topl, saved, ST)


def _logp_grad(x=P, ld=100, dt=poet.BF16, T=4, V=100, scale=1.0, tok=P, saved=P, dl=P, de=P, out=P, ldd=100):
    return poet.lib().poet_token_logprobs_grad(x, ld, dt, T, V, scale, tok, saved, dl, de, out, ldd, ST)


def _distill(x=P, ld=100, dt=poet.BF16, T=4, V=100, scale=1.0, tok=P, val=P, K=2, vs=1.0, tail=0, dl=P, loss=P,
             saved=P, out=P, ldd=100):
    return poet.lib().poet_distill_topk(x, ld, dt, T, V, scale, tok, val, K, vs, tail, dl, loss, saved, out, ldd, ST)


def _distill_grad(x=P, ld=100, dt=poet.BF16, T=4, V=100, scale=1.0, tok=P, val=P, K=2, vs=1.0, tail=0, saved=P, dl=P,
                  out=P, ldd=100):
    return poet.lib().poet_distill_topk_grad(x, ld, dt, T, V, scale, tok, val, K, vs, tail, saved, dl, out, ldd, ST)


@pytest.mark.parametrize("call", [_logp, _logp_grad, _distill, _distill_grad])
@pytest.mark.parametrize("kw", [dict(x=None), dict(x=P + 1), dict(ld=99), dict(dt=2), dict(T=-1), dict(T=(1 << 24) + 1),
                                dict(V=0), dict(V=2097153, ld=1 << 22, ), dict(scale=0.0), dict(scale=-1.0),
                                dict(scale=float("nan")), dict(scale=float("inf")), dict(saved=P + 8), dict(tok=P + 2)])
def test_logit_arguments(call, kw):
    assert call(**kw) == poet.EINVAL
    assert poet.lib().poet_last_error().decode()


@pytest.mark.parametrize("call,kw", [
    (_logp, dict(K=-1)), (_logp, dict(K=129)), (_logp, dict(top=None)), (_logp, dict(topl=None)), (_logp, dict(K=0)),
    (_logp, dict(tok=None)), (_logp, dict(H=P + 1)),
    (_logp_grad, dict(saved=None)), (_logp_grad, dict(dl=None, de=None)), (_logp_grad, dict(tok=None)),
    (_logp_grad, dict(out=None)), (_logp_grad, dict(ldd=99)), (_logp_grad, dict(out=P, ldd=101)),
    (_distill, dict(K=0)), (_distill, dict(K=129)), (_distill, dict(vs=0.0)), (_distill, dict(vs=float("nan"))),
    (_distill, dict(tail=2)), (_distill, dict(tok=None)), (_distill, dict(val=None)), (_distill, dict(loss=None)),
    (_distill, dict(out=P + 1)), (_distill, dict(out=P, ldd=104)), (_distill, dict(dl=P + 1)),
    (_distill_grad, dict(saved=None)), (_distill_grad, dict(out=None)), (_distill_grad, dict(K=0)),
])
def test_logit_arguments_of_each(call, kw):
    assert call(**kw) == poet.EINVAL


def test_no_rows_is_nothing_to_do():
    assert _logp(T=0, x=None) == poet.OK
    assert _logp_grad(T=0, x=None, out=None) == poet.OK
    assert _distill(T=0, x=None) == poet.OK
    assert _distill_grad(T=0, x=None) == poet.OK


def test_host_tensors_are_refused():
    x = torch.zeros(2, 8)
    for call in (lambda: poet.token_logprobs(x), lambda: poet.joint_forward(x, x),
                 lambda: poet.distill_topk(x, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
