"""A training step's operators together, as a user strings them: the norm
before a block, the LLaMA block around seven POET linears, the joint behind it,
a head, log probabilities of a teacher, distillation from its top tokens with
the gradient written over the logits, and the way back through all of them,
against the float64 oracles.  Bar: relative Frobenius error <= 2e-2, the block
tests' (bf16 activations between the operators); losses to 2e-2 of their size.
The same step captured into a graph and replayed gives the same bits."""
import numpy as np
import pytest

from oracle import joint as J
from oracle import llama_block as LB
from oracle import logits as G
from orthogonal_reparameterized_poet_b200 import inputs as I
from tests.harness import TOL, rel_fro
from tests.test_gpu_block import FFN, HEAD_DIM, HEADS, HIDDEN, SEQ, _build, cuda  # noqa: F401

pytestmark = pytest.mark.gpu

V, K = 1003, 12


def _step(poet, torch, blk, p):
    """(loss, perplexity, dh, gradients) of one step."""
    n0 = poet.joint_forward(None, p["h"], w_pre=p["w0"])[1]
    o, saved = blk.forward(n0)
    options = dict(w_post=p["w_post"], w_pre=p["w_pre"], gate_act=poet.GATE_SIGMOID, gate_rows=SEQ, alpha=0.9, beta=0.6)
    h1, n1 = poet.joint_forward(o, p["h"], p["gate"], **options)
    logits = n1 @ p["head"].t()
    logp = poet.token_logprobs(logits, p["tokens"])[0]
    loss, dlogits, _ = poet.distill_topk(logits, p["top"], p["top_logp"], tail=True, dloss=p["weight"], dlogits=logits)
    dn1 = dlogits @ p["head"]
    dh1, d_o, dgate, dw_post, dw_pre = poet.joint_backward(o, h1, p["gate"], None, dn1, **options)
    dn0, grads = blk.backward(saved, d_o)
    dh, _, _, _, dw0 = poet.joint_backward(None, p["h"], None, dh1, dn0, w_pre=p["w0"])
    return {"loss": loss, "logp": logp, "dh": dh, "dgate": dgate, "dw_post": dw_post, "dw_pre": dw_pre, "dw0": dw0}, n1


def test_step_matches_the_oracles(cuda):  # noqa: F811
    from orthogonal_reparameterized_poet_b200 import poet

    torch = cuda
    layers, ref = _build(torch, I.BS, 256, 0)
    blk = poet.PoetBlock(layers, SEQ, HEADS, HEAD_DIM)
    T, r = 2 * SEQ, np.random.default_rng(4)
    bf = lambda x: torch.from_numpy(x).to("cuda", torch.bfloat16)  # noqa: E731
    fl = lambda x: torch.from_numpy(x.astype(np.float32)).cuda()  # noqa: E731
    p = {"h": bf(r.standard_normal((T, HIDDEN))), "gate": bf(r.standard_normal((2, HIDDEN))),
         "head": bf(r.standard_normal((V, HIDDEN)) / np.sqrt(HIDDEN) * 2), "w0": fl(1 + 0.1 * r.standard_normal(HIDDEN)),
         "w_post": fl(1 + 0.1 * r.standard_normal(HIDDEN)), "w_pre": fl(1 + 0.1 * r.standard_normal(HIDDEN)),
         "weight": fl(r.uniform(0.5, 1.5, T) / T)}
    teacher = bf(r.standard_normal((T, V)) * 2)
    tokens = r.integers(0, V, T)
    tokens[-7:] = -1  # padding: its rows teach nothing
    p["tokens"] = torch.from_numpy(tokens.astype(np.int32)).cuda()
    _, _, p["top"], p["top_logp"], _ = poet.token_logprobs(teacher, p["tokens"], topk=K)
    got, n1 = _step(poet, torch, blk, p)
    poet.poet_sync_status()

    f = {k: v.double().cpu().numpy() for k, v in p.items()}
    shape = LB.BlockShape(HIDDEN, FFN, HEADS, HEAD_DIM, SEQ)
    n0 = J.forward(None, f["h"], w_pre=f["w0"])[1]
    o, cache = LB.block_forward(n0, ref, shape)
    options = dict(w_post=f["w_post"], w_pre=f["w_pre"], sigmoid=True, rows=SEQ, alpha=0.9, beta=0.6)
    h1, n1_ref = J.forward(o, f["h"], f["gate"], **options)[:2]
    x = n1_ref @ f["head"].T
    top = p["top"].cpu().numpy()
    logp = G.token_logprobs(x, tokens, 0, 1.0)[0]
    loss, dx, _ = G.distill(x, top, f["top_logp"], f["weight"], tail=True)
    back = J.backward(o, h1, f["gate"], None, dx @ f["head"], **options)
    dn0, _ = LB.block_backward(back["do"][0], ref, cache, shape)
    first = J.backward(None, f["h"], None, back["dh"][0], dn0, w_pre=f["w0"])
    want = {"loss": loss, "logp": logp, "dh": first["dh"][0], "dgate": back["dgate"][0], "dw_post": back["dw_post"][0],
            "dw_pre": back["dw_pre"][0], "dw0": first["dw_pre"][0]}
    errs = {k: rel_fro(v.float().cpu().numpy(), want[k]) for k, v in got.items()}
    errs["n1"] = rel_fro(n1.float().cpu().numpy(), n1_ref)
    assert all(e <= TOL[I.BF16] for e in errs.values()), errs
    assert (got["loss"][-7:] == 0).all() and (got["logp"][-7:] == 0).all()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _step(poet, torch, blk, p)  # the workspaces are there before the capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            held, _ = _step(poet, torch, blk, p)
        for v in held.values():
            v.zero_()
        graph.replay()
        graph.replay()
    s.synchronize()
    for k, v in held.items():
        if k in ("loss", "logp", "dgate", "dw_post", "dw_pre"):  # in front of the block's split sums
            assert torch.equal(v, got[k]), k
        else:
            assert rel_fro(v.float().cpu().numpy(), want[k]) <= TOL[I.BF16], k
