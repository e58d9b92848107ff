"""The first calls of a process inside a capture."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import torch
from orthogonal_reparameterized_poet_b200 import poet

o, h = (torch.randn(700, 2048, device="cuda").bfloat16() for _ in range(2))
x = torch.randn(40, 32000, device="cuda")
tk = torch.arange(40, device="cuda", dtype=torch.int32)
tt, tv, one = tk[:, None].contiguous(), torch.zeros(40, 1, device="cuda"), torch.ones(40, device="cuda")


def calls():
    a = poet.joint_forward(o, h)
    b = poet.joint_backward(o, a[0], None, h, o)
    c = poet.token_logprobs(x, tk, topk=20)
    d = poet.token_logprobs_grad(x, tk, c[4], one, one)
    e = poet.distill_topk(x, tt, tv, tail=True, grad=True)
    return [t for t in (*a, *b, *c, d, *e, poet.distill_topk_grad(x, tt, tv, e[2], tail=True)) if t is not None]


g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    held = calls()
for t in held:
    t.zero_()
g.replay()
torch.cuda.synchronize()
want = calls()
poet.poet_sync_status()
assert all(torch.equal(a, b) for a, b in zip(held, want))
print("same")
"""


def test_first_calls_in_a_capture():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
