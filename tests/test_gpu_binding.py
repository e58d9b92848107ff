"""The compiled binding of the operators around the blocks."""
import threading
import time

import pytest

from tests.test_gpu_joint import torch  # noqa: F401

pytestmark = pytest.mark.gpu


def test_calls_without_it_give_the_same(torch, monkeypatch):  # noqa: F811
    from orthogonal_reparameterized_poet_b200 import poet

    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    o, h = (torch.randn(37, 96, generator=g, device="cuda").bfloat16() for _ in range(2))
    gate = torch.randn(5, 96, generator=g, device="cuda").bfloat16()
    w = torch.rand(96, generator=g, device="cuda")
    x = torch.randn(9, 3001, generator=g, device="cuda")
    tk = torch.randint(0, 3001, (9,), generator=g, device="cuda", dtype=torch.int32)
    tt, tv = tk[:, None].contiguous(), torch.zeros(9, 1, device="cuda")
    kw = dict(w_post=w, w_pre=w, gate_act=poet.GATE_SIGMOID, gate_rows=8, alpha=0.9, beta=0.4)

    def calls():
        a = poet.joint_forward(o, h, gate, **kw)
        b = poet.joint_backward(o, a[0], gate, h, o, **kw)
        c = poet.token_logprobs(x, tk, topk=6, scale=0.7)
        d = poet.token_logprobs_grad(x, tk, c[4], tv[:, 0] + 1, tv[:, 0] - 1, scale=0.7)
        e = poet.distill_topk(x, tt, tv, grad=True)
        return [*a, *b, *c, d, *e, poet.distill_topk_grad(x, tt, tv, e[2])]

    want = calls()
    monkeypatch.setattr(poet, "_binding", poet._NoBinding)
    got = calls()
    poet.poet_sync_status()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_other_threads_run_while_a_call_waits(torch):  # noqa: F811
    """A launch into a full queue waits for the GPU; other Python threads do not."""
    from orthogonal_reparameterized_poet_b200 import poet

    x = torch.randn(4, 64, device="cuda")
    poet.joint_forward(x, x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    done = threading.Event()

    def launch():
        with torch.cuda.stream(s):
            torch.cuda._sleep(2_000_000_000)  # a second or so at 2 GHz
            for _ in range(4000):  # more launches than a queue holds
                poet.joint_forward(x, x)
        done.set()

    t = threading.Thread(target=launch)
    start = last = time.monotonic()
    t.start()
    longest = 0.0
    while not done.is_set():
        time.sleep(0.001)
        now = time.monotonic()
        longest, last = max(longest, now - last), now
    t.join()
    total = time.monotonic() - start
    torch.cuda.synchronize()
    poet.poet_sync_status()
    assert total > 0.5  # the launches did wait
    assert longest < 0.25 * total, (longest, total)


def test_calls_of_two_threads(torch):  # noqa: F811
    """Each thread's calls run on its own stream and give what they give alone."""
    from orthogonal_reparameterized_poet_b200 import poet

    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    o, h = (torch.randn(300, 256, generator=g, device="cuda") for _ in range(2))
    w = torch.rand(256, generator=g, device="cuda")
    x = torch.randn(64, 5000, generator=g, device="cuda")
    tk = torch.randint(0, 5000, (64,), generator=g, device="cuda", dtype=torch.int32)
    tt, tv = tk[:, None].contiguous(), torch.zeros(64, 1, device="cuda")

    def joint():
        return list(poet.joint_forward(o, h, w_post=w, w_pre=w)) + \
            [t for t in poet.joint_backward(o, h, None, o, h, w_post=w, w_pre=w) if t is not None]

    def logits():
        a = poet.token_logprobs(x, tk, topk=5)
        d = poet.token_logprobs_grad(x, tk, a[4], tv[:, 0].contiguous() + 1)
        c = poet.distill_topk(x, tt, tv, grad=True)
        return list(a) + [d] + list(c) + [poet.distill_topk_grad(x, tt, tv, c[2])]

    jobs = [joint, logits, joint, logits]
    want = [f() for f in jobs]
    torch.cuda.synchronize()
    streams, wrong = [torch.cuda.Stream() for _ in jobs], []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(50):
                    got = jobs[i]()
                    streams[i].synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        wrong.append(i)
        except Exception as e:  # noqa: BLE001
            wrong.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    poet.poet_sync_status()
