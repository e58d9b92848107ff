"""Cases, plain forms and 64-bit values of the operators between and after POET-trained blocks.

Three operators, each forward and backward:

* ``joint``: the joint between two blocks.  A branch's output o is normalized (RMSNorm with
  gains, optional), gated, scaled and added to the residual stream, and the stream is
  normalized for the next block:
      h' = alpha h + beta act(gate) * (o / rms(o) * w_post),   n = h' / rms(h') * w_pre.
* ``logprobs``: log probabilities of given tokens, with the entropy of each row's distribution
  and its top alternatives, from logits.
* ``distill``: the loss of a student's logits against a teacher's top logits, with its gradient.

``run`` computes them with elementary torch operations in 32 bits where ``own`` is false, and
calls the framework where it is true.  ``exact`` computes the same values in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ELEM = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def _joint(name, op, T, d, dtype, gate, act="linear", gate_rows=1, post=True, alpha=1.0, beta=1.0):
    return dict(name=name, op=op, T=T, d=d, dtype=dtype, gate=gate, act=act, gate_rows=gate_rows, post=post,
                alpha=alpha, beta=beta)


def _logits(name, op, T, V, dtype, K=0, scale=1.0, masked=False, padded=False, entropy=True, tail=False, pad_ld=0):
    return dict(name=name, op=op, T=T, V=V, dtype=dtype, K=K, scale=scale, masked=masked, padded=padded,
                entropy=entropy, tail=tail, pad_ld=pad_ld)


def listed():
    return [
        # one token between two blocks of a LLaMA-1.3B-sized model: latency
        _joint("joint_one_token", "joint", 1, 2048, "bf16", "none", beta=0.22),
        # a training step's tokens at LLaMA-1.3B width, a learned scale for each channel
        _joint("joint_train", "joint", 32768, 2048, "bf16", "channel", gate_rows=32768, beta=0.7),
        # a ragged float32 batch of odd width, one gate value computed for each token
        _joint("joint_odd_f32", "joint", 1031, 1377, "f32", "row", act="sigmoid", alpha=0.9),
        # backward of a training step at LLaMA-3B width, a gate computed for each token and channel
        _joint("joint_grad_train", "joint_grad", 16384, 2560, "bf16", "channel", act="sigmoid"),
        # backward at LLaMA-60M width, sequences of 256 tokens that each have a gate of their own
        _joint("joint_grad_sequences", "joint_grad", 2048, 512, "bf16", "channel", gate_rows=256, beta=0.5),
        # a decoding step: four rows, sampled under a grammar's mask, 20 alternatives reported
        _logits("logprobs_decode", "logprobs", 4, 32000, "bf16", K=20, scale=1.25, masked=True),
        # validation: the log probabilities behind a perplexity, padded sequences
        _logits("logprobs_eval", "logprobs", 16384, 32000, "bf16", padded=True),
        # a teacher's pass: its top 64 tokens of a large vocabulary are kept for a student
        _logits("logprobs_teacher", "logprobs", 4096, 128000, "bf16", K=64),
        # backward of log probability and entropy (a policy's step), odd vocabulary in float32
        _logits("logprobs_grad_odd", "logprobs_grad", 2047, 50257, "f32", padded=True),
        # a student's training step: loss and gradient in one call, teacher renormalized over its 64
        _logits("distill_train", "distill", 8192, 32000, "bf16", K=64),
        # the same with the teacher's remaining mass as one more outcome; odd vocabulary, padded rows
        _logits("distill_tail_odd", "distill", 1000, 50257, "bf16", K=20, scale=0.5, tail=True, padded=True),
        # the backward alone, where the loss's weights are known only later
        _logits("distill_grad_large", "distill_grad", 4096, 128000, "bf16", K=32, tail=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["joint", "joint_grad", "logprobs", "logprobs_grad", "distill", "distill_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("joint"):
        d = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:  # most widths are multiples of a vector
            d = max(64, d // 64 * 64)
        most = 32768 * 2048 // (2 if dtype == "f32" else 1)
        T = _log_int(rng, 1, min(32768, most // d))
        gate = rng.choice(["none", "channel", "channel", "row"])
        rows = rng.choice([1, T, _log_int(rng, 1, T)])
        return dict(op=op, T=T, d=d, dtype=dtype, gate=gate, act=rng.choice(["linear", "sigmoid"]), gate_rows=rows,
                    post=rng.random() < 0.7, alpha=rng.choice([1.0, 0.9]), beta=round(rng.uniform(0.1, 1.5), 3))
    V = _log_int(rng, 1000, 128000)
    if rng.random() < 0.5:
        V = V // 64 * 64
    most = 16384 * 32000 // (2 if dtype == "f32" else 1)
    T = _log_int(rng, 1, min(16384, most // V))
    K = _log_int(rng, 1, 128)
    if op == "logprobs" and rng.random() < 0.3:
        K = 0
    return dict(op=op, T=T, V=V, dtype=dtype, K=0 if op == "logprobs_grad" else K, scale=rng.choice([1.0, 0.5, 1.25]),
                masked=rng.random() < 0.3, padded=rng.random() < 0.3, entropy=rng.random() < 0.7,
                tail=rng.random() < 0.5, pad_ld=rng.choice([0, 0, 64, 3]))


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    if case["op"].startswith("joint"):
        return _prepare_joint(case, g)
    return _prepare_logits(case, g)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _prepare_joint(case, g):
    T, d, t = case["T"], case["d"], DTYPES[case["dtype"]]
    s = {"case": case}
    s["o"] = (_randn(g, T, d) * 0.8).to(t)                       # a branch's output
    s["h"] = (_randn(g, T, d) * (0.5 + 2.0 * torch.rand(T, 1, generator=g, device=DEV))).to(t)  # the stream
    G = -(-T // case["gate_rows"])
    if case["gate"] == "channel":
        s["gate"] = (_randn(g, G, d) * 0.7 + 0.3).to(t)
    elif case["gate"] == "row":
        s["gate"] = (_randn(g, G) * 0.7 + 0.3).to(t)
    else:
        s["gate"] = None
    s["w_post"] = (1.0 + 0.1 * _randn(g, d)) if case["post"] else None
    s["w_pre"] = 1.0 + 0.1 * _randn(g, d)
    if case["op"] == "joint_grad":
        s["dh"] = _randn(g, T, d).to(t)
        s["dn"] = _randn(g, T, d).to(t)
    return s


def _prepare_logits(case, g):
    T, V, K, t = case["T"], case["V"], case["K"], DTYPES[case["dtype"]]
    x = torch.empty(T, V + case["pad_ld"], dtype=t, device=DEV)[:, :V]
    s = {"case": case, "x": x}
    kk = max(K, 1)
    # distinct tokens that stand out in each row: one from each of kk equal parts of the vocabulary, in random order
    part = V // kk
    likely = torch.arange(kk, device=DEV) * part + torch.randint(0, part, (T, kk), generator=g, device=DEV)
    likely = likely.gather(1, torch.rand(T, kk, generator=g, device=DEV).argsort(1))
    heights = 9.0 - torch.rand(T, kk, generator=g, device=DEV).mul(0.3).add(0.02).cumsum(1)
    for r in range(0, T, 2048):  # in parts, to keep the float32 draws small
        z = _randn(g, min(2048, T - r), V).mul_(1.5)
        if case["masked"]:
            z[torch.rand(z.shape, generator=g, device=DEV) < 0.3] = float("-inf")
        rows = likely[r:r + 2048]
        z.scatter_(1, rows, heights[r:r + 2048] + 0.5 * _randn(g, *rows.shape))
        x[r:r + 2048] = z.to(t)
    pad = torch.zeros(T, dtype=torch.bool, device=DEV)
    if case["padded"]:
        pad[T - T // 16:] = True
    s["live"] = ~pad
    if case["op"].startswith("logprobs"):
        pick = torch.randint(0, kk, (T, 1), generator=g, device=DEV)
        tokens = likely.gather(1, pick).squeeze(1)
        s["tokens"] = torch.where(pad, -1, tokens).to(torch.int32)
    else:
        s["teacher_tokens"] = torch.where(pad[:, None], -1, likely).to(torch.int32).contiguous()
        values = heights + 0.3 * _randn(g, T, kk)
        if case["tail"]:  # log probabilities that leave a part of the mass to the other tokens
            values = torch.log_softmax(values.double(), 1).float() - 0.05 - 0.2 * torch.rand(T, 1, generator=g, device=DEV)
        s["teacher_values"] = values.contiguous()
    if case["op"].endswith("grad"):
        s["saved"] = _saved(case, s)
    if case["op"] == "logprobs_grad":
        s["dlogp"] = _randn(g, T) / T
        s["dentropy"] = 0.01 * _randn(g, T) / T if case["entropy"] else None
    if case["op"].startswith("distill"):
        s["dloss"] = (0.5 + torch.rand(T, generator=g, device=DEV)) / T
    return s


def _saved(case, s):
    """What the forward leaves for the backward, for each row: the largest logit, the logarithm of the
    sum of exp(scale (x - largest)), the entropy, and that logarithm over the tokens outside the teacher's."""
    x, c = s["x"], case["scale"]
    out = torch.zeros(x.shape[0], 4, dtype=torch.float32, device=DEV)
    for r in range(0, x.shape[0], 512):
        xr = x[r:r + 512].double()
        m = xr.amax(1, keepdim=True)
        e = ((xr - m) * c).exp()
        total = e.sum(1)
        out[r:r + 512, 0] = m[:, 0].float()
        out[r:r + 512, 1] = total.log().float()
        if case["op"] == "logprobs_grad":
            z = ((xr - m) * c).clamp(min=-1e30)
            out[r:r + 512, 2] = (total.log() - (e * z).sum(1) / total).float()
        else:
            idx = s["teacher_tokens"][r:r + 512].long().clamp(min=0)
            out[r:r + 512, 3] = e.scatter(1, idx, 0.0).sum(1).log().float()
    out[~s["live"]] = 0.0
    return out


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if op == "joint":
        return _run_joint(state)
    if op == "joint_grad":
        return _run_joint_grad(state)
    if op == "logprobs":
        return _run_logprobs(state)
    if op == "logprobs_grad":
        return _run_logprobs_grad(state)
    return _run_distill(state)


def _joint_options(s):
    from orthogonal_reparameterized_poet_b200 import poet

    case = s["case"]
    return poet, dict(w_post=s["w_post"], w_pre=s["w_pre"], post_norm=case["post"],
                      gate_act=poet.GATE_SIGMOID if case["act"] == "sigmoid" else poet.GATE_LINEAR,
                      gate_rows=case["gate_rows"], alpha=case["alpha"], beta=case["beta"], eps=EPS)


def _gate_values(s):
    """The gate of each row in 32 bits (T x d, T x 1, or 1), after its activation."""
    case = s["case"]
    if s["gate"] is None:
        return None
    v = s["gate"].float()
    if case["gate"] == "row":
        v = v[:, None]
    if case["act"] == "sigmoid":
        v = 1.0 / (1.0 + (-v).exp())
    if case["gate_rows"] > 1:
        v = v[torch.arange(case["T"], device=DEV) // case["gate_rows"]]
    return v


def _run_joint(s):
    if own:
        poet, options = _joint_options(s)
        h, n = poet.joint_forward(s["o"], s["h"], s["gate"], **options)
        return {"h": h, "n": n}
    case = s["case"]
    t = s["o"].dtype
    p = s["o"].float()
    if case["post"]:
        p = p * ((p * p).mean(1, keepdim=True) + EPS).rsqrt() * s["w_post"]
    gate = _gate_values(s)
    if gate is not None:
        p = p * gate
    h = case["alpha"] * s["h"].float() + case["beta"] * p
    n = h * ((h * h).mean(1, keepdim=True) + EPS).rsqrt() * s["w_pre"]
    return {"h": h.to(t), "n": n.to(t)}


def _run_joint_grad(s):
    if own:
        poet, options = _joint_options(s)
        dh, do, dgate, dw_post, dw_pre = poet.joint_backward(s["o"], s["h"], s["gate"], s["dh"], s["dn"], **options)
        return {"dh": dh, "do": do, "dgate": dgate, "dw_post": dw_post, "dw_pre": dw_pre}
    case = s["case"]
    t, T = s["o"].dtype, case["T"]
    # the stream after the joint, normalized
    h, dn = s["h"].float(), s["dn"].float()
    r = ((h * h).mean(1, keepdim=True) + EPS).rsqrt()
    hat = h * r
    dw_pre = (dn * hat).sum(0, dtype=torch.float64).float()
    u = dn * s["w_pre"]
    dh = s["dh"].float() + (u - hat * (u * hat).mean(1, keepdim=True)) * r
    # the branch
    o = s["o"].float()
    da = case["beta"] * dh
    if case["post"]:
        ro = ((o * o).mean(1, keepdim=True) + EPS).rsqrt()
        ohat = o * ro
        p = ohat * s["w_post"]
    else:
        p = o
    dgate = None
    dp = da
    if s["gate"] is not None:
        gate = _gate_values(s)
        dp = da * gate
        each = da * p
        if case["act"] == "sigmoid":
            each = each * (gate * (1.0 - gate))
        if case["gate"] == "row":
            each = each.sum(1)
        if case["gate_rows"] == 1:
            dgate = each.to(t)
        elif case["gate_rows"] >= T:
            dgate = each.sum(0, keepdim=True, dtype=torch.float64).to(t)
        else:
            at = torch.arange(T, device=DEV) // case["gate_rows"]
            dgate = torch.zeros(s["gate"].shape, dtype=torch.float64, device=DEV).index_add_(0, at, each.double()).to(t)
    dw_post = None
    if case["post"]:
        dw_post = (dp * ohat).sum(0, dtype=torch.float64).float()
        v = dp * s["w_post"]
        do = (v - ohat * (v * ohat).mean(1, keepdim=True)) * ro
    else:
        do = dp
    return {"dh": (case["alpha"] * dh).to(t), "do": do.to(t), "dgate": dgate, "dw_post": dw_post, "dw_pre": dw_pre}


def _run_logprobs(s):
    case = s["case"]
    if own:
        from orthogonal_reparameterized_poet_b200 import poet

        logp, entropy, top_tokens, top_logp, _ = poet.token_logprobs(
            s["x"], s["tokens"], topk=case["K"], scale=case["scale"], entropy=case["entropy"])
        return {"logp": logp, "entropy": entropy, "top_tokens": top_tokens, "top_logp": top_logp}
    live = s["tokens"] >= 0
    x = s["x"].float()
    m = x.amax(1, keepdim=True)
    z = (x - m) * case["scale"]
    e = z.exp()
    total = e.sum(1)
    at = s["tokens"].long().clamp(min=0)[:, None]
    logp = torch.where(live, z.gather(1, at)[:, 0] - total.log(), 0.0)
    entropy = top_tokens = top_logp = None
    if case["entropy"]:
        entropy = total.log() - (e * z.clamp(min=-1e30)).sum(1) / total
        entropy = torch.where(live, entropy, 0.0)
    if case["K"]:
        order = s["x"].sort(dim=1, descending=True, stable=True)[1][:, :case["K"]]  # ties: the lower token first
        top_logp = z.gather(1, order) - total.log()[:, None]
        fine = live[:, None] & (top_logp > float("-inf"))
        top_tokens = torch.where(fine, order, -1).to(torch.int32)
        top_logp = torch.where(fine, top_logp, float("-inf"))
    return {"logp": logp, "entropy": entropy, "top_tokens": top_tokens, "top_logp": top_logp}


def _run_logprobs_grad(s):
    case = s["case"]
    if own:
        from orthogonal_reparameterized_poet_b200 import poet

        return {"dlogits": poet.token_logprobs_grad(s["x"], s["tokens"], s["saved"], s["dlogp"], s["dentropy"],
                                                    scale=case["scale"])}
    live = s["tokens"] >= 0
    logp = (s["x"].float() - s["saved"][:, :1]) * case["scale"] - s["saved"][:, 1:2]
    p = logp.exp()
    d = -s["dlogp"][:, None] * p
    if s["dentropy"] is not None:
        d -= s["dentropy"][:, None] * (p * (logp.clamp(min=-1e30) + s["saved"][:, 2:3]))
    at = s["tokens"].long().clamp(min=0)[:, None]
    d.scatter_add_(1, at, s["dlogp"][:, None])
    return {"dlogits": torch.where(live[:, None], d * case["scale"], 0.0).to(s["x"].dtype)}


def _run_distill(s):
    case = s["case"]
    if own:
        from orthogonal_reparameterized_poet_b200 import poet

        options = dict(tail=case["tail"], scale=case["scale"])
        if case["op"] == "distill_grad":
            return {"dlogits": poet.distill_topk_grad(s["x"], s["teacher_tokens"], s["teacher_values"], s["saved"],
                                                      s["dloss"], **options)}
        loss, dlogits, _ = poet.distill_topk(s["x"], s["teacher_tokens"], s["teacher_values"], dloss=s["dloss"],
                                             grad=True, **options)
        return {"loss": loss, "dlogits": dlogits}
    x, values = s["x"].float(), s["teacher_values"]
    live = s["teacher_tokens"][:, :1] >= 0
    at = s["teacher_tokens"].long().clamp(min=0)
    if case["tail"]:
        q = values.exp()
        rest = (1.0 - q.sum(1, keepdim=True)).clamp(min=0.0)
        logq = values
    else:
        logq = values - values.amax(1, keepdim=True)
        logq = logq - logq.exp().sum(1, keepdim=True).log()
        q = logq.exp()
    known = case["op"] == "distill_grad"
    m = s["saved"][:, :1] if known else x.amax(1, keepdim=True)
    z = (x - m) * case["scale"]
    e = z.exp()
    total = s["saved"][:, 1:2].exp() if known else e.sum(1, keepdim=True)
    p = e / total
    factor = 1.0
    if case["tail"]:
        others = s["saved"][:, 3:4].exp() if known else e.scatter(1, at, 0.0).sum(1, keepdim=True)
        factor = 1.0 - rest * (total / others)
    d = (p * factor).scatter(1, at, p.gather(1, at) - q) * (s["dloss"][:, None] * case["scale"])
    dlogits = torch.where(live, d, 0.0).to(s["x"].dtype)
    if known:
        return {"dlogits": dlogits}
    loss = (q * (logq - (z.gather(1, at) - total.log()))).sum(1)
    if case["tail"]:
        loss = loss + (rest * (rest.log() - (others / total).log()))[:, 0]
    return {"loss": torch.where(live[:, 0], loss, 0.0), "dlogits": dlogits}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    T, es = case["T"], ELEM[case["dtype"]]
    if case["op"].startswith("joint"):
        d = case["d"]
        grad = case["op"] == "joint_grad"
        rows = T * d * es * (6 if grad else 4)  # forward: o, h, h', n; backward: o, h, dh', dn, dh, do
        G = -(-T // case["gate_rows"])
        gate = {"none": 0, "row": G, "channel": G * d}[case["gate"]] * es
        gains = 4 * d * (1 + case["post"])
        return {"bytes": rows + (2 if grad else 1) * (gate + gains), "flops": T * d * (30 if grad else 14)}
    V, K = case["V"], case["K"]
    live = T - T // 16 if case["padded"] else T
    if case["op"] == "logprobs":
        return {"bytes": live * V * es + T * (8 + 4 * case["entropy"] + 8 * K), "flops": live * V * 6}
    grad = (live + T) * V * es  # the logits read, the gradient written (zeros in padded rows)
    if case["op"] == "logprobs_grad":
        return {"bytes": grad + T * (24 + 4 * case["entropy"]), "flops": live * V * (8 if case["entropy"] else 5)}
    return {"bytes": grad + T * (8 * K + 20), "flops": live * V * (10 if case["op"] == "distill" else 5)}


# ------------------------------------------------------------------ the same values in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("joint"):
        return _exact_joint(case, s)
    parts = [_exact_logits(case, s, slice(r, r + 512)) for r in range(0, case["T"], 512)]
    names = {"logprobs": ("logp", "entropy", "top_tokens", "top_logp"), "distill": ("loss", "dlogits")}
    names = names.get(case["op"], ("dlogits",))
    return {k: torch.cat([p[k] for p in parts]) if parts[0].get(k) is not None else None for k in names}


def _exact_joint(case, s):
    """By torch's own derivatives of the definition in float64."""
    T, d, rows = case["T"], case["d"], case["gate_rows"]
    leaf = {k: v.double().requires_grad_() for k, v in s.items() if isinstance(v, torch.Tensor)}

    def norm(v, w):
        return v / torch.sqrt(torch.sum(v ** 2, -1, keepdim=True) / d + EPS) * w

    def branch():
        p = norm(leaf["o"], leaf["w_post"]) if case["post"] else leaf["o"]
        if case["gate"] == "none":
            return p
        v = torch.sigmoid(leaf["gate"]) if case["act"] == "sigmoid" else leaf["gate"]
        v = v.reshape(v.shape[0], -1).repeat_interleave(rows, 0)[:T]
        return p * v

    if case["op"] == "joint":
        with torch.no_grad():
            h = case["alpha"] * leaf["h"] + case["beta"] * branch()
            return {"h": h, "n": norm(h, leaf["w_pre"])}
    after, w_pre = leaf["h"], leaf["w_pre"]  # the stream after the joint
    through, dw_pre = torch.autograd.grad(norm(after, w_pre), (after, w_pre), leaf["dn"].detach())
    total = leaf["dh"].detach() + through
    inputs = ["o"] + (["gate"] if case["gate"] != "none" else []) + (["w_post"] if case["post"] else [])
    found = dict(zip(inputs, torch.autograd.grad(branch(), [leaf[k] for k in inputs], case["beta"] * total)))
    return {"dh": case["alpha"] * total, "do": found["o"], "dgate": found.get("gate"), "dw_post": found.get("w_post"),
            "dw_pre": dw_pre}


def _exact_logits(case, s, rows):
    """Some rows of an operator on logits, in float64."""
    c = case["scale"]
    x = s["x"][rows].double() * c
    logp = torch.log_softmax(x, 1)
    p = logp.exp()
    live = s["live"][rows]
    zero = torch.zeros((), dtype=torch.float64, device=DEV)
    if case["op"].startswith("logprobs"):
        at = s["tokens"][rows].long().clamp(min=0)[:, None]
        H = -torch.nan_to_num(p * logp, nan=0.0).sum(1)
        if case["op"] == "logprobs":
            got = {"logp": torch.where(live, logp.gather(1, at)[:, 0], zero)}
            if case["entropy"]:
                got["entropy"] = torch.where(live, H, zero)
            if case["K"]:
                top = logp.topk(case["K"], 1)[0]
                got["top_logp"] = torch.where(live[:, None], top, -torch.inf)
            return got
        hot = torch.zeros_like(p).scatter_(1, at, 1.0)
        d = s["dlogp"][rows].double()[:, None] * (hot - p)
        if case["entropy"]:
            d -= s["dentropy"][rows].double()[:, None] * (torch.nan_to_num(p * logp, nan=0.0) + p * H[:, None])
        return {"dlogits": torch.where(live[:, None], d * c, zero)}
    at = s["teacher_tokens"][rows].long().clamp(min=0)
    values = s["teacher_values"][rows].double()
    q = torch.exp(values) if case["tail"] else torch.softmax(values, 1)
    dense = torch.zeros_like(p).scatter_(1, at, q)
    d = p - dense
    loss = (q * (q.log() - logp.gather(1, at))).sum(1)
    if case["tail"]:
        inside = torch.zeros_like(p).scatter_(1, at, 1.0) > 0
        others = torch.where(inside, zero, p).sum(1, keepdim=True)
        rest = (1.0 - q.sum(1, keepdim=True)).clamp(min=0.0)
        loss = loss + (rest * (rest / others).log())[:, 0]
        d = torch.where(inside, d, p * (1.0 - rest / others))
    d = torch.where(live[:, None], d * (s["dloss"][rows].double()[:, None] * c), zero)
    return {"loss": torch.where(live, loss, zero), "dlogits": d}
