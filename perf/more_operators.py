"""Cases of the operators around a language model's head and between its blocks, for timing and comparing them.

Two operators: the log probabilities of given tokens with the distribution's entropy and its top alternatives, from the
last hidden states and the head (`logprobs`, with the gradient of both), and the norms after and before a block with
its gate and the residual's scale (`norm`, with the gradient). `run` computes each from elementary torch operations in
32 bits, or, with `own` set, through the package's entry points.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_IGNORE = -100
_EPS = 1e-6

# width 768 and vocabulary 50304 are those of the 124M-parameter model whose matrices this package's benchmark updates
_WIDTH, _VOCAB = 768, 50304

# the dearest listed case; drawn ones stay under it
_MOST_PRODUCT = 8192 * _VOCAB * _WIDTH
_MOST_ELEMENTS = 8192 * 2048


def listed():
    return [
        # one sampled token of a conversation: its log probability and what else was likely; latency counts
        dict(name="logprobs_one_token", op="logprobs", n=1, v=_VOCAB, d=_WIDTH, type="bf16", grad=False, top=8,
             ignored=0.0, softcap=0.0),
        # held-out text scored with alternatives, a quarter of the positions padding
        dict(name="logprobs_evaluation", op="logprobs", n=2048, v=_VOCAB, d=_WIDTH, type="bf16", grad=False, top=5,
             ignored=0.25, softcap=0.0),
        # a teacher's twenty best words a position, of a wider model with a soft cap
        dict(name="logprobs_wide_capped", op="logprobs", n=3000, v=_VOCAB, d=2048, type="bf16", grad=False, top=20,
             ignored=0.0, softcap=30.0),
        # one micro-batch of training on rewards: log probabilities and entropy, then both gradients
        dict(name="logprobs_policy_124m", op="logprobs", n=8192, v=_VOCAB, d=_WIDTH, type="bf16", grad=True, top=0,
             ignored=0.0, softcap=0.0),
        # the same of a small full-precision model, odd sizes everywhere, prompts masked
        dict(name="logprobs_policy_odd_fp32", op="logprobs", n=777, v=8191, d=331, type="fp32", grad=True, top=3,
             ignored=0.1, softcap=0.0),
        # between two blocks for one new token; latency counts
        dict(name="norm_one_token", op="norm", n=1, d=_WIDTH, x="bf16", y="bf16", grad=False, post=True, gate="vector",
             scale="none", pre=True),
        # the same for a batch of prompts
        dict(name="norm_prompts", op="norm", n=8192, d=_WIDTH, x="bf16", y="bf16", grad=False, post=True,
             gate="vector", scale="none", pre=True),
        # a training step of the 124M model: learnt scalars weigh the residual and the block
        dict(name="norm_train_124m", op="norm", n=8192, d=_WIDTH, x="bf16", y="bf16", grad=True, post=False,
             gate="scalar", scale="scalar", pre=True),
        # a wider model that keeps its residual in 32 bits, norms on both sides and a learnt gate for each channel
        dict(name="norm_train_wide_mixed", op="norm", n=8192, d=2048, x="fp32", y="bf16", grad=True, post=True,
             gate="vector", scale="none", pre=True),
        # gates computed for each token, odd sizes, full precision
        dict(name="norm_train_gated_odd_fp32", op="norm", n=1001, d=1023, x="fp32", y="fp32", grad=True, post=True,
             gate="matrix", scale="vector", pre=True),
        # the norm before the first block, with its gradient
        dict(name="norm_train_first", op="norm", n=8192, d=_WIDTH, x="bf16", y="none", grad=True, post=False,
             gate="none", scale="none", pre=True),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    if rng.random() < 0.5:
        kind = rng.choice(["bf16", "bf16", "fp32"])
        grad = rng.random() < 0.5
        # the matrix rate of 32-bit inputs is a sixteenth of that of 16 bits
        most = _MOST_PRODUCT // (1 if kind == "bf16" else 16)
        n, v, d = _log_int(rng, 1, 8192), _log_int(rng, 200, _VOCAB), _log_int(rng, 32, 2048)
        if rng.random() < 0.6:
            d = max(32, d // 32 * 32)
        while n * v * d > most:
            n = max(1, n // 2)
        top = rng.choice([0, 1, 5, rng.randint(2, 32)])
        while n * (top + 8) * d > 2 ** 28:
            n //= 2
        return dict(op="logprobs", n=n, v=v, d=d, type=kind, grad=grad, top=top,
                    ignored=rng.choice([0.0, 0.1, 0.5]) if n >= 64 else 0.0, softcap=rng.choice([0.0, 0.0, 30.0]))
    x, y = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")])
    d = _log_int(rng, 32, 8192)
    if rng.random() < 0.6:
        d = max(32, d // 32 * 32)
    n = min(_log_int(rng, 1, 16384), _MOST_ELEMENTS // d)
    if rng.random() < 0.2:
        return dict(op="norm", n=n, d=d, x=x, y="none", grad=rng.random() < 0.5, post=False, gate="none", scale="none",
                    pre=True)
    return dict(op="norm", n=n, d=d, x=x, y=y, grad=rng.random() < 0.6, post=rng.random() < 0.6,
                gate=rng.choice(["none", "scalar", "vector", "matrix"]), scale=rng.choice(["none", "scalar", "vector"]),
                pre=rng.random() < 0.8)


def _normal(shape, gen, sd=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * sd


def _prepare_logprobs(case, gen):
    kind = _TYPES[case["type"]]
    n, v, d = case["n"], case["v"], case["d"]
    weight = _normal((v, d), gen, 1.0 / math.sqrt(d))
    # frequent words come often; what the model has learnt shows in the state: part of it points to the token
    tokens = (v * torch.rand(n, generator=gen, device="cuda") ** 3).to(torch.int64).clamp_(0, v - 1)
    learnt = 16.0 * torch.rand((n, 1), generator=gen, device="cuda")
    hidden = _normal((n, d), gen) + learnt * weight[tokens]
    if case["ignored"]:
        tokens[torch.rand(n, generator=gen, device="cuda") < case["ignored"]] = _IGNORE
    state = dict(case=case, hidden=hidden.to(kind), weight=weight.to(kind), tokens=tokens)
    if case["grad"]:
        # rewards less their mean, and an entropy bonus
        state["grad_logprobs"] = _normal((n,), gen, 1.0 / n)
        state["grad_entropy"] = torch.full((n,), -0.01 / n, device="cuda")
    return state


def _prepare_norm(case, gen):
    n, d = case["n"], case["d"]
    kx = _TYPES[case["x"]]
    ky = kx if case["y"] == "none" else _TYPES[case["y"]]
    # tokens and channels of uneven size, as a residual stream has them
    uneven = lambda: _normal((n, d), gen) * torch.exp(0.5 * _normal((n, 1), gen)) * torch.exp(0.5 * _normal((d,), gen))  # noqa: E731
    gain = lambda: (1.0 + 0.2 * _normal((d,), gen)).to(ky)  # noqa: E731
    state = dict(case=case, x=(3.0 * uneven()).to(kx), y=None, post=None, gate=None, scale=None, pre=None)
    if case["y"] != "none":
        state["y"] = uneven().to(ky)
    if case["post"]:
        state["post"] = gain()
    if case["gate"] == "scalar":
        state["gate"] = 1.0 + 0.1 * _normal((1,), gen)
    elif case["gate"] == "vector":
        state["gate"] = (0.5 * _normal((d,), gen)).to(ky)
    elif case["gate"] == "matrix":
        state["gate"] = torch.sigmoid(_normal((n, d), gen)).to(ky)
    if case["scale"] == "scalar":
        state["scale"] = 1.0 + 0.1 * _normal((1,), gen)
    elif case["scale"] == "vector":
        state["scale"] = (1.0 + 0.1 * _normal((d,), gen)).to(ky)
    if case["pre"]:
        state["pre"] = gain()
    if case["grad"]:
        state["dout"] = _normal((n, d), gen, 1e-3).to(kx) if case["y"] != "none" else None
        state["dhidden"] = _normal((n, d), gen, 1e-3).to(ky) if case["pre"] else None
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (_prepare_logprobs if case["op"] == "logprobs" else _prepare_norm)(case, gen)


def _there(*outputs):
    return [x for x in outputs if x is not None]


def _run_own(state):
    import muon_newton_schulz_update_amd as mu

    case = state["case"]
    if case["op"] == "logprobs":
        h, w, t, more = state["hidden"], state["weight"], state["tokens"], dict(ignore_index=_IGNORE, softcap=case["softcap"])
        out = mu.linear_logprobs(h, w, t, top=case["top"], **more)
        grads = ()
        if case["grad"]:
            grads = mu.linear_logprobs_grad(h, w, t, out.stats, grad_logprobs=state["grad_logprobs"],
                                            grad_entropy=state["grad_entropy"], **more)
        return _there(out.logprobs, out.entropy, out.top_logprobs, out.top_tokens, *grads)
    if case["y"] == "none":
        grads = mu.rms_norm_grad(state["x"], state["dhidden"], state["pre"], eps=_EPS) if case["grad"] else ()
        return _there(mu.rms_norm(state["x"], state["pre"], eps=_EPS), *grads)
    more = dict(post_norm=case["post"], post_gain=state["post"], gate=state["gate"], scale=state["scale"],
                pre_norm=case["pre"], pre_gain=state["pre"], eps=_EPS)
    out = mu.residual_norm(state["x"], state["y"], **more)
    grads = mu.residual_norm_grad(state["x"], state["y"], state["dout"], state["dhidden"], **more) if case["grad"] else ()
    return _there(*out, *grads)


def _logprobs(state):
    case, kind = state["case"], _TYPES[state["case"]["type"]]
    cap, top = case["softcap"], case["top"]
    kept = state["tokens"] != _IGNORE
    at = torch.where(kept, state["tokens"], 0)[:, None]
    h, w = state["hidden"].float(), state["weight"].float()
    raw = h @ w.t()
    z = cap * torch.tanh(raw / cap) if cap else raw
    most = z.max(dim=1, keepdim=True).values
    e = torch.exp(z - most)
    total = e.sum(dim=1, keepdim=True)
    lse = most + torch.log(total)
    logp = z - lse
    p = e / total
    entropy = -(p * logp).sum(dim=1)
    out = [torch.where(kept, logp.gather(1, at)[:, 0], 0.0), torch.where(kept, entropy, 0.0)]
    if top:
        # neighbours in rank are nearer than the rounding of 32-bit sums now and then: a few more, in 64 bits, decide
        near = raw.topk(min(top + 8, case["v"]), dim=1).indices.sort(dim=1).values
        fine = (state["hidden"].double()[:, None, :] * state["weight"][near].double()).sum(dim=2)
        fine, order = fine.sort(dim=1, descending=True, stable=True)
        best = fine[:, :top]
        best = (cap * torch.tanh(best / cap) if cap else best) - lse
        out.append(torch.where(kept[:, None], best, 0.0).float())
        out.append(torch.where(kept[:, None], near.gather(1, order)[:, :top], -1))
    if case["grad"]:
        g, ge = torch.where(kept, state["grad_logprobs"], 0.0)[:, None], torch.where(kept, state["grad_entropy"], 0.0)[:, None]
        dz = -p * (g + ge * (logp + entropy[:, None]))
        dz.scatter_add_(1, at, g)
        if cap:
            dz *= 1 - (z / cap).square()
        out += [(dz @ w).to(kind), (dz.t() @ h).to(kind)]
    return out


def _norm(state):
    case = state["case"]
    f = lambda t: None if t is None else t.float()  # noqa: E731
    x, y, post, gate, scale, pre = (f(state[k]) for k in ("x", "y", "post", "gate", "scale", "pre"))
    kx = state["x"].dtype
    ky = kx if y is None else state["y"].dtype
    out, hidden, n, yh, ry, xh, rx = x if scale is None else x * scale, None, None, None, None, None, None
    if y is not None:
        n = y
        if case["post"]:
            ry = torch.rsqrt(y.square().mean(dim=1, keepdim=True) + _EPS)
            yh = y * ry
            n = yh * post
        out = out + (n if gate is None else gate * n)
    if case["pre"]:
        rx = torch.rsqrt(out.square().mean(dim=1, keepdim=True) + _EPS)
        xh = out * rx
        hidden = (xh * pre).to(ky)
    results = _there(None if y is None else out.to(kx), hidden)
    if not case["grad"]:
        return results
    d, grads = f(state["dout"]), {}
    if case["pre"]:
        dh = state["dhidden"].float()
        dn = dh * pre
        back = rx * (dn - xh * (dn * xh).mean(dim=1, keepdim=True))
        d = back if d is None else d + back
        grads["pre"] = (dh * xh).sum(dim=0).to(ky)
    grads["x"] = (d if scale is None else d * scale).to(kx)
    if scale is not None:
        part = (d * x).sum(dim=0)
        grads["scale"] = (part.sum().reshape(1) if scale.numel() == 1 else part).to(state["scale"].dtype)
    if y is not None:
        dn = d if gate is None else d * gate
        if gate is not None:
            part = d * n
            grads["gate"] = (part if gate.dim() == 2 else part.sum().reshape(1) if gate.numel() == 1 else part.sum(dim=0)).to(
                state["gate"].dtype)
        if case["post"]:
            grads["post"] = (dn * yh).sum(dim=0).to(ky)
            dn = dn * post
            dn = ry * (dn - yh * (dn * yh).mean(dim=1, keepdim=True))
        grads["y"] = dn.to(ky)
    return results + _there(*(grads.get(k) for k in ("x", "y", "post", "gate", "scale", "pre")))


def run(state):
    if own:
        return _run_own(state)
    return (_logprobs if state["case"]["op"] == "logprobs" else _norm)(state)


def work(case):
    if case["op"] == "logprobs":
        size = 2 if case["type"] == "bf16" else 4
        n, v, d = case["n"], case["v"], case["d"]
        rows = n * (1 - case["ignored"])
        moved = (rows + v) * d * size + 8 * n + 8 * n + 12 * n * case["top"]
        if case["grad"]:
            return {"bytes": moved + 8 * n + (n + v) * d * size, "flops": 6 * rows * v * d}
        return {"bytes": moved, "flops": 2 * rows * v * d}
    n, d = case["n"], case["d"]
    ex = 2 if case["x"] == "bf16" else 4
    ey = ex if case["y"] == "none" else 2 if case["y"] == "bf16" else 4
    there = case["y"] != "none"
    # x, out; y, hidden; a gate for each element
    moved = ex * (2 if there else 1) + ey * ((1 if there else 0) + (1 if case["pre"] else 0))
    moved += ey if case["gate"] == "matrix" else 0
    if case["grad"]:
        # dout, dx; dhidden, dy; the gate's gradient
        moved += ex * (2 if there else 1) + ey * ((1 if there else 0) + (1 if case["pre"] else 0))
        moved += ey if case["gate"] == "matrix" else 0
    return {"bytes": n * d * moved, "flops": n * d * (34 if case["grad"] else 10)}


def _exact_logprobs(state):
    """Token by token in blocks, in 64 bits: log-softmax, and the gradient by differentiating it."""
    case = state["case"]
    cap, top = case["softcap"], case["top"]
    t = state["tokens"]
    w = state["weight"].double().requires_grad_(case["grad"])
    parts, dh, dw = [], [], torch.zeros_like(w)
    for i in range(0, case["n"], 2048):
        h = state["hidden"][i:i + 2048].double().requires_grad_(case["grad"])
        kept = t[i:i + 2048] != _IGNORE
        raw = torch.matmul(h, w.t())
        logp = torch.log_softmax(torch.tanh(raw / cap) * cap if cap else raw, dim=1)
        chosen = logp.gather(1, t[i:i + 2048].clamp(min=0)[:, None])[:, 0].masked_fill(~kept, 0)
        entropy = torch.special.entr(logp.exp()).sum(dim=1).masked_fill(~kept, 0)
        block = [chosen.detach(), entropy.detach()]
        if top:
            order = raw.detach().sort(dim=1, descending=True, stable=True).indices[:, :top]
            block += [logp.detach().gather(1, order).masked_fill(~kept[:, None], 0), order.masked_fill(~kept[:, None], -1)]
        parts.append(block)
        if case["grad"]:
            g = torch.autograd.grad([chosen, entropy], [h, w], [state["grad_logprobs"][i:i + 2048].double(),
                                                                state["grad_entropy"][i:i + 2048].double()])
            dh.append(g[0])
            dw += g[1]
    out = [torch.cat(x) for x in zip(*parts)]
    return out + ([torch.cat(dh), dw.detach()] if case["grad"] else [])


def _exact_norm(state):
    case = state["case"]
    names = [k for k in ("x", "y", "post", "gate", "scale", "pre") if state[k] is not None]
    leaves = {k: state[k].double().requires_grad_(case["grad"]) for k in names}
    unit = lambda t: t / (t.pow(2).sum(dim=-1, keepdim=True) / t.shape[-1] + _EPS).sqrt()  # noqa: E731
    out = leaves["x"] * leaves.get("scale", 1)
    if "y" in leaves:
        block = unit(leaves["y"]) * leaves["post"] if case["post"] else leaves["y"]
        out = out + block * leaves.get("gate", 1)
    results, into = ([out], [state.get("dout")]) if "y" in leaves else ([], [])
    if case["pre"]:
        results.append(unit(out) * leaves["pre"])
        into.append(state.get("dhidden"))
    grads = torch.autograd.grad(results, [leaves[k] for k in names], [g.double() for g in into]) if case["grad"] else ()
    return [r.detach() for r in results] + list(grads)


def exact(case, seed):
    state = prepare(case, seed)
    return (_exact_logprobs if case["op"] == "logprobs" else _exact_norm)(state)
