"""Cases of the operators at the end of a training step, for timing and comparing them.

Three operators: the softmax cross entropy of a language-model head with its gradient (`loss`), the global gradient
norm with clipping (`clip`) and the AdamW update of the parameters that are not Muon's (`adamw`). `run` computes each
from elementary torch operations in 32 bits, or, with `own` set, through the package's entry points.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_IGNORE = -100

# width 768 and vocabulary 50304 are those of the 124M-parameter model whose matrices this package's benchmark updates
_WIDTH, _VOCAB = 768, 50304

# the dearest listed case; drawn ones stay under it
_MOST_PRODUCT = 8192 * 50304 * 2048
_MOST_ELEMENTS = 2 * _VOCAB * _WIDTH


def listed():
    return [
        # one token scored against the whole vocabulary: the weight is read once, latency counts
        dict(name="loss_one_token", op="loss", n=1, v=_VOCAB, d=_WIDTH, type="bf16", grad=False, each=True, ignored=0.0,
             softcap=0.0),
        # held-out text: losses of every token, no gradient; a quarter of the positions is padding
        dict(name="loss_evaluation", op="loss", n=2048, v=_VOCAB, d=_WIDTH, type="bf16", grad=False, each=True,
             ignored=0.25, softcap=0.0),
        # a small full-precision model with odd sizes everywhere
        dict(name="loss_grad_odd_fp32", op="loss", n=777, v=8191, d=331, type="fp32", grad=True, each=False, ignored=0.1,
             softcap=0.0),
        # one micro-batch of the 124M model, eight sequences of 1024
        dict(name="loss_grad_124m", op="loss", n=8192, v=_VOCAB, d=_WIDTH, type="bf16", grad=True, each=False,
             ignored=0.0, softcap=0.0),
        # a wider model with a soft cap on its logits and masked prompts
        dict(name="loss_grad_wide_capped", op="loss", n=8192, v=_VOCAB, d=2048, type="bf16", grad=True, each=False,
             ignored=0.15, softcap=30.0),
        # the gains of a small model: a few kilobytes a tensor, latency counts
        dict(name="clip_gains", op="clip", shapes="gains", count=24, type="fp32", max_norm=1.0, scale=0.1, apart=True),
        # most of the 124M model's gradients, matrices with both embeddings, over the limit; kept beside the clipped ones
        dict(name="clip_124m", op="clip", shapes="model", count=8, type="bf16", max_norm=1.0, scale=1e-2, apart=True),
        # an ordinary step of a full-precision model with odd sizes: under the limit, in place
        dict(name="clip_under_limit_odd", op="clip", shapes="odd", count=9, type="fp32", max_norm=1e4, scale=1e-3,
             apart=False),
        # the gains' update
        dict(name="adamw_gains", op="adamw", shapes="gains", count=16, type="fp32", scaled=False, copies=False),
        # both embeddings and the gains of the 124M model, with the clipping coefficient from the device
        dict(name="adamw_embeddings", op="adamw", shapes="embeddings", count=12, type="bf16", scaled=True, copies=False),
        # 32-bit weights of odd sizes with the 16-bit copies that the model computes with
        dict(name="adamw_odd_copies", op="adamw", shapes="odd", count=9, type="fp32", scaled=True, copies=True),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["loss", "loss", "loss", "clip", "adamw"])
    kind = rng.choice(["bf16", "bf16", "fp32"])
    if op == "loss":
        grad = rng.random() < 0.6
        # the matrix rate of 32-bit inputs is a sixteenth of that of 16 bits
        most = _MOST_PRODUCT // (1 if kind == "bf16" else 16)
        n, v, d = _log_int(rng, 1, 8192), _log_int(rng, 200, _VOCAB), _log_int(rng, 32, 2048)
        if rng.random() < 0.6:
            d = max(32, d // 32 * 32)
        while n * v * d > most:
            n = max(1, n // 2)
        return dict(op="loss", n=n, v=v, d=d, type=kind, grad=grad, each=rng.random() < 0.4,
                    ignored=rng.choice([0.0, 0.1, 0.5]) if n >= 64 else 0.0, softcap=rng.choice([0.0, 0.0, 30.0]))
    shapes = dict(shapes="drawn", count=rng.randint(1, 15), largest=_log_int(rng, 64, _MOST_ELEMENTS // 15),
                  seed=rng.randrange(1 << 20))
    if op == "clip":
        apart = rng.random() < 0.6
        return dict(op="clip", **shapes, type=kind, max_norm=1.0 if apart else 1e6, scale=10 ** rng.uniform(-3, 0),
                    apart=apart)
    return dict(op="adamw", **shapes, type=kind, scaled=rng.random() < 0.5, copies=kind == "fp32" and rng.random() < 0.5)


def _shapes(case):
    """The tensors' shapes and types of a clip or adamw case."""
    kind = _TYPES[case["type"]]
    count = case["count"]
    if case["shapes"] == "gains":
        return [((_WIDTH,), kind)] * count
    if case["shapes"] == "model":
        layer = [((_WIDTH, _WIDTH), kind)] * 4 + [((4 * _WIDTH, _WIDTH), kind), ((_WIDTH, 4 * _WIDTH), kind)]
        return [((_VOCAB, _WIDTH), kind)] * 2 + layer * count
    if case["shapes"] == "embeddings":
        return [((_VOCAB, _WIDTH), kind)] * 2 + [((_WIDTH,), torch.float32)] * count
    if case["shapes"] == "odd":
        return [((1021 + 2 * i, 1023 + 202 * i) if i % 3 else (4099 + i,), kind) for i in range(count)]
    rng = random.Random(case["seed"])
    sizes = [_log_int(rng, max(1, case["largest"] // 1000), case["largest"]) for _ in range(count)]
    cols = [_log_int(rng, 1, 3000) for _ in range(count)]
    return [((s,) if rng.random() < 0.3 else (max(1, s // c), c), kind) for s, c in zip(sizes, cols)]


def _normal(shape, gen, sd=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * sd


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = _TYPES[case["type"]]
    if case["op"] == "loss":
        n, v, d = case["n"], case["v"], case["d"]
        weight = _normal((v, d), gen, 1.0 / math.sqrt(d))
        # frequent words come often; what the model has learnt shows in the state: part of it points to the target
        targets = (v * torch.rand(n, generator=gen, device="cuda") ** 3).to(torch.int64).clamp_(0, v - 1)
        learnt = 16.0 * torch.rand((n, 1), generator=gen, device="cuda")
        hidden = _normal((n, d), gen) + learnt * weight[targets]
        if case["ignored"]:
            targets[torch.rand(n, generator=gen, device="cuda") < case["ignored"]] = _IGNORE
        return dict(case=case, hidden=hidden.to(kind), weight=weight.to(kind), targets=targets)
    shapes = _shapes(case)
    if case["op"] == "clip":
        # uneven rows, as gradients have them
        grads = [(_normal(s, gen, case["scale"]) * torch.exp(_normal(s[:1] + (1,) * (len(s) - 1), gen))).to(k)
                 for s, k in shapes]
        return dict(case=case, grads=grads, out=[torch.empty_like(g) for g in grads] if case["apart"] else None)
    return dict(case=case, weights=[_normal(s, gen, 0.02).to(k) for s, k in shapes],
                grads=[_normal(s, gen, 1e-3).to(k) for s, k in shapes],
                firsts=[_normal(s, gen, 5e-4) for s, _ in shapes],
                seconds=[_normal(s, gen, 1e-3).square() for s, _ in shapes],
                scale=torch.rand((), generator=gen, device="cuda") if case["scaled"] else None,
                copies=[torch.empty(s, device="cuda", dtype=torch.bfloat16) for s, _ in shapes]
                if case["copies"] else None)


_STEP, _LR, _BETA1, _BETA2, _EPS, _DECAY = 100, 3e-3, 0.8, 0.95, 1e-10, 0.01


def _run_own(state):
    import muon_newton_schulz_update_amd as mu

    case = state["case"]
    if case["op"] == "loss":
        reduction = "none" if case["each"] else "mean"
        call = mu.linear_cross_entropy_grad if case["grad"] else mu.linear_cross_entropy
        return call(state["hidden"], state["weight"], state["targets"], ignore_index=_IGNORE, reduction=reduction,
                    softcap=case["softcap"])
    if case["op"] == "clip":
        norm = mu.clip_grad_norm(state["grads"], case["max_norm"], out=state["out"])
        return [norm, state["out"] if case["apart"] else state["grads"]]
    mu.adamw_update(state["grads"], state["firsts"], state["seconds"], state["weights"], step=_STEP, lr=_LR,
                    beta1=_BETA1, beta2=_BETA2, eps=_EPS, weight_decay=_DECAY, grad_scale=state["scale"],
                    copies=state["copies"])
    return [state["weights"], state["firsts"], state["seconds"], state["copies"]]


def _loss(state):
    case, kind = state["case"], _TYPES[state["case"]["type"]]
    kept = state["targets"] != _IGNORE
    targets = torch.where(kept, state["targets"], 0)[:, None]
    h, w = state["hidden"].float(), state["weight"].float()
    z = h @ w.t()
    cap = case["softcap"]
    if cap:
        z = cap * torch.tanh(z / cap)
    top = z.max(dim=1, keepdim=True).values
    e = torch.exp(z - top)
    total = e.sum(dim=1, keepdim=True)
    loss = torch.where(kept, (top + torch.log(total) - z.gather(1, targets))[:, 0], 0.0)
    share = kept.float() if case["each"] else kept.float() / kept.sum().clamp(min=1)
    value = loss if case["each"] else (loss * share).sum()
    if not case["grad"]:
        return value
    dz = e / total
    dz.scatter_add_(1, targets, torch.full_like(targets, -1, dtype=torch.float32))
    dz *= share[:, None]
    if cap:
        dz *= 1 - (z / cap).square()
    return value, (dz @ w).to(kind), (dz.t() @ h).to(kind)


def _clip(state):
    grads, limit = state["grads"], state["case"]["max_norm"]
    norm = torch.sqrt(torch.stack([g.float().square().sum() for g in grads]).sum())
    coef = torch.clamp(limit / (norm + 1e-6), max=1.0)
    out = state["out"] if state["case"]["apart"] else grads
    return [norm, [o.copy_(g.float() * coef) for o, g in zip(out, grads)]]


def _adamw(state):
    s = state["scale"]
    grads = [g.float() if s is None else g.float() * s for g in state["grads"]]
    firsts = [m.mul_(_BETA1).add_((1 - _BETA1) * g) for m, g in zip(state["firsts"], grads)]
    seconds = [v.mul_(_BETA2).add_((1 - _BETA2) * g.square()) for v, g in zip(state["seconds"], grads)]
    c1, c2 = 1 - _BETA1 ** _STEP, 1 - _BETA2 ** _STEP
    weights = [w.copy_(w.float() * (1 - _LR * _DECAY) - _LR * (m / c1) / (torch.sqrt(v / c2) + _EPS))
               for w, m, v in zip(state["weights"], firsts, seconds)]
    copies = None if state["copies"] is None else [c.copy_(w) for c, w in zip(state["copies"], weights)]
    return [weights, firsts, seconds, copies]


def run(state):
    if own:
        return _run_own(state)
    return {"loss": _loss, "clip": _clip, "adamw": _adamw}[state["case"]["op"]](state)


def work(case):
    size = 2 if case["type"] == "bf16" else 4
    if case["op"] == "loss":
        n, v, d = case["n"], case["v"], case["d"]
        rows = n * (1 - case["ignored"])
        read = (rows + v) * d * size + 8 * n
        written = 4 * (n if case["each"] else 1)
        if case["grad"]:
            return {"bytes": read + written + (n + v) * d * size, "flops": 6 * rows * v * d}
        return {"bytes": read + written, "flops": 2 * rows * v * d}
    counts = [(math.prod(s), 2 if k == torch.bfloat16 else 4) for s, k in _shapes(case)]
    if case["op"] == "clip":
        return {"bytes": sum(c * e for c, e in counts) * (2 if case["apart"] else 1), "flops": 3 * sum(c for c, _ in counts)}
    return {"bytes": sum(c * (3 * e + 16 + (2 if case["copies"] else 0)) for c, e in counts),
            "flops": 14 * sum(c for c, _ in counts)}


def _exact_loss(state):
    """Token by token in blocks: log-sum-exp and its derivative in 64 bits."""
    case = state["case"]
    h, w, t = state["hidden"].double(), state["weight"].double(), state["targets"]
    n, cap = case["n"], case["softcap"]
    kept = (t != _IGNORE).double()
    weight_of = kept if case["each"] else kept / max(1.0, float(kept.sum()))
    losses, dh, dw = [], [], torch.zeros_like(w)
    for i in range(0, n, 2048):
        hi, ti, gi = h[i:i + 2048], t[i:i + 2048], weight_of[i:i + 2048]
        raw = torch.matmul(hi, w.t().contiguous())
        z = raw if not cap else torch.tanh(raw / cap) * cap
        at = torch.where(ti == _IGNORE, torch.zeros_like(ti), ti)[:, None]
        lse = torch.logsumexp(z, dim=1)
        losses.append(torch.where(ti == _IGNORE, torch.zeros_like(lse), lse - z.gather(1, at)[:, 0]))
        if not case["grad"]:
            continue
        dz = torch.exp(z - lse[:, None])
        dz.scatter_(1, at, torch.expm1(z.gather(1, at) - lse[:, None]))
        if cap:
            dz = dz * (1 - torch.tanh(raw / cap) ** 2)
        dz = dz * gi[:, None]
        dh.append(torch.matmul(dz, w))
        dw += torch.matmul(dz.t().contiguous(), hi)
    loss = torch.cat(losses)
    value = loss if case["each"] else (loss * weight_of).sum()
    return (value, torch.cat(dh), dw) if case["grad"] else value


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "loss":
        return _exact_loss(state)
    grads = [g.double() for g in state["grads"]]
    if case["op"] == "clip":
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g) for g in grads]))
        factor = min(1.0, case["max_norm"] / (float(norm) + 1e-6))
        return [norm, [g * factor for g in grads]]
    factor = 1.0 if state["scale"] is None else float(state["scale"])
    grads = [g * factor for g in grads]
    firsts = [m.double() + (1 - _BETA1) * (g - m.double()) for m, g in zip(state["firsts"], grads)]
    seconds = [v.double() + (1 - _BETA2) * (g ** 2 - v.double()) for v, g in zip(state["seconds"], grads)]
    unbias1, unbias2 = 1 / (1 - _BETA1 ** _STEP), 1 / math.sqrt(1 - _BETA2 ** _STEP)
    weights = [(1 - _LR * _DECAY) * w.double() - _LR * m * unbias1 / (v.sqrt() * unbias2 + _EPS)
               for w, m, v in zip(state["weights"], firsts, seconds)]
    return [weights, firsts, seconds, weights if case["copies"] else None]
