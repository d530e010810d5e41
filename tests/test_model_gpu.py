"""The norms around a block and the head's log probabilities together, as a model uses them: each operator's part of a
chain against its own 64-bit oracle, on what the chain has there."""
import importlib.util
import math
import os

import pytest
import torch

import muon_newton_schulz_update_amd as mu
from test_logprobs_gpu import BF, F32, Oracle, gen, normal, within
from test_norms_gpu import oracle

pytestmark = pytest.mark.gpu


def chain(n, v, d, tx, ty, seed):
    """A block's end and the model's: residual stream, the block's result, norms and head."""
    x, y = (2 * normal((n, d), seed)).to(tx).requires_grad_(), normal((n, d), seed + 1).to(ty).requires_grad_()
    params = dict(post_gain=(1 + 0.2 * normal((d,), seed + 2)).to(ty), gate=0.5 * normal((1,), seed + 3),
                  scale=1 + 0.1 * normal((1,), seed + 4), pre_gain=(1 + 0.2 * normal((d,), seed + 5)).to(ty))
    head = normal((v, d), seed + 6, 1 / math.sqrt(d)).to(ty).requires_grad_()
    tokens = torch.randint(0, v, (n,), generator=gen(seed + 7), device="cuda")
    tokens[::7] = -100
    for t in params.values():
        t.requires_grad_()
    return x, y, params, head, tokens


@pytest.mark.parametrize("tx,ty", [(BF, BF), (F32, BF), (F32, F32)], ids=["bf16", "mixed", "fp32"])
@pytest.mark.parametrize("n,v,d", [(1, 300, 64), (150, 1003, 200), (700, 5000, 768)])
def test_block_end_head_and_back(tx, ty, n, v, d):
    x, y, params, head, tokens = chain(n, v, d, tx, ty, seed=n)
    out, hidden = mu.residual_norm(x, y, **params)
    hidden.retain_grad()
    found = mu.linear_logprobs(hidden, head, tokens, top=4)
    advantage, dout = normal((n,), 60), normal((n, d), 61).to(tx)
    loss = -(advantage * found.logprobs + 0.01 * found.entropy).sum()
    torch.autograd.backward([loss, out], [None, dout])
    o = Oracle(hidden.detach(), head.detach(), tokens)
    o.check(found, 4)
    kept = tokens != -100
    dh, dh_err, dw, dw_err = o.gradients(torch.where(kept, -advantage, 0.0), torch.full((n,), -0.01, device="cuda"))
    within(hidden.grad, dh, dh_err, "dhidden")
    within(head.grad, dw, dw_err, "dhead")
    plain = {k: t.detach() for k, t in params.items()}
    want = oracle(x.detach(), y.detach(), post_norm=True, pre_norm=True, eps=1e-6, dout=dout, dhidden=hidden.grad, **plain)
    for name, t in dict(dx=x, dy=y, **{"d" + k: t for k, t in params.items()}).items():
        within(t.grad, *want[name], name)
    within(out, *want["out"], "out")
    within(hidden, *want["hidden"], "hidden")


def test_a_step_of_all_in_a_graph():
    """Norms, log probabilities, both gradients, the gradients' norm and AdamW, captured and replayed."""
    n, v, d = 260, 900, 128
    x, y, params, head, tokens = (t for t in chain(n, v, d, F32, BF, seed=90))
    x, y, head = (t.detach() for t in (x, y, head))
    params = {k: t.detach() for k, t in params.items()}
    g = normal((n,), 91, 1 / n)
    handle, s = mu.Handle(), torch.cuda.Stream()

    def fresh():
        return dict(w=head.clone(), m=torch.zeros((v, d), device="cuda"), v=torch.zeros((v, d), device="cuda"))

    def step(state):
        out, hidden = mu.residual_norm(x, y, handle=handle, **params)
        found = mu.linear_logprobs(hidden, state["w"], tokens, top=2, handle=handle)
        dh, dw = mu.linear_logprobs_grad(hidden, state["w"], tokens, found.stats, grad_logprobs=g, grad_entropy=g, handle=handle)
        grads = mu.residual_norm_grad(x, y, None, dh, handle=handle, **params)
        norm, coef = mu.grad_norm([dw, *grads], max_norm=0.1, handle=handle)
        mu.adamw_update([dw], [state["m"]], [state["v"]], [state["w"]], step=3, lr=1e-2, grad_scale=coef, handle=handle)
        return [*found, dh, dw, *grads, norm]

    eager, captured = fresh(), fresh()
    with torch.cuda.stream(s):
        step(fresh())
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = step(captured)
        for k in range(4):
            graph.replay()
            want = step(eager)
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), k
            assert all(torch.equal(eager[name], captured[name]) for name in eager), k
    s.synchronize()
    handle.close()


def test_example_looks_at_what_it_learnt():
    """examples/train_small_lm.py runs, and its gradients come through the norms."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_small_lm.py")
    spec = importlib.util.spec_from_file_location("train_small_lm", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    model = module.Model()
    words = module.text(5, module.language())
    loss = mu.linear_cross_entropy(model.hidden(words[:-1]), model.copies[1], words[1:])
    loss.backward()
    for p in model.matrices + model.copies:
        assert p.grad.shape == p.shape and bool(torch.isfinite(p.grad.float()).all()) and bool(p.grad.any())
        p.grad = None
    module.train(2, say=None, model=model)
    found = module.look(model, say=None)
    assert all(math.isfinite(x) for x in found.values()) and 0 <= found["among_four"] <= 1
    out = model.score(words[:-1], words[1:])
    mean = mu.linear_cross_entropy(model.hidden(words[:-1]).detach(), model.copies[1].detach(), words[1:])
    # the same log probabilities, each within a loss's bound (its sum of 4096 exponentials and its logits' 258 roundings)
    assert abs(float(out.logprobs.mean()) + float(mean)) <= 2 * (512 + 4096 / 64 + 4 * 64 + 258 * 64) * 2.0 ** -24
