"""Backward passes of the norms and the log probabilities by autograd, captured into a graph; and calls that the shapes
of their tensors refuse."""
import gc

import pytest
import torch

import muon_newton_schulz_update_amd as mu
from test_logprobs_gpu import BF, make, normal

pytestmark = pytest.mark.gpu


def leaves(n, v, d, seed):
    h, w, t = make(n, v, d, BF, seed=seed, ignored=0.1)
    gain = (1 + 0.2 * normal((d,), seed + 1)).to(BF)
    return [x.requires_grad_() for x in (h, w, gain)], t


def gradients(h, w, gain, t, into):
    out, hidden = mu.residual_norm(h, h, pre_gain=gain)
    found = mu.linear_logprobs(mu.rms_norm(hidden, gain), w, t)
    return torch.autograd.grad([found.logprobs, found.entropy, out], [h, w, gain], into)


def test_forward_and_backward_in_a_graph():
    """Shared leaves (x is y too, one gain in two norms): every replay is the eager result of the same values."""
    xs, t = leaves(130, 700, 96, 201)
    into = [normal((130,), 205), normal((130,), 206), normal((130, 96), 207).to(BF)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            gradients(*xs, t, into)
        s.synchronize()
        gc.collect()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = gradients(*xs, t, into)
        for k in range(4):
            with torch.no_grad():
                xs[0].copy_(normal((130, 96), 210 + k))
            for g in got:
                g.fill_(7)
            graph.replay()
            s.synchronize()
            want = gradients(*xs, t, into)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), k
    s.synchronize()


@pytest.mark.parametrize("op", ["residual_norm", "rms_norm", "linear_logprobs"])
def test_an_eager_result_of_the_same_leaf_on_another_stream_is_refused(op):
    """In the forward call, before anything of it is recorded; the capture goes on, and works once the result is gone."""
    (h, w, gain), t = leaves(40, 300, 64, 220)
    call = dict(residual_norm=lambda: mu.residual_norm(h, h, pre_gain=gain)[1], rms_norm=lambda: mu.rms_norm(h, gain),
                linear_logprobs=lambda: mu.linear_logprobs(h, w, t).entropy)[op]
    s, seen = torch.cuda.Stream(), torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call()                             # buffers grow outside the capture
        s.synchronize()
    eager = call()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call()                             # (outside a capture it is torch's to order)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            with pytest.raises(RuntimeError, match="another stream"):
                call()
            seen.add_(1)
        del eager
        gc.collect()
        graph2 = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph2, stream=s):
            got = call().detach()
        graph.replay()
        graph2.replay()
        s.synchronize()
        assert torch.equal(seen, torch.ones_like(seen)) and torch.equal(got, call().detach())
    s.synchronize()


def test_a_gate_is_of_the_tokens_shape():
    """As many rows in another order are not: they would be taken for other tokens'."""
    y = normal((2, 3, 64), 230).to(BF)
    gate = normal((3, 2, 64), 231).to(BF)
    for call in (lambda: mu.residual_norm(y, y, gate=gate), lambda: mu.residual_norm(y, y, gate=gate.view(6, 64)),
                 lambda: mu.residual_norm_grad(y, y, y, y, gate=gate)):
        with pytest.raises(ValueError, match="gate"):
            call()
    one = mu.residual_norm(y, y, gate=gate[:1, :1].contiguous())
    assert all(torch.equal(a, b) for a, b in zip(one, mu.residual_norm(y, y, gate=gate[0, 0])))
