"""A backward pass cannot be captured beside an eager result of the same leaf on another stream, whoever made that result:
the operators refuse it in their forward call."""
import gc

import pytest
import torch

import muon_newton_schulz_update_amd as mu
from test_captured_backward_gpu import leaves

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("op", ["residual_norm", "rms_norm", "linear_logprobs"])
@pytest.mark.parametrize("leaf", [0, 1])
def test_a_result_of_torch_on_another_stream_is_refused(op, leaf):
    """An embedding tied to the head, a gain that something else used before: the first use of the leaf is not ours."""
    (h, w, gain), t = leaves(40, 300, 64, 320)
    uses = dict(residual_norm=(h, gain), rms_norm=(h, gain), linear_logprobs=(h, w))[op]
    call = dict(residual_norm=lambda: mu.residual_norm(h, h, pre_gain=gain)[1], rms_norm=lambda: mu.rms_norm(h, gain),
                linear_logprobs=lambda: mu.linear_logprobs(h, w, t).entropy)[op]
    s, seen = torch.cuda.Stream(), torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s), torch.no_grad():
        call()                             # buffers grow outside the capture
        s.synchronize()
    eager = uses[leaf] * 2                 # torch's own, on the default stream
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call()                             # (outside a capture it is torch's to order)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            with pytest.raises(RuntimeError, match="another stream"):
                call()
            seen.add_(1)
        with torch.no_grad():              # nothing to differentiate, nothing to refuse
            graph1 = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph1, stream=s):
                alone = call()
        del eager
        gc.collect()
        graph2 = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph2, stream=s):
            got = call().detach()
        for g in (graph, graph1, graph2):
            g.replay()
        s.synchronize()
        assert torch.equal(seen, torch.ones_like(seen)) and torch.equal(got, call().detach()) and torch.equal(alone, got)
    s.synchronize()


def test_a_result_on_the_same_stream_is_no_reason():
    (h, w, gain), t = leaves(40, 300, 64, 330)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        eager = h * 2, gain * 2
        mu.rms_norm(h, gain)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = mu.rms_norm(h, gain).detach()
        graph.replay()
        s.synchronize()
        assert torch.equal(got, mu.rms_norm(h, gain).detach()) and all(x.requires_grad for x in eager)
    s.synchronize()
