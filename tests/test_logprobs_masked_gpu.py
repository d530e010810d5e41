"""The gradient beside words that the head masks with logits as low as their type goes: these have no part in it."""
import pytest
import torch

import muon_newton_schulz_update_amd as mu
from test_logprobs_gpu import BF, F32, Oracle, gen, make, normal, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [3, 150])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("low", [-3e38, -1e20, -1000.0])
def test_gradient_beside_masked_words(n, low, softcap, dtype):
    """A channel of ones in the hidden states, in which 680 of 700 words have `low`: their probability is 0 as far as 32 bits
    go (with a soft cap their slope is), so the channel's gradient is that of zeros, and the others' that of the kept words."""
    v, d = 700, 32
    h, w, _ = make(n, v, d, dtype, seed=22)
    h[:, 0], w[:, 0] = 1.0, 0.0
    words = torch.randperm(v, generator=gen(23), device="cuda")
    masked, kept = words[20:], words[:20].sort().values
    at = torch.arange(n, device="cuda") % 20
    w2 = w.clone()
    w2[masked, 0] = low
    out = mu.linear_logprobs(h, w2, kept[at], softcap=softcap)
    gl, ge = normal((n,), 24), normal((n,), 25)
    for a, b in ((gl, ge), (gl, None), (None, ge)):
        dh, dw = mu.linear_logprobs_grad(h, w2, kept[at], out.stats, grad_logprobs=a, grad_entropy=b, softcap=softcap)
        if softcap:
            # capped words keep exp(-2 cap) of the sum; their slope is 0, so the channel of `low` has nothing of them
            assert not bool(dh[:, 0].any()) and not bool(dw[masked].any())
            continue
        o = Oracle(h, w[kept], at)
        oh, eh, ow, ew = o.gradients(a, b)
        assert not bool(dh[:, 0].any()) and not bool(dw[masked].any())
        within(dh, oh, eh, "dhidden")
        within(dw[kept], ow, ew, "dweight")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_gradient_of_a_masked_target(dtype):
    """A given word that the head masks: its log probability's gradient is its row less the mean of the others', and the
    entropy's does not know it."""
    v, d, n = 300, 32, 70
    h, w, _ = make(n, v, d, dtype, seed=26)
    h[:, 0], w[:, 0] = 1.0, 0.0
    w2 = w.clone()
    w2[11, 0] = -1000.0
    t = torch.full((n,), 11, device="cuda")
    out = mu.linear_logprobs(h, w2, t)
    g = normal((n,), 27)
    dh, dw = mu.linear_logprobs_grad(h, w2, t, out.stats, grad_entropy=g)
    assert not bool(dh[:, 0].any()) and not bool(dw[11].any())
    o = Oracle(h, w2, t)
    for a in (dict(grad_logprobs=g), dict(grad_logprobs=g, grad_entropy=g)):
        dh, dw = mu.linear_logprobs_grad(h, w2, t, out.stats, **a)
        oh, eh, ow, ew = o.gradients(g, a.get("grad_entropy"))
        within(dh, oh, eh, "dhidden")
        within(dw, ow, ew, "dweight")
