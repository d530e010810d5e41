"""The cross entropy's gradient beside words that the head masks with logits as low as their type goes: these have no part
in it, as in the log probabilities' (test_logprobs_masked_gpu.py)."""
import pytest
import torch

import muon_newton_schulz_update_amd as mu
from test_logprobs_gpu import BF, F32, Oracle, gen, make, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,v", [(3, 700), (150, 700), (600, 9000)])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("low", [-3e38, -1e20, -1000.0])
def test_gradient_beside_masked_words(n, v, low, softcap, dtype):
    """A channel of ones in the hidden states, in which all but 20 words have `low`: its gradient is that of zeros."""
    h, w, _ = make(n, v, 32, dtype, seed=22)
    h[:, 0], w[:, 0] = 1.0, 0.0
    words = torch.randperm(v, generator=gen(23), device="cuda")
    masked, kept = words[20:], words[:20].sort().values
    at = torch.arange(n, device="cuda") % 20
    w2 = w.clone()
    w2[masked, 0] = low
    loss, dh, dw = mu.linear_cross_entropy_grad(h, w2, kept[at], reduction="sum", softcap=softcap)
    assert not bool(dh[:, 0].any()) and not bool(dw[masked].any())
    if softcap:
        return
    o = Oracle(h, w[kept], at)
    oh, eh, ow, ew = o.gradients(torch.full((n,), -1.0, device="cuda"), None)
    # (a kept exponential has 10 bits of mantissa and is rounded again: half as much again of a 16-bit gradient's error)
    within(dh, oh, 2 * eh, "dhidden")
    within(dw[kept], ow, 2 * ew, "dweight")
    assert bool(torch.isfinite(loss))
