"""Log probability and entropy where the model is sure of the target: its logit counts in more than 32 bits.

The other words' logits are single products, exact in 32 bits; the target's is a long sum whose parts cancel, which a
32-bit sum misses by far more than the bounds. In units of U = 2^-24, relative: a tile's exponentials of differences of at
most 2 take 2 * 3 for their exponents, with a soft cap 12 * 2 for the capped logits, and 4 for themselves; their sums at
most 64 + 16 additions; the joins and logarithms 16: 128 together. The entropy, a sum of positive terms p |log p| of these,
twice that."""
import pytest
import torch

import muon_newton_schulz_update_amd as mu
from test_logprobs_gpu import BF, F32, normal

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("softcap", [0.0, 50.0])
@pytest.mark.parametrize("n,v,d,top", [(1, 300, 512, 0), (1, 300, 512, 3), (40, 300, 509, 2), (700, 200, 512, 0), (700, 200, 512, 1)])
def test_a_sure_target(n, v, d, top, softcap, dtype):
    h, w = normal((n, d), 1).to(dtype), torch.zeros((v, d), device="cuda")
    t = torch.arange(n, device="cuda") % 7
    h[:, 0] = h[:, 1] = 1
    w[:, 1] = (2 * torch.rand(v, generator=torch.Generator("cuda").manual_seed(2), device="cuda") - 1).to(dtype).float()
    w[:7, 2:] = 4 * normal((7, d - 2), 3)
    w = w.to(dtype)
    # seven targets; each token's own ones differ by the hidden state: one channel brings the sum to about 20
    raw = h.double() @ w.double().t()
    h[:, 0] = 1
    keep = torch.full((n, 7), -30.0, device="cuda", dtype=torch.float64)
    keep[torch.arange(n, device="cuda"), t] = 20.0
    # (a channel a target, so that every token can set all seven)
    room = torch.zeros((v, 7), device="cuda")
    room[:7] = torch.eye(7, device="cuda")
    w = torch.cat([w, room.to(dtype)], 1).contiguous()
    h = torch.cat([h, (keep - raw[:, :7]).to(dtype)], 1).contiguous()
    z = h.double() @ w.double().t()
    z = softcap * torch.tanh(z / softcap) if softcap else z
    lp = torch.log_softmax(z, dim=1)
    others = torch.logsumexp(z.scatter(1, t[:, None], -float("inf")), 1) - z.gather(1, t[:, None])[:, 0]
    want = -torch.log1p(others.exp())
    entropy = torch.special.entr(lp.exp()).scatter(1, t[:, None], (-want * want.exp())[:, None]).sum(1)
    out = mu.linear_logprobs(h, w, t, top=top, softcap=softcap)
    assert float(((out.logprobs - want) / want).abs().max()) <= 128 * U
    assert float(((out.entropy - entropy) / entropy).abs().max()) <= 256 * U
    if top:
        assert torch.equal(out.top_tokens[:, 0], t) and torch.equal(out.top_logprobs[:, 0], out.logprobs)
