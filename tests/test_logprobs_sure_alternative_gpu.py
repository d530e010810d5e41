"""Log probabilities and entropy where the model is sure of another word than the given one.

As for a sure target (test_logprobs_sure_gpu.py): the sure words' logits are long sums whose parts cancel, which 32-bit sums
miss by far more than the bounds; the others' are single products, exact in 32 bits. In units of U = 2^-24, relative: in a
tile without the sure word exponentials of differences of at most 2 take 2 * 3 for their exponents, with a soft cap 12 * 2 for
the capped logits, and 4 for themselves; their sums at most 64 + 16 additions; the joins and logarithms 16: 128 together. In
the sure word's own tile the differences are up to D = its logit + 2: one rounding of the difference (D), one of its product
with log2 e (D, too) and that constant's own (D / 4): `bound`. The entropy, a sum of positive terms p |log p| of these, twice
that."""
import pytest
import torch

import muon_newton_schulz_update_amd as mu
from test_logprobs_gpu import BF, F32, normal

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def bound(high):
    return (128 + 2.25 * (high + 2)) * U


def sure_words(n, v, d, dtype, high, seed=1):
    """A head whose word i % 7 has a logit of about `high` for token i, its six like -30, the others between -1 and 1."""
    h, w = normal((n, d), seed).to(dtype), torch.zeros((v, d), device="cuda")
    t = torch.arange(n, device="cuda") % 7
    h[:, 0] = h[:, 1] = 1
    w[:, 1] = (2 * torch.rand(v, generator=torch.Generator("cuda").manual_seed(seed + 1), device="cuda") - 1).to(dtype).float()
    w[:7, 2:] = 4 * normal((7, d - 2), seed + 2)
    w = w.to(dtype)
    raw = torch.matmul(h.double(), w.double().t().contiguous())
    keep = torch.full((n, 7), -30.0, device="cuda", dtype=torch.float64)
    keep[torch.arange(n, device="cuda"), t] = high
    room = torch.zeros((v, 7), device="cuda")
    room[:7] = torch.eye(7, device="cuda")
    w = torch.cat([w, room.to(dtype)], 1).contiguous()
    h = torch.cat([h, (keep - raw[:, :7]).to(dtype)], 1).contiguous()
    return h, w, t


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("softcap", [0.0, 50.0])
@pytest.mark.parametrize("high", [8.0, 12.0, 20.0, 40.0])
@pytest.mark.parametrize("n,v,d,top", [(1, 300, 512, 1), (1, 300, 512, 3), (40, 300, 509, 2), (700, 200, 512, 1), (70, 5000, 512, 2)])
def test_a_sure_alternative(n, v, d, top, high, softcap, dtype):
    h, w, sure = sure_words(n, v, d, dtype, high)
    z = torch.matmul(h.double(), w.double().t().contiguous())
    z = softcap * torch.tanh(z / softcap) if softcap else z
    at = sure[:, None]
    others = torch.logsumexp(z.scatter(1, at, -float("inf")), 1) - z.gather(1, at)[:, 0]
    first = -torch.log1p(others.exp())
    lp = torch.log_softmax(z, dim=1)
    entropy = torch.special.entr(lp.exp()).scatter(1, at, (-first * first.exp())[:, None]).sum(1)
    other = 7 + torch.arange(n, device="cuda") % (v - 7)
    for target in (other, torch.full_like(other, -1), sure):         # (-1: outside the vocabulary)
        out = mu.linear_logprobs(h, w, target, top=top, softcap=softcap)
        assert torch.equal(out.top_tokens[:, 0], sure)
        got = out.top_logprobs[:, 0].double()
        assert bool((got <= 0).all())
        assert float(((got - first) / first).abs().max()) <= bound(high)
        assert float(((out.entropy - entropy) / entropy).abs().max()) <= 2 * bound(high)
        assert bool((out.top_logprobs[:, 1:] <= out.top_logprobs[:, :-1]).all())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("top", [0, 2])
@pytest.mark.parametrize("high", [8, 16, 32])
@pytest.mark.parametrize("n,v", [(1, 300), (50, 5000), (700, 640)])
def test_entropy_beside_an_exact_sure_word(n, v, high, top, dtype):
    """Every logit a single product, and one by far the largest, or two or nine equal ones: the entropy is a small sum of
    small terms, none of which may go under beside the large one's."""
    for equal in (1, 2, 9):
        h, w = torch.zeros((n, 64), device="cuda"), torch.zeros((v, 64), device="cuda")
        h[:, 5] = 1
        w[:, 5] = (torch.rand(v, generator=torch.Generator("cuda").manual_seed(4), device="cuda") - 1).to(dtype).float()
        words = torch.tensor([130, 131, 2, 299, 77, 200, 64, 65, 32][:equal], device="cuda")
        w[words, 5] = float(high)
        h, w = h.to(dtype), w.to(dtype)
        lp = torch.log_softmax(torch.matmul(h.double(), w.double().t().contiguous()), 1)
        rest = torch.ones(v, device="cuda", dtype=torch.bool)
        rest[words] = False
        small = lp[:, rest].exp().sum(1)                                # p of all others
        entropy = torch.special.entr(lp[:, rest].exp()).sum(1) - (1 - small) * (torch.log1p(-small) - torch.log(torch.tensor(float(equal))))
        t = torch.arange(n, device="cuda") % 30 + 3
        out = mu.linear_logprobs(h, w, t, top=top)
        assert float(((out.entropy - entropy) / entropy).abs().max()) <= 2 * bound(high), equal
        assert bool((out.entropy > 0).all())
