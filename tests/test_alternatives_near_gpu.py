"""Alternatives whose 32-bit sums are off by more than they differ, several of them in one lane's set.

A sum over products of 2^26 loses everything below 2 (a spacing of fp32 there is 8, or 4 just under it), however small it
ends: the words made so come out as 0 in 32 bits and have their exact logits in 64 alone. The other words' logits are single
products, exact in 32 bits. As long as a call's `top` + 8 largest 32-bit sums have all of these words among them, the
alternatives are those of the exact logits.
"""
import pytest
import torch

import muon_newton_schulz_update_amd as mu
from test_logprobs_gpu import BF, F32, gen

pytestmark = pytest.mark.gpu

# one lane's set of 16-bit heads (fp32: its first half, and half of another): rows in fours, every second four
SET = [8 * i + j for i in range(8) for j in range(4)]


def cancelling(n, v, words, logits, plain, seed, dtype, d=320):
    """Hidden states of ones and 2^13s, and a head: `words` have products 2^26, their logit and -2^26, far apart in the
    width, the others one product: `plain`, a dict, or between -6 and -5."""
    h, w = torch.zeros((n, d), device="cuda"), torch.zeros((v, d), device="cuda")
    h[:, 3], h[:, 150] = 2.0 ** 13, 2.0 ** 13
    h[:, 70], h[:, 300] = 1.0, 1.0
    w[:, 300] = -5 - torch.rand(v, generator=gen(seed), device="cuda")
    for word, z in plain.items():
        w[word, 300] = z
    words = torch.tensor(words, device="cuda")
    w[words, 300] = 0
    w[words, 3], w[words, 150] = 2.0 ** 13, -2.0 ** 13
    w[words, 70] = torch.tensor(logits, device="cuda", dtype=torch.float32)
    return h.to(dtype), w.to(dtype)


def order(h, w, top):
    raw = torch.matmul(h.double(), w.double().t().contiguous())
    return raw.sort(dim=1, descending=True, stable=True).indices[:, :top]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 40, 300])
@pytest.mark.parametrize("given", ["neither", "first", "second"])
def test_a_set_mate_behind_in_32_bits(n, given, dtype):
    """Two words of one set: 0.625 in both precisions, and 0 in 32 bits, 1 in 64."""
    first, second = 512 + SET[5], 512 + SET[2]
    h, w = cancelling(n, 2000, [second], [1.0], {first: 0.625}, 1, dtype)
    t = torch.full((n,), {"neither": 7, "first": first, "second": second}[given], device="cuda")
    for top in (1, 2, 5):
        assert torch.equal(mu.linear_logprobs(h, w, t, top=top).top_tokens, order(h, w, top))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 40, 300])
@pytest.mark.parametrize("top", [1, 3, 7, 12])
@pytest.mark.parametrize("where", ["one set", "two sets", "apart"])
def test_words_that_are_equal_in_32_bits(n, top, where, dtype):
    """Eight words, 0 in 32 bits, of exact logits in another order than the words' (steps of 2^-6 from 0.5), behind a few
    of larger sums, some of which the exact ones pass: all are among the `top` + 8 largest sums in 32 bits."""
    places = {"one set": SET[3:11], "two sets": SET[1:5] + [4 + x for x in SET[6:10]], "apart": [0, 130, 257, 400, 901, 902, 1333, 1999]}[where]
    words = [(640 if where != "apart" else 0) + x for x in places]
    logits = [0.5 + 2.0 ** -6 * k for k in (3, 6, 0, 7, 1, 5, 2, 4)]
    plain = {640 + SET[14]: 0.53125 + 2.0 ** -7, 1100: 0.25, 1500: 0.125}
    plain = dict(list(plain.items())[:min(top, 3)])
    h, w = cancelling(n, 2000, words, logits, plain, 2, dtype)
    t = torch.arange(n, device="cuda") % 2000
    t[0] = words[1]
    assert torch.equal(mu.linear_logprobs(h, w, t, top=top).top_tokens, order(h, w, top))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [2, 90])
def test_an_infinite_target_leaves_the_alternatives(n, dtype):
    """Its values are no numbers, as another word's infinity makes them; the alternatives are in order behind it."""
    h = torch.randn((n, 32), generator=gen(3), device="cuda").to(dtype)
    w = torch.randn((700, 32), generator=gen(4), device="cuda").to(dtype)
    h[:, 0], w[:, 0], w[7, 0] = 1, 0, float("inf")
    t = torch.full((n,), 7, device="cuda")
    out = mu.linear_logprobs(h, w, t, top=9)
    assert bool(out.logprobs.isnan().all()) and bool(out.entropy.isnan().all())
    assert torch.equal(out.top_tokens, order(h, w, 9)) and bool((out.top_logprobs[:, 1:] == -float("inf")).all())
    t[0] = 3
    out = mu.linear_logprobs(h, w, t, top=9)
    assert bool(out.logprobs.isnan().all()) and bool((out.top_tokens[0] == -1).all()) and torch.equal(out.top_tokens[1:], order(h, w, 9)[1:])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 300])
def test_no_log_probability_is_above_0(n, dtype):
    """A word of logit 3.5 that is 0 in 32 bits is found first, and its probability, which the sums do not know, is no
    more than 1."""
    h, w = cancelling(n, 2000, [512 + SET[2]], [3.5], {700: 0.125}, 5, dtype)
    out = mu.linear_logprobs(h, w, torch.full((n,), 7, device="cuda"), top=3)
    assert torch.equal(out.top_tokens, order(h, w, 3)) and bool((out.top_logprobs <= 0).all())
