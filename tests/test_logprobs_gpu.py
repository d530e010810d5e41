"""Log probabilities, entropy and alternatives on the GPU against plain 64-bit implementations.

Tolerances are element-wise bounds derived from the arithmetic, not fitted. With u = 2^-24:

* logits: a fp32 sum of D products (exact for bf16 inputs) is within dz = (D + 2) u sum_k |h_k w_k|, a capped one
  a dozen roundings of itself more;
* log probability: two logits, a sum of exponentials of at most 512 serial additions and one per tile, and the
  rounding of references up to the largest logit;
* entropy H = log S - sum p (z - t): each logit's error counts p |log p + H|; the exponent's rounding, (z - t) u,
  once in a term's factor and once in its exponential; the sums as above, relative to 1 + sum p |z - t|;
* the logits' gradient -p (b + g log p): p's error (twice a log probability's), and g p times log p's and H's;
  in bf16 one rounding (2^-8);
* the gradients are sums of K such terms: that error plus K u times the sum of absolute products, and the output's
  rounding (bf16 2^-8).

The alternatives' tokens are those of 64-bit logits, sorted with equal ones in rising order, exactly.
"""
import math

import pytest
import torch

import muon_newton_schulz_update_amd as mu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(shape, seed, sd=1.0):
    return torch.randn(shape, generator=gen(seed), device="cuda") * sd


def mm(a, b):
    return torch.matmul(a.contiguous(), b.contiguous())


def within(got, want, err, what):
    got = got.double()
    bad = ~((got - want).abs() <= err)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, worst {float(((got - want).abs() / err).max()):.3g}x")


def make(n, v, d, dtype, seed=0, learnt=12.0, ignored=0.0, ignore=-100):
    w = normal((v, d), seed * 7 + 1, 1 / math.sqrt(d))
    t = torch.randint(0, v, (n,), generator=gen(seed * 7 + 2), device="cuda")
    h = normal((n, d), seed * 7 + 3) + learnt * torch.rand((n, 1), generator=gen(seed * 7 + 4), device="cuda") * w[t]
    if ignored:
        t[torch.rand(n, generator=gen(seed * 7 + 5), device="cuda") < ignored] = ignore
    return h.to(dtype), w.to(dtype), t


class Oracle:
    """Results, gradients and their element-wise error bounds, in 64 bits."""

    def __init__(self, h, w, t, ignore=-100, softcap=0.0):
        D, V = w.shape[1], w.shape[0]
        self.valid = t != ignore
        self.h, self.w, self.bf, self.cap = torch.where(self.valid[:, None], h.double(), 0.0), w.double(), h.dtype == BF, softcap
        self.raw = mm(self.h, self.w.t())
        z = softcap * torch.tanh(self.raw / softcap) if softcap else self.raw
        self.at = torch.where(self.valid, t, 0)[:, None].long()
        self.dz = (D + 2) * U * mm(self.h.abs(), self.w.abs().t()).amax(1) + (12 * U * z.abs().amax(1) if softcap else 0)
        self.lse = torch.logsumexp(z, 1)
        zt = z.gather(1, self.at)[:, 0]
        others = torch.logsumexp((z - zt[:, None]).scatter(1, self.at, float("-inf")), 1)
        self.logp = -torch.logaddexp(others, torch.zeros_like(others))
        self.others, self.z = others, z
        self.lp = z - self.lse[:, None]
        self.p = torch.exp(self.lp)
        self.sum_err = (512 + V / 64) * U
        self.each = 2 * self.dz + self.sum_err + 4 * U * (self.lse.abs() + zt.abs() + z.abs().amax(1))
        self.H = -(self.p * self.lp).sum(1)
        far = z.amax(1, keepdim=True) - z
        a, b = (self.p * far).sum(1), (self.p * far * far).sum(1)
        self.H_err = (2 * self.dz * (self.p * (self.lp + self.H[:, None]).abs()).sum(1) + (self.sum_err + 16 * U) * (1 + a)
                      + 8 * U * (a + b) + 4 * U * self.H.abs() + V * 1e-17)

    def check(self, out, top):
        v = self.valid
        zero = lambda x: torch.where(v, x, 0.0)
        within(out.logprobs, zero(self.logp), zero(self.each) + 1e-37, "logprobs")
        within(out.entropy, zero(self.H), zero(self.H_err) + 1e-37, "entropy")
        if not top:
            assert out.top_logprobs is None and out.top_tokens is None
            return
        order = self.raw.sort(dim=1, descending=True, stable=True).indices[:, :top]
        want = torch.where(v[:, None], order, -1)
        assert out.top_tokens.dtype == torch.int64 and torch.equal(out.top_tokens, want), (
            int((out.top_tokens != want).sum()), out.top_tokens[(out.top_tokens != want).any(1)][:2], want[(out.top_tokens != want).any(1)][:2])
        within(out.top_logprobs, torch.where(v[:, None], self.lp.gather(1, order), 0.0), zero(self.each)[:, None] + 1e-37, "top_logprobs")

    def gradients(self, gl, ge):
        v = self.valid
        gl, ge = (torch.where(v, torch.zeros_like(self.H) if g is None else g.double(), 0.0)[:, None] for g in (gl, ge))
        H = self.H[:, None]
        slope = 1 / torch.cosh(self.raw / self.cap) ** 2 if self.cap else torch.ones((), dtype=torch.float64, device="cuda")
        q = -self.p * (gl + ge * (self.lp + H))
        pt = torch.exp(self.logp)[:, None]
        q.scatter_(1, self.at, gl * torch.sigmoid(self.others)[:, None] - ge * pt * (self.logp[:, None] + H))
        s = q * slope
        # absolute parts: nothing may cancel in a bound
        size = self.p * (gl.abs() + ge.abs() * (self.lp + H).abs())
        size.scatter_(1, self.at, gl.abs() * torch.sigmoid(self.others)[:, None] + ge.abs() * pt * (self.logp[:, None] + H).abs())
        e = self.each[:, None]
        s_err = size * (2 * e + 24 * U) + ge.abs() * self.p * (e + self.H_err[:, None] + 8 * U * (self.lp.abs() + H))
        if self.cap:
            # a slope's own roundings and what the logit's error does to it
            x = (self.raw / self.cap).abs()
            s_err = (s_err + size * ((8 * x + 24) * U + 4 * self.dz[:, None] / self.cap)) * slope.clamp(max=1.0)
        s_err = s_err + (2.0 ** -8 * s.abs() if self.bf else 0) + (gl.abs() + ge.abs()) * 1e-36
        V, n = self.w.shape[0], self.h.shape[0]
        out = 2.0 ** -8 if self.bf else 2 * U
        dh, dw = mm(s, self.w), mm(s.t(), self.h)
        dh_err = mm(s_err + (V + 8) * U * s.abs(), self.w.abs()) + out * dh.abs() + 1e-37
        dw_err = mm((s_err + (n + 8) * U * s.abs()).t(), self.h.abs()) + out * dw.abs() + 1e-37
        return dh, dh_err, dw, dw_err


def check(h, w, t, top=0, ignore=-100, softcap=0.0, grads=True, seed=50, **kw):
    out = mu.linear_logprobs(h, w, t, top=top, ignore_index=ignore, softcap=softcap, **kw)
    o = Oracle(h, w, t, ignore, softcap)
    o.check(out, top)
    if not grads:
        return out
    n = len(t)
    gl, ge = normal((n,), seed), normal((n,), seed + 1)
    for a, b in ((gl, ge), (gl, None), (None, ge)):
        dh, dw = mu.linear_logprobs_grad(h, w, t, out.stats, grad_logprobs=a, grad_entropy=b, ignore_index=ignore, softcap=softcap)
        oh, eh, ow, ew = o.gradients(a, b)
        assert dh.dtype == h.dtype and dw.dtype == w.dtype
        within(dh, oh, eh, "dhidden")
        within(dw, ow, ew, "dweight")
    return out


SHAPES = [(1, 1, 1), (1, 2, 3), (2, 63, 8), (3, 64, 31), (17, 65, 64), (33, 100, 40), (63, 255, 33), (64, 256, 96), (65, 257, 128),
          (127, 511, 192), (128, 1000, 65), (255, 300, 64), (256, 512, 256), (257, 1025, 320), (300, 5003, 768),
          (1, 50304, 768), (5, 20000, 200), (700, 777, 1030), (1100, 640, 64), (33, 4099, 2048), (2500, 1030, 72)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,v,d", SHAPES)
def test_shapes(n, v, d, dtype):
    h, w, t = make(n, v, d, dtype, seed=n + v + d)
    check(h, w, t, top=min(v, 7))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("top", [0, 1, 2, 31, 32])
@pytest.mark.parametrize("softcap", [0.0, 15.0])
@pytest.mark.parametrize("n,v", [(3, 40), (211, 1003), (70, 9000)])
def test_options(dtype, top, softcap, n, v):
    h, w, t = make(n, v, 160, dtype, seed=3, ignored=0.3, ignore=7)
    check(h, w, t.to(torch.int32), top=top, ignore=7, softcap=softcap, grads=top == 2)


def test_large_tiles():
    """256-tiles: many tokens and words."""
    h, w, t = make(3500, 14000, 128, BF, seed=4, ignored=0.1)
    check(h, w, t, top=9, softcap=0.0)
    check(h, w, t, top=0, softcap=20.0)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [2, 70, 300])
def test_equal_logits_come_by_rising_token(dtype, n):
    """Small whole numbers: every logit is exact, and most are equal to others; a row of zeros makes all equal."""
    v, d = 1500, 16
    h = torch.randint(-2, 3, (n, d), generator=gen(5), device="cuda").to(dtype)
    w = torch.randint(-1, 2, (v, d), generator=gen(6), device="cuda").to(dtype)
    w[700:] = w[:800].clone()                               # the same words again
    h[1] = 0
    t = torch.randint(0, v, (n,), generator=gen(7), device="cuda")
    out = check(h, w, t, top=32, grads=False)
    assert out.top_tokens[1].tolist() == list(range(32))
    assert abs(float(out.entropy[1]) - math.log(v)) <= 600 * U and abs(float(out.top_logprobs[1, 3]) + math.log(v)) <= 600 * U


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_neighbours_nearer_than_a_sum_of_32_bits(dtype):
    """Eight words whose logits differ by 2^-16 on top of 4096 (a spacing of fp32 there is 2^-11), some of them in one
    wave's rows: the order is that of 64 bits."""
    v, d = 3001, 64
    h, w = torch.zeros((40, d), device="cuda"), torch.zeros((v, d), device="cuda")
    h[:, 0], h[:, 1] = 64.0, 2.0 ** -8
    words = torch.tensor([2999, 5, 6, 14, 1200, 1201, 77, 1999], device="cuda")
    w[:, 0] = 1.0
    w[words, 0] = 64.0
    rank = torch.tensor([3, 7, 0, 5, 1, 6, 2, 4], device="cuda")
    w[words, 1] = rank.float() * 2.0 ** -8
    t = torch.randint(0, v, (40,), generator=gen(8), device="cuda")
    t[3] = 1200
    out = mu.linear_logprobs(h.to(dtype), w.to(dtype), t, top=8)
    assert torch.equal(out.top_tokens, words[rank.argsort(descending=True)].expand(40, 8))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_alternatives_side_by_side(dtype):
    """All of the best words in one wave's rows, in one lane's set, and given themselves."""
    v, d, n = 2100, 48, 90
    w = torch.zeros((v, d), device="cuda")
    h = torch.zeros((n, d), device="cuda")
    h[:, 0] = 1.0
    w[:, 0] = -torch.rand(v, generator=gen(9), device="cuda")
    # lane sets: rows of a block in fours, every second four
    one_set = torch.tensor([b + 32 * m + 8 * i + j for b in (256, 1024) for m in range(2) for i in range(4) for j in range(4)], device="cuda")
    side = torch.arange(640, 680, device="cuda")
    for words in (one_set, side):
        x = w.clone()
        x[words, 0] = 1 + torch.rand(len(words), generator=gen(10), device="cuda")
        t = words[torch.arange(n, device="cuda") % len(words)]
        check(h.to(dtype), x.to(dtype), t, top=32, grads=False)


def test_target_outside_the_vocabulary():
    h, w, t = make(70, 500, 64, BF, seed=11)
    good = mu.linear_logprobs(h, w, t, top=3)
    bad = t.clone()
    bad[5], bad[6], bad[7] = 500, -1, 2 ** 40
    out = mu.linear_logprobs(h, w, bad, top=3)
    rest = torch.ones(70, dtype=torch.bool, device="cuda")
    rest[5:8] = False
    assert bool(out.logprobs[5:8].isnan().all()) and torch.equal(out.logprobs[rest], good.logprobs[rest])
    assert torch.equal(out.top_tokens, good.top_tokens)
    o = Oracle(h, w, t)
    within(out.entropy, o.H, o.H_err, "entropy")
    g, e = normal((70,), 12), normal((70,), 13)
    dh, dw = mu.linear_logprobs_grad(h, w, bad, out.stats, grad_logprobs=g, grad_entropy=e)
    oh, eh, ow, ew = o.gradients(torch.where(rest, g, 0.0), e)
    within(dh, oh, eh, "dhidden")
    within(dw, ow, ew, "dweight")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("where", ["all", "all but last", "all but first", "blocks"])
@pytest.mark.parametrize("n", [60, 520, 2600])
def test_ignored_rows_are_never_read(dtype, where, n):
    h, w, t = make(n, 300, 64, dtype, seed=14)
    keep = torch.zeros(n, dtype=torch.bool, device="cuda")
    if where == "all but last":
        keep[-1] = True
    elif where == "all but first":
        keep[0] = True
    elif where == "blocks":
        keep[20:40] = True
        keep[n - 9:n - 7] = True
    t = torch.where(keep, t, -100)
    h2 = torch.where(keep[:, None], h, float("nan"))
    g = torch.where(keep, normal((n,), 15), float("nan"))
    a, b = check(h, w, t, top=4, grads=False), mu.linear_logprobs(h2, w, t, top=4)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    x = mu.linear_logprobs_grad(h, w, t, a.stats, grad_logprobs=g.nan_to_num(), grad_entropy=g.nan_to_num())
    y = mu.linear_logprobs_grad(h2, w, t, torch.where(keep[:, None], b.stats, float("nan")), grad_logprobs=g, grad_entropy=g)
    assert all(torch.equal(p, q) for p, q in zip(x, y)) and not bool(y[0][~keep].any())
    for z in (a.logprobs, a.entropy, a.top_logprobs):
        assert not bool(z[~keep].any())
    assert bool((a.top_tokens[~keep] == -1).all())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_no_tokens(dtype):
    h, w, t = torch.empty((0, 64), device="cuda", dtype=dtype), normal((300, 64), 1).to(dtype), torch.empty(0, device="cuda", dtype=torch.int64)
    out = mu.linear_logprobs(h, w, t, top=3)
    assert out.logprobs.shape == (0,) and out.top_tokens.shape == (0, 3) and out.stats.shape == (0, 4)
    g = torch.empty(0, device="cuda")
    dh, dw = mu.linear_logprobs_grad(h, w, t, out.stats, grad_logprobs=g, dweight=torch.full_like(w, float("nan")))
    assert dh.shape == (0, 64) and not bool(dw.any())
    assert mu.linear_logprobs_grad(h, w, t, out.stats, grad_logprobs=g, dweight=False)[0].shape == (0, 64)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,v,d,pad,shift", [(70, 333, 64, 8, 0), (70, 333, 64, 3, 0), (130, 257, 128, 5, 1), (9, 600, 40, 1, 3)])
def test_strides_and_alignment(dtype, n, v, d, pad, shift):
    """Rows inside wider buffers, starts off 16 bytes, NaN all around."""
    h, w, t = make(n, v, d, dtype, seed=16)

    def inside(x):
        buf = torch.full((x.shape[0] * (d + pad) + shift + 64,), float("nan"), device="cuda", dtype=dtype)
        y = buf[shift:shift + x.shape[0] * (d + pad)].view(x.shape[0], d + pad)[:, :d]
        y.copy_(x)
        return buf, y

    (_, h2), (_, w2) = inside(h), inside(w)
    a, b = check(h, w, t, top=5, grads=False), mu.linear_logprobs(h2, w2, t, top=5)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    bh, dh = inside(torch.zeros_like(h))
    bw, dw = inside(torch.zeros_like(w))
    nan = int(bh.isnan().sum()), int(bw.isnan().sum())
    g, e = normal((n,), 17), normal((n,), 18)
    mu.linear_logprobs_grad(h2, w2, t, b.stats, grad_logprobs=g, grad_entropy=e, dhidden=dh, dweight=dw)
    ref = mu.linear_logprobs_grad(h, w, t, a.stats, grad_logprobs=g, grad_entropy=e)
    assert nan == (int(bh.isnan().sum()), int(bw.isnan().sum()))
    assert torch.equal(dh, ref[0]) and torch.equal(dw, ref[1])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("spread", [1e-3, 50.0, 1000.0])
def test_logit_ranges(dtype, spread):
    """Logits far apart: exponentials of whole tiles vanish, and the alternatives behind a sure one are in order."""
    h, w, t = make(150, 900, 64, dtype, seed=19, learnt=0.0)
    check((h.float() * spread).to(dtype), w, t, top=12)
    h, w, t = make(150, 900, 64, dtype, seed=20, learnt=spread)
    check(h, w, t, top=12)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("softcap", [0.02, 1.0, 30.0, 1e5])
def test_soft_caps(dtype, softcap):
    h, w, t = make(150, 900, 64, dtype, seed=21)
    check(h, w, t, top=6, softcap=softcap)


@pytest.mark.parametrize("n", [3, 150])
@pytest.mark.parametrize("low", [-float("inf"), -3e38])
def test_masked_words(n, low):
    """Words whose logit is minus infinity, or as low as 32 bits go: no part of the sums; behind every other word, or
    no alternative at all."""
    v, d = 700, 32
    h, w, t = make(n, v, d, F32, seed=22)
    h[:, 0], w[:, 0] = 1.0, 0.0
    words = torch.randperm(v, generator=gen(23), device="cuda")
    masked, kept = words[20:], words[:20].sort().values
    place = torch.full((v,), -1, device="cuda")
    place[kept] = torch.arange(20, device="cuda")
    t = kept[torch.arange(n, device="cuda") % 20]
    small = mu.linear_logprobs(h, w[kept], place[t], top=20)
    w2 = w.clone()
    w2[masked, 0] = low
    out = mu.linear_logprobs(h, w2, t, top=32)
    o = Oracle(h, w[kept], place[t])
    within(out.logprobs, o.logp, o.each, "logprobs")
    within(out.entropy, o.H, o.H_err, "entropy")
    assert torch.equal(out.top_tokens[:, :20], kept[small.top_tokens])
    if low == -float("inf"):
        assert bool((out.top_tokens[:, 20:] == -1).all()) and bool((out.top_logprobs[:, 20:] == low).all())
    else:
        assert bool((out.top_logprobs[:, 20:] <= -2e38).all()) and bool(torch.isfinite(out.top_logprobs).all())
        assert bool((place[out.top_tokens[:, 20:]] == -1).all())
    masked_target = torch.full((n,), int(masked[0]), device="cuda")
    assert bool((mu.linear_logprobs(h, w2, masked_target).logprobs <= -2e38).all())


@pytest.mark.parametrize("n", [2, 90])
def test_infinite_logits_under_a_soft_cap(n):
    """They count as the cap, and come first, by rising token: several of them in one lane's set, and one given."""
    v, d, cap = 900, 16, 5.0
    h, w, t = make(n, v, d, F32, seed=47)
    h[:, 0] = 1.0
    words = torch.tensor([256, 257, 264, 290, 400, 777], device="cuda")
    raw = mm(h.double(), w.double().t())
    w[words, 0] = float("inf")
    raw[:, words] = float("inf")
    t[0] = 264
    out = mu.linear_logprobs(h, w, t, top=9, softcap=cap)
    assert torch.equal(out.top_tokens, raw.sort(dim=1, descending=True, stable=True).indices[:, :9])
    z = cap * torch.tanh(raw / cap)
    lp = torch.log_softmax(z, 1)
    err = (512 + v / 64 + 40) * U + 12 * U * cap + 2 * (d + 2) * U * mm(h.abs().double(), w.nan_to_num(0, 0, 0).abs().double().t()).amax(1)
    within(out.logprobs, lp.gather(1, t[:, None])[:, 0], err + 12 * U * cap, "logprobs")
    within(out.top_logprobs, lp.gather(1, out.top_tokens), (err + 12 * U * cap)[:, None], "top_logprobs")


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_bad_hidden_row(value):
    h, w, t = make(100, 800, 64, BF, seed=24)
    good = mu.linear_logprobs(h, w, t, top=4)
    h2 = h.clone()
    h2[33, 7] = value
    out = mu.linear_logprobs(h2, w, t, top=4)
    rest = torch.arange(100, device="cuda") != 33
    for a, b in zip(out, good):
        assert torch.equal(a[rest], b[rest])
    assert bool(out.logprobs[33].isnan()) and bool(out.entropy[33].isnan())
    assert out.top_tokens[33].tolist() == [-1] * 4 and bool(out.top_logprobs[33].isnan().all())


@pytest.mark.parametrize("n", [5, 200, 3000])
def test_a_token_does_not_depend_on_its_batch_and_calls_repeat(n):
    h, w, t = make(n, 2000, 96, BF, seed=25)
    a, b = mu.linear_logprobs(h, w, t, top=8), mu.linear_logprobs(h, w, t, top=8)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    g = normal((n,), 26)
    x, y = (mu.linear_logprobs_grad(h, w, t, a.stats, grad_logprobs=g, grad_entropy=g) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(x, y))
    assert torch.equal(mu.linear_logprobs(h[:1], w, t[:1], top=8).top_tokens, a.top_tokens[:1])
    assert torch.equal(mu.linear_logprobs(h, w, t, top=3).top_tokens, a.top_tokens[:, :3])


def test_agrees_with_the_cross_entropy():
    h, w, t = make(300, 3000, 128, BF, seed=27, ignored=0.2)
    out = mu.linear_logprobs(h, w, t)
    loss = mu.linear_cross_entropy(h, w, t, reduction="none")
    # (both are within `each` of the value: they join the tiles' sums in another order)
    within(out.logprobs, -loss.double(), 2 * Oracle(h, w, t).each, "logprobs")


def test_autograd():
    h, w, t = make(120, 700, 64, F32, seed=28, ignored=0.1)
    gl, ge = normal((4, 30), 29), normal((4, 30), 30)
    x, y = h.view(4, 30, 64).clone().requires_grad_(), w.clone().requires_grad_()
    out = mu.linear_logprobs(x, y, t.view(4, 30), top=2, softcap=9.0)
    assert out.logprobs.requires_grad and out.entropy.requires_grad and not out.top_logprobs.requires_grad and not out.stats.requires_grad
    assert out.top_tokens.shape == (4, 30, 2) and out.stats.shape == (4, 30, 4)
    got = torch.autograd.grad([out.logprobs, out.entropy], [x, y], [gl, ge], retain_graph=True)
    want = mu.linear_logprobs_grad(h, w, t, out.stats, grad_logprobs=gl.view(-1), grad_entropy=ge.view(-1), softcap=9.0)
    assert torch.equal(got[0].view(120, 64), want[0]) and torch.equal(got[1], want[1])
    # one result alone, with a broadcast gradient; one input alone
    (a,) = torch.autograd.grad(out.entropy.sum(), [y], retain_graph=True)
    b = mu.linear_logprobs_grad(h, w, t, out.stats, grad_entropy=torch.ones(120, device="cuda"), softcap=9.0, dhidden=False)
    assert b[0] is None and torch.equal(a, b[1])
    out = mu.linear_logprobs(x, w, t.view(4, 30))
    (a,) = torch.autograd.grad(out.logprobs.mean(), [x])
    assert a.shape == x.shape and bool(torch.isfinite(a).all())
    with torch.no_grad():
        assert not mu.linear_logprobs(x, y, t.view(4, 30)).logprobs.requires_grad


def test_gradient_by_differences():
    """Central differences of 64-bit values along random directions: the formula's gradient, which the kernels' are held
    to elsewhere, and theirs (fp32: within their own bounds' share)."""
    h, w, t = make(60, 400, 48, F32, seed=31)
    out = mu.linear_logprobs(h, w, t, softcap=8.0)
    gl, ge = normal((60,), 32), normal((60,), 33)
    dh, dw = mu.linear_logprobs_grad(h, w, t, out.stats, grad_logprobs=gl, grad_entropy=ge, softcap=8.0)

    def value(a, b):
        z = 8.0 * torch.tanh(mm(a, b.t()) / 8.0)
        lp = torch.log_softmax(z, 1)
        return float((gl * lp.gather(1, t[:, None])[:, 0]).sum() + (ge * -(lp.exp() * lp).sum(1)).sum())

    for name, x, g in (("hidden", h, dh), ("weight", w, dw)):
        way, e = normal(x.shape, 34).double(), 1e-6
        at = lambda k: value(h.double() + (k * way if name == "hidden" else 0), w.double() + (k * way if name == "weight" else 0))
        slope = (at(e) - at(-e)) / (2 * e)
        mine = float((g.double() * way).sum())
        assert abs(slope - mine) <= 2e-5 * float((g.double() * way).abs().sum()), (name, slope, mine)


def test_in_a_graph_and_beside_other_calls():
    h, w, t = make(300, 1000, 128, BF, seed=35, ignored=0.1)
    big = make(3000, 1500, 128, BF, seed=36)
    g, e = normal((300,), 37), normal((300,), 38)
    handle, s = mu.Handle(), torch.cuda.Stream()
    hs = h.clone()

    def call():
        out = mu.linear_logprobs(hs, w, t, top=6, handle=handle)
        return (*out, *mu.linear_logprobs_grad(hs, w, t, out.stats, grad_logprobs=g, grad_entropy=e, handle=handle))

    with torch.cuda.stream(s):
        call()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            captured = call()
        for k in range(4):
            hs.copy_(h * (1 + k / 4))
            for x in captured:
                x.fill_(-7)
            graph.replay()
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(captured, call())), k
            mu.linear_cross_entropy_grad(*big, handle=handle)          # the same workspace, which it outgrows
    s.synchronize()
    handle.close()


def test_one_token_in_a_graph():
    h, w, t = make(1, 50304, 768, BF, seed=39)
    handle, s = mu.Handle(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        mu.linear_logprobs(h, w, t, top=8, handle=handle)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = mu.linear_logprobs(h, w, t, top=8, handle=handle)
        for k in range(3):
            h.copy_(normal((1, 768), 40 + k, 2.0))
            t.fill_(11 * k)
            graph.replay()
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, mu.linear_logprobs(h, w, t, top=8, handle=handle))), k
    s.synchronize()
    handle.close()


def test_several_pieces():
    """More tokens than a gibibyte of statistics or of logits' gradients holds."""
    h, w, t = make(520, 1 << 22, 16, BF, seed=41, learnt=4.0)
    t[100:110] = -100
    out = mu.linear_logprobs(h, w, t, top=5)
    rows = torch.tensor([0, 99, 105, 255, 256, 511, 512, 519], device="cuda")
    Oracle(h[rows], w, t[rows]).check(mu.LogProbs(*(x[rows] for x in out)), 5)
    h, w, t = make(600, 1 << 20, 16, BF, seed=42, learnt=4.0)
    t[100:110] = -100
    out = mu.linear_logprobs(h, w, t)
    g, e = normal((600,), 43), normal((600,), 44)
    dh, dw = mu.linear_logprobs_grad(h, w, t, out.stats, grad_logprobs=g, grad_entropy=e)
    oh, eh, ow, ew = Oracle(h, w, t).gradients(g, e)
    within(dh, oh, eh, "dhidden")
    within(dw, ow, ew, "dweight")


def test_refusals():
    h, w, t = make(10, 50, 64, BF, seed=45)
    out = mu.linear_logprobs(h, w, t)
    g = normal((10,), 46)
    grad = lambda *a, **kw: mu.linear_logprobs_grad(*a, **{**dict(grad_logprobs=g), **kw})
    bad = [
        lambda: mu.linear_logprobs(h, w.float(), t),
        lambda: mu.linear_logprobs(h, w[:, :32], t),
        lambda: mu.linear_logprobs(h, w, t[:9]),
        lambda: mu.linear_logprobs(h, w.view(5, 10, 64), t),
        lambda: mu.linear_logprobs(h, w, t.to(torch.int16)),
        lambda: mu.linear_logprobs(h, w, t, softcap=-1.0),
        lambda: mu.linear_logprobs(h, w, t, softcap=float("nan")),
        lambda: mu.linear_logprobs(h, w, t, top=-1),
        lambda: mu.linear_logprobs(h, w, t, top=33),
        lambda: mu.linear_logprobs(h, w[:5], t, top=6),
        lambda: mu.linear_logprobs(h.half(), w.half(), t),
        lambda: mu.linear_logprobs(h.t().contiguous().t(), w, t),
        lambda: mu.linear_logprobs(h, w, t.cpu()),
        lambda: mu.linear_logprobs(h.cpu(), w.cpu(), t.cpu()),
        lambda: grad(h, w, t, out.stats, grad_logprobs=None),
        lambda: grad(h, w, t, out.stats, grad_logprobs=g[:9]),
        lambda: grad(h, w, t, out.stats, grad_logprobs=g.to(BF)),
        lambda: grad(h, w, t, out.stats, grad_entropy=g.cpu()),
        lambda: grad(h, w, t, out.stats[:9]),
        lambda: grad(h, w, t, out.stats.double()),
        lambda: grad(h, w, t, out.stats, dhidden=h),
        lambda: grad(h, w, t, out.stats, dweight=w),
        lambda: grad(h, w, t, out.stats, dweight=w.float()),
        lambda: grad(h, w, t, out.stats, dhidden=False, dweight=False),
        lambda: grad(h, w, t, out.stats, dhidden=torch.empty((9, 64), device="cuda", dtype=BF)),
    ]
    keep = h.clone(), w.clone()
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            f()
            pytest.fail(f"call {i} was accepted")
    torch.cuda.synchronize()
    assert torch.equal(h, keep[0]) and torch.equal(w, keep[1])
