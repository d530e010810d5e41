"""Training-step operators on the GPU against plain 64-bit implementations.

Tolerances are element-wise bounds derived from the arithmetic, not fitted:

* logits: a fp32 sum of D products (exact for bf16 inputs) is within
  dz = (D + 2) u sum_k |h_k w_k|, u = 2^-24;
* loss: two logits (2 dz), a sum of exponentials of at most 512 serial
  additions and one per tile, and the rounding of references up to |lse|;
* the logits' gradient is relative to 2 (dz + loss terms) and, in bf16, one
  rounding (2^-8, unit roundoff 2^-8 / 2 doubled for the kept exponential's
  own 2^-11) of each term;
* the gradients are sums of K such terms: that relative error plus K u times
  the sum of absolute products, and the output's rounding.
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


def oracle(h, w, t, ignore, reduction, softcap, grad_out=None):
    """Loss, gradients and their element-wise error bounds, in 64 bits."""
    bf = h.dtype == BF
    valid = t != ignore
    h64 = torch.where(valid[:, None], h.double(), 0.0)
    w64 = w.double()
    D, V = w.shape[1], w.shape[0]
    raw = mm(h64, w64.t())
    z = softcap * torch.tanh(raw / softcap) if softcap else raw
    at = torch.where(valid, t, 0)[:, None].long()
    lse = torch.logsumexp(z, 1)
    zt = z.gather(1, at)[:, 0]
    # the other words' mass against the target's, without the difference of two
    # large logarithms: even 64 bits lose a confident token's loss in it
    others = torch.logsumexp((z - zt[:, None]).scatter(1, at, float("-inf")), 1)
    each = torch.where(valid, torch.logaddexp(others, torch.zeros_like(others)), 0.0)
    n = int(valid.sum())
    g = torch.ones_like(each) if grad_out is None else grad_out.double().expand_as(each).clone()
    if reduction == "mean":
        g = g / max(n, 1)
    g = torch.where(valid, g, 0.0)
    dz_err = (D + 2) * U * mm(h64.abs(), w64.abs().t()).amax(1) if V else 0
    # tanh and the product around it: a few roundings of a value up to the cap
    dz_err = dz_err + (8 * U * softcap if softcap else 0)
    each_err = torch.where(valid, 2 * dz_err + (512 + V / 64) * U + 4 * U * (lse.abs() + zt.abs() + z.abs().amax(1)), 0.0)
    p = torch.exp(z - lse[:, None])
    q = p.clone()
    q.scatter_(1, at, -torch.sigmoid(others)[:, None])
    f = 1 - (z / softcap) ** 2 if softcap else torch.ones((), dtype=torch.float64, device=h.device)
    s = q * f * g[:, None]
    rel = 2 * each_err[:, None] + 16 * U + (2.0 ** -8 + 2.0 ** -11 if bf else 0)
    s_err = s.abs() * rel + g.abs()[:, None] * 2.0 ** -62
    if softcap:
        back = 2.0 ** -11 if bf else 4 * U * (2 + z.abs() + lse.abs()[:, None])
        s_err = s_err + (q * g[:, None]).abs() * 4 * (back + dz_err[:, None]) / softcap
    dh, dw = mm(s, w64), mm(s.t(), h64)
    out = 2.0 ** -8 if bf else 2 * U
    dh_err = mm(s_err + (V + 8) * U * s.abs(), w64.abs()) + out * dh.abs() + 1e-38
    dw_err = mm((s_err + (len(t) + 8) * U * s.abs()).t(), h64.abs()) + out * dw.abs() + 1e-38
    if reduction == "none":
        loss, loss_err = each, each_err
    else:
        k = max(n, 1) if reduction == "mean" else 1
        loss, loss_err = each.sum() / k, each_err.sum() / k + 2 * U * each.abs().sum() / k
    return loss, loss_err + 1e-38, dh, dh_err, dw, dw_err


def within(got, want, err, what):
    got = got.double()
    bad = ~((got - want).abs() <= err)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, worst {float(((got - want).abs() / err).max()):.3g}x")


def check_loss(h, w, t, ignore=-100, reduction="mean", softcap=0.0, grad_out=None, **kw):
    loss, dh, dw = mu.linear_cross_entropy_grad(h, w, t, ignore_index=ignore, reduction=reduction, softcap=softcap,
                                                grad_out=grad_out, **kw)
    only = mu.linear_cross_entropy(h, w, t, ignore_index=ignore, reduction=reduction, softcap=softcap)
    ol, el, oh, eh, ow, ew = oracle(h, w, t, ignore, reduction, softcap, grad_out)
    assert loss.dtype == F32 and loss.shape == ol.shape and dh.dtype == h.dtype and dw.dtype == w.dtype
    within(loss, ol, el, "loss")
    within(only, ol, el, "loss alone")
    within(dh, oh, eh, "dhidden")
    within(dw, ow, ew, "dweight")
    return loss, dh, dw


def make(n, v, d, dtype, seed=0, learnt=12.0, ignored=0.0, ignore=-100):
    w = normal((v, d), seed * 7 + 1, 1 / math.sqrt(d))
    t = torch.randint(0, v, (n,), generator=gen(seed * 7 + 2), device="cuda")
    h = normal((n, d), seed * 7 + 3) + learnt * torch.rand((n, 1), generator=gen(seed * 7 + 4), device="cuda") * w[t]
    if ignored:
        t[torch.rand(n, generator=gen(seed * 7 + 5), device="cuda") < ignored] = ignore
    return h.to(dtype), w.to(dtype), t


SHAPES = [(1, 1, 1), (1, 2, 3), (2, 63, 8), (3, 64, 31), (17, 65, 64), (63, 255, 33), (64, 256, 96), (65, 257, 128),
          (127, 511, 192), (128, 1000, 65), (255, 300, 64), (256, 512, 256), (257, 1025, 320), (300, 5003, 768),
          (1, 50304, 768), (5, 20000, 200), (700, 777, 1030), (1100, 640, 64), (33, 4099, 2048)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,v,d", SHAPES)
def test_cross_entropy_shapes(n, v, d, dtype):
    check_loss(*make(n, v, d, dtype, seed=n + v + d))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("softcap", [0.0, 15.0])
def test_cross_entropy_options(dtype, reduction, softcap):
    h, w, t = make(211, 1003, 160, dtype, seed=3, ignored=0.3, ignore=7)
    go = None
    if reduction == "none":
        go = normal((211,), 11)
    elif reduction == "sum":
        go = torch.tensor(0.37, device="cuda")
    check_loss(h, w, t.to(torch.int32), ignore=7, reduction=reduction, softcap=softcap, grad_out=go)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("softcap", [1e-40, 0.02, 1.0, 5.0, 30.0, 1e3, 1e5, 1e6, 1e8, 1e30, 3e38])
@pytest.mark.parametrize("n,v,d", [(1, 3000, 64), (150, 900, 64)])
def test_cross_entropy_soft_cap_of_any_size(n, v, d, softcap, dtype):
    """A capped logit is off by the raw one's error and a dozen roundings of itself, not of the cap: one for the
    product with 1 / cap and for that value, at most four of a quotient's two sides, two of a reciprocal, one of each
    product after it (and, where exp(-2 x) is taken, x below 1 in it for each rounding of its argument)."""
    h, w, t = make(n, v, d, dtype, seed=17)
    raw = mm(h.double(), w.double().t())
    cap = float(torch.tensor(softcap, dtype=F32))
    z = cap * torch.tanh(raw / cap)
    zt = z.gather(1, t[:, None])[:, 0]
    others = torch.logsumexp((z - zt[:, None]).scatter(1, t[:, None], float("-inf")), 1)
    want = torch.logaddexp(others, torch.zeros_like(others))
    dz = (d + 2) * U * mm(h.double().abs(), w.double().abs().t()).amax(1) + 12 * U * z.abs().amax(1)
    err = 2 * dz + (512 + v / 64) * U + 4 * U * (torch.logsumexp(z, 1).abs() + zt.abs() + z.abs().amax(1))
    within(mu.linear_cross_entropy(h, w, t, reduction="none", softcap=softcap), want, err, "loss alone")
    within(mu.linear_cross_entropy_grad(h, w, t, reduction="none", softcap=softcap)[0], want, err, "loss")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("cap", [1e8, 1e16, 1e30])
@pytest.mark.parametrize("spread", [0.025, 1e-6])
def test_cross_entropy_huge_logits_under_a_huge_soft_cap(cap, spread, dtype):
    """Around the place where the cap's two forms meet, which may differ by more than a logit's spacing there: results
    stay finite, and every token's gradients sum to nothing (their roundings: 2^-8 and 2^-11 of each in bf16)."""
    n, v = 40, 700
    h = (cap * (0.625 + spread * (2 * torch.rand((n, v), generator=gen(38), device="cuda") - 1))).to(dtype)
    t = torch.randint(0, v, (n,), generator=gen(39), device="cuda")
    w = torch.eye(v, device="cuda").to(dtype)
    loss, dz, _ = mu.linear_cross_entropy_grad(h, w, t, reduction="none", softcap=cap)
    only = mu.linear_cross_entropy(h, w, t, reduction="none", softcap=cap)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(dz).all()) and bool((only >= 0).all())
    # every probability is in [0, 1] and a slope in [0.66, 0.71] (tanh^2 of 0.6 to 0.65)
    x = dz.double() / (1 - torch.tanh(h.double() / cap) ** 2)
    assert bool((x.abs() <= 1.02).all())
    assert bool((x.sum(1).abs() <= x.abs().sum(1) * (2.0 ** -7 + 16 * U) + 1e-6).all())


@pytest.mark.parametrize("first,cap", [(547008118784.0, 1e12), (273504059392.0, 5e11), (8962170817609728.0, 1e16)])
def test_cross_entropy_huge_logits_whose_caps_fall(first, cap):
    """Neighbouring 32-bit logits, whose capped values, a rounding each, need not rise with them and are thousands
    apart: the largest logit's exponential still bounds the others'."""
    n, v = 400, 200
    low = torch.full((n,), first, device="cuda").view(torch.int32) + torch.arange(n, device="cuda", dtype=torch.int32)
    h = low.view(F32)[:, None].repeat(1, v)
    h[:, 5::16] = (low + 1).view(F32)[:, None]        # some in every wave's rows
    t = torch.full((n,), 7, device="cuda")
    w = torch.eye(v, device="cuda")
    loss, dz, _ = mu.linear_cross_entropy_grad(h, w, t, reduction="none", softcap=cap)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(dz).all()) and bool((dz.abs() <= 1.0).all())
    assert bool(torch.isfinite(mu.linear_cross_entropy(h, w, t, reduction="none", softcap=cap)).all())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("softcap", [1.0, 5.0, 30.0, 1000.0])
@pytest.mark.parametrize("v", [96, 640])
def test_cross_entropy_soft_cap_slope_of_saturated_logits(v, softcap, dtype):
    """The weight is the identity, so dhidden is the logits' gradient itself, value by value, of raw logits (exact) up
    to 6.5 caps. Its bound has no absolute part but that of a kept exponential of 2^-63 and less: the cap as above; the
    slope 4 e / (1 + e)^2, e = exp(-2 x), with 4 roundings of x twice in its exponent and 8 of its own; the
    probability as in the other tests; in bf16 the kept value's 2^-11 and a rounding, and the output's."""
    n = 70
    cap = softcap
    h = (cap * 13 * (torch.rand((n, v), generator=gen(18), device="cuda") - 0.5)).to(dtype)
    t = torch.randint(0, v, (n,), generator=gen(19), device="cuda")
    w = torch.eye(v, device="cuda").to(dtype)
    raw = h.double()
    z = cap * torch.tanh(raw / cap)
    lse = torch.logsumexp(z, 1)
    zt = z.gather(1, t[:, None])[:, 0]
    others = torch.logsumexp((z - zt[:, None]).scatter(1, t[:, None], float("-inf")), 1)
    q = torch.exp(z - lse[:, None]).scatter(1, t[:, None], -torch.sigmoid(others)[:, None])
    want = q / torch.cosh(raw / cap) ** 2
    x = (raw / cap).abs()
    each = 24 * U * z.abs().amax(1) + (512 + v / 64) * U + 4 * U * (lse.abs() + zt.abs() + z.abs().amax(1))
    rel = 2 * each[:, None] + 16 * U + (8 * x + 8) * U + (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -8 if dtype == BF else 2 * U)
    got = mu.linear_cross_entropy_grad(h, w, t, reduction="sum", softcap=softcap, dweight=False)[1]
    within(got, want, want.abs() * rel * (1 + 2.0 ** -7) + 2.0 ** -62, "dhidden")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("where", ["all", "all but last", "all but first", "blocks"])
def test_cross_entropy_ignored_rows_are_never_read(dtype, where):
    h, w, t = make(520, 300, 64, dtype, seed=5)
    keep = torch.zeros(520, dtype=torch.bool, device="cuda")
    if where == "all but last":
        keep[-1] = True
    elif where == "all but first":
        keep[0] = True
    elif where == "blocks":
        keep[64:128] = True
        keep[300:301] = True
    t = torch.where(keep, t, -100)
    clean = check_loss(h, w, t)
    h2 = torch.where(keep[:, None], h, float("nan"))
    h2[~keep, 0] = float("inf")
    dirty = mu.linear_cross_entropy_grad(h2, w, t)
    for a, b in zip(clean, dirty):
        assert torch.equal(a, b)
    assert not bool(dirty[1][~keep].any())
    if where == "all":
        assert float(dirty[0]) == 0.0 and not bool(dirty[2].any())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_cross_entropy_no_tokens(dtype):
    h, w, t = torch.empty((0, 64), device="cuda", dtype=dtype), normal((300, 64), 1).to(dtype), torch.empty(
        0, device="cuda", dtype=torch.int64)
    dw = torch.full((300, 64), float("nan"), device="cuda", dtype=dtype)
    loss, dh, _ = mu.linear_cross_entropy_grad(h, w, t, dweight=dw)
    assert float(loss) == 0.0 and dh.shape == (0, 64) and not bool(dw.any())
    assert mu.linear_cross_entropy(h, w, t, reduction="none").shape == (0,)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_cross_entropy_no_tokens_and_one_gradient(dtype, reduction):
    """An empty batch whose only gradient has no elements (a frozen head), or only the weight's."""
    h, w, t = torch.empty((0, 64), device="cuda", dtype=dtype), normal((300, 64), 1).to(dtype), torch.empty(
        0, device="cuda", dtype=torch.int64)
    shape = (0,) if reduction == "none" else ()
    for got in (mu.linear_cross_entropy(h, w, t, reduction=reduction),
                mu.linear_cross_entropy_grad(h, w, t, reduction=reduction, dweight=False)[0],
                mu.linear_cross_entropy_grad(h, w, t, reduction=reduction, dhidden=False)[0]):
        assert got.shape == shape and not bool(got.any())
    assert not bool(mu.linear_cross_entropy_grad(h, w, t, reduction=reduction, dhidden=False)[2].any())
    loss = mu.linear_cross_entropy(h.requires_grad_(), w, t, reduction=reduction)
    loss.sum().backward()
    assert loss.shape == shape and h.grad.shape == (0, 64)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,v,d,pad,shift", [(70, 333, 64, 8, 0), (70, 333, 64, 3, 0), (130, 257, 128, 5, 1), (9, 600, 40, 1, 3)])
def test_cross_entropy_strides_and_alignment(dtype, n, v, d, pad, shift):
    """Rows inside wider buffers, starts off 16 bytes, NaN all around."""
    h, w, t = make(n, v, d, dtype, seed=9)

    def inside(x):
        buf = torch.full((x.shape[0] * (d + pad) + shift + 64,), float("nan"), device="cuda", dtype=dtype)
        y = buf[shift:shift + x.shape[0] * (d + pad)].view(x.shape[0], d + pad)[:, :d]
        y.copy_(x)
        return buf, y

    (_, h2), (_, w2) = inside(h), inside(w)
    bh, dh = inside(torch.zeros_like(h))
    bw, dw = inside(torch.zeros_like(w))
    nan_h, nan_w = int(bh.isnan().sum()), int(bw.isnan().sum())
    loss, _, _ = check_loss(h2, w2, t, dhidden=dh, dweight=dw)
    assert int(bh.isnan().sum()) == nan_h and int(bw.isnan().sum()) == nan_w
    ref = mu.linear_cross_entropy_grad(h, w, t)
    assert torch.equal(loss, ref[0]) and torch.equal(dh, ref[1]) and torch.equal(dw, ref[2])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("spread", [1e-3, 50.0, 1000.0])
def test_cross_entropy_logit_ranges(dtype, spread):
    """Logits far apart: exponentials of whole tiles vanish; a token sure of its target keeps a relative gradient."""
    h, w, t = make(150, 900, 64, dtype, seed=13, learnt=0.0)
    check_loss((h.float() * spread).to(dtype), w, t)
    h, w, t = make(150, 900, 64, dtype, seed=14, learnt=spread)
    check_loss(h, w, t, reduction="sum")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("log2", [20, 25, 30, 37, 60, 120])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("n,v", [(1, 300), (70, 20000)])
def test_cross_entropy_of_huge_logits(n, v, sign, log2, dtype):
    """Logits that 32 bits hold exactly, up to three spacings apart and in every tile: each difference is exact, so
    the loss and probabilities are as good as those of small logits."""
    step = max(1.0, 2.0 ** (log2 - 23))
    k = torch.randint(0, 4, (v,), generator=gen(28), device="cuda") * (torch.rand(v, generator=gen(29), device="cuda") < 0.02)
    t = torch.randint(0, v, (n,), generator=gen(30), device="cuda")
    half = log2 // 2
    h = torch.zeros((n, 8), device="cuda")
    h[:, 0], h[:, 5] = 2.0 ** (log2 - half), 1.0
    w = torch.zeros((v, 8), device="cuda")
    w[:, 0], w[:, 5] = sign * 2.0 ** half, k * step
    h, w = h.to(dtype), w.to(dtype)
    z = mm(h.double(), w.double().t())
    assert torch.equal(z, z.float().double())
    zt = z.gather(1, t[:, None])[:, 0]
    others = torch.logsumexp((z - zt[:, None]).scatter(1, t[:, None], float("-inf")), 1)
    each = torch.logaddexp(others, torch.zeros_like(others))
    err = (512 + v / 64) * U + 8 * U * each
    loss, _, dw = mu.linear_cross_entropy_grad(h, w, t, reduction="none", dhidden=None)
    within(loss, each, err, "loss")
    within(mu.linear_cross_entropy(h, w, t, reduction="none"), each, err, "loss alone")
    p = torch.exp(z - zt[:, None] - each[:, None]).scatter(1, t[:, None], -torch.sigmoid(others)[:, None])
    rel = 2 * err[:, None] + 16 * U + (2.0 ** -8 + 2.0 ** -11 if dtype == BF else 0)
    want = p.sum(0)                                   # the gradient of the last column's weights
    bound = (p.abs() * (rel + (n + 8) * U) + 2.0 ** -62).sum(0) + (2.0 ** -8 if dtype == BF else 2 * U) * want.abs()
    within(dw[:, 5], want, bound, "dweight")


def test_cross_entropy_target_out_of_range():
    h, w, t = make(100, 300, 64, BF, seed=15)
    good = mu.linear_cross_entropy_grad(h, w, t, reduction="none")
    for bad in (300, -1, 2 ** 40, -2 ** 62):
        t2 = t.clone()
        t2[17] = bad
        loss, dh, dw = mu.linear_cross_entropy_grad(h, w, t2, reduction="none")
        assert bool(loss[17].isnan()) and not bool(dh[17].any()) and bool(torch.isfinite(dw).all())
        keep = torch.arange(100, device="cuda") != 17
        assert torch.equal(loss[keep], good[0][keep]) and torch.equal(dh[keep], good[1][keep])


def test_cross_entropy_non_finite_values_stay_visible():
    h, w, t = make(100, 300, 64, BF, seed=16)
    h2 = h.clone()
    h2[3, 5] = float("nan")
    loss, dh, dw = mu.linear_cross_entropy_grad(h2, w, t, reduction="none")
    good = mu.linear_cross_entropy_grad(h, w, t, reduction="none")
    assert bool(loss[3].isnan()) and bool(dh[3].isnan().all()) and bool(dw.isnan().all())
    keep = torch.arange(100, device="cuda") != 3
    assert torch.equal(loss[keep], good[0][keep]) and torch.equal(dh[keep], good[1][keep])
    w2 = w.clone()
    w2[250] = float("inf")
    assert not bool(torch.isfinite(mu.linear_cross_entropy(h, w2, t)))


@pytest.mark.parametrize("n,v,d,dtype", [(600, 1 << 20, 32, BF), (13000, 50000, 40, BF), (1200, 300000, 24, F32)])
def test_cross_entropy_in_pieces(n, v, d, dtype):
    """More tokens than one piece holds: the weight's gradient is summed over pieces."""
    check_loss(*make(n, v, d, dtype, seed=21, ignored=0.2), reduction="sum")


@pytest.mark.parametrize("n,v,d,dtype", [
    (1500, 300, 72, BF), (1500, 300, 72, F32), (2100, 257, 33, F32), (5000, 200, 64, BF), (70000, 200, 32, BF),
    (66000, 210, 40, F32)])
def test_cross_entropy_of_many_tokens_and_a_small_weight(n, v, d, dtype):
    """The weight's gradient is summed over the tokens in parts (past 65536 tokens in pieces too)."""
    check_loss(*make(n, v, d, dtype, seed=24, ignored=0.2))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,v,d,ignored", [(1, 700, 64, 0.0), (2, 257, 72, 0.5), (31, 5000, 768, 0.3), (33, 300, 200, 0.6),
                                           (63, 30000, 128, 0.4), (64, 50304, 768, 0.2), (64, 1000, 40, 0.0),
                                           (65, 1000, 40, 0.3)])
def test_cross_entropy_of_few_tokens(n, v, d, ignored, dtype):
    """The loss alone of up to 64 tokens reads their rows in place: those of a wider buffer too, never the ignored ones."""
    h, w, t = make(n, v, d, dtype, seed=25, ignored=ignored)
    check_loss(h, w, t, reduction="none")
    wide = torch.full((n, d + 24), float("nan"), device="cuda", dtype=dtype)
    wide[:, 8:8 + d] = h
    wide[t == -100] = float("nan")
    for reduction in ("none", "mean"):
        want = mu.linear_cross_entropy(h, w, t, reduction=reduction)
        assert torch.equal(mu.linear_cross_entropy(wide[:, 8:8 + d], w, t, reduction=reduction), want)
        assert torch.equal(mu.linear_cross_entropy(h, w, t.int(), reduction=reduction), want)
    none = torch.full_like(t, -100)
    assert mu.linear_cross_entropy(wide[:, 8:8 + d], w, none).item() == 0.0
    assert not mu.linear_cross_entropy(wide[:, 8:8 + d], w, none, reduction="none").any()
    t[0] = v                       # outside the vocabulary
    assert bool(mu.linear_cross_entropy(h, w, t, reduction="none")[0].isnan())


@pytest.mark.parametrize("n", [1, 64, 128, 129])
def test_cross_entropy_of_few_tokens_and_a_large_vocabulary(n):
    """Either side of the tokens from which the widest tiles are taken, at a vocabulary that has many of them."""
    h, w, t = make(n, 250001, 64, BF, seed=36)
    check_loss(h, w, t, reduction="none")


@pytest.mark.parametrize("n,v,d,pad,words,softcap", [
    (65, 3000, 64, 0, 3000, 0.0), (64, 3000, 64, 0, 3000, 0.0), (300, 5003, 136, 0, 40, 0.0), (300, 5003, 129, 3, 5003, 20.0),
    (1000, 200, 72, 0, 200, 0.0), (5000, 300, 64, 0, 1, 0.0), (5000, 300, 40, 5, 300, 0.0), (9000, 40000, 256, 0, 40000, 0.0),
    (9000, 40000, 256, 1, 300, 0.0), (20000, 700, 128, 0, 700, 0.0), (13000, 50000, 40, 0, 50000, 0.0)])
def test_cross_entropy_targets_gradient_keeps_sixteen_bits(n, v, d, pad, words, softcap):
    """A token's gradient is mostly its target's: in 16-bit calls too that term has 2^-17 of itself (its rounding's
    remainder is added, in 16 bits again) and the softmax's 32-bit error, for any number of tokens, also of one word,
    in rows of whole 16-byte pieces or not. The other words' terms have the 2^-8 and 2^-11 of their roundings."""
    h, w, t = make(n, v, d, BF, seed=35, ignored=0.1)
    t = torch.where(t == -100, t, t % words)
    buf = torch.zeros((n, d + pad), device="cuda", dtype=BF)
    buf[:, :d] = h
    _, dh, dw = mu.linear_cross_entropy_grad(buf[:, :d], w, t, reduction="sum", softcap=softcap)
    w64 = w.double()
    want_w, err_w = torch.zeros_like(w64), torch.zeros_like(w64)
    for i in range(0, n, 4096):
        hi, ti = h[i:i + 4096].double(), t[i:i + 4096]
        keep = (ti != -100)[:, None]
        raw = mm(hi, w64.t())
        z = softcap * torch.tanh(raw / softcap) if softcap else raw
        at = torch.where(ti == -100, 0, ti)[:, None]
        zt = z.gather(1, at)
        lse = torch.logsumexp(z, 1, keepdim=True)
        others = torch.logsumexp((z - zt).scatter(1, at, float("-inf")), 1, keepdim=True)
        dz = (d + 2) * U * mm(hi.abs(), w64.abs().t()).amax(1, keepdim=True) + (12 * U * z.abs().amax(1, keepdim=True) if softcap else 0)
        each = 2 * dz + (512 + v / 64) * U + 4 * U * (lse.abs() + zt.abs() + z.abs().amax(1, keepdim=True))
        f = 1 - (z / softcap) ** 2 if softcap else 1.0
        q = torch.exp(z - lse).scatter(1, at, -torch.sigmoid(others)) * f * keep
        rel = (2 * each + 16 * U + (4 * dz / softcap / f if softcap else 0) + 2.0 ** -8 + 2.0 ** -11).expand_as(q)
        rel = rel.scatter(1, at, (rel - 2.0 ** -8 - 2.0 ** -11 + 2.0 ** -17).gather(1, at))
        q_err = q.abs() * rel + 2.0 ** -62 * keep
        want_h = mm(q, w64)
        within(dh[i:i + 4096], want_h, mm(q_err + (v + 8) * U * q.abs(), w64.abs()) + 2.0 ** -8 * want_h.abs() + 1e-38, "dhidden")
        want_w += mm(q.t(), hi)
        err_w += mm((q_err + (n + 8) * U * q.abs()).t(), hi.abs())
        del raw, z, f, q, rel, q_err
    within(dw, want_w, err_w + 2.0 ** -8 * want_w.abs() + 1e-38, "dweight")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,v,d", [(70, 300, 136), (700, 900, 72), (1, 77, 8), (1500, 5000, 328)])
def test_cross_entropy_rows_that_end_with_their_allocation(n, v, d, dtype):
    """Rows of whole 16-byte pieces, whose width is no multiple of a stage, as the last bytes of a buffer: no kernel
    reads a row past its width."""
    h, w, t = make(n, v, d, dtype, seed=37)

    def last(x):
        buf = torch.empty(32 << 20, device="cuda", dtype=torch.uint8).view(dtype)
        y = buf[buf.numel() - x.numel():].view_as(x)
        assert y.data_ptr() % 16 == 0
        return y.copy_(x)

    want = mu.linear_cross_entropy_grad(h, w, t)
    got = mu.linear_cross_entropy_grad(last(h), last(w), t, dhidden=last(h), dweight=last(w))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(mu.linear_cross_entropy(last(h), last(w), t), mu.linear_cross_entropy(h, w, t))


def test_cross_entropy_repeats_bit_for_bit_and_on_other_streams():
    h, w, t = make(700, 3001, 192, BF, seed=22, ignored=0.1)
    first = mu.linear_cross_entropy_grad(h, w, t)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = mu.linear_cross_entropy_grad(h, w, t)
    s.synchronize()
    again = mu.linear_cross_entropy_grad(h, w, t)
    for a, b, c in zip(first, other, again):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_cross_entropy_one_gradient_only():
    h, w, t = make(300, 700, 96, BF, seed=23)
    loss, dh, dw = mu.linear_cross_entropy_grad(h, w, t)
    a = mu.linear_cross_entropy_grad(h, w, t, dweight=False)
    b = mu.linear_cross_entropy_grad(h, w, t, dhidden=False)
    assert a[2] is None and b[1] is None
    assert torch.equal(a[1], dh) and torch.equal(b[2], dw) and torch.equal(a[0], loss) and torch.equal(b[0], loss)


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_cross_entropy_autograd(reduction):
    h, w, t = make(6 * 35, 400, 64, BF, seed=24, ignored=0.2)
    hp = h.view(6, 35, 64).clone().requires_grad_()
    wp = w.clone().requires_grad_()
    loss = mu.linear_cross_entropy(hp, wp, t.view(6, 35), reduction=reduction)
    up = normal(loss.shape, 25).abs()
    loss.backward(up)
    go = up.reshape(-1) if reduction == "none" else None
    _, dh, dw = mu.linear_cross_entropy_grad(h, w, t, reduction=reduction, grad_out=go)
    if reduction == "none":
        assert torch.equal(hp.grad.view(-1, 64), dh) and torch.equal(wp.grad, dw)
    else:
        assert torch.equal(hp.grad.view(-1, 64), (dh.float() * up).to(BF)) and torch.equal(wp.grad, (dw.float() * up).to(BF))
    # a frozen head
    hp.grad = None
    mu.linear_cross_entropy(hp, w, t.view(6, 35), reduction="sum").backward()
    assert torch.equal(hp.grad.view(-1, 64), mu.linear_cross_entropy_grad(h, w, t, reduction="sum")[1])


def test_cross_entropy_second_backward_is_refused():
    h, w, t = make(50, 100, 64, BF, seed=26)
    loss = mu.linear_cross_entropy(h.requires_grad_(), w, t)
    loss.backward(retain_graph=True)
    with pytest.raises(RuntimeError, match="taken before"):
        loss.backward()


@pytest.mark.parametrize("reduction", ["sum", "mean", "none"])
def test_cross_entropy_saved_tensor_hooks(reduction):
    """Hooks on saved tensors see all that a forward keeps, and backward uses what they give back."""
    h, w, t = make(90, 300, 64, BF, seed=33)
    h.requires_grad_(), w.requires_grad_()
    mu.linear_cross_entropy(h, w, t, reduction=reduction).sum().mul(0.5).backward()
    want, h.grad, w.grad = (h.grad, w.grad), None, None
    kept = []

    def pack(x):
        kept.append(x.shape)
        return x.cpu()

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda x: x.cuda()):
        loss = mu.linear_cross_entropy(h, w, t, reduction=reduction)
    assert h.shape in kept and w.shape in kept
    loss.sum().mul(0.5).backward()
    assert torch.equal(h.grad, want[0]) and torch.equal(w.grad, want[1])
    # without hooks the gradients become the leaves' own, uncopied
    if reduction != "none":
        h.grad = w.grad = None
        loss = mu.linear_cross_entropy(h, w, t, reduction=reduction)
        own = [x.data_ptr() for x in loss.grad_fn.saved_tensors]
        loss.backward()
        assert [h.grad.data_ptr(), w.grad.data_ptr()] == own


@pytest.mark.parametrize("reduction", ["sum", "none"])
def test_cross_entropy_backward_uses_the_given_handle(reduction, monkeypatch):
    """(Its own thread's handle would have a second workspace.)"""
    h, w, t = make(90, 300, 64, BF, seed=34)
    want = mu.linear_cross_entropy_grad(h, w, t, reduction=reduction)
    handle = mu.Handle()

    def other(device=None):
        raise AssertionError("another handle was asked for")

    monkeypatch.setattr(mu.training, "get_handle", other)
    loss = mu.linear_cross_entropy(h.requires_grad_(), w.requires_grad_(), t, reduction=reduction, handle=handle)
    loss.sum().backward()
    torch.cuda.synchronize()
    assert torch.equal(h.grad, want[1]) and torch.equal(w.grad, want[2])
    handle.close()


@pytest.mark.parametrize("needs_grad", [False, True])
def test_cross_entropy_refuses_forward_mode(needs_grad):
    import torch.autograd.forward_ad as fwd

    h, w, t = make(20, 100, 64, F32, seed=32)
    h.requires_grad_(needs_grad)
    with fwd.dual_level():
        for a, b in ((fwd.make_dual(h, torch.ones_like(h)), w), (h, fwd.make_dual(w, torch.ones_like(w)))):
            with pytest.raises((ValueError, RuntimeError)):
                mu.linear_cross_entropy(a, b, t)
    with pytest.raises((ValueError, RuntimeError)):
        torch.func.jvp(lambda x: mu.linear_cross_entropy(x, w, t), (h.detach(),), (torch.ones_like(h),))


@pytest.mark.parametrize("softcap", [0.0, 6.0])
def test_cross_entropy_gradient_against_differences(softcap):
    """Central differences of the 32-bit loss along random directions. With
    step s the difference is off by s^2 / 6 times a third derivative (at most
    that of a sum of N functions of logit changes bounded by m along the
    direction: N m^3) and by the losses' rounding over s."""
    h, w, t = make(40, 120, 33, F32, seed=27, learnt=3.0)
    loss, dh, dw = mu.linear_cross_entropy_grad(h, w, t, reduction="sum", softcap=softcap)
    step = 2.0 ** -7
    for k in range(4):
        vh, vw = normal(h.shape, 100 + k), normal(w.shape, 200 + k)
        vh, vw = vh / vh.norm(dim=1, keepdim=True), vw / vw.norm(dim=1, keepdim=True)
        up = mu.linear_cross_entropy(h + step * vh, w + step * vw, t, reduction="none", softcap=softcap).double().sum()
        dn = mu.linear_cross_entropy(h - step * vh, w - step * vw, t, reduction="none", softcap=softcap).double().sum()
        slope = (dh.double() * vh.double()).sum() + (dw.double() * vw.double()).sum()
        m = float((vh @ w.t()).abs().amax() + (h @ vw.t()).abs().amax()) + 1
        tol = step ** 2 * 40 * m ** 3 + 40 * 2.0 ** -20 / step
        assert abs(float((up - dn) / (2 * step) - slope)) <= tol


# ---------------------------------------------------------------------------
# norm, clipping, scaling
# ---------------------------------------------------------------------------
def tensors(seed, dtype=None):
    shapes = [(1,), (7,), (8,), (768,), (1000, 3), (129, 257), (8192,), (8193,), (3, 5, 7), (), (0,), (4, 0), (2049, 1023)]
    return [normal(s, seed + i, 10.0 ** (i % 5 - 2)).to(dtype or (BF if i % 2 else F32)) for i, s in enumerate(shapes)]


def norm64(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


@pytest.mark.parametrize("dtype", [None, BF, F32])
@pytest.mark.parametrize("max_norm", [0.5, 1e6])
@pytest.mark.parametrize("apart", [False, True])
def test_clip(dtype, max_norm, apart):
    ts = tensors(31, dtype)
    want = norm64(ts)
    before = [t.clone() for t in ts]
    # squares and sums in 64 bits: the norm is off by its rounding to 32
    n, coef = mu.grad_norm(ts, max_norm=max_norm)
    assert abs(float(n) - want) <= 2 * U * want and float(mu.grad_norm(ts)) == float(n)
    c = min(1.0, max_norm / (want + 1e-6))
    assert abs(float(coef) - c) <= 6 * U * c
    out = [torch.full_like(t, float("nan")) for t in ts] if apart else None
    assert float(mu.clip_grad_norm(ts, max_norm, out=out)) == float(n)
    for a, b in zip(out if apart else ts, before):
        assert torch.equal(a, (b.float() * coef).to(b.dtype))
    if apart:
        assert all(torch.equal(a, b) for a, b in zip(ts, before))


def test_clip_list_longer_than_a_launch():
    ts = [normal((5 + i % 300,), i) for i in range(400)]
    n = mu.clip_grad_norm(ts, 1.0)
    assert abs(norm64(ts) - 1.0) <= 1e-5 and float(n) > 1.0
    assert float(mu.grad_norm([normal((5 + i % 300,), i) for i in range(400)])) == float(n)


def test_norm_workspace_grows_between_calls():
    """Each growth is a new buffer, wherever it lies, whose count of finished blocks has to start at 0."""
    handle, one = mu.Handle(), torch.full((3,), 2.0, device="cuda")
    for n in (1, 9000, 1, 14000, 22000, 33000, 2):
        for _ in range(2):
            torch.full((1 << 20,), float("nan"), device="cuda")
            assert float(mu.grad_norm([one] * n, handle=handle)) == float(torch.tensor(math.sqrt(12.0 * n), dtype=F32))
    handle.close()


def test_norm_of_strided_and_unaligned_tensors():
    base = normal((300, 1000), 41)
    views = [base[:, 1:998], base[3:200:2, 8:16], base.view(-1)[1:777], base[:, 5:6], base.to(BF)[:, 3:900]]
    want = norm64(views)
    assert abs(float(mu.grad_norm(views)) - want) <= 2 * U * want
    keep = base.clone()
    mu.clip_grad_norm([base[:, 1:501]], 1.0)
    assert torch.equal(base[:, 501:], keep[:, 501:]) and torch.equal(base[:, :1], keep[:, :1])
    assert abs(norm64([base[:, 1:501]]) - 1.0) <= 1e-5


def test_norm_edges():
    assert float(mu.grad_norm([])) == 0.0
    n, c = mu.grad_norm([torch.zeros(5, device="cuda"), torch.empty(0, device="cuda")], max_norm=1.0)
    assert float(n) == 0.0 and float(c) == 1.0
    big = [torch.full((1000,), 3e38, device="cuda")]          # the squares overflow 32 bits, the norm only just
    assert float(mu.grad_norm(big)) == float("inf")
    big = [torch.full((1000,), 1e30, device="cuda")]
    assert abs(float(mu.grad_norm(big)) / (1e30 * math.sqrt(1000)) - 1) <= 4 * U
    small = [torch.full((1000,), 1e-30, device="cuda")]
    assert abs(float(mu.grad_norm(small)) / (1e-30 * math.sqrt(1000)) - 1) <= 4 * U
    for x in (float("nan"), float("inf")):
        ts = [normal((100,), 3), torch.tensor([1.0, x], device="cuda")]
        n, c = mu.grad_norm(ts, max_norm=1.0)
        assert not math.isfinite(float(n)) and (math.isnan(float(c)) if x != x else float(c) == 0.0)
    assert abs(float(mu.grad_norm([normal((100,), 3)])) - norm64([normal((100,), 3)])) <= 1e-5


def test_scale_by_device_scalar():
    ts = tensors(51)
    out = [torch.empty_like(t) for t in ts]
    coef = torch.tensor(-0.3, device="cuda")
    mu.scale(ts, coef, out=out)
    assert all(torch.equal(o, (t.float() * coef).to(t.dtype)) for o, t in zip(out, ts))
    mu.scale(ts, coef)
    assert all(torch.equal(o, t) for o, t in zip(out, ts))


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------
def adam64(g, m, v, w, step, lr, b1, b2, eps, wd, s):
    g = g.double() * s
    m = b1 * m.double() + (1 - b1) * g
    v = b2 * v.double() + (1 - b2) * g * g
    w = w.double() * (1 - lr * wd) - lr * (m / (1 - b1 ** step)) / ((v / (1 - b2 ** step)).sqrt() + eps)
    return m, v, w


@pytest.mark.parametrize("wt,gt,cp", [(F32, F32, None), (BF, BF, None), (F32, BF, BF), (BF, F32, F32)])
@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("strided", [False, True])
def test_adamw(wt, gt, cp, scaled, strided):
    shapes = [(768,), (1,), (130, 257), (0,), (8193,), (2, 3, 4), (1030, 1023)] + [(33,)] * 40
    f = lambda x: x[:, 1:-1] if strided and x.dim() == 2 else x
    mk = lambda k, sd, dt: [f(normal(s, 60 * k + i, sd).to(dt)) for i, s in enumerate(shapes)]
    g, w, m = mk(1, 1e-3, gt), mk(2, 0.02, wt), mk(3, 1e-3, F32)
    v = [f(normal(s, 240 + i, 1e-3).square()) for i, s in enumerate(shapes)]
    copies = None if cp is None else [torch.empty_like(x, dtype=cp) for x in w]
    s = torch.tensor(0.7, device="cuda") if scaled else None
    hp = dict(lr=3e-3, beta1=0.9, beta2=0.97, eps=1e-8, weight_decay=0.1)
    # the library takes its constants as 32-bit values
    r = {k: float(torch.tensor(x, dtype=F32)) for k, x in hp.items()}
    for step in (1, 2, 50):
        want = [adam64(a, b, c, d, step, r["lr"], r["beta1"], r["beta2"], r["eps"], r["weight_decay"],
                       float(s) if scaled else 1.0) for a, b, c, d in zip(g, m, v, w)]
        old = [x.double() for x in w]
        mu.adamw_update(g, m, v, w, step=step, grad_scale=s, copies=copies, **hp)
        for i in range(len(w)):
            wm, wv, ww = want[i]
            # a handful of roundings of each sum's terms
            within(m[i], wm, 4 * U * (wm.abs() + g[i].double().abs() + m[i].double().abs()) + 1e-44, "exp_avg")
            within(v[i], wv, 8 * U * wv.abs() + 1e-44, "exp_avg_sq")
            move = (ww - old[i]).abs()
            mterm = 8 * U * hp["lr"] * (g[i].double().abs() + m[i].double().abs()) / (wv.sqrt() + 1e-8) * 20
            e = 16 * U * (move + old[i].abs()) + mterm + 1e-44
            within(w[i], ww, e + (2.0 ** -8 * ww.abs() if wt == BF else 0), "weight")
            if copies is not None:
                within(copies[i], ww, e + (2.0 ** -8 * ww.abs() if cp == BF else 0), "copy")


def test_adamw_mixed_list_and_copies_left_out():
    w = [normal((64, 64), 1).to(BF), normal((99,), 2), normal((5, 5), 3)]
    g = [normal((64, 64), 4), normal((99,), 5).to(BF), normal((5, 5), 6)]
    m, v = [torch.zeros(x.shape, device="cuda") for x in w], [torch.zeros(x.shape, device="cuda") for x in w]
    one = [x.clone() for x in w]
    c = [None, torch.zeros(99, device="cuda", dtype=BF), None]
    mu.adamw_update(g, m, v, w, step=1, lr=0.1, copies=c)
    # step 1 from zero moments moves every weight by lr against its gradient's sign
    for a, b, x in zip(w, one, g):
        within(a, b.double() - float(torch.tensor(0.1)) * x.double().sign(), 2.0 ** -8 * (b.double().abs() + 0.1), "weight")
    assert torch.equal(c[1], w[1].to(BF))


@pytest.mark.parametrize("wt", [F32, BF])
@pytest.mark.parametrize("ct", [F32, BF])
def test_adamw_weight_and_copy_are_roundings_of_one_value(wt, ct):
    x = normal((257, 130), 1, 0.02).to(wt).float()
    g = [normal((257, 130), 2, 1e-2)]
    got = []
    for wide in (True, False):
        w, c = [x.clone() if wide else x.to(wt)], [torch.empty(257, 130, device="cuda", dtype=F32 if wide else ct)]
        m, v = [torch.zeros(257, 130, device="cuda")], [torch.zeros(257, 130, device="cuda")]
        mu.adamw_update(g, m, v, w, step=1, lr=1e-2, copies=c)
        got.append((w[0], c[0]))
    value = got[0][0]
    assert torch.equal(got[0][1], value) and torch.equal(got[1][0], value.to(wt)) and torch.equal(got[1][1], value.to(ct))


def test_adamw_non_finite_gradient_stays_with_its_element():
    w, g = [torch.ones(1000, device="cuda", dtype=BF)], [torch.ones(1000, device="cuda")]
    m, v = [torch.zeros(1000, device="cuda")], [torch.zeros(1000, device="cuda")]
    g[0][17] = float("nan")
    mu.adamw_update(g, m, v, w, step=1, lr=0.01)
    bad = torch.arange(1000, device="cuda") == 17
    assert bool(w[0][bad].isnan().all()) and bool(torch.isfinite(w[0][~bad]).all())


# ---------------------------------------------------------------------------
# together, captured, on long offsets
# ---------------------------------------------------------------------------
def test_training_step_in_a_graph():
    """The whole chain, captured once and replayed, against the same calls made eagerly."""
    h, w, t = make(300, 1000, 128, BF, seed=71, ignored=0.1)
    s = torch.cuda.Stream()

    def fresh():
        return dict(w=w.clone(), m=torch.zeros(w.shape, device="cuda"), v=torch.zeros(w.shape, device="cuda"),
                    dw=torch.empty_like(w), dh=torch.empty_like(h))

    def step(x):
        loss, _, _ = mu.linear_cross_entropy_grad(h, x["w"], t, dhidden=x["dh"], dweight=x["dw"])
        norm, coef = mu.grad_norm([x["dw"]], max_norm=0.1)
        mu.adamw_update([x["dw"]], [x["m"]], [x["v"]], [x["w"]], step=3, lr=1e-2, grad_scale=coef)
        mu.clip_grad_norm([x["dh"]], 1e-3)
        return loss, norm

    eager, captured = fresh(), fresh()
    with torch.cuda.stream(s):
        step(fresh())                      # the handle's buffers grow outside the capture
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = step(captured)
        for k in range(4):
            graph.replay()
            want = step(eager)
            s.synchronize()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), k
            for name in eager:
                assert torch.equal(eager[name], captured[name]), (k, name)
            torch.zeros(1 << 20, device="cuda").sum()


def test_outgrown_workspace_is_freed():
    """Calls of growing size on one handle hold one workspace at the end, not all that they outgrew."""
    v, d = 50304, 64
    h, w, t = make(8192, v, d, BF, seed=72)
    handle = mu.Handle()
    torch.cuda.synchronize()
    held = lambda: torch.cuda.mem_get_info()[1] - torch.cuda.mem_get_info()[0] - torch.cuda.memory_reserved()
    before = held()
    for n in (256, 512, 1024, 2048, 4096, 8192):
        got = mu.linear_cross_entropy_grad(h[:n], w, t[:n], handle=handle)
    torch.cuda.synchronize()
    # the exponentials, and at most as much again of the rest as they may grow by
    assert held() - before <= 8192 * 50432 * 2 + (320 << 20)
    handle.close()
    want = mu.linear_cross_entropy_grad(h, w, t)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph_replays_on_a_workspace_that_was_outgrown():
    h, w, t = make(300, 1000, 128, BF, seed=73, ignored=0.1)
    big = make(3000, 1500, 128, BF, seed=74)
    many = [normal((33,), i) for i in range(3000)]
    handle, s = mu.Handle(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        call = lambda: (*mu.linear_cross_entropy_grad(h, w, t, handle=handle), mu.grad_norm([h, w], handle=handle))
        want = call()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = call()
        for k in range(3):
            for x in out:
                x.fill_(float("nan"))
            graph.replay()
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), k
            mu.linear_cross_entropy_grad(*big, handle=handle)          # outgrows the captured workspace
            mu.grad_norm(many * (k + 1), handle=handle)
            torch.full((1 << 22,), float("nan"), device="cuda")
        s.synchronize()
    handle.close()


@pytest.mark.parametrize("wt", [F32, BF])
def test_adamw_in_a_graph_counts_its_steps(wt):
    """Step and rate on the device, changed between the replays, against the call with their numbers. The moments do
    not depend on them; the weight's three constants are each one rounding from those made on the host."""
    shapes = [(130, 257), (8193,), (5,)]
    g = [normal(s, 90 + i, 1e-2) for i, s in enumerate(shapes)]
    w = [normal(s, 93 + i).to(wt) for i, s in enumerate(shapes)]
    m, v = [torch.zeros(s, device="cuda") for s in shapes], [torch.zeros(s, device="cuda") for s in shapes]
    step, lr = torch.zeros((), device="cuda", dtype=torch.int64), torch.full((1,), 0.01, device="cuda")
    hp = dict(beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)
    clone = lambda xs: [x.clone() for x in xs]

    def run(m, v, w):
        step.add_(1)
        mu.adamw_update(g, m, v, w, step=step, lr=lr, **hp)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run(clone(m), clone(v), clone(w))
        step.zero_()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            run(m, v, w)
        for k in (1, 2, 3, 40, 41, 100000):
            step.fill_(k - 1)
            rate = 0.01 / k
            lr.fill_(rate)
            m2, v2, w2, old = clone(m), clone(v), clone(w), clone(w)
            mu.adamw_update(g, m2, v2, w2, step=k, lr=rate, **hp)
            graph.replay()
            s.synchronize()
            assert int(step) == k
            for i in range(len(shapes)):
                assert torch.equal(m[i], m2[i]) and torch.equal(v[i], v2[i])
                move = 4 * U * ((w2[i].double() - old[i].double()).abs() + old[i].double().abs())
                within(w[i], w2[i].double(), move + (2.0 ** -7 * w2[i].double().abs() if wt == BF else 0) + 1e-44, f"weight, step {k}")
                if wt == F32:                  # (a late step's rate is too small to move 16-bit weights)
                    assert not torch.equal(w[i], old[i])
    with pytest.raises(ValueError, match="step"):
        mu.adamw_update(g, m, v, w, step=step.int(), lr=0.1)
    with pytest.raises(ValueError, match="lr"):
        mu.adamw_update(g, m, v, w, step=1, lr=lr.cpu())


def test_lists_past_32_bit_offsets():
    n = (1 << 32) + 12345
    g = torch.zeros(n, device="cuda", dtype=BF)
    g[-1], g[-12340], g[7], g[1 << 31] = 3.0, 4.0, 12.0, 84.0
    norm, coef = mu.grad_norm([g], max_norm=8.5)
    assert float(norm) == 85.0
    mu.clip_grad_norm([g], 8.5)
    for i, x in ((-1, 3.0), (-12340, 4.0), (7, 12.0), (1 << 31, 84.0)):
        assert abs(float(g[i]) - x * 0.1) <= 2.0 ** -8 * x
    assert abs(float(mu.grad_norm([g])) - 8.5) <= 2.0 ** -8 * 8.5


# ---------------------------------------------------------------------------
# refusals: nothing is written
# ---------------------------------------------------------------------------
def test_refusals():
    h, w, t = make(10, 50, 64, BF, seed=81)
    bad = [
        lambda: mu.linear_cross_entropy(h, w.float(), t),
        lambda: mu.linear_cross_entropy(h, w[:, :32], t),
        lambda: mu.linear_cross_entropy(h, w, t[:9]),
        lambda: mu.linear_cross_entropy(h, w, t.to(torch.int16)),
        lambda: mu.linear_cross_entropy(h, w, t, softcap=-1.0),
        lambda: mu.linear_cross_entropy(h, w, t, softcap=float("nan")),
        lambda: mu.linear_cross_entropy(h, w, t, reduction="max"),
        lambda: mu.linear_cross_entropy(h.half(), w.half(), t),
        lambda: mu.linear_cross_entropy(h.t().contiguous().t(), w, t),
        lambda: mu.linear_cross_entropy(h, w, t.cpu()),
        lambda: mu.linear_cross_entropy(h.cpu(), w.cpu(), t.cpu()),
        lambda: mu.linear_cross_entropy_grad(h, w, t, dhidden=h),
        lambda: mu.linear_cross_entropy_grad(h, w, t, dweight=w),
        lambda: mu.linear_cross_entropy_grad(h, w, t, dhidden=False, dweight=False),
        lambda: mu.linear_cross_entropy_grad(h, w, t, dhidden=torch.empty(10, 64, device="cuda")),
        lambda: mu.linear_cross_entropy_grad(h, w, t, reduction="none", grad_out=torch.ones((), device="cuda")),
        lambda: mu.linear_cross_entropy_grad(h, w, t, grad_out=torch.ones((), device="cuda", dtype=BF)),
        lambda: mu.clip_grad_norm([h], 0.0),
        lambda: mu.clip_grad_norm([h], float("nan")),
        lambda: mu.clip_grad_norm([h, h], 1.0),
        lambda: mu.clip_grad_norm([h], 1.0, out=[w]),
        lambda: mu.clip_grad_norm([h.half()], 1.0),
        lambda: mu.grad_norm([h, h.cpu()]),
        lambda: mu.scale([h], torch.ones(2, device="cuda")),
        lambda: mu.adamw_update([h], [h], [h], [h], step=1),
        lambda: mu.adamw_update([h], [h.float()], [h.float()], [w], step=1),
        lambda: mu.adamw_update([h], [h.float()], [h.float()], [h.clone()], step=0),
        lambda: mu.adamw_update([h], [h.float()], [h.float()], [h.clone()], step=1, beta1=1.0),
        lambda: mu.adamw_update([h], [h.float()], [h.float()], [h], step=1),
    ]
    keep = h.clone(), w.clone()
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            f()
            pytest.fail(f"call {i} was accepted")
    torch.cuda.synchronize()
    assert torch.equal(h, keep[0]) and torch.equal(w, keep[1])


def test_example_trains():
    """examples/train_small_lm.py: every operator in one program; the loss falls from log(vocabulary)."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_small_lm.py")
    spec = importlib.util.spec_from_file_location("train_small_lm", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    losses = module.train(40, say=None)
    assert abs(losses[0] - math.log(module.VOCAB)) < 1.0 and losses[-1] < losses[0] - 3.0, (losses[0], losses[-1])
