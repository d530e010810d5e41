"""The gradient of a single gate or scale where the tokens' parts cancel.

All rows of y (and of x) are the same and the first half of dout's is the other half with the other sign, so each product of
the sum has its exact opposite, whatever its rounding: a sum in 64 bits is what one more row adds. That row's own error: in
units of U = 2^-24 yhat 26, the products 2 and their sums of at most 16 16, out of its absolute sum; the parts of the blocks
are two floats, and the sums of 64 bits: 2^-46 of the absolute sum over all rows.
"""
import pytest
import torch

import muon_newton_schulz_update_amd as mu
from test_norms_gpu import BF, F32, U, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tx,ty", [(BF, BF), (F32, BF), (F32, F32)], ids=["bf16", "mixed", "fp32"])
@pytest.mark.parametrize("scale", ["one", "channels"])
@pytest.mark.parametrize("d", [96, 509, 768, 1023, 2048, 8192, 16384])
def test_sums_over_tokens_that_cancel(d, scale, tx, ty):
    n = 2 * max(300, (1 << 23) // d) + 1
    y = normal((1, d), 1).to(ty).expand(n, d).contiguous()
    x = normal((1, d), 2).to(tx).expand(n, d).contiguous()
    half = normal((1, d), 3).to(tx).expand(n // 2, d)
    dout = torch.cat([half, -half, normal((1, d), 4).to(tx)]).contiguous()
    gain = (1 + 0.2 * normal((d,), 5)).to(ty)
    gate = torch.full((1,), 0.75, device="cuda")
    s = torch.full((1,), 1.25, device="cuda") if scale == "one" else 1 + 0.1 * normal((d,), 6)
    yh = y[-1].double() / torch.sqrt(y[-1].double().square().mean() + float(torch.tensor(1e-6, dtype=F32)))
    for post_norm, post_gain in ((True, gain), (True, None), (False, None)):
        got = mu.residual_norm_grad(x, y, dout, None, post_norm=post_norm, post_gain=post_gain, gate=gate, scale=s, pre_norm=False)
        of = (yh if post_norm else y[-1].double()) * (1 if post_gain is None else gain.double())
        part, every = dout[-1].double() * of, 2 * (n // 2) * (dout[0].double() * of).abs().sum()
        err = 44 * U * part.abs().sum() + 2.0 ** -46 * every + U * part.sum().abs()
        assert abs(float(got.gate) - float(part.sum())) <= float(err), (post_norm, post_gain is not None)
    if scale == "one":
        part, every = (dout[-1] * x[-1].float()).double(), 2 * (n // 2) * (dout[0].double() * x[0].double()).abs().sum()
        want = (dout[-1].double() * x[-1].double()).sum()
        assert abs(float(got.scale) - float(want)) <= float(8 * U * part.abs().sum() + 2.0 ** -46 * every + U * want.abs())


@pytest.mark.parametrize("d", [96, 768, 1023, 16384])
def test_infinities_of_y_stay_out_of_its_gradient_without_a_norm(d):
    y, dout = normal((40, d), 7), normal((40, d), 8)
    y[3, 5], y[7, d - 1] = float("inf"), float("nan")
    gate = torch.full((1,), 0.75, device="cuda")
    for g, want in ((gate, dout * 0.75), (None, dout)):
        got = mu.residual_norm_grad(normal((40, d), 9), y, dout, None, post_norm=False, gate=g, pre_norm=False)
        assert torch.equal(got.y, want)
