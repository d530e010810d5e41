"""The norms' native binding refuses before it calls: no device, no library needed."""
import pytest
import torch

import muon_newton_schulz_update_amd as mu

T = torch.zeros
X, V = T(4, 8), T(8)


def forward(x=X, y=X, post_gain=None, gate=None, scale=None, pre_gain=None, dtype=None):
    # (an entry of 0 would be a fault if it were ever called)
    return mu.training._describe().residual_norm(0, 0, 0, (x, y, post_gain, gate, scale, pre_gain), True, True, 1e-6, dtype)


def backward(dout=X, dhidden=X, wanted=(True,) * 6, x=X, y=X, gate=None):
    return mu.training._describe().residual_norm_grad(0, 0, 0, (x, y, None, gate, None, None), dout, dhidden, wanted, True, True, 1e-6)


@pytest.mark.parametrize("call,error,match", [
    (lambda: forward(), ValueError, "x: expected a tensor on GPU 0, got one on cpu"),
    (lambda: forward(x=None), TypeError, "x: expected a tensor"),
    (lambda: forward(y=3), TypeError, "y: expected a tensor"),
    (lambda: forward(y=T(4, 9)), ValueError, r"y of shape \[4, 9\] beside x of \[4, 8\]"),
    (lambda: forward(x=T(2, 3, 8), y=T(2, 3, 8), gate=T(3, 2, 8)), ValueError, "gate of shape"),
    (lambda: forward(x=X.half(), y=X.half()), TypeError, "x: dtype Half"),
    (lambda: forward(x=X.t(), y=X.t()), ValueError, "x: columns must be contiguous"),
    (lambda: forward(x=T(2, 3, 8).transpose(0, 1), y=T(3, 2, 8)), ValueError, "x: a tensor that is not a matrix"),
    (lambda: backward(x=T(0, 8), y=T(0, 8), dout=T(0, 7)), ValueError, "dout of shape"),
    (lambda: backward(x=T(0, 8), y=T(0, 8), dout=T(0, 8), dhidden=T(8, 0)), ValueError, "dhidden of shape"),
    (lambda: backward(wanted=(True,) * 5), ValueError, "six"),
    (lambda: backward(wanted=[True] * 6), TypeError, "tuple"),
    (lambda: backward(gate=T(8, 4)), ValueError, "gate of shape"),
    (lambda: backward(dhidden=1.0), ValueError, "x: expected a tensor on GPU 0"),
])
def test_refusals(call, error, match):
    with pytest.raises(error, match=match):
        call()


def test_refusals_leave_no_references():
    import sys
    x = T(4, 8)
    before = sys.getrefcount(x)
    for _ in range(50):
        with pytest.raises(ValueError):
            forward(x=x)
        with pytest.raises(ValueError):
            backward(x=x)
    assert sys.getrefcount(x) == before
