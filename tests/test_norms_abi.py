"""Host-side rules of the norms around a block (no GPU): what is refused and with which status, and the validation of
these and of the log probabilities under sanitizers."""
import ctypes
import os
import shutil
import subprocess

import pytest

import muon_newton_schulz_update_amd as mu
from muon_newton_schulz_update_amd import MuonMatrix

OK, INVALID, DTYPE, SHAPE = 0, -1, -2, -3
F32, BF16 = 0, 1
AT = [x << 32 for x in range(1, 20)]       # far apart addresses

pytestmark = pytest.mark.skipif(not os.path.exists(mu.library_path()), reason="libmuon.so not built")


def M(k, rows=4, cols=8, ld=None, dtype=F32, shift=0):
    return MuonMatrix(AT[k] + shift if rows * cols else None, rows, cols, cols if ld is None else ld, dtype)


def V(k, n=8, dtype=F32):
    return M(k, 1, n, dtype=dtype)


def expect(result, code, text=""):
    rc, msg = result
    assert rc == code and text in msg, (rc, msg)


def test_defaults():
    p = mu.NormParams()
    mu.load_library().muon_norm_params_default(ctypes.byref(p))
    assert (p.post_gain, p.pre_gain, p.gate, p.scale, p.post_norm, p.pre_norm) == (None,) * 4 + (1, 1)
    assert p.eps == pytest.approx(1e-6)


def test_forward_rules():
    check = mu.check_residual_norm_args
    x, y, out, hid = (M(k) for k in range(4))
    half = lambda k, **kw: M(k, dtype=BF16, **kw)
    expect(check(x, y, out, hid), OK)
    expect(check(x, y, out, hid, post_gain=V(5), pre_gain=V(6, dtype=BF16), gate=V(7), scale=V(8)), OK)
    expect(check(x, y, out, hid, gate=V(7, 1), scale=V(8, 1)), OK)
    expect(check(x, y, out, hid, gate=M(7)), OK)
    expect(check(half(0), half(1), half(2), half(3), gate=half(7)), OK)
    expect(check(x, half(1), out, half(3), gate=half(7)), OK)           # 32-bit residual, 16-bit block
    expect(check(x, None, None, hid), OK)                               # the norm before the first block
    expect(check(x, None, None, half(3)), OK)
    expect(check(x, None, out, None, pre_norm=0, scale=V(8, 1)), OK)
    expect(check(x, y, out, None, pre_norm=0), OK)
    expect(check(M(0, 0), M(1, 0), M(2, 0), M(3, 0), gate=M(7, 0)), OK)  # no tokens
    expect(check(None, y, out, hid), INVALID, "NULL x")
    expect(check(x, y, None, hid), INVALID, "NULL out")
    expect(check(x, y, out, None), INVALID, "NULL hidden")
    expect(check(x, None, None, None, pre_norm=0), INVALID, "NULL out and hidden")
    expect(check(x, y, out, hid, pre_norm=0), INVALID, "without a norm")
    expect(check(x, y, out, hid, post_norm=0, post_gain=V(5)), INVALID, "post_gain")
    expect(check(x, None, None, hid, post_gain=V(5)), INVALID, "post_gain")
    expect(check(x, None, None, hid, gate=V(5)), INVALID, "gate")
    expect(check(x, y, out, None, pre_norm=0, pre_gain=V(5)), INVALID, "pre_gain")
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        expect(check(x, y, out, hid, eps=eps), INVALID, "eps")
    expect(check(M(0, 4, 16385), M(1, 4, 16385), M(2, 4, 16385), M(3, 4, 16385)), SHAPE, "16384")
    expect(check(M(0, 4, 0), M(1, 4, 0), M(2, 4, 0), M(3, 4, 0)), SHAPE)
    expect(check(M(0, 1 << 31), M(1, 1 << 31), M(2, 1 << 31), M(3, 1 << 31)), SHAPE, "2^31")
    expect(check(x, M(1, 5), out, hid), SHAPE)
    expect(check(x, y, M(2, 4, 7), hid), SHAPE)
    expect(check(x, y, out, M(3, 3)), SHAPE)
    expect(check(M(0, ld=7), y, out, hid), SHAPE, "ld")
    expect(check(half(0), y, half(2), hid), DTYPE)                      # 32-bit block on a 16-bit residual
    expect(check(x, y, half(2), hid), DTYPE, "out")
    expect(check(x, y, out, half(3)), DTYPE, "hidden")
    expect(check(half(0), None, None, hid), DTYPE, "hidden")
    expect(check(M(0, dtype=2), y, out, hid), DTYPE)
    expect(check(x, y, out, hid, post_gain=V(5, 7)), SHAPE, "post_gain")
    expect(check(x, y, out, hid, post_gain=V(5, 1)), SHAPE, "post_gain")
    expect(check(x, y, out, hid, pre_gain=M(5)), SHAPE, "pre_gain")
    expect(check(x, y, out, hid, scale=M(5)), SHAPE, "scale")
    expect(check(x, y, out, hid, gate=M(5, 2)), SHAPE, "gate")
    expect(check(x, half(1), out, half(3), gate=M(7)), DTYPE, "gate")
    expect(check(x, y, out, hid, gate=MuonMatrix(None, 1, 8, 8, F32)), INVALID, "NULL pointer")
    expect(check(x, y, out, hid, gate=MuonMatrix(AT[5] + 2, 1, 8, 8, F32)), INVALID, "aligned")
    # outputs share nothing; what is read may
    expect(check(x, x, out, hid, post_gain=V(5), pre_gain=V(5), gate=V(5), scale=V(5)), OK)
    expect(check(x, y, x, hid), INVALID, "share memory")
    expect(check(x, y, out, y), INVALID, "share memory")
    expect(check(x, y, out, M(2, shift=64)), INVALID, "share memory")
    expect(check(x, y, out, hid, pre_gain=V(3)), INVALID, "share memory")
    expect(check(M(0, ld=16), M(0, ld=16, shift=32), out, hid), OK)     # columns of one buffer


def test_gradient_rules():
    def check(x=M(0), y=M(1), dout=M(2), dhidden=M(3), grads=None, **kw):
        return mu.check_residual_norm_grad_args(x, y, dout, dhidden, {"x": M(4)} if grads is None else grads, **kw)

    every = dict(post_gain=V(9), pre_gain=V(10), gate=V(11), scale=V(12))
    expect(check(), OK)
    expect(check(dout=None), OK)
    expect(check(dhidden=None), OK)
    expect(check(dout=None, dhidden=None), INVALID, "NULL dout")
    expect(check(pre_norm=0), INVALID, "without a norm")
    expect(check(dhidden=None, pre_norm=0), OK)
    expect(check(grads={}), INVALID, "no gradient")
    expect(mu.check_residual_norm_grad_args(M(0), M(1), M(2), M(3), None), INVALID, "NULL gradients")
    expect(check(grads={"x": M(4), "y": M(5), "post_gain": V(6), "pre_gain": V(7), "gate": V(8), "scale": V(13)}, **every), OK)
    for name in every:
        expect(check(grads={name: V(6)}), INVALID, "without")
        expect(check(grads={name: V(6, 7)}, **every), SHAPE)
        expect(check(grads={name: V(6, dtype=BF16)}, **every), DTYPE)
    expect(check(y=None, grads={"y": M(5)}), INVALID, "without y")
    expect(check(y=None, dout=None, dhidden=M(3, dtype=BF16)), OK)
    expect(check(dhidden=M(3, dtype=BF16)), DTYPE, "dhidden")
    expect(check(dout=M(2, dtype=BF16)), DTYPE, "dout")
    expect(check(dout=M(2, 5)), SHAPE)
    expect(check(grads={"x": M(4, dtype=BF16)}), DTYPE, "dx")
    expect(check(grads={"y": M(4, 4, 9)}), SHAPE, "dy")
    expect(check(grads={"x": M(4), "y": M(4)}), INVALID, "share memory")
    expect(check(grads={"x": M(2)}), INVALID, "share memory")
    expect(check(grads={"gate": V(11)}, gate=V(11)), INVALID, "share memory")
    expect(check(grads={"gate": M(5)}, gate=M(11)), OK)
    expect(check(grads={"gate": V(5)}, gate=M(11)), SHAPE, "dgate")


def test_rows_of_tensors_on_the_host_are_refused():
    import torch

    pack = mu.training._describe().pack_rows
    words, at = pack((None, torch.empty(0, 3, 4), torch.empty(0)), ("a", "b", "c"), 0)
    m = [MuonMatrix.from_buffer_copy(words[40 * i:40 * i + 40]) for i in range(3)]
    assert [(x.rows, x.cols) for x in m] == [(0, 0), (0, 4), (1, 0)] and isinstance(at, int)
    for bad in (torch.ones(2, 3), torch.ones(2, 3, 4), torch.ones(())):
        with pytest.raises(ValueError, match="x: expected a tensor on GPU 0"):
            pack((bad,), ("x",), 0)
    with pytest.raises(ValueError, match="contiguous"):
        pack((torch.ones(2, 3, 4).transpose(0, 1),), ("x",), 0)
    with pytest.raises(ValueError, match="differ in length"):
        pack((None,), ("x", "y"), 0)
    with pytest.raises(TypeError, match="x: expected a tensor"):
        pack((3,), ("x",), 0)
    with pytest.raises(TypeError, match="dtype"):
        pack((torch.ones(3, dtype=torch.float16),), ("x",), 0)


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_validation_under_asan_ubsan(tmp_path):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = tmp_path / "model_validate_fuzz"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           f"-I{root}/include", f"-I{root}/muon_newton_schulz_update_amd/csrc",
           f"{root}/tests/native/model_validate_fuzz.cpp", f"{root}/muon_newton_schulz_update_amd/csrc/validate.cpp",
           "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 and "sanitizer" in (r.stderr or "").lower() and "cannot find" in r.stderr:
        pytest.skip("sanitizer runtime not installed")
    assert r.returncode == 0, r.stderr[-2000:]
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, (run.stdout[-2000:], run.stderr[-4000:])
    assert run.stdout.splitlines()[-1].startswith("ok "), run.stdout
