"""Host-side rules of the training-step entry points (no GPU): defaults, what
is refused and with which status, and the validation under sanitizers."""
import ctypes
import os
import shutil
import subprocess

import pytest

import muon_newton_schulz_update_amd as mu
from muon_newton_schulz_update_amd import MuonMatrix

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, DTYPE, SHAPE = 0, -1, -2, -3
F32, BF16 = 0, 1
A, B, C, D, E = (x << 32 for x in range(1, 6))       # far apart addresses

pytestmark = pytest.mark.skipif(not os.path.exists(mu.library_path()), reason="libmuon.so not built")


def M(ptr=A, rows=4, cols=8, ld=None, dtype=F32):
    return MuonMatrix(ptr, rows, cols, cols if ld is None else ld, dtype)


def expect(result, code, text=""):
    rc, msg = result
    assert rc == code and text in msg, (rc, msg)


def test_defaults():
    c = mu.AdamWConfig()
    mu.load_library().muon_adamw_config_default(ctypes.byref(c))
    assert [round(x, 9) for x in (c.lr, c.beta1, c.beta2, c.weight_decay)] == pytest.approx([0.01, 0.8, 0.95, 0.0])
    assert c.eps == pytest.approx(1e-10) and c.step == 1
    c = mu.LossConfig()
    mu.load_library().muon_loss_config_default(ctypes.byref(c))
    assert (c.reduction, c.softcap, c.ignore_index) == (2, 0.0, -100)


def test_norm_rules():
    check = mu.check_norm_args
    expect(check([]), OK)
    expect(check([M(), M(B, 0, 5), M(None, 3, 0), M(C, 70000, 70000, dtype=BF16)]), OK)   # no Newton-Schulz limits
    expect(check([M(), M()]), OK)                                  # read only: the same tensor twice
    expect(check([M()], norm=None), INVALID, "NULL norm")
    expect(check([M()], coef=8192, max_norm=0.0), INVALID, "max_norm")
    expect(check([M()], coef=8192, max_norm=float("nan")), INVALID, "max_norm")
    expect(check([M()], coef=8194), INVALID, "aligned")
    expect(check([M(dtype=2)]), DTYPE, "grad[0]")
    expect(check([M(rows=-1)]), SHAPE)
    expect(check([M(ld=7)]), SHAPE, "ld 7 < cols 8")
    expect(check([M(rows=1, ld=0)]), OK)                           # a single row has no stride
    expect(check([M(rows=1 << 40, cols=8, ld=8)]), SHAPE, "2^42")
    expect(check([M(ld=(1 << 40) + 1)]), SHAPE, "2^40")
    expect(check([M(None)]), INVALID, "NULL pointer")
    expect(check([M(A + 2)]), INVALID, "aligned")
    # outputs
    expect(check([M()], [M(B)]), OK)
    expect(check([M()], [M()]), OK)                                # in place, element for element
    expect(check([M()], [M(B, dtype=BF16)]), OK)
    expect(check([M()], [M(B, 4, 7)]), SHAPE)
    expect(check([M()], [M(A + 16)]), INVALID, "share memory")
    expect(check([M()], [M(dtype=BF16)]), INVALID, "share memory")  # the same bytes as another type
    expect(check([M(), M(B)], [M(C), M(C)]), INVALID, "share memory")
    expect(check([M(), M(B)], [M(B), M(A)]), INVALID, "share memory")
    expect(check([M()], [M(B)], norm=B), INVALID, "share memory")
    # column slices of one buffer
    expect(check([M(A, 4, 4, 8)], [M(A + 16, 4, 4, 8)]), OK)


def test_norm_scalars_are_outputs():
    """Norm and coefficient at one address, or in a tensor's place: the second write would destroy the first, or a
    gradient."""
    check = mu.check_norm_args
    for out in (None, [M(B)], [M()]):
        expect(check([M()], out, norm=C, coef=C + 4), OK)
        expect(check([M()], out, norm=C, coef=C), INVALID, "share memory")
        expect(check([M()], out, norm=C, coef=C + 2), INVALID, "aligned")
        expect(check([M()], out, norm=A, coef=A), INVALID, "share memory")
        expect(check([M()], out, norm=A + 8, coef=C), INVALID, "share memory")
        expect(check([M()], out, norm=C, coef=A + 8), INVALID, "share memory")
    expect(check([], norm=C, coef=C), INVALID, "share memory")


def test_norm_rules_of_a_list_in_place():
    check = mu.check_norm_args
    for twice in ([M(), M()], [M(), M(A + 16)], [M(A, 4, 8, 16), M(A, 4, 9, 16)]):
        expect(check(twice), OK)                                   # a norm reads
        expect(check(twice, twice), INVALID, "share memory")       # a clip in place writes
    expect(check([M(), M(B)], [M(), M(B)]), OK)


def test_adamw_rules():
    def check(g=None, m=None, v=None, w=None, copies=None, scale=None, **cfg):
        c = mu.AdamWConfig()
        mu.load_library().muon_adamw_config_default(ctypes.byref(c))
        for k, x in cfg.items():
            setattr(c, k, x)
        return mu.check_adamw_args([g or M(A, dtype=BF16)], [m or M(B)], [v or M(C)], [w or M(D, dtype=BF16)], copies,
                                   c, scale)

    expect(check(), OK)
    expect(mu.check_adamw_args([], [], [], []), OK)
    expect(check(copies=[M(E, dtype=BF16)], scale=4096), OK)
    expect(check(copies=[M(None, 0, 0)]), OK)
    expect(check(step=0), INVALID, "step")
    expect(check(beta1=1.0), INVALID, "beta")
    expect(check(beta2=-0.1), INVALID, "beta")
    expect(check(beta2=float("nan")), INVALID, "beta")
    expect(check(eps=-1.0), INVALID, "eps")
    expect(check(lr=float("inf")), INVALID, "lr")
    expect(check(weight_decay=-1.0), INVALID, "weight_decay")
    expect(check(m=M(B, dtype=BF16)), DTYPE, "exp_avg[0]")
    expect(check(v=M(C, dtype=BF16)), DTYPE, "exp_avg_sq[0]")
    expect(check(g=M(A, 4, 9)), SHAPE)
    expect(check(copies=[M(E, 8, 4)]), SHAPE)
    expect(check(m=M(C)), INVALID, "share memory")
    expect(check(g=M(D, dtype=BF16)), INVALID, "share memory")     # the gradient in the weight's place
    expect(check(copies=[M(D, dtype=BF16)]), INVALID, "share memory")
    expect(check(scale=B), INVALID, "share memory")
    expect(check(scale=4097), INVALID, "aligned")


def test_adamw_rules_of_device_step_and_rate():
    def check(**cfg):
        c = mu.AdamWConfig()
        mu.load_library().muon_adamw_config_default(ctypes.byref(c))
        assert c.step_at is None and c.lr_at is None
        for k, x in cfg.items():
            setattr(c, k, x)
        return mu.check_adamw_args([M(A)], [M(B)], [M(C)], [M(D)], None, c, None)

    expect(check(step_at=E, lr_at=E + 8), OK)
    expect(check(step_at=E, step=0), OK)                           # not read
    expect(check(lr_at=E, lr=float("nan")), OK)
    expect(check(lr_at=E, step=0), INVALID, "step")
    expect(check(step_at=E, lr=float("nan")), INVALID, "lr")
    expect(check(step_at=E + 4), INVALID, "aligned")
    expect(check(lr_at=E + 2), INVALID, "aligned")
    expect(check(step_at=B), INVALID, "share memory")
    expect(check(lr_at=D + 4), INVALID, "share memory")
    expect(check(lr_at=A + 4), OK)                                 # the gradient is only read


def test_loss_rules():
    def check(h=None, w=None, **kw):
        return mu.check_loss_args(h or M(A, 10, 64, dtype=BF16), w or M(B, 50, 64, dtype=BF16), **kw)

    dh, dw = M(C, 10, 64, dtype=BF16), M(D, 50, 64, dtype=BF16)
    expect(check(), OK)
    expect(check(dhidden=dh, dweight=dw), OK)
    expect(check(dhidden=dh), OK)
    expect(check(h=M(None, 0, 64, dtype=BF16), targets=None), OK)
    expect(mu.check_loss_args(None, dw), INVALID, "NULL")
    expect(check(loss=None), INVALID, "NULL loss")
    expect(check(targets=None), INVALID, "NULL targets")
    expect(check(target_bytes=2), DTYPE, "targets")
    expect(check(targets=4098), INVALID, "aligned")
    expect(check(cfg=mu.LossConfig(3, 0.0, 0)), INVALID, "reduction")
    expect(check(cfg=mu.LossConfig(2, -1.0, 0)), INVALID, "softcap")
    expect(check(cfg=mu.LossConfig(2, float("inf"), 0)), INVALID, "softcap")
    expect(check(h=M(A, 10, 32, dtype=BF16)), SHAPE, "columns")
    expect(check(h=M(A, 10, 64)), DTYPE, "types")
    expect(check(w=M(B, 0, 64, dtype=BF16)), SHAPE)
    expect(check(w=M(B, (1 << 22) + 1, 64, dtype=BF16)), SHAPE, "2^22")
    expect(check(h=M(A, (1 << 24) + 1, 64, dtype=BF16)), SHAPE, "2^24")
    expect(check(h=M(A, 10, 65537, dtype=BF16), w=M(B, 50, 65537, dtype=BF16)), SHAPE)
    expect(check(dhidden=M(C, 10, 64)), DTYPE, "dhidden")
    expect(check(dweight=M(D, 49, 64, dtype=BF16)), SHAPE)
    expect(check(dhidden=M(A, 10, 64, dtype=BF16)), INVALID, "share memory")
    expect(check(dweight=M(B, 50, 64, dtype=BF16)), INVALID, "share memory")
    expect(check(dhidden=dh, dweight=M(C, 50, 64, dtype=BF16)), INVALID, "share memory")
    expect(check(loss=A), INVALID, "share memory")
    expect(check(targets=C, dhidden=dh), INVALID, "share memory")
    # per-token losses take N values: one in front of the weight runs into it
    expect(check(loss=B - 8), OK)
    expect(check(loss=B - 8, cfg=mu.LossConfig(0, 0.0, 0)), INVALID, "share memory")


def test_negated_views_are_refused():
    """Their memory holds the other sign."""
    import torch

    pack = mu.training._describe().pack
    z = torch.ones(4, 1, dtype=torch.complex64)
    for view in (torch.imag(z.conj()), torch._neg_view(torch.ones(2, 3)), torch._neg_view(torch.ones(0, 3))):
        assert view.is_neg()
        with pytest.raises(ValueError, match="negated"):
            pack((view,), "hidden", 0)


def test_tensors_with_a_forward_tangent_are_refused():
    """Describing one would drop its tangent without a word."""
    import torch
    import torch.autograd.forward_ad as fwd

    pack = mu.training._describe().pack
    with fwd.dual_level():
        for shape in ((2, 3), (3,), (0, 3)):
            with pytest.raises(ValueError, match="tangent"):
                pack((fwd.make_dual(torch.ones(shape), torch.ones(shape)),), "hidden", 0)
        pack((torch.ones(0, 3),), "hidden", 0)


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_training_validation_under_asan_ubsan(tmp_path):
    exe = tmp_path / "train_validate_fuzz"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           f"-I{ROOT}/include", f"-I{ROOT}/muon_newton_schulz_update_amd/csrc",
           f"{ROOT}/tests/native/train_validate_fuzz.cpp", f"{ROOT}/muon_newton_schulz_update_amd/csrc/validate.cpp",
           "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 and "sanitizer" in (r.stderr or "").lower() and "cannot find" in r.stderr:
        pytest.skip("sanitizer runtime not installed")
    assert r.returncode == 0, r.stderr[-2000:]
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, (run.stdout[-2000:], run.stderr[-4000:])
    assert run.stdout.splitlines()[-1].startswith("ok "), run.stdout


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_validation_when_memory_runs_out(tmp_path):
    exe = tmp_path / "check_alloc"
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", f"-I{ROOT}/include", f"-I{ROOT}/muon_newton_schulz_update_amd/csrc",
                        f"{ROOT}/tests/native/check_alloc.cpp", f"{ROOT}/muon_newton_schulz_update_amd/csrc/validate.cpp",
                        "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0 and run.stdout == "ok\n", (run.returncode, run.stdout[-500:], run.stderr[-500:])
