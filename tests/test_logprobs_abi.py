"""Host-side rules of the head's log probabilities (no GPU): what is refused and with which status."""
import ctypes
import os

import pytest

import muon_newton_schulz_update_amd as mu
from muon_newton_schulz_update_amd import MuonMatrix

OK, INVALID, DTYPE, SHAPE = 0, -1, -2, -3
F32, BF16 = 0, 1
A, B, C, D, E, F, G, H = (x << 32 for x in range(1, 9))       # far apart addresses

pytestmark = pytest.mark.skipif(not os.path.exists(mu.library_path()), reason="libmuon.so not built")


def M(ptr=A, rows=10, cols=64, ld=None, dtype=BF16):
    return MuonMatrix(ptr if rows * cols else None, rows, cols, cols if ld is None else ld, dtype)


def W(rows=50, cols=64, dtype=BF16, ptr=B):
    return M(ptr, rows, cols, dtype=dtype)


def expect(result, code, text=""):
    rc, msg = result
    assert rc == code and text in msg, (rc, msg)


def config(top=0, softcap=0.0, ignore=-100):
    return mu.LogProbConfig(top, softcap, ignore)


def test_defaults():
    c = config(7, 1.0, 3)
    mu.load_library().muon_logprob_config_default(ctypes.byref(c))
    assert (c.top, c.softcap, c.ignore_index) == (0, 0.0, -100)


def test_forward_rules():
    def check(h=None, w=None, **kw):
        return mu.check_logprob_args(h or M(), w or W(), **{**dict(targets=C, logprobs=D), **kw})

    top = dict(top_logprobs=G, top_tokens=H)
    expect(check(), OK)
    expect(check(entropy=E, stats=F, cfg=config(5), **top), OK)
    expect(check(cfg=config(32), **top), OK)
    expect(check(h=M(rows=0), targets=None, logprobs=None), OK)
    expect(check(h=M(dtype=F32), w=W(dtype=F32)), OK)
    expect(mu.check_logprob_args(None, W()), INVALID, "NULL")
    expect(mu.check_logprob_args(M(), None), INVALID, "NULL")
    expect(check(logprobs=None), INVALID, "NULL logprobs")
    expect(check(targets=None), INVALID, "NULL targets")
    expect(check(target_bytes=2), DTYPE, "targets")
    expect(check(targets=C + 2), INVALID, "aligned")
    expect(check(logprobs=D + 2), INVALID, "aligned")
    expect(check(entropy=E + 1), INVALID, "aligned")
    expect(check(stats=F + 8), INVALID, "aligned")
    expect(check(cfg=config(5), top_logprobs=G + 2, top_tokens=H), INVALID, "aligned")
    expect(check(cfg=config(5), top_logprobs=G, top_tokens=H + 4), INVALID, "aligned")
    expect(check(cfg=config(5), top_logprobs=G), INVALID, "NULL top")
    expect(check(cfg=config(5), top_tokens=H), INVALID, "NULL top")
    expect(check(top_logprobs=G + 1, top_tokens=H + 1), OK)                # not looked at
    for n, v in ((-1, 50), (33, 50), (6, 5)):
        expect(check(w=W(v), cfg=config(n), **top), INVALID, "alternatives")
    expect(check(w=W(5), cfg=config(5), **top), OK)
    for cap in (-1.0, float("inf"), float("nan")):
        expect(check(cfg=config(0, cap)), INVALID, "softcap")
    expect(check(h=M(cols=32)), SHAPE, "columns")
    expect(check(h=M(dtype=F32)), DTYPE, "types")
    expect(check(w=W(0)), SHAPE)
    expect(check(w=W((1 << 22) + 1)), SHAPE, "2^22")
    expect(check(h=M(rows=(1 << 24) + 1)), SHAPE, "2^24")
    expect(check(h=M(cols=65537), w=W(cols=65537)), SHAPE)
    # outputs: 40, 40, 160, 200 and 400 bytes
    expect(check(entropy=D), INVALID, "share memory")
    expect(check(entropy=D + 40), OK)
    expect(check(entropy=D + 36), INVALID, "share memory")
    expect(check(stats=E, entropy=E + 156), INVALID, "share memory")
    expect(check(logprobs=A), INVALID, "share memory")
    expect(check(logprobs=B + 8), INVALID, "share memory")
    expect(check(logprobs=C), INVALID, "share memory")
    expect(check(cfg=config(5), top_logprobs=G, top_tokens=G + 192), INVALID, "share memory")
    expect(check(cfg=config(5), top_logprobs=G, top_tokens=G + 200), OK)
    expect(check(cfg=config(5), top_logprobs=G, top_tokens=D), INVALID, "share memory")


def test_gradient_rules():
    dh, dw = M(G), W(ptr=H)

    def check(h=None, w=None, **kw):
        return mu.check_logprob_grad_args(h or M(), w or W(), **{**dict(targets=C, stats=D, grad_logprobs=E, dhidden=dh, dweight=dw), **kw})

    expect(check(), OK)
    expect(check(grad_entropy=F), OK)
    expect(check(grad_logprobs=None, grad_entropy=F), OK)
    expect(check(grad_entropy=E), OK)                                      # both are only read
    expect(check(dhidden=None), OK)
    expect(check(dweight=None), OK)
    expect(check(h=M(rows=0), dhidden=M(rows=0), targets=None, stats=None, grad_logprobs=None), OK)
    expect(check(dhidden=None, dweight=None), INVALID, "NULL dhidden")
    expect(check(stats=None), INVALID, "NULL stats")
    expect(check(grad_logprobs=None), INVALID, "NULL grad")
    expect(check(stats=D + 4), INVALID, "aligned")
    expect(check(grad_logprobs=E + 2), INVALID, "aligned")
    expect(check(grad_entropy=F + 2), INVALID, "aligned")
    expect(check(dhidden=M(G, dtype=F32)), DTYPE, "dhidden")
    expect(check(dweight=W(49, ptr=H)), SHAPE, "dweight")
    expect(check(dhidden=M(A)), INVALID, "share memory")
    expect(check(dweight=W(ptr=B)), INVALID, "share memory")
    expect(check(dweight=W(ptr=G)), INVALID, "share memory")
    expect(check(stats=G), INVALID, "share memory")
    expect(check(grad_logprobs=H), INVALID, "share memory")
    expect(check(targets=G), INVALID, "share memory")
    expect(check(cfg=config(0, -1.0)), INVALID, "softcap")
