"""The norms around a block on the GPU against plain 64-bit implementations.

Tolerances are element-wise bounds derived from the arithmetic, not fitted. With
u = 2^-24: a mean of squares takes at most 16 serial additions in a thread, 6
across a wave and 16 across waves, so it is within 42 u of itself and its
1 / sqrt, two roundings more, within 24 u; every other operation adds u of its
result, and errors of what goes in are carried through. A result is rounded once
to its type (bf16: 2^-8 of itself). Sums over n tokens take at most n / 256 + 72
serial additions of a channel (16 times as many where one value sums all of them).
"""
import pytest
import torch

import muon_newton_schulz_update_amd as mu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
STEP = {BF: 2.0 ** -8, F32: U}
TINY = 1e-37


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(shape, seed, sd=1.0):
    return torch.randn(shape, generator=gen(seed), device="cuda") * sd


def within(got, want, err, what):
    bad = ~((got.double() - want).abs() <= err)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, worst {float(((got.double() - want).abs() / err).max()):.3g}x")


def oracle(x, y, post_gain, gate, scale, pre_gain, post_norm, pre_norm, eps, dout=None, dhidden=None, like=None):
    """{name: (value, bound)} of results and gradients in 64 bits."""
    eps = float(torch.tensor(eps, dtype=F32))
    n, d = x.shape
    f = lambda t: None if t is None else t.double()
    one = torch.ones((), dtype=torch.float64, device="cuda")
    X, Y, g1, g, s, g2 = (f(t) for t in (x, y, post_gain, gate, scale, pre_gain))
    s, g, g1, g2 = (one if t is None else t for t in (s, g, g1, g2))
    ty = like if like is not None else x.dtype if y is None else y.dtype
    found = {}
    put = lambda name, value, err, t: found.__setitem__(name, (value, err + STEP[t] * value.abs() + TINY))
    o, o_err = s * X, 2 * U * (s * X).abs()
    r1 = yh = yh_err = None
    if y is not None:
        r1 = 1 / torch.sqrt(Y.square().mean(1, keepdim=True) + eps) if post_norm else one
        yh = Y * r1
        yh_err = yh.abs() * (26 * U if post_norm else 0)
        part = g * g1 * yh
        o = o + part
        o_err = o_err + (g * g1).abs() * yh_err + 3 * U * part.abs() + U * o.abs()
        put("out", o, o_err, x.dtype)
    if pre_norm:
        mean = o.square().mean(1, keepdim=True) + eps
        r2 = 1 / torch.sqrt(mean)
        rel2 = (o.abs() * o_err).mean(1, keepdim=True) / mean + 24 * U
        xh = o * r2
        xh_err = r2 * o_err + xh.abs() * (rel2 + U)
        put("hidden", xh * g2, xh_err * g2.abs() + 3 * U * (xh * g2).abs(), ty)
    if dout is None and dhidden is None:
        return found
    D = torch.zeros_like(X) if dout is None else dout.double()
    dt, dt_err = D, torch.zeros_like(X)
    sums = n / 256 + 72
    total = lambda t, err, k=1: (t.sum(0), err.sum(0) + (k * sums + 30) * U * t.abs().sum(0))
    if dhidden is not None:
        dh = dhidden.double()
        u = dh * g2
        m = (u * xh).mean(1, keepdim=True)
        m_err = (u.abs() * xh_err + 44 * U * (u * xh).abs()).mean(1, keepdim=True)
        back = r2 * (u - xh * m)
        dt = D + back
        dt_err = r2 * (2 * U * u.abs() + xh_err * m.abs() + xh.abs() * m_err) + (rel2 + 5 * U) * r2 * (u.abs() + (xh * m).abs())
        dt_err = dt_err + 2 * U * (D.abs() + back.abs())
        if pre_gain is not None:
            put("dpre_gain", *total(dh * xh, dh.abs() * xh_err + U * (dh * xh).abs()), pre_gain.dtype)
    elif pre_gain is not None:
        put("dpre_gain", torch.zeros_like(g2), torch.zeros_like(g2), pre_gain.dtype)
    put("dx", s * dt, s.abs() * dt_err + 2 * U * (s * dt).abs(), x.dtype)
    if scale is not None:
        t, e = dt * X, dt_err * X.abs() + U * (dt * X).abs()
        if scale.numel() == 1 and d > 1:
            put("dscale", t.sum().view(scale.shape), e.sum() + (16 * sums + 60) * U * t.abs().sum(), scale.dtype)
        else:
            a, b = total(t, e, 16)
            put("dscale", a.view(scale.shape), b.view(scale.shape), scale.dtype)
    if y is None:
        return found
    t, e = dt * yh, dt_err * yh.abs() + dt.abs() * yh_err + 3 * U * (dt * yh).abs()
    if gate is not None:
        a, b = t * g1, e * g1.abs() + 3 * U * (t * g1).abs()
        if gate.numel() == 1 and d > 1:
            put("dgate", a.sum().view(gate.shape), b.sum() + (16 * sums + 60) * U * a.abs().sum(), gate.dtype)
        elif gate.dim() == 2 and n > 1:
            put("dgate", a, b, gate.dtype)
        else:
            a, b = total(a, b, 16)
            put("dgate", a.view(gate.shape), b.view(gate.shape), gate.dtype)
    if post_gain is not None:
        put("dpost_gain", *total(t * g, e * g.abs() + 3 * U * (t * g).abs()), post_gain.dtype)
    v = g * dt * g1
    v_err = (g * g1).abs() * dt_err + 3 * U * v.abs()
    if not post_norm:
        put("dy", v, v_err, y.dtype)
        return found
    m = (v * yh).mean(1, keepdim=True)
    m_err = (v_err * yh.abs() + v.abs() * yh_err + 44 * U * (v * yh).abs()).mean(1, keepdim=True)
    put("dy", r1 * (v - yh * m), r1 * (v_err + yh_err * m.abs() + yh.abs() * m_err) + 30 * U * r1 * (v.abs() + (yh * m).abs()),
        y.dtype)
    return found


def check(x, y, *, dout=True, dhidden=True, seed=900, **kw):
    """Results and gradients of one call, against the oracle; returns them."""
    options = dict(dict(post_gain=None, gate=None, scale=None, pre_gain=None, post_norm=y is not None, pre_norm=True, eps=1e-6), **kw)
    ty = x.dtype if y is None else y.dtype
    dout = normal(x.shape, seed).to(x.dtype) if dout is True else dout
    dhidden = normal(x.shape, seed + 1).to(ty) if dhidden is True and options["pre_norm"] else dhidden if options["pre_norm"] else None
    if y is None:
        dout = None
        got = {"hidden": mu.rms_norm(x, options["pre_gain"], eps=options["eps"])}
        got.update(zip(("dx", "dpre_gain"), mu.rms_norm_grad(x, dhidden, options["pre_gain"], eps=options["eps"])))
    else:
        got = dict(zip(("out", "hidden"), mu.residual_norm(x, y, **options)))
        grads = mu.residual_norm_grad(x, y, dout, dhidden, **options)
        got.update({"d" + k: t for k, t in grads._asdict().items()})
    want = oracle(x, y, dout=dout, dhidden=dhidden, **options)
    for name, t in got.items():
        assert (t is None) == (name not in want), name
        if t is not None:
            within(t, *want[name], name)
    kinds = {"out": x, "hidden": y if y is not None else x, "dx": x, "dy": y, **{"d" + k: options[k] for k in ("post_gain", "gate", "scale", "pre_gain")}}
    for name, t in got.items():
        if t is not None:
            assert t.dtype == kinds[name].dtype and t.shape == kinds[name].shape, name
    return got


TYPES = [(BF, BF), (F32, BF), (F32, F32)]
IDS = ["bf16", "mixed", "fp32"]


def tensors(n, d, tx, ty, seed=0, gate="vector", scale="scalar", post=True, pre=True, tp=None):
    tp = tp or ty
    x, y = (3 * normal((n, d), seed)).to(tx), (normal((n, d), seed + 1) * torch.exp(normal((n, 1), seed + 2))).to(ty)
    shapes = {"scalar": (1,), "vector": (d,), "matrix": (n, d)}
    kw = dict(post_gain=(1 + 0.3 * normal((d,), seed + 3)).to(tp) if post else None,
              pre_gain=(1 + 0.3 * normal((d,), seed + 4)).to(tp) if pre else None,
              gate=None if gate is None else normal(shapes[gate], seed + 5).to(ty if gate == "matrix" else tp),
              scale=None if scale is None else (1 + 0.2 * normal(shapes[scale], seed + 6)).to(tp))
    return x, y, kw


@pytest.mark.parametrize("tx,ty", TYPES, ids=IDS)
@pytest.mark.parametrize("n,d", [(1, 1), (3, 2), (2, 7), (17, 8), (33, 31), (5, 64), (40, 128), (9, 129), (65, 200), (6, 512),
                                 (7, 513), (70, 768), (4, 1000), (3, 1024), (5, 1025), (9, 2048), (2, 2050), (3, 4096),
                                 (2, 4099), (3, 8192), (2, 8200), (5, 16383), (3, 16384), (1000, 96), (2600, 40)])
def test_shapes(n, d, tx, ty):
    x, y, kw = tensors(n, d, tx, ty, seed=n + d)
    check(x, y, **kw)
    check(x, None, pre_gain=kw["pre_gain"])


@pytest.mark.parametrize("tx,ty", TYPES, ids=IDS)
@pytest.mark.parametrize("gate", [None, "scalar", "vector", "matrix"])
@pytest.mark.parametrize("scale", [None, "scalar", "vector"])
@pytest.mark.parametrize("post_norm,pre_norm", [(True, True), (True, False), (False, True), (False, False)])
def test_options(tx, ty, gate, scale, post_norm, pre_norm):
    for n, d in ((37, 100), (19, 1100)):
        x, y, kw = tensors(n, d, tx, ty, seed=5, gate=gate, scale=scale, post=post_norm, pre=pre_norm, tp=F32 if gate == "scalar" else None)
        check(x, y, post_norm=post_norm, pre_norm=pre_norm, **kw)


@pytest.mark.parametrize("dout,dhidden", [(None, True), (True, None)])
@pytest.mark.parametrize("d", [96, 2000])
def test_one_gradient_comes_in(dout, dhidden, d):
    x, y, kw = tensors(50, d, F32, BF, seed=8, gate="matrix", scale="vector")
    check(x, y, dout=dout, dhidden=dhidden, **kw)


def test_without_gains():
    for gate in (None, "matrix"):
        x, y, kw = tensors(70, 768, BF, BF, seed=9, gate=gate, post=False, pre=False)
        check(x, y, **kw)


@pytest.mark.parametrize("eps", [1e-12, 1e-2, 10.0])
def test_eps_and_zero_rows(eps):
    x, y, kw = tensors(20, 300, F32, F32, seed=11, scale=None)
    x[3], y[3], y[7], x[9] = 0, 0, 0, 0
    got = check(x, y, eps=eps, **kw)
    assert not bool(got["out"][3].any()) and not bool(got["hidden"][3].any())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_value_stays_in_its_row(value):
    for d in (96, 768, 3000):
        x, y, kw = tensors(30, d, BF, BF, seed=12)
        clean = mu.residual_norm(x, y, **kw)
        dirty = x.clone()
        dirty[11, 5] = value
        out, hidden = mu.residual_norm(dirty, y, **kw)
        grads = mu.residual_norm_grad(dirty, y, out.nan_to_num(0, 0, 0), hidden.nan_to_num(0, 0, 0), **kw)
        rest = torch.arange(30, device="cuda") != 11
        assert torch.equal(out[rest], clean[0][rest]) and torch.equal(hidden[rest], clean[1][rest])
        assert bool(torch.isfinite(grads.x[rest].float()).all()) and not bool(torch.isfinite(out[11, 5]))


def test_no_tokens():
    for tp in (F32, BF):
        x, y, kw = tensors(0, 300, F32, BF, gate="vector", tp=tp)
        out, hidden = mu.residual_norm(x, y, **kw)
        assert out.shape == hidden.shape == (0, 300) and hidden.dtype == BF
        grads = mu.residual_norm_grad(x, y, out, hidden, **kw)
        for k in ("post_gain", "gate", "scale", "pre_gain"):
            assert getattr(grads, k).shape == kw[k].shape and not bool(getattr(grads, k).any())
    full = torch.empty((0, 300), device="cuda", dtype=BF)
    assert mu.residual_norm_grad(x, y, out, hidden, gate=full).gate.shape == (0, 300)


def test_shapes_of_more_dimensions_and_a_single_row():
    x, y, kw = tensors(24, 96, BF, BF, seed=14, gate="matrix")
    flat = mu.residual_norm(x, y, **kw)
    kw3 = dict(kw, gate=kw["gate"].view(2, 3, 4, 96))
    deep = mu.residual_norm(x.view(2, 3, 4, 96), y.view(2, 3, 4, 96), **kw3)
    assert all(a.shape == (2, 3, 4, 96) and torch.equal(a.view(24, 96), b) for a, b in zip(deep, flat))
    g = mu.residual_norm_grad(x.view(2, 3, 4, 96), y.view(2, 3, 4, 96), *deep, **kw3)
    h = mu.residual_norm_grad(x, y, *flat, **kw)
    assert g.gate.shape == (2, 3, 4, 96) and all(torch.equal(a.flatten(), b.flatten()) for a, b in zip(g, h))
    one = mu.residual_norm(x[7], y[7], **dict(kw, gate=kw["gate"][7]))
    assert all(torch.equal(a, b[7]) for a, b in zip(one, flat))
    assert torch.equal(mu.rms_norm(x.float(), dtype=BF), mu.rms_norm(x.float()).to(BF))


@pytest.mark.parametrize("tx,ty", TYPES, ids=IDS)
@pytest.mark.parametrize("d,pad,shift", [(96, 8, 0), (97, 3, 1), (768, 5, 3), (2100, 1, 1)])
def test_strides_and_alignment(tx, ty, d, pad, shift):
    """Rows inside wider buffers, starts off 16 bytes, NaN all around."""
    n = 23
    x, y, kw = tensors(n, d, tx, ty, seed=16, gate="matrix", scale="vector")

    def inside(t):
        buf = torch.full((n * (d + pad) + shift + 64,), float("nan"), device="cuda", dtype=t.dtype)
        view = buf[shift:shift + n * (d + pad)].view(n, d + pad)[:, :d]
        view.copy_(t)
        return buf, view

    off = lambda t: None if t is None else torch.cat((t[:1], t))[1:]
    kw2 = {k: inside(t)[1] if t.dim() == 2 else off(t) for k, t in kw.items()}
    (_, x2), (_, y2) = inside(x), inside(y)
    a, b = mu.residual_norm(x, y, **kw), mu.residual_norm(x2, y2, **kw2)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    (_, do), (_, dh) = inside(a[0]), inside(a[1])
    g, h = mu.residual_norm_grad(x, y, *a, **kw), mu.residual_norm_grad(x2, y2, do, dh, **kw2)
    assert all(torch.equal(p, q) for p, q in zip(g, h))


@pytest.mark.parametrize("d", [100, 1500])
def test_outputs_leave_what_is_around_them(d):
    """The C call into strided outputs."""
    import ctypes

    from muon_newton_schulz_update_amd import MuonMatrix

    n, handle = 21, mu.get_handle()
    handle._bind_stream()
    x, y, kw = tensors(n, d, F32, BF, seed=18)
    desc = lambda t: MuonMatrix(t.data_ptr(), t.shape[0], t.shape[1], t.stride(0), int(t.dtype == BF))
    bufs = [torch.full((n + 2, d + 9), 7.0, device="cuda", dtype=t) for t in (F32, BF, F32, BF)]
    views = [b[1:-1, 4:4 + d] for b in bufs]
    m = [desc(t) for t in (x, y, *views)]
    p = mu.NormParams(None, None, None, None, 1, 1, 1e-6)
    ref = ctypes.byref
    assert handle._lib.residual_norm(handle.ptr, ref(m[0]), ref(m[1]), ref(p), ref(m[2]), ref(m[3])) == 0
    grads = mu.norms._GradPointers(ctypes.addressof(m[4]), ctypes.addressof(m[5]))
    assert handle._lib.residual_norm_grad(handle.ptr, ref(m[0]), ref(m[1]), ref(p), ref(m[2]), ref(m[3]), ref(grads)) == 0
    want = mu.residual_norm(x, y)
    want += tuple(mu.residual_norm_grad(x, y, *want))[:2]
    for b, v, w in zip(bufs, views, want):
        assert torch.equal(v, w)
        v.fill_(7.0)
        assert bool((b == 7.0).all())


def test_gradient_of_autograd_and_by_differences():
    """autograd gives what the explicit calls do; 64-bit differences of the results along random directions give the
    gradients' products with them (central differences of step e: e^2 of third derivatives, below 1e-8 here)."""
    x, y, kw = tensors(40, 200, F32, F32, seed=21, gate="matrix", scale="vector")
    leaves = dict(x=x, y=y, **kw)
    for t in leaves.values():
        t.requires_grad_()
    out, hidden = mu.residual_norm(x, y, **kw)
    co, ch = normal(out.shape, 22), normal(out.shape, 23)
    got = torch.autograd.grad([out, hidden], list(leaves.values()), [co, ch])
    plain = {k: t.detach() for k, t in kw.items()}
    want = mu.residual_norm_grad(x.detach(), y.detach(), co, ch, **plain)._asdict()
    assert all(torch.equal(g, want[k]) for k, g in zip(leaves, got))

    def value(**t):
        r = oracle(t["x"], t["y"], t["post_gain"], t["gate"], t["scale"], t["pre_gain"], True, True, 1e-6)
        return float((r["out"][0] * co).sum() + (r["hidden"][0] * ch).sum())

    for i, (name, t) in enumerate(leaves.items()):
        way = normal(t.shape, 30 + i).double()
        base = {k: v.detach().double() for k, v in leaves.items()}
        STEP[torch.float64] = 0.0
        e = 1e-5
        slope = (value(**dict(base, **{name: base[name] + e * way})) - value(**dict(base, **{name: base[name] - e * way}))) / (2 * e)
        mine = float((want[name].double() * way).sum())
        size = float((want[name].double() * way).abs().sum())
        assert abs(slope - mine) <= 1e-5 * size, (name, slope, mine)
    # one of the two results alone, a broadcast gradient, and inputs that need none
    out, hidden = mu.residual_norm(x, y, **kw)
    g = torch.autograd.grad(hidden.sum(), [x, kw["gate"]], retain_graph=True)
    w = mu.residual_norm_grad(x.detach(), y.detach(), None, torch.ones_like(hidden), **plain)
    assert torch.equal(g[0], w.x) and torch.equal(g[1], w.gate)
    out, hidden = mu.residual_norm(x.detach(), y, **plain)
    (g,) = torch.autograd.grad(out.square().sum(), [y])
    assert torch.equal(g, mu.residual_norm_grad(x.detach(), y.detach(), 2 * out.detach(), None, **plain).y)
    h = mu.rms_norm(x, kw["pre_gain"])
    g = torch.autograd.grad(h, [x, kw["pre_gain"]], ch)
    assert all(torch.equal(a, b) for a, b in zip(g, mu.rms_norm_grad(x.detach(), ch, plain["pre_gain"])))
    with torch.no_grad():
        assert not mu.rms_norm(x, kw["pre_gain"]).requires_grad


def test_first_norm_of_a_32_bit_residual_for_16_bit_blocks():
    x, gain = (3 * normal((70, 300), 41)).requires_grad_(), (1 + 0.3 * normal((300,), 42)).to(BF).requires_grad_()
    h = mu.rms_norm(x, gain, dtype=BF)
    dh = normal((70, 300), 43).to(BF)
    dx, dgain = torch.autograd.grad(h, [x, gain], dh)
    want = oracle(x.detach(), None, None, None, None, gain.detach(), False, True, 1e-6, dhidden=dh, like=BF)
    assert h.dtype == BF and dx.dtype == F32 and dgain.dtype == BF
    for name, t in (("hidden", h), ("dx", dx), ("dpre_gain", dgain)):
        within(t, *want[name], name)
    explicit = mu.rms_norm_grad(x.detach(), dh, gain.detach())
    assert torch.equal(explicit[0], dx) and torch.equal(explicit[1], dgain)


def test_repeats_bit_for_bit_and_on_another_stream():
    x, y, kw = tensors(3000, 768, BF, BF, seed=25)
    first = (*mu.residual_norm(x, y, **kw), *mu.residual_norm_grad(x, y, x, y, **kw))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = (*mu.residual_norm(x, y, **kw), *mu.residual_norm_grad(x, y, x, y, **kw))
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_in_a_graph():
    x, y, kw = tensors(500, 320, F32, BF, seed=26, gate="matrix")
    handle, s = mu.Handle(), torch.cuda.Stream()
    xs = x.clone()

    def call():
        out, hidden = mu.residual_norm(xs, y, handle=handle, **kw)
        return (out, hidden, *mu.residual_norm_grad(xs, y, out, hidden, handle=handle, **kw))

    with torch.cuda.stream(s):
        call()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            captured = call()
        for k in range(4):
            xs.copy_(x * (k + 1))
            for t in captured:
                t.fill_(float("nan"))
            graph.replay()
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(captured, call())), k
            # an eager call of more channels grows the workspace, which the graph keeps
            mu.rms_norm_grad(normal((5000, 2000 * (k + 1)), k), normal((5000, 2000 * (k + 1)), k), normal((2000 * (k + 1),), 3), handle=handle)
    s.synchronize()
    handle.close()


def test_past_32_bit_offsets():
    n, d = (1 << 20) + 3, 4099
    x = torch.zeros((n, d), device="cuda", dtype=BF)
    y = torch.zeros((n, d), device="cuda", dtype=BF)
    rows = torch.tensor([0, 5, 524287, 524288, n - 2, n - 1], device="cuda")
    a, b, kw = tensors(len(rows), d, BF, BF, seed=28)
    x[rows], y[rows] = a, b
    out, hidden = mu.residual_norm(x, y, **kw)
    want = mu.residual_norm(a, b, **kw)
    assert torch.equal(out[rows], want[0]) and torch.equal(hidden[rows], want[1])
    grads = mu.residual_norm_grad(x, y, out, hidden, **kw)
    small = mu.residual_norm_grad(a, b, *want, **kw)
    assert torch.equal(grads.x[rows], small.x) and torch.equal(grads.y[rows], small.y)
    # the other rows add zeros: the same sums in another order, each rounded once more
    for k in ("post_gain", "gate", "pre_gain"):
        p, q = getattr(grads, k).float(), getattr(small, k).float()
        assert float((p - q).norm() / q.norm()) <= 2.0 ** -8


def test_refusals():
    x, y, kw = tensors(10, 64, BF, BF, seed=31)
    f32 = x.float()
    bad = [
        lambda: mu.residual_norm(x, y.float()),
        lambda: mu.residual_norm(x, y[:9]),
        lambda: mu.residual_norm(x, y[:, :32]),
        lambda: mu.residual_norm(x, y.view(2, 5, 64)),
        lambda: mu.residual_norm(x.half(), y.half()),
        lambda: mu.residual_norm(x.cpu(), y.cpu()),
        lambda: mu.residual_norm(x, y.cpu()),
        lambda: mu.residual_norm(x, y, gate=kw["gate"].cpu()),
        lambda: mu.residual_norm(x, y, gate=f32),
        lambda: mu.residual_norm(x, y, gate=kw["gate"][:32]),
        lambda: mu.residual_norm(x, y, gate=y[:1].expand(10, 64)),
        lambda: mu.residual_norm(x, y, scale=x),
        lambda: mu.residual_norm(x, y, pre_gain=kw["gate"][:1]),
        lambda: mu.residual_norm(x, y, pre_norm=False, pre_gain=kw["pre_gain"]),
        lambda: mu.residual_norm(x, y, post_norm=False, post_gain=kw["post_gain"]),
        lambda: mu.residual_norm(x, y, eps=0.0),
        lambda: mu.residual_norm(x, y, eps=float("nan")),
        lambda: mu.residual_norm(x.t().contiguous().t(), y),
        lambda: mu.rms_norm(x, dtype=F32),
        lambda: mu.rms_norm(x, dtype=torch.float16),
        lambda: mu.rms_norm(torch.zeros((2, 16385), device="cuda")),
        lambda: mu.rms_norm(torch.zeros((2, 0), device="cuda")),
        lambda: mu.residual_norm_grad(x, y, None, None),
        lambda: mu.residual_norm_grad(x, y, f32, y),
        lambda: mu.residual_norm_grad(x, y, x, f32),
        lambda: mu.residual_norm_grad(x, y, x[:9], y),
        lambda: mu.residual_norm_grad(x, y, x, y, pre_norm=False),
        lambda: mu.rms_norm_grad(x, f32),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            f()
            pytest.fail(f"call {i} was accepted")
