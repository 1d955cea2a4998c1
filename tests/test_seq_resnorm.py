"""The norms around a block with its gate and residual scale, forward and backward, through the C-ABI against float64."""
import ctypes
import itertools

import pytest

# unit roundoff (half a last place over the value): 24, 8 and 11 significant bits
U = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
U32 = 2.0 ** -24
# A float32 sum of a row: each thread adds at most 32 values (rows of up to 16384; 16 + d / 1024 beyond) and a
# tree of 10 levels follows; with the few roundings of the formulas, 64 units of the terms' sizes bound it.
E = 64 * U32
# the activations are good to 16 units of the argument's size, their slopes to four times that
AEVAL = 16 * U32
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def _torch():
    import torch
    return torch


@pytest.fixture(scope="module")
def seq():
    import mixed_precision_refinement_gb300 as zs
    s = zs.Seq()
    yield s
    zs.zsolve_seq_check(s.seq)  # no wait gave up in any of the tests
    s.close()


def _inputs(rows, d, dtype, wdtype, gate=True, scaled=True, weights=True, seed=0, pad=0, shift=0):
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(seed)

    def rand(n=rows):
        buf = torch.randn(n * (d + pad) + shift, generator=gen, device="cuda").to(dtype)
        return buf[shift:].view(n, d + pad)[:, :d]

    def vec(mean, size):
        return (mean + size * torch.randn(d, generator=gen, device="cuda")).to(wdtype)

    i = dict(x=rand(), o=rand(), z=rand() if gate else None, c=vec(0.5, 0.2) if scaled else None)
    for n, m in (("w1", 1), ("b1", 0), ("w2", 1), ("b2", 0)):
        i[n] = vec(m, 0.3) if weights else None
    return i, rand(), rand()


def _act64(z, act):
    torch = _torch()
    f = torch.nn.functional
    z = z.detach().requires_grad_()
    a = {"none": lambda t: t * 1, "relu": torch.relu, "silu": f.silu, "gelu": f.gelu,
         "gelu_tanh": lambda t: f.gelu(t, approximate="tanh")}[act](z)
    s, = torch.autograd.grad(a.sum(), z)
    return a.detach(), s


def _mean(t):
    return t.mean(1, keepdim=True)


def _near(got, ref, tol, dtype, what):
    tol = tol + U[dtype] * (ref.abs() + tol) + (2.0 ** -25 if dtype == "float16" else 1e-30)  # float16: half its smallest step
    off = (got.double() - ref).abs() / tol
    assert bool((off <= 1).all()), (what, float(off.max()), int((off > 1).sum()))


def _check(seq, i, dy, dh, act, kind, after, types, eps=1e-5):
    torch = _torch()
    dt, wdt = types
    D = {n: None if t is None else t.double() for n, t in i.items()}
    one, zero = torch.ones_like(D["o"][0]), torch.zeros_like(D["o"][0])
    w1, b1, c, w2, b2 = (D[n] if D[n] is not None else e for n, e in (("w1", one), ("b1", zero), ("c", one), ("w2", one), ("b2", zero)))
    args = dict(z=i["z"], act=act, c=i["c"], w2=i["w2"], b2=i["b2"], kind=kind, after=after)
    y, h, stats = seq.resnorm(i["x"], i["o"], i["w1"], i["b1"], eps=eps, **args)

    def standard(v):
        mu = _mean(v) if kind == "layer" else torch.zeros_like(v[:, :1])
        rs = 1 / (_mean((v - mu).square()) + eps).sqrt()
        return (v - mu) * rs, mu, rs, (v.abs().amax(1, keepdim=True) + mu.abs()) * rs  # the last: what a mean's error is relative to

    o, x = D["o"], D["x"]
    h1, mu1, rs1, size1 = standard(o) if after else (o, 0 * o[:, :1], 0 * o[:, :1] + 1, o.abs())
    t = h1 * w1 + b1
    a, slope = _act64(D["z"], act) if i["z"] is not None else (torch.ones_like(o), torch.zeros_like(o))
    aev = AEVAL * (1 + D["z"].abs()) if i["z"] is not None else torch.zeros_like(o)
    ttol = E * (1 + size1 + h1.abs()) * w1.abs() + E * t.abs()
    yref = x + c * a * t
    ytol = c.abs() * (a.abs() * ttol + aev * (t.abs() + ttol)) + E * ((c * a * t).abs() + x.abs())
    _near(y, yref, ytol, dt, "y")
    h2, mu2, rs2, size2 = standard(yref)
    worst = ytol.amax(1, keepdim=True)
    h2tol = rs2 * 2 * worst * (1 + h2.abs()) + E * (1 + size2 + h2.abs())
    _near(h, h2 * w2 + b2, h2tol * w2.abs() + E * b2.abs(), dt, "h")
    for k, (ref, tol) in enumerate(((mu1, E * o.abs().amax(1, keepdim=True)), (rs1, E * (1 + size1.amax(1, keepdim=True)) * rs1),
                                    (mu2, worst + E * yref.abs().amax(1, keepdim=True)), (rs2, (E * (1 + size2) + 2 * worst * rs2) * rs2))):
        if kind == "rms" and k % 2 == 0 or not after and k < 2:
            assert torch.equal(stats[:, k:k + 1].double(), ref)
        elif i["o"].shape[1] > 1:
            _near(stats[:, k:k + 1], ref, tol, "float32", f"stats {k}")

    got = seq.resnorm_bwd(dh, y, i["o"], stats, i["w1"], i["b1"], dy=dy, **args)
    mu1, rs1, mu2, rs2 = stats.double().split(1, 1)
    yd, dh, dy = y.double(), dh.double(), dy.double() if dy is not None else torch.zeros_like(o)
    layer = kind == "layer"

    def slope_of(v, g, rs):
        return rs * (g - (_mean(g) if layer else 0) - v * _mean(g * v))

    def slope_tol(v, g, gtol, rs, size):
        whole = g.abs() + _mean(g.abs()) + (v.abs() + E * size) * _mean(g.abs() * (v.abs() + E * size))
        return rs * (gtol + _mean(gtol) + v.abs() * _mean(gtol * v.abs()) + E * whole * (1 + size))

    h2, size2 = (yd - mu2) * rs2, (yd.abs().amax(1, keepdim=True) + mu2.abs()) * rs2
    a2 = dh * w2
    dx = dy + slope_of(h2, a2, rs2)
    xtol = slope_tol(h2, a2, U32 * a2.abs(), rs2, size2) + E * dy.abs()
    h1 = (o - mu1) * rs1
    size1 = (o.abs().amax(1, keepdim=True) + mu1.abs()) * rs1 if after else 0 * rs1
    t = h1 * w1 + b1
    ttol = E * (1 + size1 + h1.abs()) * w1.abs() + E * t.abs()
    u, utol = dx * a, a.abs() * xtol + aev * (dx.abs() + xtol)
    p, ptol = u * c, c.abs() * utol + E * (u * c).abs()
    a1 = p * w1
    do, dotol = (slope_of(h1, a1, rs1), slope_tol(h1, a1, ptol * w1.abs() + E * a1.abs(), rs1, size1)) if after else (a1, ptol * w1.abs() + E * a1.abs())
    dz = dx * c * t * slope
    dztol = (c * t).abs() * (slope.abs() * xtol + 4 * aev * (dx.abs() + xtol)) + (c * slope * dx).abs() * ttol + E * dz.abs()
    sums = E + i["o"].shape[0] * U32
    cols = dict(w1=(p * h1, ptol * h1.abs() + (p * size1).abs() * E + sums * (p * h1).abs()), b1=(p, ptol + sums * p.abs()),
                c=(u * t, (utol + sums * u.abs() * (1 + size1)) * ((h1 * w1).abs() + b1.abs()) + u.abs() * ttol),
                w2=(dh * h2, dh.abs() * E * size2 + sums * (dh * h2).abs()), b2=(dh, sums * dh.abs()))
    _near(got[0], dx, xtol, dt, "dx")
    _near(got[1], do, dotol, dt, "do")
    if i["z"] is None:
        assert got[2] is None
    else:
        _near(got[2], dz, dztol, dt, "dz")
    for n, g in zip(("w1", "b1", "c", "w2", "b2"), got[3:]):
        if i[n] is None:
            assert g is None
        else:
            _near(g, cols[n][0].sum(0), cols[n][1].sum(0), wdt, "d" + n)


WIDTHS = [1, 2, 7, 8, 64, 255, 256, 257, 512, 520, 1000, 1024, 1025, 2048, 2157, 4096, 4104, 8192, 8200, 16384, 16392]
TYPES = [("float32", "float32"), ("bfloat16", "bfloat16"), ("bfloat16", "float32"), ("float16", "float16")]


@pytest.mark.gpu
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_widths(seq, d, types):
    torch = _torch()
    rows = 700 if d <= 4104 else 9
    i, dy, dh = _inputs(rows, d, *(getattr(torch, t) for t in types), seed=d)
    _check(seq, i, dy, dh, ACTS[d % 5], "rms" if d % 3 == 1 else "layer", True, types)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(12001, 1), (12000, 5), (12003, 64), (9001, 250), (5000, 520), (3001, 1111), (1501, 4100), (900, 8192)])
@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_many_rows_a_block(seq, rows, d, types):
    torch = _torch()
    i, dy, dh = _inputs(rows, d, *(getattr(torch, t) for t in types), seed=d + 1)
    _check(seq, i, dy, dh, ACTS[d % 5], "layer" if d % 3 == 1 else "rms", True, types)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [5, 264, 2157])
def test_statistics_off_16_bytes(seq, d):
    """Statistics that start anywhere give what aligned ones do, but for the order of the sums."""
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    i, dy, dh = _inputs(300, d, torch.float32, torch.float32, seed=3)
    weights = dict(z=i["z"], act="silu", c=i["c"], w2=i["w2"], b2=i["b2"])
    y, _, stats = seq.resnorm(i["x"], i["o"], i["w1"], i["b1"], **weights)
    moved = torch.empty(1201, device="cuda")[1:].view(300, 4)
    moved.copy_(stats)
    one, other = (seq.resnorm_bwd(dh, y, i["o"], t, i["w1"], i["b1"], dy=dy, **weights) for t in (stats, moved))
    for a, b in zip(one, other):
        # each is off by at most a few hundred float32 roundings of its terms, which are of a few times the largest result
        assert float((a - b).abs().max()) <= 2.0 ** -24 * 600 * 4 * float(a.abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("after", [True, False])
@pytest.mark.parametrize("gate", [None] + ACTS)
def test_forms(seq, kind, after, gate):
    torch = _torch()
    for n, (scaled, weights, grad_y, d) in enumerate(itertools.product([True, False], [True, False], [True, False], [72, 8200])):
        types = TYPES[n % 4]
        i, dy, dh = _inputs(5, d, *(getattr(torch, t) for t in types), gate=gate is not None, scaled=scaled, weights=weights, seed=n)
        _check(seq, i, dy if grad_y else None, dh, gate or "silu", kind, after, types)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (8, 8), (1, 16)])
@pytest.mark.parametrize("d", [264, 3, 1500])
def test_strides_and_alignment(seq, dtype, pad, shift, d):
    torch = _torch()
    dt = getattr(torch, dtype)
    i, dy, dh = _inputs(300, d, dt, dt, seed=3, pad=pad, shift=shift)
    _check(seq, i, dy, dh, "silu", "layer", True, (dtype, dtype))


@pytest.mark.gpu
def test_an_offset_costs_no_digits(seq):
    """A residual stream with a large offset: h keeps float32's digits of the differences."""
    torch = _torch()
    i, dy, dh = _inputs(20, 1000, torch.float32, torch.float32, seed=8)
    i["x"] += 512.0
    i["x"], i["o"] = (i["x"] * 64).round() / 64, i["o"] + 256.0
    y, h, stats = seq.resnorm(i["x"], i["o"], c=torch.zeros(1000, device="cuda"))
    ref = torch.nn.functional.layer_norm(i["x"].double(), (1000,))
    assert float((h.double() - ref).abs().max()) <= E * 8
    t = seq.resnorm(torch.zeros_like(i["x"]), i["o"])[0]
    assert float((t.double() - torch.nn.functional.layer_norm(i["o"].double(), (1000,))).abs().max()) <= E * 8


@pytest.mark.gpu
@pytest.mark.parametrize("d", [200, 4096, 20000])
def test_sum_in_place(seq, d):
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    i, _, _ = _inputs(11, d, torch.bfloat16, torch.bfloat16, seed=d)
    y, h, _ = seq.resnorm(i["x"], i["o"], i["w1"], i["b1"], z=i["z"], c=i["c"], w2=i["w2"], b2=i["b2"])
    x, h2 = i["x"].clone(), torch.empty_like(i["x"])
    zs.zsolve_resnorm(seq.seq, x, i["o"], i["w1"], i["b1"], i["z"], "silu", i["c"], i["w2"], i["b2"], "layer", True, 1e-5, x, h2)
    assert torch.equal(x, y) and torch.equal(h, h2)


@pytest.mark.gpu
def test_some_gradients_only_and_the_same_twice(seq):
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    for d, rows in ((200, 20011), (2157, 500), (8200, 70)):
        i, dy, dh = _inputs(rows, d, torch.float32, torch.float32, seed=5)
        w = {n: i[n] for n in ("w1", "b1", "z", "c", "w2", "b2")}
        y, _, stats = seq.resnorm(i["x"], i["o"], **w)
        ref = seq.resnorm_bwd(dh, y, i["o"], stats, dy=dy, **w)
        for got, want in zip(seq.resnorm_bwd(dh, y, i["o"], stats, dy=dy, **w), ref):
            assert torch.equal(got, want)
        for which in (None, 2, 3, 4, 5, 6, 7):
            dx, do = torch.empty_like(y), torch.empty_like(y)
            rest = [torch.zeros_like(t) if n == which else None for n, t in enumerate(ref)][2:]
            zs.zsolve_resnorm_bwd(seq.seq, dh, dy, y, i["o"], stats, i["w1"], i["b1"], i["z"], "silu", i["c"], i["w2"], i["b2"], "layer",
                                  True, dx, do, *rest)
            assert torch.equal(dx, ref[0]) and torch.equal(do, ref[1])
            assert which is None or torch.equal(rest[which - 2], ref[which])


@pytest.mark.gpu
def test_no_rows_constant_rows_and_nonfinite(seq):
    torch = _torch()
    i, dy, dh = _inputs(6, 96, torch.float32, torch.float32, seed=6)
    w = {n: i[n] for n in ("w1", "b1", "c", "w2", "b2")}
    none = torch.empty(0, 96, device="cuda")
    y, h, stats = seq.resnorm(none, none, z=none, **w)
    assert y.shape == h.shape == (0, 96) and stats.shape == (0, 4)
    dx, do, dz, *sums = seq.resnorm_bwd(none, none, none, stats, z=none, **w)
    assert dx.shape == do.shape == dz.shape == (0, 96) and not any(bool(t.any()) for t in sums)

    const = torch.full((3, 40), 7.25, device="cuda")
    y, h, stats = seq.resnorm(const, const)  # no variance: both norms are zero
    assert torch.equal(y, const) and not h.any() and float((stats[:, 1::2] - 1e-5 ** -0.5).abs().max()) < 1e-3

    # a row that is not finite spoils that row alone, in each of the tensors
    args = {n: i[n] for n in ("x", "o", "z")}
    y, h, stats = seq.resnorm(**args, **w)
    keep = [0, 1, 3, 5]
    for name in args:
        bad = {n: t.clone() for n, t in args.items()}
        bad[name][2, 5], bad[name][4, 0] = float("inf"), float("nan")
        y2, h2, _ = seq.resnorm(**bad, **w)
        assert torch.isnan(h2[2]).all() and torch.isnan(h2[4]).all() and torch.equal(h2[keep], h[keep]) and torch.equal(y2[keep], y[keep])
    ref = seq.resnorm_bwd(dh, y, i["o"], stats, z=i["z"], dy=dy, **w)
    for name in ("dh", "dy", "y", "o", "z"):
        bad = {n: t.clone() for n, t in dict(dh=dh, dy=dy, y=y, o=i["o"], z=i["z"]).items()}
        bad[name][2, 5] = float("nan")
        for p, q in zip(seq.resnorm_bwd(stats=stats, **bad, **w)[:3], ref):
            assert torch.equal(p[keep + [4]], q[keep + [4]])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gradient_against_differences(seq, kind):
    """The derivative of a sum of the outputs along a direction, from forward values at +- h and +- 2 h (Richardson): off by
    the outputs' rounding over h and by at most the difference of the two estimates."""
    torch = _torch()
    i, dy, dh = _inputs(4, 48, torch.float32, torch.float32, seed=9)
    names = ("x", "o", "z", "w1", "b1", "c", "w2", "b2")
    y, _, stats = seq.resnorm(**i, act="gelu", kind=kind)
    dx, do, dz, *sums = seq.resnorm_bwd(dh, y, i["o"], stats, i["w1"], i["b1"], i["z"], "gelu", i["c"], i["w2"], i["b2"], dy, kind)
    step = 2.0 ** -6
    for name, grad in zip(names, (dx, do, dz, *sums)):
        along = torch.randn(i[name].shape, generator=torch.Generator("cuda").manual_seed(1), device="cuda") / 4

        def value(t):
            a, b, _ = seq.resnorm(**{**i, name: i[name] + t * along}, act="gelu", kind=kind)
            return float((a.double() * dy.double()).sum() + (b.double() * dh.double()).sum())

        val = {t: value(t * step) for t in (-2, -1, 1, 2)}
        d1, d2 = (val[1] - val[-1]) / (2 * step), (val[2] - val[-2]) / (4 * step)
        terms = grad.double() * along.double()
        noise = 2 / step * E * float((y.abs() * dy.abs()).sum() + 8 * dh.abs().sum())
        assert abs((4 * d1 - d2) / 3 - float(terms.sum())) <= noise + abs(d1 - d2) + E * float(terms.abs().sum()), name


@pytest.mark.gpu
@pytest.mark.parametrize("wtype", ["bfloat16", "float32"])
def test_autograd(seq, wtype):
    torch = _torch()
    i, dy, dh = _inputs(60, 72, torch.bfloat16, getattr(torch, wtype), seed=1)
    i = {n: t.view(3, 20, 72) if t.dim() == 2 else t for n, t in i.items()}
    dy, dh = dy.view(3, 20, 72), dh.view(3, 20, 72)
    w = {n: i[n] for n in ("w1", "b1", "z", "c", "w2", "b2")}
    y0, h0, stats = seq.resnorm(**i)
    assert stats.shape == (3, 20, 4)
    names = ("x", "o", "z", "w1", "b1", "c", "w2", "b2")
    for grads, use in (((dy, dh), 3), ((None, dh), 2), ((dy, None), 1)):
        leaves = {n: t.clone().requires_grad_() for n, t in i.items()}
        y, h, st = seq.resnorm(**leaves)
        assert torch.equal(y, y0) and torch.equal(h, h0)
        torch.autograd.backward([t for n, t in enumerate((y, h)) if use >> n & 1], [g for g in grads if g is not None])
        ref = seq.resnorm_bwd(grads[1] if grads[1] is not None else torch.zeros_like(dh), y0, i["o"], stats, dy=grads[0], **w)
        for n, want in zip(names, ref):
            assert torch.equal(leaves[n].grad, want), n
    with pytest.raises(RuntimeError, match="stats"):
        seq.resnorm(**{n: t.clone().requires_grad_() for n, t in i.items()})[2].sum().backward()
    C = i["c"].clone().requires_grad_()  # one of them alone
    seq.resnorm(**{**i, "c": C})[1].float().sum().backward()
    assert torch.equal(C.grad, seq.resnorm_bwd(torch.ones_like(dh), y0, i["o"], stats, **w)[5])


@pytest.mark.gpu
def test_refusals(seq):
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    x, w = torch.ones(4, 16, device="cuda"), torch.ones(16, device="cuda")
    for bad in (dict(o=x[:3]), dict(o=x[:, :8]), dict(o=x, z=x[:3]), dict(o=x, w1=w[:8]), dict(o=x, act="swish", z=x), dict(o=x, kind="batch"),
                dict(o=x, c=torch.ones(32, device="cuda")[::2])):
        with pytest.raises(ValueError):
            seq.resnorm(x, **bad)
    for bad in (dict(o=x.half()), dict(o=x, z=x.bfloat16()), dict(o=x, w1=w.half()), dict(o=x, w1=w, b2=w.half())):
        with pytest.raises(TypeError):
            seq.resnorm(x, **bad)
    y, h, stats = seq.resnorm(x, x)
    with pytest.raises(ValueError):
        seq.resnorm_bwd(h, y, x, stats[:, :3])
    with pytest.raises(ValueError):  # as many values, in another order (of as many rows as values it could not be told)
        seq.resnorm_bwd(h[:3], y[:3], x[:3], stats[:3].T.contiguous())
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(zs.ZsolveError) as e:
            seq.resnorm(x, x, eps=eps)
        assert e.value.status == zs.ZSOLVE_EINVAL


def _calls(lib, handle):
    p = 64  # never read: every call below is refused before the device is touched
    good = dict(type=1, wtype=1, kind=0, after=1, act=0, rows=4, d=8, o=p, z=None, ldo=8, ldz=8, w1=None, b1=None, c=None, w2=None, b2=None,
                eps=1e-5)

    def args(**over):
        from mixed_precision_refinement_gb300 import seq as binding
        a = {**good, **over}
        return binding.zsolve_resnorm_args(*(a[n] for n, _ in binding.zsolve_resnorm_args._fields_))

    def fwd(x=p, ldx=8, y=p, ldy=8, h=p, ldh=8, a=None, **over):
        a = ctypes.byref(args(**over)) if a is None else a or None
        return lib.zsolve_resnorm(handle, a, x, ldx, y, ldy, h, ldh, None)

    def bwd(dh=p, lddh=8, dy=None, lddy=8, y=p, ldy=8, stats=p, dx=p, lddx=8, do=p, lddo=8, dz=None, lddz=8, a=None, **over):
        a = ctypes.byref(args(**over)) if a is None else a or None
        return lib.zsolve_resnorm_bwd(handle, a, dh, lddh, dy, lddy, y, ldy, stats, dx, lddx, do, lddo, dz, lddz, *([None] * 5))

    both = [dict(a=0), dict(type=3), dict(wtype=2), dict(type=0, wtype=1), dict(kind=2), dict(kind=-1), dict(act=5), dict(act=-1), dict(rows=-1),
            dict(d=0), dict(d=1 << 25), dict(rows=1 << 31), dict(o=None), dict(ldo=7), dict(z=p, ldz=7), dict(y=None), dict(ldy=7),
            dict(eps=float("nan"))]
    return ((fwd, both + [dict(x=None), dict(h=None), dict(ldx=7), dict(ldh=7)]),
            (bwd, both + [dict(dh=None), dict(stats=None), dict(dx=None), dict(do=None), dict(lddh=7), dict(dy=p, lddy=7), dict(lddx=7),
                          dict(lddo=7), dict(dz=p), dict(z=p, dz=p, lddz=7)]))


@pytest.mark.gpu
def test_refusals_of_the_library(seq):
    import mixed_precision_refinement_gb300 as zs
    for call, bad in _calls(zs.raw_lib(), seq.seq):
        for args in bad:
            assert call(**args) == zs.ZSOLVE_EINVAL, args


def test_null_handle_is_refused_without_a_device():
    import mixed_precision_refinement_gb300 as zs
    for call, _ in _calls(zs.raw_lib(), None):
        assert call() == zs.ZSOLVE_EINVAL
