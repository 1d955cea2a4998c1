"""The gated feed-forward projections, forward and backward, through the C-ABI against float64."""
import pytest

# unit roundoff (half a last place over the value): 8 and 11 significant bits
U = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
# one addition of the tensor cores' float32 sums, which need not round to nearest
UADD = 2.0 ** -23
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
# the activations' slopes are at most 1.13; their own evaluation is good to 16 units of the argument's size
SLOPE, AEVAL = 1.13, 16 * 2.0 ** -24


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


def _act64(z, act):
    torch = _torch()
    f = torch.nn.functional
    return {"none": lambda t: t, "relu": torch.relu, "silu": f.silu, "gelu": f.gelu,
            "gelu_tanh": lambda t: f.gelu(t, approximate="tanh")}[act](z)


def _randn(gen, shape, dt, pad=0, shift=0):
    """Rows of shape[-1] values `pad` apart, from `shift` values into their storage."""
    torch = _torch()
    m, d = shape
    buf = torch.randn(m * (d + pad) + shift, generator=gen, device="cuda").to(dt)
    return buf[shift:].view(m, d + pad)[:, :d]


def _close(got, ref, tol, u):
    tol = tol + u * (ref.abs() + tol) + (2.0 ** -25 if u == U["float16"] else 1e-30)  # float16: half its smallest step
    bad = (got.double() - ref).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), float(((got.double() - ref).abs() / tol).max()))


def _check(seq, m, n, k, dtype, act, bias=True, seed=0, pads=(0, 0, 0), shifts=(0, 0, 0)):
    torch = _torch()
    dt, u = getattr(torch, dtype), U[dtype]
    gen = torch.Generator("cuda").manual_seed(seed)
    x = _randn(gen, (m, k), dt, pads[0], shifts[0])
    wg, wu = (_randn(gen, (n, k), dt, p, s) / 4 if not p and not s else _randn(gen, (n, k), dt, p, s)
              for p, s in ((pads[1], shifts[1]), (pads[2], shifts[2])))
    bg, bu = (_randn(gen, (1, n), dt)[0] if bias else None for _ in range(2))
    y, zg, zu = seq.glu(x, wg, wu, bg, bu, act=act, keep=True)
    assert torch.equal(seq.glu(x, wg, wu, bg, bu, act=act), y)
    X, G, W = x.double(), wg.double(), wu.double()
    gref, uref = X @ G.T + (bg.double() if bias else 0), X @ W.T + (bu.double() if bias else 0)
    gtol = k * UADD * (X.abs() @ G.abs().T) + UADD * gref.abs()
    utol = k * UADD * (X.abs() @ W.abs().T) + UADD * uref.abs()
    _close(zg, gref, gtol, u)
    _close(zu, uref, utol, u)
    a = _act64(gref, act)
    atol = SLOPE * gtol + AEVAL * (1 + gref.abs())
    _close(y, a * uref, atol * (uref.abs() + utol) + a.abs() * utol + UADD * (a * uref).abs(), u)

    dy = _randn(gen, (m, n), dt, pads[0], shifts[1])
    dx, dwg, dwu, dbg, dbu = seq.glu_bwd(dy, x, wg, wu, zg, zu, act=act)
    zz = zg.double().requires_grad_()
    slope, = torch.autograd.grad(_act64(zz, act).sum(), zz)
    D, Z, zz = dy.double(), zu.double(), zz.detach()
    dg, du = D * Z * slope, D * _act64(zz, act)
    # evaluated in float32, then rounded to the operands' type (float16: to its smallest steps too)
    small = 2.0 ** -25 if dtype == "float16" else 0.0
    evg, evu = AEVAL * 4 * (D * Z).abs() * (1 + zz.abs()), AEVAL * D.abs() * (1 + zz.abs())
    og, ou = (e + u * (d.abs() + e) + small for e, d in ((evg, dg), (evu, du)))
    A, B = dg.abs() + og, du.abs() + ou
    _close(dx, dg @ G + du @ W, og @ G.abs() + ou @ W.abs() + 2 * n * UADD * (A @ G.abs() + B @ W.abs()), u)
    _close(dwg, dg.T @ X, og.T @ X.abs() + m * UADD * (A.T @ X.abs()), u)
    _close(dwu, du.T @ X, ou.T @ X.abs() + m * UADD * (B.T @ X.abs()), u)
    _close(dbg, dg.sum(0), evg.sum(0) + m * UADD * dg.abs().sum(0), u)
    _close(dbu, du.sum(0), evu.sum(0) + m * UADD * du.abs().sum(0), u)


SHAPES = [(1, 1, 1), (1, 8, 16), (3, 5, 7), (8, 1000, 2157), (12, 72, 40), (128, 64, 64), (129, 130, 65), (200, 65, 1000),
          (64, 1024, 2048), (1000, 264, 72), (2, 40, 5000), (300, 1077, 331), (2500, 1500, 136), (4000, 1200, 64),
          (2600, 3300, 1900), (5000, 300, 700)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_shapes(seq, m, n, k, dtype):
    _check(seq, m, n, k, dtype, ACTS[(m + n + k) % 5], seed=m + n + k)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias", [True, False])
def test_epilogues(seq, act, bias, dtype):
    _check(seq, 150, 200, 96, dtype, act, bias, seed=7)
    _check(seq, 20, 200, 1500, dtype, act, bias, seed=8)  # split along k
    _check(seq, 5, 60, 96, dtype, act, bias, seed=9)  # a few rows


@pytest.mark.gpu
@pytest.mark.parametrize("m", [4, 140, 3000])
@pytest.mark.parametrize("pads,shifts", [((8, 8, 8), (0, 0, 0)), ((1, 3, 5), (0, 0, 0)), ((0, 0, 0), (1, 1, 1)),
                                         ((8, 0, 0), (4, 0, 8)), ((0, 7, 0), (0, 8, 3))])
def test_strides_and_alignment(seq, pads, shifts, m):
    _check(seq, m, 136, 80, "bfloat16", "silu", seed=9, pads=pads, shifts=shifts)


@pytest.mark.gpu
def test_one_weight_in_two_halves(seq):
    """Both weights as views of one matrix, and outputs in places of the caller's own with rows apart."""
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(2)
    w = _randn(gen, (2 * 72, 40), torch.bfloat16)
    x = _randn(gen, (90, 40), torch.bfloat16)
    wide = torch.full((90, 300), 7.0, device="cuda", dtype=torch.bfloat16)
    y, zg, zu = wide[:, :72], wide[:, 80:152], wide[:, 161:233]
    zs.zsolve_glu(seq.seq, x, w[:72], w[72:], None, None, "silu", y, zg, zu)
    ref = seq.glu(x, w[:72].clone(), w[72:].clone(), keep=True)
    for got, want in zip((y, zg, zu), ref):
        assert torch.equal(got, want)
    kept = torch.ones(300, dtype=torch.bool, device="cuda")
    kept[:72] = kept[80:152] = kept[161:233] = False
    assert bool((wide[:, kept] == 7).all())


@pytest.mark.gpu
def test_nonfinite_rows_stay_alone(seq):
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(4)
    x, wg, wu = (_randn(gen, s, torch.bfloat16) for s in ((200, 77), (150, 77), (150, 77)))
    y, zg, zu = seq.glu(x, wg, wu, keep=True)
    bad = x.clone()
    bad[130, 3], bad[131, 76] = float("nan"), float("inf")
    yb = seq.glu(bad, wg, wu)
    keep = [i for i in range(200) if i not in (130, 131)]
    assert torch.equal(yb[keep], y[keep]) and torch.isnan(yb[130]).all()
    dy = _randn(gen, (200, 150), torch.bfloat16)
    dx = seq.glu_bwd(dy, x, wg, wu, zg, zu)[0]
    dyb = dy.clone()
    dyb[7, 149] = float("nan")
    dxb = seq.glu_bwd(dyb, x, wg, wu, zg, zu)[0]
    keep = [i for i in range(200) if i != 7]
    assert torch.equal(dxb[keep], dx[keep]) and torch.isnan(dxb[7]).all()


@pytest.mark.gpu
def test_no_rows(seq):
    torch = _torch()
    x, w = torch.empty(0, 32, device="cuda", dtype=torch.float16), torch.ones(48, 32, device="cuda", dtype=torch.float16)
    y, zg, zu = seq.glu(x, w, w, keep=True)
    assert y.shape == (0, 48)
    dx, *rest = seq.glu_bwd(y, x, w, w, zg, zu)
    assert dx.shape == (0, 32) and not any(bool(t.any()) for t in rest)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(70, 500, 900), (4100, 1030, 2100), (2100, 2000, 2304)])
def test_some_gradients_only_and_the_same_twice(seq, m, n, k):
    """Each gradient alone, both weights' without the input's, and all of them: the same bits (the last two sizes
    on pairs of SMs, together and apart)."""
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(6)
    x, wg, wu, dy, zg, zu = (_randn(gen, s, torch.bfloat16) for s in ((m, k), (n, k), (n, k), (m, n), (m, n), (m, n)))
    ref = seq.glu_bwd(dy, x, wg, wu, zg, zu)
    for got, want in zip(seq.glu_bwd(dy, x, wg, wu, zg, zu), ref):
        assert torch.equal(got, want)
    for which in [(0,), (1,), (2,), (3,), (4,), (1, 2), (0, 2, 4)]:
        out = [torch.zeros_like(t) if i in which else None for i, t in enumerate(ref)]
        zs.zsolve_glu_bwd(seq.seq, dy, x, wg, wu, "silu", zg, zu, *out)
        for i in which:
            assert torch.equal(out[i], ref[i]), (which, i)


@pytest.mark.gpu
def test_gradient_against_differences(seq):
    """Derivatives of single outputs along a direction, from forward values at x +- h p and x +- 2 h p
    (Richardson): off by the outputs' rounding over h, by at most the difference of the two estimates,
    and by the gradient's own rounding."""
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(3)
    m, n, k, h = 20, 24, 40, 2.0 ** -3
    u = U["float16"]

    def grid(*shape):  # multiples of 1/16, so that x +- 2 h p is exact
        return (torch.randint(-24, 25, shape, generator=gen, device="cuda") / 16).half()

    x, wg, wu, bg, bu = grid(m, k), grid(n, k) / 4, grid(n, k) / 4, grid(n), grid(n)
    for act in ACTS[2:]:
        y, zg, zu = seq.glu(x, wg, wu, bg, bu, act=act, keep=True)
        for i, j in ((0, 0), (12, 7), (19, 23)):
            dy = torch.zeros_like(y)
            dy[i, j] = 1.0
            grads = seq.glu_bwd(dy, x, wg, wu, zg, zu, act=act)
            p = torch.zeros_like(x)
            p[i] = torch.randint(-1, 2, (k,), generator=gen, device="cuda").half() / 4
            q, one = p[i].expand(n, k), torch.ones_like(bg) / 4
            forms = (lambda t: (x + t * p, wg, wu, bg, bu), lambda t: (x, wg + t * q, wu, bg, bu), lambda t: (x, wg, wu + t * q, bg, bu),
                     lambda t: (x, wg, wu, bg + t * one, bu), lambda t: (x, wg, wu, bg, bu + t * one))
            for grad, along, f in zip(grads, (p, q, q, one, one), forms):
                val = {t: float(seq.glu(*f(t * h), act=act)[i, j]) for t in (-2, -1, 1, 2)}
                d1, d2 = (val[1] - val[-1]) / (2 * h), (val[2] - val[-2]) / (4 * h)
                terms = grad.double() * along.double()
                # zg and zu are rounded before they are used: at most u |z| times derivatives below 1.2 of the other factor's size
                own = 4 * u * float(terms.abs().sum())
                w = (wg.double().abs()[j] * along.double().abs().max()).sum() + (wu.double().abs()[j] * along.double().abs().max()).sum() + 1
                own += 1.2 * u * float((1 + zu[i, j].double().abs()) * (1 + zg[i, j].double().abs()) * w * x.double().abs().max().clamp(min=1))
                noise = 1.5 / h * u * max(abs(v) for v in val.values())
                assert abs((4 * d1 - d2) / 3 - float(terms.sum())) <= noise + abs(d1 - d2) + own, (act, i, j)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("keep", [False, True])
def test_autograd(seq, act, keep):
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(3)

    def randn(*s):
        return torch.randn(*s, generator=gen, device="cuda").bfloat16()

    ins = x, wg, wu, bg, bu = randn(2, 30, 40), randn(24, 40), randn(24, 40), randn(24), randn(24)
    dy = randn(2, 30, 24)
    y0, zg, zu = seq.glu(*ins, act=act, keep=True)
    leaves = [t.clone().requires_grad_() for t in ins]
    out = seq.glu(*leaves, act=act, keep=keep)
    y = out[0] if keep else out
    assert torch.equal(y, y0)
    y.backward(dy)
    for leaf, want in zip(leaves, seq.glu_bwd(dy, x, wg, wu, zg, zu, act=act)):
        assert torch.equal(leaf.grad, want)
    if keep:
        with pytest.raises(RuntimeError, match="zg and zu"):
            seq.glu(*(t.clone().requires_grad_() for t in ins), act=act, keep=True)[1].sum().backward()
    W = wu.clone().requires_grad_()  # one weight alone
    seq.glu(x, wg, W, bg, act=act).sum().backward()
    y1, zg1, zu1 = seq.glu(x, wg, wu, bg, act=act, keep=True)
    assert torch.equal(W.grad, seq.glu_bwd(torch.ones_like(y1), x, wg, wu, zg1, zu1, act=act)[2])


@pytest.mark.gpu
def test_refusals(seq):
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    x, w = torch.ones(4, 16, device="cuda", dtype=torch.bfloat16), torch.ones(8, 16, device="cuda", dtype=torch.bfloat16)
    z = torch.ones(4, 8, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        seq.glu(x, w, w, act="swish")
    with pytest.raises(ValueError):
        seq.glu(x, w, w[:7])
    with pytest.raises(ValueError):
        seq.glu(x, w[:, :15], w)
    with pytest.raises(TypeError):
        seq.glu(x, w, w.half())
    with pytest.raises(ValueError):
        seq.glu(x, w, w, bu=torch.ones(7, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        seq.glu_bwd(z, x, w, w, z[:3], z)
    with pytest.raises(zs.ZsolveError) as e:
        seq.glu(x.float(), w.float(), w.float())
    assert e.value.status == zs.ZSOLVE_EINVAL and "BF16" in str(e.value)
    with pytest.raises(zs.ZsolveError):
        zs.zsolve_glu(seq.seq, x, w, w, None, None, "silu", z, z.clone(), None)


def _calls(lib, handle):
    p = 64  # never read: every call below is refused before the device is touched

    def fwd(type=1, m=4, n=8, k=16, x=p, ldx=16, wg=p, ldwg=16, wu=p, ldwu=16, act=0, y=p, ldy=8, zg=None, ldzg=8, zu=None, ldzu=8):
        return lib.zsolve_glu(handle, type, m, n, k, x, ldx, wg, ldwg, wu, ldwu, None, None, act, y, ldy, zg, ldzg, zu, ldzu)

    def bwd(type=1, m=4, n=8, k=16, dy=p, lddy=8, x=p, ldx=16, wg=p, ldwg=16, wu=p, ldwu=16, act=0, zg=p, ldzg=8, zu=p, ldzu=8, dx=p,
            lddx=16, dwg=p, lddwg=16, dwu=p, lddwu=16):
        return lib.zsolve_glu_bwd(handle, type, m, n, k, dy, lddy, x, ldx, wg, ldwg, wu, ldwu, act, zg, ldzg, zu, ldzu, dx, lddx, dwg,
                                  lddwg, dwu, lddwu, p, p)

    sizes = [dict(type=0), dict(m=-1), dict(n=0), dict(k=0), dict(k=1 << 30), dict(ldx=15), dict(ldwg=15), dict(ldwu=15), dict(act=5),
             dict(act=-1), dict(x=None), dict(wg=None), dict(wu=None)]
    return ((fwd, sizes + [dict(y=None), dict(ldy=7), dict(zg=p), dict(zu=p), dict(zg=p, zu=p, ldzg=7), dict(zg=p, zu=p, ldzu=7)]),
            (bwd, sizes + [dict(dy=None), dict(zg=None), dict(zu=None), dict(lddy=7), dict(ldzg=7), dict(ldzu=7), dict(lddx=15),
                           dict(lddwg=15), dict(lddwu=15)]))


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
