"""The matrix product with its epilogue, forward and backward, through the C-ABI against float64."""
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
    tol = tol + u * (ref.abs() + tol) + 1e-12
    bad = (got.double() - ref).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), float(((got.double() - ref).abs() / tol).max()))


def _check(seq, m, n, k, dtype, act, bias=True, res=True, seed=0, pads=(0, 0, 0), shifts=(0, 0, 0)):
    torch = _torch()
    dt, u = getattr(torch, dtype), U[dtype]
    gen = torch.Generator("cuda").manual_seed(seed)
    x = _randn(gen, (m, k), dt, pads[0], shifts[0])
    w = _randn(gen, (n, k), dt, pads[1], shifts[1])
    b = _randn(gen, (1, n), dt)[0] if bias else None
    r = _randn(gen, (m, n), dt, pads[2], shifts[2]) if res else None
    y, z = seq.linear(x, w, b, act=act, r=r, keep=True)
    X, W = x.double(), w.double()
    zref = X @ W.T + (b.double() if bias else 0)
    ztol = k * UADD * (X.abs() @ W.abs().T) + UADD * zref.abs()
    _close(z, zref, ztol, u)
    ref = _act64(zref, act) + (r.double() if res else 0)
    _close(y, ref, SLOPE * ztol + (AEVAL + UADD) * (1 + zref.abs() + ref.abs()), u)

    dy = _randn(gen, (m, n), dt, pads[2], shifts[2])
    dx, dw, db = seq.linear_bwd(dy, x, w, z, act=act)
    zz = z.double().requires_grad_()
    slope, = torch.autograd.grad(_act64(zz, act).sum(), zz)
    dz = dy.double() * slope
    # evaluated in float32, then rounded to the operands' type (float16: to its smallest steps too)
    dztol = (AEVAL * 4 * dy.double().abs() * (1 + zz.detach().abs()))
    op = dztol + u * dz.abs() + (2.0 ** -25 if dtype == "float16" else 0.0)
    if act == "none":
        op = torch.zeros_like(op)
    A = dz.abs() + op
    _close(dx, dz @ W, op @ W.abs() + n * UADD * (A @ W.abs()), u)
    _close(dw, dz.T @ X, op.T @ X.abs() + m * UADD * (A.T @ X.abs()), u)
    _close(db, dz.sum(0), dztol.sum(0) + m * UADD * dz.abs().sum(0), u)
    return y


SHAPES = [(1, 1, 1), (1, 8, 16), (3, 5, 7), (128, 128, 64), (129, 257, 65), (200, 130, 1000), (64, 1024, 2048),
          (1000, 520, 72), (2, 40, 5000), (300, 2157, 331), (2500, 1500, 136), (4000, 2300, 64),
          (2600, 3300, 1900)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_shapes(seq, m, n, k, dtype):
    _check(seq, m, n, k, dtype, ACTS[(m + n + k) % 5], seed=m + n + k)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,res", [(True, True), (False, False)])
def test_epilogues(seq, act, bias, res, dtype):
    _check(seq, 150, 200, 96, dtype, act, bias, res, seed=7)
    _check(seq, 9, 200, 1500, dtype, act, bias, res, seed=8)  # split along k


@pytest.mark.gpu
@pytest.mark.parametrize("pads,shifts", [((8, 8, 8), (0, 0, 0)), ((1, 3, 5), (0, 0, 0)), ((0, 0, 0), (1, 1, 1)),
                                         ((8, 0, 0), (4, 0, 8)), ((0, 7, 0), (0, 8, 3))])
def test_strides_and_alignment(seq, pads, shifts):
    _check(seq, 140, 136, 80, "bfloat16", "silu", seed=9, pads=pads, shifts=shifts)


@pytest.mark.gpu
def test_gradient_against_differences(seq):
    """Derivatives of single outputs along a direction, from forward values at x +- h p and x +- 2 h p
    (Richardson): off by the outputs' rounding over h, by at most the difference of the two estimates,
    and by the gradient's own rounding."""
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(3)
    m, n, k, h = 5, 24, 40, 2.0 ** -3
    u = U["float16"]

    def grid(*shape):  # multiples of 1/16, so that x +- 2 h p is exact
        return (torch.randint(-24, 25, shape, generator=gen, device="cuda") / 16).half()

    x, w, b = grid(m, k), (grid(n, k) / 4), grid(n)
    for act in ACTS[2:]:
        y, z = seq.linear(x, w, b, act=act, keep=True)
        for i, j in ((0, 0), (2, 7), (4, 23)):
            dy = torch.zeros_like(y)
            dy[i, j] = 1.0
            dx, dw, db = seq.linear_bwd(dy, x, w, z, act=act)
            p = torch.zeros_like(x)
            p[i] = torch.randint(-1, 2, (k,), generator=gen, device="cuda").half() / 4
            for grad, along, f in ((dx, p, lambda t: seq.linear(x + t * p, w, b, act=act)),
                                   (dw, p[i].expand(n, k), lambda t: seq.linear(x, w + t * p[i], b, act=act)),
                                   (db, torch.ones_like(b) / 4, lambda t: seq.linear(x, w, b + t / 4, act=act))):
                val = {t: float(f(t * h)[i, j]) for t in (-2, -1, 1, 2)}
                d1, d2 = (val[1] - val[-1]) / (2 * h), (val[2] - val[-2]) / (4 * h)
                terms = grad.double() * along.double()
                # z is rounded before its slope is taken: at most u |z| times a second derivative below 1.2
                own = (3 * u + 1.2 * u * abs(float(z[i, j]))) * float(terms.abs().sum())
                noise = 1.5 / h * u * max(abs(v) for v in val.values())
                assert abs((4 * d1 - d2) / 3 - float(terms.sum())) <= noise + abs(d1 - d2) + own, (act, i, j)


@pytest.mark.gpu
def test_nonfinite_rows_stay_alone_and_residual_in_place(seq):
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(4)
    x, w = _randn(gen, (200, 77), torch.bfloat16), _randn(gen, (150, 77), torch.bfloat16)
    r = _randn(gen, (200, 150), torch.bfloat16)
    y = seq.linear(x, w, r=r, act="silu")
    bad = x.clone()
    bad[130, 3], bad[131, 76] = float("nan"), float("inf")
    yb = seq.linear(bad, w, r=r, act="silu")
    keep = [i for i in range(200) if i not in (130, 131)]
    assert torch.equal(yb[keep], y[keep])
    assert torch.isnan(yb[130]).all() and not torch.isfinite(yb[131]).any() | torch.isfinite(yb[131]).all()
    inplace = r.clone()
    zs.zsolve_linear(seq.seq, x, w, None, "silu", inplace, inplace)
    assert torch.equal(inplace, y)


@pytest.mark.gpu
def test_no_rows(seq):
    torch = _torch()
    x, w = torch.empty(0, 32, device="cuda", dtype=torch.float16), torch.ones(48, 32, device="cuda", dtype=torch.float16)
    y, z = seq.linear(x, w, keep=True)
    assert y.shape == (0, 48)
    dx, dw, db = seq.linear_bwd(y, x, w, z, act="silu")
    assert dx.shape == (0, 32) and not dw.any() and not db.any()


@pytest.mark.gpu
def test_same_result_twice(seq):
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(5)
    x, w = _randn(gen, (70, 3000), torch.bfloat16), _randn(gen, (500, 3000), torch.bfloat16)
    dy = _randn(gen, (70, 500), torch.bfloat16)
    one, two = ((seq.linear(x, w),) + seq.linear_bwd(dy, x, w) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(one, two))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(1024, 1032, 5000), (4100, 1030, 4100), (1030, 4100, 4100)])
def test_both_gradients_in_one_launch(seq, m, n, k):
    """Large products whose tiles are dealt together, with sums of the same and of different lengths; each as
    it is alone."""
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(k)
    x, w, dy = (_randn(gen, s, torch.bfloat16) for s in ((m, k), (n, k), (m, n)))
    x, w, dy = (t.contiguous() for t in (x, w, dy))
    import mixed_precision_refinement_gb300 as zs
    both = torch.empty_like(x), torch.empty_like(w)
    alone = torch.empty_like(x), torch.empty_like(w)
    before = zs.zsolve_seq_launches(seq.seq)
    zs.zsolve_linear_bwd(seq.seq, dy, x, w, "none", None, *both)
    assert n % 8 or zs.zsolve_seq_launches(seq.seq) == before + 1
    zs.zsolve_linear_bwd(seq.seq, dy, x, w, "none", None, alone[0], None)
    zs.zsolve_linear_bwd(seq.seq, dy, x, w, "none", None, None, alone[1])
    for got, one, ref, size in ((both[0], alone[0], dy.double() @ w.double(), dy.double().abs() @ w.double().abs()),
                                (both[1], alone[1], dy.double().T @ x.double(), dy.double().abs().T @ x.double().abs())):
        assert torch.equal(got, one)
        # float32 sums of max(m, n) terms on the tensor cores, which cut instead of rounding, and one rounding
        assert bool(((got.double() - ref).abs() <= max(m, n) * 2.0 ** -23 * size + 2.0 ** -8 * ref.abs()).all())


@pytest.mark.gpu
def test_some_gradients_only(seq):
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(6)
    x, w, dy = (_randn(gen, s, torch.float16) for s in ((90, 40), (56, 40), (90, 56)))
    dx, dw, db = seq.linear_bwd(dy, x, w)
    for which in range(3):
        out = [torch.zeros_like(t) if i == which else None for i, t in enumerate((dx, dw, db))]
        zs.zsolve_linear_bwd(seq.seq, dy, x, w, "none", None, *out)
        assert torch.equal(out[which], (dx, dw, db)[which])


@pytest.mark.gpu
def test_refusals(seq):
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    x, w = torch.ones(4, 16, device="cuda", dtype=torch.bfloat16), torch.ones(8, 16, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        seq.linear(x, w, act="swish")
    with pytest.raises(ValueError):
        seq.linear(x, w[:, :15])
    with pytest.raises(TypeError):
        seq.linear(x, w.half())
    with pytest.raises(ValueError):
        seq.linear(x, w, b=torch.ones(7, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(zs.ZsolveError) as e:
        seq.linear(x.float(), w.float())
    assert e.value.status == zs.ZSOLVE_EINVAL and "BF16" in str(e.value)
    with pytest.raises(zs.ZsolveError):
        seq.linear_bwd(torch.ones(4, 8, device="cuda", dtype=torch.bfloat16), x, w, act="silu")  # no z
    lib, p = zs.raw_lib(), x.data_ptr()

    def call(type=1, m=4, n=8, k=16, x=p, ldx=16, w=p, ldw=16, act=0, y=p, ldy=8):
        return lib.zsolve_linear(seq.seq, type, m, n, k, x, ldx, w, ldw, None, act, None, 0, y, ldy, None, 0)

    for bad in (dict(type=0), dict(m=-1), dict(n=0), dict(k=0), dict(k=1 << 30), dict(x=None), dict(w=None),
                dict(y=None), dict(ldx=15), dict(ldw=15), dict(ldy=7), dict(act=5), dict(act=-1)):
        assert call(**bad) == zs.ZSOLVE_EINVAL, bad


def test_null_handle_is_refused_without_a_device():
    import mixed_precision_refinement_gb300 as zs
    lib = zs.raw_lib()
    assert lib.zsolve_linear(None, 1, 1, 1, 1, None, 1, None, 1, None, 0, None, 0, None, 1, None, 0) == zs.ZSOLVE_EINVAL
    assert lib.zsolve_seq_check(None) == zs.ZSOLVE_EINVAL
