"""Layer norm forward and backward through the C-ABI against float64."""
import ctypes

import pytest

# unit roundoff (half a last place over the value): 24, 8 and 11 significant bits
U = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
U32 = 2.0 ** -24
# A float32 sum of a row: each thread adds at most 32 values (rows of up to
# 16384; 16 + d / 1024 beyond) and a tree of 10 levels follows; with the few
# roundings of the output formula, 64 units of the terms' sizes bound it.
ADDS = 64


def _torch():
    import torch
    return torch


@pytest.fixture(scope="module")
def seq():
    import mixed_precision_refinement_gb300 as zs
    s = zs.Seq()
    yield s
    s.close()


def _inputs(rows, d, dtype, wdtype, seed=0, pad=0, shift=0):
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(seed)
    buf = torch.randn(rows * (d + pad) + shift, generator=gen, device="cuda").to(dtype)
    x = buf[shift:].view(rows, d + pad)[:, :d]
    w = (1 + 0.3 * torch.randn(d, generator=gen, device="cuda")).to(wdtype)
    b = (0.3 * torch.randn(d, generator=gen, device="cuda")).to(wdtype)
    dy = torch.randn(rows, d, generator=gen, device="cuda").to(dtype)
    return x, w, b, dy


def _forward64(x, w, b, eps):
    x = x.double()
    mu = x.mean(1, keepdim=True)
    rs = 1 / ((x - mu).square().mean(1, keepdim=True) + eps).sqrt()
    h = (x - mu) * rs
    y = h if w is None else h * w.double()
    return (y if b is None else y + b.double()), mu, rs, h


# widths around each number of threads a row is given, odd ones, one value,
# and rows longer than the registers hold
WIDTHS = [1, 2, 7, 8, 64, 255, 256, 257, 512, 520, 1000, 1024, 2048, 2157, 4096, 4104, 8192, 8200, 16384, 16385, 20000]


@pytest.mark.gpu
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("types", [("float32", "float32"), ("bfloat16", "bfloat16"), ("bfloat16", "float32"),
                                   ("float16", "float16")], ids="-".join)
def test_forward_and_backward(seq, d, types):
    torch = _torch()
    dt, wdt = (getattr(torch, t) for t in types)
    rows = 37 if d < 5000 else 5
    x, w, b, dy = _inputs(rows, d, dt, wdt, seed=d)
    y, mean, rstd = seq.layernorm(x, w, b, eps=1e-5)
    ref, mu, rs, h = _forward64(x, w, b, 1e-5)
    size = (x.double().abs().amax(1, keepdim=True) + mu.abs()) * rs  # what the mean's error is relative to
    tol = ADDS * U32 * (1 + size + h.abs()) * (w.double().abs() + 1) + U[types[0]] * ref.abs() + 1e-30
    assert bool(((y.double() - ref).abs() <= tol).all())
    assert bool(((mean.double() - mu[:, 0]).abs() <= ADDS * U32 * x.double().abs().amax(1)).all())
    if d > 1:
        assert bool(((rstd.double() / rs[:, 0] - 1).abs() <= ADDS * U32 * (1 + size[:, 0])).all())

    dx, dw, db = seq.layernorm_bwd(dy, x, mean, rstd, w)
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    a = dy.double() * w.double()
    m1, m2 = a.mean(1, keepdim=True), (a * h).mean(1, keepdim=True)
    ref = rstd.double()[:, None] * (a - m1 - h * m2)
    hsize = h.abs() + ADDS * U32 * size
    terms = rstd.double()[:, None] * (a.abs() + a.abs().mean(1, keepdim=True) + hsize * (a * h).abs().mean(1, keepdim=True))
    # an error in h (relative to the mean's size) enters through h and mean(a h)
    terms = terms * (1 + size)
    assert bool(((dx.double() - ref).abs() <= ADDS * U32 * terms + U[types[0]] * ref.abs() + 1e-30).all())
    # the columns' sums: at most `rows` additions in a chain, then 32
    for got, t in ((dw, dy.double() * h), (db, dy.double())):
        tol = (rows + ADDS) * U32 * (t.abs() * (1 + size)).sum(0) + U[types[1]] * t.sum(0).abs() + 1e-30
        assert bool(((got.double() - t.sum(0)).abs() <= tol).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (8, 8)])
def test_strided_and_unaligned_rows_equal_packed_ones(seq, dtype, pad, shift):
    torch = _torch()
    dt = getattr(torch, dtype)
    x, w, b, dy = _inputs(19, 264, dt, dt, seed=3, pad=pad, shift=shift)
    packed = x.contiguous()
    ref, mean, rstd = seq.layernorm(packed, w, b)
    y, mean2, rstd2 = seq.layernorm(x, w, b)
    tol = 4 * U[dtype] * (1 + ref.double().abs()) if dtype != "float32" else ADDS * U32 * 8
    assert bool(((y.double() - ref.double()).abs() <= tol).all())
    g1, g2 = seq.layernorm_bwd(dy, packed, mean, rstd, w), seq.layernorm_bwd(dy, x, mean, rstd, w)
    for p, q in zip(g1, g2):
        scale = p.double().abs().max()
        assert float((p.double() - q.double()).abs().max()) <= (4 * U[dtype] + ADDS * U32) * float(scale)


@pytest.mark.gpu
def test_many_rows_give_the_same_gradients_twice(seq):
    torch = _torch()
    x, w, b, dy = _inputs(20011, 200, torch.float32, torch.float32, seed=5)
    _, mean, rstd = seq.layernorm(x, w, b)
    one, two = seq.layernorm_bwd(dy, x, mean, rstd, w), seq.layernorm_bwd(dy, x, mean, rstd, w)
    assert all(torch.equal(p, q) for p, q in zip(one, two))
    t = dy.double() * ((x.double() - mean.double()[:, None]) * rstd.double()[:, None])
    # chains of at most 20011 / (152 * 8) / 1 + 4 rows a thread and 4 * 1216 / 32 parts
    assert bool(((one[1].double() - t.sum(0)).abs() <= 256 * U32 * t.abs().sum(0)).all())


@pytest.mark.gpu
def test_no_weights_no_rows_constant_rows_and_nonfinite(seq):
    torch = _torch()
    x, _, _, dy = _inputs(6, 96, torch.float32, torch.float32, seed=6)
    y, mean, rstd = seq.layernorm(x)
    ref, *_ = _forward64(x, None, None, 1e-5)
    assert float((y.double() - ref).abs().max()) <= ADDS * U32 * 16
    dx, dw, db = seq.layernorm_bwd(dy, x, mean, rstd)
    assert float((db.double() - dy.double().sum(0)).abs().max()) <= 16 * U32 * 30

    none = torch.empty(0, 96, device="cuda")
    y, mean, rstd = seq.layernorm(none)
    assert y.shape == (0, 96) and mean.shape == (0,)
    dx, dw, db = seq.layernorm_bwd(none, none, mean, rstd)
    assert dx.shape == (0, 96) and not dw.any() and not db.any()

    const = torch.full((3, 40), 7.25, device="cuda")
    y, mean, rstd = seq.layernorm(const)  # no variance: h = 0, rstd = eps^-1/2
    assert not y.any() and float((rstd - 1e-5 ** -0.5).abs().max()) < 1e-3

    # a row that is not finite spoils that row alone
    bad = x.clone()
    bad[2, 5] = float("inf")
    bad[4, 0] = float("nan")
    y2, *_ = seq.layernorm(bad)
    assert torch.isnan(y2[2]).all() and torch.isnan(y2[4]).all()
    keep = [0, 1, 3, 5]
    assert torch.equal(y2[keep], seq.layernorm(x)[0][keep])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [200, 4096, 20000])
def test_forward_in_place(seq, d):
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    x, w, b, _ = _inputs(9, d, torch.bfloat16, torch.float32, seed=12)
    ref, _, _ = seq.layernorm(x, w, b)
    y = x.clone()
    zs.zsolve_layernorm(seq.seq, y, w, b, 1e-5, y)
    assert torch.equal(y, ref)


@pytest.mark.gpu
def test_large_offset_keeps_the_variance(seq):
    torch = _torch()
    x = torch.randn(9, 1000, device="cuda") + 4096.0
    y, *_ = seq.layernorm(x)
    ref, mu, rs, _ = _forward64(x, None, None, 1e-5)
    # the mean is off by at most ADDS units of 4096 at worst; the variance around it by that squared
    assert float((y.double() - ref).abs().max()) <= ADDS * U32 * 4200 * 1.1


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(5, 1000), (2000, 1000), (2000, 1001), (700, 4096), (3, 20000)])
def test_large_offset_keeps_the_gradient(seq, rows, d):
    """With x and the mean on one grid, x - mean is exact: nothing is relative to the mean's size."""
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(d)
    x, dy, w = (torch.randn(n, d, device="cuda", generator=gen) for n in (rows, rows, 1))
    x, w = x + 4096.0, w[0]
    mean = x.double().mean(1).float()
    rstd = torch.rsqrt((x.double() - mean.double()[:, None]).square().mean(1)).float()
    dx, dw, db = seq.layernorm_bwd(dy, x, mean, rstd, w)
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    a = dy.double() * w.double()
    m1, m2 = a.mean(1, keepdim=True), (a * h).mean(1, keepdim=True)
    ref = rstd.double()[:, None] * (a - m1 - h * m2)
    terms = rstd.double()[:, None] * (a.abs() + a.abs().mean(1, keepdim=True) + h.abs() * (a * h).abs().mean(1, keepdim=True))
    assert bool(((dx.double() - ref).abs() <= ADDS * U32 * terms + 1e-30).all())
    # a column's sum: its rows' errors and those of a sum of `rows` terms, of random signs
    t = dy.double() * h
    assert bool(((dw.double() - t.sum(0)).abs() <= ADDS * U32 * t.abs().sum(0)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("d", [48, 700])
def test_gradient_against_differences(seq, d):
    """The directional derivative of sum(c * y) from values of the forward kernel at x +- h p and
    x +- 2 h p (Richardson): off by the values' rounding over h, and by at most the difference of
    the two estimates."""
    torch = _torch()
    x, w, b, c = _inputs(3, d, torch.float32, torch.float32, seed=9)
    p = torch.randn(3, d, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    _, mean, rstd = seq.layernorm(x, w, b)
    dx, dw, db = seq.layernorm_bwd(c, x, mean, rstd, w)
    h = 2.0 ** -6

    def val(t, ww=w, bb=b):
        return float((c.double() * seq.layernorm(t, ww, bb)[0].double()).sum())

    def rich(f):
        d1, d2 = (f(h) - f(-h)) / (2 * h), (f(2 * h) - f(-2 * h)) / (4 * h)
        return (4 * d1 - d2) / 3, abs(d1 - d2)

    noise = 1.5 / h * float(c.double().abs().sum()) * ADDS * U32 * 8
    got, slack = rich(lambda t: val(x + t * p))
    assert abs(got - float((dx.double() * p.double()).sum())) <= noise + slack
    pw = p[0]
    got, slack = rich(lambda t: val(x, ww=w + t * pw))
    assert abs(got - float((dw.double() * pw.double()).sum())) <= noise + slack
    got, slack = rich(lambda t: val(x, bb=b + t * pw))
    assert abs(got - float((db.double() * pw.double()).sum())) <= noise + slack


@pytest.mark.gpu
def test_refusals(seq):
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    x = torch.randn(4, 16, device="cuda")
    with pytest.raises(TypeError):
        seq.layernorm(x.double())
    with pytest.raises(ValueError):
        seq.layernorm(x.cpu())
    with pytest.raises(ValueError):
        seq.layernorm(x.T)
    with pytest.raises(ValueError):
        seq.layernorm(x, torch.ones(15, device="cuda"))
    with pytest.raises(TypeError):
        seq.layernorm(x, torch.ones(16, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(zs.ZsolveError) as e:
        seq.layernorm(x, eps=-1.0)
    assert e.value.status == zs.ZSOLVE_EINVAL and "eps" in str(e.value)
    lib, p = zs.raw_lib(), x.data_ptr()
    assert lib.zsolve_layernorm(seq.seq, 9, 9, 4, 16, p, 16, None, None, 1e-5, p, 16, None, None) == zs.ZSOLVE_EINVAL
    assert lib.zsolve_layernorm(seq.seq, 0, 1, 4, 16, p, 16, None, None, 1e-5, p, 16, None, None) == zs.ZSOLVE_EINVAL
    assert lib.zsolve_layernorm(seq.seq, 0, 0, 4, 0, p, 16, None, None, 1e-5, p, 16, None, None) == zs.ZSOLVE_EINVAL
    assert lib.zsolve_layernorm(seq.seq, 0, 0, -1, 16, p, 16, None, None, 1e-5, p, 16, None, None) == zs.ZSOLVE_EINVAL
    assert lib.zsolve_layernorm(seq.seq, 0, 0, 4, 16, None, 16, None, None, 1e-5, p, 16, None, None) == zs.ZSOLVE_EINVAL
    assert lib.zsolve_layernorm(seq.seq, 0, 0, 4, 16, p, 15, None, None, 1e-5, p, 16, None, None) == zs.ZSOLVE_EINVAL
    assert lib.zsolve_layernorm_bwd(seq.seq, 0, 0, 4, 16, p, 16, p, 16, None, p, None, p, 16, None,
                                    None) == zs.ZSOLVE_EINVAL
    assert zs.zsolve_seq_last_error(seq.seq)


def test_null_handle_is_refused_without_a_device():
    import mixed_precision_refinement_gb300 as zs
    lib = zs.raw_lib()
    assert lib.zsolve_layernorm(None, 0, 0, 1, 1, None, 1, None, None, 0.0, None, 1, None, None) == zs.ZSOLVE_EINVAL
    assert lib.zsolve_seq_create(None) == zs.ZSOLVE_EINVAL
    assert lib.zsolve_seq_set_stream(None, None) == zs.ZSOLVE_EINVAL
    assert lib.zsolve_seq_reserve(None, 1) == zs.ZSOLVE_EINVAL
    lib.zsolve_seq_destroy(ctypes.c_void_p())


@pytest.mark.gpu
def test_streams_workspace_and_capture():
    """Work on one stream after the other on one handle; a capture refuses to grow the workspace and
    replays once it is large enough."""
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    x, w, b, dy = _inputs(500, 128, torch.float32, torch.float32, seed=11)
    with zs.Seq() as s:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        _, mean, rstd = s.layernorm(x, w, b)
        ref = s.layernorm_bwd(dy, x, mean, rstd, w)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = s.layernorm_bwd(dy, x, mean, rstd, w)
        torch.cuda.current_stream().wait_stream(side)
        third = s.layernorm_bwd(dy, x, mean, rstd, w)
        torch.cuda.synchronize()
        for p, q, r in zip(ref, again, third):
            assert torch.equal(p, q) and torch.equal(p, r)
        assert zs.zsolve_seq_launches(s.seq) == 7
    with zs.Seq() as s:
        out = [torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)]
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            zs.zsolve_seq_set_stream(s.seq, stream)
            with pytest.raises(zs.ZsolveError) as e:
                zs.zsolve_layernorm_bwd(s.seq, dy, x, mean, rstd, w, *out)
            x.add(0)
        assert e.value.status == zs.ZSOLVE_ESTATE
        zs.zsolve_seq_reserve(s.seq, 1 << 24)
        assert zs.zsolve_seq_workspace_bytes(s.seq) == 1 << 24
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            zs.zsolve_layernorm_bwd(s.seq, dy, x, mean, rstd, w, *out)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(ref, out):
            assert torch.equal(p, q)
