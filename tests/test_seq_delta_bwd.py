"""Gradients of the gated delta rule through the C-ABI: against the derivative of the float64
recurrence, and against differences of it.

Tolerances.  As for the forward pass (keys of norm at most 1, steps in 0 .. 1, decays at most 1), the
adjoint recurrence is not expansive, and the errors of the chunks of both recurrences add up: with
n = 2 chunks + 2 of them, each held to e = 64 2^-21 of the sizes of what it multiplies.  With A, B the
largest Frobenius norms of a state and of a state's gradient, and u, x, d the largest norms of a
token's u, dX and dO, the products are bounded by
  dq: scale d A + scale 64 d u,  dk: u B + x A + 64 (scale d u + x u),  dv: B + 64 scale d,
  dbeta: the same with the values' norm, dg: A B + 64 times dk's,  ds0: B + scale d tokens
and 16-bit gradients are rounded once more.
"""
import ctypes

import pytest

from test_seq_delta import E32, U, _inputs

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


@pytest.fixture(scope="module")
def seq():
    import mixed_precision_refinement_gb300 as zs
    s = zs.Seq()
    yield s
    s.close()


def _loss(x, dout, ds, scale, keep=None):
    """sum(dout * o) + sum(ds * s) of the recurrence, in the inputs' type (float64)."""
    torch = _torch()
    group = x["v"].shape[1] // x["k"].shape[1]
    q, k = (x[n].repeat_interleave(group, 1) for n in ("q", "k"))
    total = 0.0
    off = x["offsets"].tolist()
    for i in range(len(off) - 1):
        s = x["s0"][i]
        for t in range(off[i], off[i + 1]):
            s = s * torch.exp(x["g"][t])[:, None, None]
            u = x["beta"][t][:, None] * (x["v"][t] - torch.einsum("hkv,hk->hv", s, k[t]))
            s = s + k[t][..., None] * u[:, None, :]
            if keep is not None:
                s.retain_grad()
                u.retain_grad()
                keep.append((s, u))
            total = total + scale * (torch.einsum("hkv,hk->hv", s, q[t]) * dout[t]).sum()
        total = total + (s * ds[i]).sum()
    return total


NAMES = ("q", "k", "v", "g", "beta", "s0")


def _case(lens, hk, hv, dk, dv, dtype, seed, ds=True, **kw):
    torch = _torch()
    x = _inputs(lens, hk, hv, dk, dv, dtype, seed, **kw)
    x["s0"] *= 0.2
    gen = torch.Generator("cuda").manual_seed(seed + 1)
    dout = torch.randn(x["v"].shape, generator=gen, device="cuda").to(x["v"].dtype)
    dstate = 0.2 * torch.randn(x["s0"].shape, generator=gen, device="cuda") * (1.0 if ds else 0.0)
    return x, dout, dstate


def _reference(x, dout, ds, scale):
    y = {n: (t if n == "offsets" else t.double().requires_grad_()) for n, t in x.items()}
    keep = []
    _loss(y, dout.double(), ds.double(), scale, keep).backward()
    A = max([float(s.detach().norm(dim=(-2, -1)).max()) for s, _ in keep] + [float(x["s0"].double().norm(dim=(-2, -1)).max())])
    B = max([float(s.grad.norm(dim=(-2, -1)).max()) for s, _ in keep] + [float(ds.double().norm(dim=(-2, -1)).max())])
    un = max([float(u.detach().norm(dim=-1).max()) for _, u in keep] + [0.0])
    xn = max([float(u.grad.norm(dim=-1).max()) for _, u in keep] + [0.0])
    return {n: y[n].grad for n in NAMES}, (A, B, un, xn)


def _tolerances(x, dout, sizes, scale, chunks):
    A, B, un, xn = sizes
    group = x["v"].shape[1] // x["k"].shape[1]
    d = float(dout.double().norm(dim=-1).max()) if dout.numel() else 0.0
    vn = float(x["v"].double().norm(dim=-1).max()) if dout.numel() else 0.0
    e = (2 * chunks + 2) * E32
    tk = un * B + xn * A + 64 * (scale * d * un + xn * un)
    tv = B + 64 * scale * d
    return {"q": e * group * (scale * d * A + 64 * scale * d * un), "k": e * group * tk, "v": e * tv,
            "beta": e * (tv * (vn + A) + 64 * xn * un), "g": e * (A * B + 64 * tk),
            "s0": e * (B + scale * d * 64 * chunks)}


def _check(seq, lens, hk, hv, dk, dv, dtype, seed=0, **kw):
    x, dout, ds = _case(lens, hk, hv, dk, dv, dtype, seed, **kw)
    scale = 0.6
    ref, sizes = _reference(x, dout, ds, scale)
    got = seq.delta_bwd(dout, x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], ds, x["offsets"], scale)
    tol = _tolerances(x, dout, sizes, scale, max(-(-n // 64) for n in lens))
    for n, y in zip(NAMES, got):
        u = U[dtype] if n in "qkv" else U["float32"]
        err = (y.double() - ref[n]).abs() - u * ref[n].abs()
        assert float(err.max()) <= tol[n], (n, float(err.max()), tol[n])
        # the errors are of both signs: their root mean square is held to a hundredth of the bound
        assert float(err.clamp(min=0).square().mean().sqrt()) <= tol[n] / 100, n
    return x, dout, ds, got


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (32, 32), (96, 80), (100, 33), (1, 1), (17, 130)])
def test_head_sizes(seq, dk, dv, dtype):
    _check(seq, [70, 130], 2, 2, dk, dv, dtype, seed=dk + dv)


@pytest.mark.parametrize("lens", [[1], [63], [64], [65], [128], [1, 0, 2, 64, 0, 130]], ids=lambda x: "-".join(map(str, x)))
def test_lengths(seq, lens):
    _check(seq, lens, 1, 2, 48, 40, "float32", seed=sum(lens))
    _check(seq, lens, 1, 2, 48, 40, "bfloat16", seed=sum(lens) + 1)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("hk,hv", [(1, 1), (1, 6), (3, 3), (2, 8)])
def test_shared_key_heads(seq, hk, hv, dtype):
    _check(seq, [80], hk, hv, 64, 32, dtype, seed=hk * hv)


def test_long_memory_and_no_last_gradient(seq):
    _check(seq, [300], 1, 1, 128, 64, "float32", seed=4, decay=0.0, positive=True)
    x, dout, ds, got = _check(seq, [150], 1, 2, 32, 64, "bfloat16", seed=5, ds=False)
    again = seq.delta_bwd(dout, x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], None, x["offsets"], 0.6)
    torch = _torch()
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_strong_and_infinite_decays(seq):
    torch = _torch()
    x, dout, ds = _case([150], 1, 2, 32, 32, "float32", 6)
    x["g"][40, 0] = -300.0
    x["g"][90, 1] = -5000.0
    x["beta"][20] = 0.0
    ref, sizes = _reference(x, dout, ds, 0.6)
    tol = _tolerances(x, dout, sizes, 0.6, 3)
    got = seq.delta_bwd(dout, x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], ds, x["offsets"], 0.6)
    for n, y in zip(NAMES, got):
        assert float((y.double() - ref[n]).abs().max()) <= tol[n], n
    x["g"][40, 0] = -float("inf")  # empties the state as exp(-300) does: the same gradients, and none is NaN
    got = seq.delta_bwd(dout, x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], ds, x["offsets"], 0.6)
    for n, y in zip(NAMES, got):
        assert float((y.double() - ref[n]).abs().max()) <= tol[n], n


@pytest.mark.parametrize("name", NAMES)
def test_gradient_against_differences(seq, name):
    """Along a random direction, from differences of the float64 recurrence (steps h and 2 h, Richardson:
    off by h^4, below the tolerance by far)."""
    torch = _torch()
    x, dout, ds = _case([75, 20], 1, 2, 16, 12, "float32", 7)
    scale, h = 0.6, 1e-3
    _, sizes = _reference(x, dout, ds, scale)
    tol = _tolerances(x, dout, sizes, scale, 2)
    got = dict(zip(NAMES, seq.delta_bwd(dout, x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], ds, x["offsets"], scale)))
    p = torch.randn(x[name].shape, generator=torch.Generator("cuda").manual_seed(8), device="cuda").double()
    y = {n: (t if n == "offsets" else t.double()) for n, t in x.items()}

    def val(s):
        return float(_loss(dict(y, **{name: y[name] + s * h * p}), dout.double(), ds.double(), scale))

    d1, d2 = (val(1) - val(-1)) / (2 * h), (val(2) - val(-2)) / (4 * h)
    along = float((got[name].double() * p).sum())
    # the elements' errors along p: of both signs, ten times their root mean square bound
    assert abs((4 * d1 - d2) / 3 - along) <= 10 * tol[name] / 100 * float(p.norm()) + 1e-6 * abs(along)


def test_strided_inputs_and_no_tokens(seq):
    torch = _torch()
    x, dout, ds = _case([50, 50], 2, 2, 32, 24, "bfloat16", 9)
    ref = seq.delta_bwd(dout, x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], ds, x["offsets"])
    for pad in (0, 5):
        wide = torch.empty(2, 50, pad + 2 * 64 + 2 * 48, device="cuda", dtype=torch.bfloat16)
        parts = [wide[..., pad + a:pad + b] for a, b in ((0, 64), (64, 128), (128, 176), (176, 224))]
        q, k, v, do = (p.unflatten(-1, (2, d)) for p, d in zip(parts, (32, 32, 24, 24)))
        for d, src in ((q, x["q"]), (k, x["k"]), (v, x["v"]), (do, dout)):
            d.copy_(src.view(d.shape))
        got = seq.delta_bwd(do, q, k, v, x["g"].view(2, 50, 2), x["beta"].view(2, 50, 2), x["s0"], ds)
        assert all(torch.equal(a.reshape(b.shape), b) for a, b in zip(got, ref))
    none = [t[:0] for t in (dout, x["q"], x["k"], x["v"], x["g"], x["beta"])]
    off = torch.zeros(3, dtype=torch.int64, device="cuda")
    got = seq.delta_bwd(*none, x["s0"], ds, off)
    assert torch.equal(got[5], ds) and got[0].shape == (0, 2, 32)


def test_same_result_twice(seq):
    torch = _torch()
    x, dout, ds = _case([200, 130], 2, 4, 128, 64, "bfloat16", 10)
    args = (dout, x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], ds, x["offsets"])
    one, two = seq.delta_bwd(*args), seq.delta_bwd(*args)
    assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_refusals(seq):
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    x, dout, ds = _case([10], 2, 4, 16, 8, "float32", 11)
    args = (x["q"], x["k"], x["v"], x["g"], x["beta"])
    with pytest.raises(TypeError):
        seq.delta_bwd(dout.half(), *args)
    with pytest.raises(ValueError):
        seq.delta_bwd(dout[:9], *args)
    with pytest.raises(ValueError):
        seq.delta_bwd(dout, *args, ds=ds[..., :7])
    lib, p = zs.raw_lib(), dout.data_ptr()
    a = zs.zsolve_delta_args(type=0, hk=2, hv=4, dk=16, dv=8, nseq=1, tokens=10, offsets=None, q=p, k=p, v=p, ldq=32,
                             ldk=32, ldv=32, g=p, beta=p, s0=None, scale=1.0)
    good = [p, 32, None, p, p, p, p, p, None]
    for i, v in ((0, None), (1, 31), (3, None), (4, None), (5, None), (6, None), (7, None)):
        bad = list(good)
        bad[i] = v
        assert lib.zsolve_delta_bwd(seq.seq, ctypes.byref(a), *bad) == zs.ZSOLVE_EINVAL, i
    assert lib.zsolve_delta_bwd(None, ctypes.byref(a), *good) == zs.ZSOLVE_EINVAL


def test_many_sequences_equal_one_alone(seq):
    """One sequence's recurrences run side by side, those of many one after the other: the same gradients."""
    torch = _torch()
    x, dout, ds = _case([200] * 40, 1, 2, 64, 64, "bfloat16", 12)
    order = ("q", "k", "v", "g", "beta")
    many = seq.delta_bwd(dout, *(x[n] for n in order), x["s0"], ds=ds, offsets=x["offsets"])
    for i in (0, 39):
        at = slice(200 * i, 200 * i + 200)
        one = seq.delta_bwd(dout[at], *(x[n][at] for n in order), x["s0"][i:i + 1], ds=ds[i:i + 1])
        for a, b in zip(many[:5], one):
            assert torch.equal(a[at], b)
        assert torch.equal(many[5][i], one[5][0])
