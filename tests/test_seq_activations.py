"""The activations' tails: values and slopes far from zero, where a cancellation would leave no digits, held to
bounds relative to the value itself.

Tolerances.  With X the exponent's size (z^2 / 2, |z|, or 2 sqrt(2 / pi) |z + 0.044715 z^3|), the argument's
roundings are at most 2^-22 X of the result, the exponential's own error 2 + 1.2 X units in the last place, and the
other factors' 16 2^-24: together below (X + 4) 2^-21.  The result is rounded once; the slope twice, since it is the
products' operand.  A quotient whose divisor is above 2^126 is 0.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

U = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
STEP = {"bfloat16": 0.0, "float16": 2.0 ** -25}  # half of float16's smallest step; bfloat16 has float32's range
FAR = {"bfloat16": 12.0, "float16": 6.0}


@pytest.fixture(scope="module")
def seq():
    import mixed_precision_refinement_gb300 as zs
    s = zs.Seq()
    yield s
    zs.zsolve_seq_check(s.seq)
    s.close()


def _parts(z, act):
    """Value, slope, the size of the slope's two terms, X, and what the slope loses with a quotient of 2^-126, in
    float64 without cancellation."""
    import torch
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
        q = z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return z * p, p + q, p.abs() + q.abs(), 0.5 * z * z, 0.0 * z
    c, a = (1.0, 0.0) if act == "silu" else (2 * math.sqrt(2 / math.pi), 0.044715)
    x, inner = c * (z + a * z ** 3), z.abs() * c * (1 + 3 * a * z * z)
    p = torch.sigmoid(x)
    q = inner * z.sign() * p * torch.sigmoid(-x)
    return z * p, p + q, p.abs() + q.abs(), x.abs(), (1 + inner) * 2.0 ** -126


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("rows", [7, 700])
def test_tails(seq, act, dtype, rows):
    import torch
    dt, u = getattr(torch, dtype), U[dtype]
    z = torch.linspace(-FAR[dtype], FAR[dtype], rows, device="cuda").to(dt)[:, None]
    one = torch.ones(1, 1, device="cuda", dtype=dt)
    value, slope, size, x, lost = _parts(z.double(), act)
    tol = (x + 4) * 2.0 ** -21
    for n in (1, 8):  # one output, or eight at once
        y = seq.linear(z, one.expand(n, 1).contiguous(), act=act)
        for i in range(n):
            err = (y[:, i:i + 1].double() - value).abs()
            assert bool((err <= (tol * (1 + u) + u) * value.abs() + STEP[dtype] + lost).all()), (act, n)
    dx, _, db = seq.linear_bwd(one.expand(rows, 1).contiguous(), z, one, z, act=act)
    err = (dx.double() - slope).abs()
    assert bool((err <= tol * size * (1 + 2 * u) + (2 * u + u * u) * slope.abs() + 3 * STEP[dtype] + lost).all())


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_very_large_values(seq, act):
    """Where z^2 or z^3 is no longer a float32: the values are z and 0, the slopes 1 and 0."""
    import torch
    z = torch.tensor([1e4, 1e15, 1e20, 3e38], device="cuda").bfloat16()[:, None]
    z = torch.cat([z, -z])
    one = torch.ones(1, 1, device="cuda", dtype=torch.bfloat16)
    y = seq.linear(z, one, act=act)
    assert torch.equal(y[:4], z[:4]) and not y[4:].any()
    dx, _, _ = seq.linear_bwd(torch.full_like(z, 3.0), z, one, z, act=act)
    assert bool((dx[:4] == 3.0).all()) and not dx[4:].any()
