"""Layer norm of rows with a common offset: outputs, mean and rstd as exact as without one.

Tolerance.  x - m is exact where x and m are within a factor of two of each other, so all errors are relative
to the deviations: float32 sums of them (at most 64 roundings in a chain, as for the operator without an
offset), which enter the output as mean |h| and through rstd as |h| / 2, and the output's own few roundings.
"""
import pytest

pytestmark = pytest.mark.gpu

U32, ADDS = 2.0 ** -24, 64


@pytest.fixture(scope="module")
def seq():
    import mixed_precision_refinement_gb300 as zs
    s = zs.Seq()
    yield s
    zs.zsolve_seq_check(s.seq)
    s.close()


@pytest.mark.parametrize("offset", [100.0, 1e4, -1e4, 1e5])
@pytest.mark.parametrize("d", [40, 200, 512, 1000, 1001, 2048, 4096, 4099, 8192, 16384, 20000])
def test_offset_costs_no_digits(seq, d, offset):
    import torch
    gen = torch.Generator("cuda").manual_seed(d)
    x = torch.randn(33, d, device="cuda", generator=gen) + offset
    y, mean, rstd = seq.layernorm(x, eps=0.0)
    x = x.double()
    mu = x.mean(1, keepdim=True)
    z = x - mu
    rs = z.square().mean(1, keepdim=True).rsqrt()
    h = z * rs
    size = h.abs().mean(1, keepdim=True) + h.abs()
    assert bool(((y.double() - h).abs() <= ADDS * U32 * size).all())
    assert bool(((rstd.double()[:, None] / rs - 1).abs() <= ADDS * U32).all())
    # the mean is rounded once to float32
    assert bool(((mean.double()[:, None] - mu).abs() <= U32 * mu.abs() + ADDS * U32 * z.abs().mean(1, keepdim=True)).all())


@pytest.mark.parametrize("d", [7, 40, 1000, 4096, 20000])
def test_constant_rows_with_no_variance(seq, d):
    """No deviation at all: h = 0 with rstd = eps^-1/2, whatever the mean's rounding."""
    import torch
    for value in (0.1, 7.3, -123.456, 3e5):
        y, mean, rstd = seq.layernorm(torch.full((3, d), value, device="cuda"), eps=1e-5)
        x = torch.full((1,), value, device="cuda")
        # m may be off by the sum's error, of which the second pass leaves a float32's rounding
        left = ADDS * U32 * ADDS * U32 * abs(value) + 2.0 ** -126
        assert float(y.abs().max()) <= left * 1e-5 ** -0.5
        assert float((rstd * 1e-5 ** 0.5 - 1).abs().max()) <= 8 * U32
        assert bool((mean == x).all())
