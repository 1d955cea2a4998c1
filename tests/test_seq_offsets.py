"""Offsets of the gated delta rule that leave tokens to no sequence, as a buffer filled in part has: the
sequences' results are those of the tokens alone, and the outputs and gradients of the others are zero."""
import pytest

from test_seq_delta import _inputs

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "g", "beta")


@pytest.fixture(scope="module")
def seq():
    import mixed_precision_refinement_gb300 as zs
    s = zs.Seq()
    yield s
    zs.zsolve_seq_check(s.seq)
    s.close()


# tokens before, the sequences' lengths, tokens after; the small ones go token by token
CASES = [(5, [35, 0, 30], 30), (0, [64], 1), (200, [70], 0), (130, [0], 70), (1, [0, 1, 0], 1), (2, [3], 3), (4, [0], 4)]
HEADS = [(2, 2, 32, 40, "float32"), (1, 3, 128, 64, "bfloat16"), (2, 4, 17, 33, "float16")]


def _case(before, lens, after, hk, hv, dk, dv, dtype):
    import torch
    x = _inputs([before + sum(lens) + after], hk, hv, dk, dv, dtype, seed=before + after)
    x["s0"] = torch.randn(len(lens), hv, dk, dv, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    x["offsets"] = torch.tensor([before + sum(lens[:i]) for i in range(len(lens) + 1)], device="cuda")
    inner = dict(x, offsets=x["offsets"] - before)
    for n in NAMES:
        # what lies outside is not read
        inner[n] = x[n][before:before + sum(lens)].clone()
        x[n][:before] = x[n][before + sum(lens):] = float("nan")
    return x, inner


@pytest.mark.parametrize("before,lens,after", CASES)
@pytest.mark.parametrize("hk,hv,dk,dv,dtype", HEADS)
@pytest.mark.parametrize("form", ["delta", "step"])
def test_outputs(seq, before, lens, after, hk, hv, dk, dv, dtype, form):
    import torch

    import mixed_precision_refinement_gb300 as zs
    x, inner = _case(before, lens, after, hk, hv, dk, dv, dtype)
    call = zs.zsolve_delta_step if form == "step" else zs.zsolve_delta
    # zsolve_delta takes up to 8 tokens one by one
    same_way = form == "step" or (sum(lens) <= 8) == (before + sum(lens) + after <= 8)
    o, s = torch.full_like(x["v"], 7.0), torch.full_like(x["s0"], 7.0)
    call(seq.seq, *(x[n] for n in NAMES), o, s, x["s0"], x["offsets"])
    oi, si = torch.full_like(inner["v"], 7.0), torch.full_like(x["s0"], 7.0)
    call(seq.seq, *(inner[n] for n in NAMES), oi, si, x["s0"], inner["offsets"])
    at = slice(before, before + sum(lens))
    if same_way:
        assert torch.equal(o[at], oi) and torch.equal(s, si)
    else:
        assert bool(torch.isfinite(o).all()) and float((s - si).abs().max()) <= 1e-4
    assert not o[:before].any() and not o[at.stop:].any()


@pytest.mark.parametrize("before,lens,after", CASES)
@pytest.mark.parametrize("hk,hv,dk,dv,dtype", HEADS)
def test_gradients(seq, before, lens, after, hk, hv, dk, dv, dtype):
    import torch

    import mixed_precision_refinement_gb300 as zs
    x, inner = _case(before, lens, after, hk, hv, dk, dv, dtype)
    gen = torch.Generator("cuda").manual_seed(3)
    dout = torch.randn(x["v"].shape, generator=gen, device="cuda").to(x["v"].dtype)
    ds = torch.randn(x["s0"].shape, generator=gen, device="cuda")
    at = slice(before, before + sum(lens))
    # the workspace holds something else before: the gradients of all tokens as one sequence, NaN
    everything = torch.full_like(x["offsets"], dout.shape[0])
    everything[0] = 0
    seq.delta_bwd(dout, *(x[n] for n in NAMES), x["s0"], ds, everything)

    def grads(y, d):
        out = [torch.full_like(y[n], 7.0) for n in NAMES] + [torch.full_like(y["s0"], 7.0)]
        zs.zsolve_delta_bwd(seq.seq, d, *(y[n] for n in NAMES), *out, s0=y["s0"], ds=ds, offsets=y["offsets"])
        return out

    got, ref = grads(x, dout), grads(inner, dout[at].clone())
    assert torch.equal(got[5], ref[5])
    for n, a, b in zip(NAMES, got, ref):
        assert torch.equal(a[at], b), n
        assert not a[:before].any() and not a[at.stop:].any(), n
