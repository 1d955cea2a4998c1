"""Gradients of tensors whose leading dimensions differ from one another's (a batch of sequences beside its rows, states in one
piece): each has the shape of what it is the gradient of, and the values of the call on one layout."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def seq():
    import mixed_precision_refinement_gb300 as zs
    s = zs.Seq()
    yield s
    zs.zsolve_seq_check(s.seq)
    s.close()


def _randn(gen, *shape, dtype=None):
    import torch
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype or torch.float32)


def _same(call, tensors, shapes):
    """call's gradients with its tensors in `shapes`, against those in their own."""
    import torch
    grads = []
    for form in (lambda n, t: t, lambda n, t: t.reshape(shapes.get(n, t.shape))):
        leaves = {n: form(n, t).detach().clone().requires_grad_() for n, t in tensors.items()}
        outs = call(**leaves)
        torch.autograd.backward(outs, [torch.linspace(-1, 1, o.numel(), device="cuda").view(o.shape).to(o.dtype) for o in outs])
        for n, t in leaves.items():
            assert t.grad.shape == t.shape, n
        grads.append({n: t.grad.flatten() for n, t in leaves.items()})
    for n in tensors:
        assert torch.equal(grads[0][n], grads[1][n]), n


@pytest.mark.parametrize("shapes", [dict(x=(2, 3, 40)), dict(o=(2, 3, 40)), dict(z=(1, 6, 40)), dict(x=(3, 2, 40), z=(2, 3, 40))], ids=str)
def test_resnorm(seq, shapes):
    import torch
    gen = torch.Generator("cuda").manual_seed(1)
    t = {n: _randn(gen, 6, 40) for n in "xoz"}
    _same(lambda x, o, z: seq.resnorm(x, o, z=z)[:2], t, shapes)
    _same(lambda x, o, z: seq.resnorm(x, o, z=z)[:1], t, shapes)
    x, o, z = (t[n].reshape(shapes.get(n, (6, 40))) for n in "xoz")
    y, h, stats = seq.resnorm(x, o, z=z)
    dx, do, dz, *_ = seq.resnorm_bwd(h, y, o, stats, z=z)
    assert (dx.shape, do.shape, dz.shape) == (x.shape, o.shape, z.shape)


def test_linear_with_rows_added(seq):
    import torch
    gen = torch.Generator("cuda").manual_seed(2)
    t = dict(x=_randn(gen, 2, 6, 32, dtype=torch.bfloat16), r=_randn(gen, 2, 6, 16, dtype=torch.bfloat16))
    w = _randn(gen, 16, 32, dtype=torch.bfloat16)
    _same(lambda x, r: [seq.linear(x, w, r=r)], t, dict(r=(12, 16)))
    _same(lambda x, r: [seq.linear(x, w, act="silu", r=r)], t, dict(x=(12, 32)))


@pytest.mark.parametrize("form", ["decay", "delta"])
def test_states_in_one_piece(seq, form):
    import torch
    gen = torch.Generator("cuda").manual_seed(3)
    b, n, hk, hv, dk, dv = 2, 20, 1, 2, 16, 8
    t = dict(q=_randn(gen, b, n, hk, dk), k=_randn(gen, b, n, hk, dk) / 4, v=_randn(gen, b, n, hv, dv), g=-_randn(gen, b, n, hv).abs(),
             s0=_randn(gen, b, hv, dk, dv))
    if form == "delta":
        t["beta"] = torch.rand(b, n, hv, generator=gen, device="cuda")
    _same(getattr(seq, form), t, dict(s0=(b * hv * dk * dv,), g=(b * n, hv)))
