"""What the binding refuses before the library is called: tensors of another device, and shapes that have the
right number of values in another order."""
import pytest

from mixed_precision_refinement_gb300 import seq as binding


class Elsewhere:
    """A tensor of another device, as far as the checks ask."""

    is_cuda = True
    device = "cuda:1"

    def get_device(self):
        return 1

    def __getattr__(self, name):
        raise AssertionError(f"{name}: nothing of the tensor is used")


@pytest.mark.parametrize("check", [lambda t: binding._rows(t, "x"), lambda t: binding._vector(t, "w", 4, None),
                                   lambda t: binding._tokens(t, "q")])
def test_a_tensor_of_another_device_is_refused(check, monkeypatch):
    monkeypatch.setattr(binding, "_device", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="current device, 0.*cuda:1"):
        check(Elsewhere())


@pytest.fixture(scope="module")
def seq():
    import mixed_precision_refinement_gb300 as zs
    with zs.Seq() as s:
        yield s


@pytest.mark.gpu
def test_delta_shapes_in_another_order(seq):
    import torch
    b, t, hk, hv, dk, dv = 2, 6, 1, 3, 8, 4

    def make(*shape):
        return torch.rand(*shape, device="cuda")

    q, k, v = make(b, t, hk, dk), make(b, t, hk, dk), make(b, t, hv, dv)
    g, beta, s0 = -make(b, t, hv), make(b, t, hv), make(b, hv, dk, dv)
    good = dict(q=q, k=k, v=v, g=g, beta=beta, s0=s0)
    o, _ = seq.delta(**good)
    # other shapes with the same order
    for same in (dict(g=g.view(b * t, hv)), dict(beta=beta.flatten()), dict(s0=s0.view(b * hv, dk, dv)), dict(s0=s0.flatten())):
        assert torch.equal(seq.delta(**{**good, **same})[0], o)
    # the same number of values in another one
    other = [dict(g=make(b, hv, t)), dict(g=make(t, b, hv)), dict(g=make(hv, b * t)), dict(beta=make(t, b, hv)),
             dict(beta=make(hv, b, t)), dict(s0=make(b, hv, dv, dk)), dict(s0=make(b, dk, hv, dv)), dict(s0=make(hv, b, dk, dv)),
             dict(k=make(t, b, hk, dk)), dict(v=make(t, b, hv, dv))]
    for bad in other:
        with pytest.raises(ValueError):
            seq.delta(**{**good, **bad})
        with pytest.raises(ValueError):
            seq.delta_bwd(o, **{**good, **bad})
    with pytest.raises(ValueError):
        seq.delta_bwd(make(t, b, hv, dv), **good)
    with pytest.raises(ValueError):
        seq.delta_bwd(o, **good, ds=make(b, hv, dv, dk))
    step = [x[:, 0].contiguous() for x in (q, k, v, g, beta)]
    seq.delta_step(*step, s0)
    with pytest.raises(ValueError):
        seq.delta_step(*step[:3], make(hv, b), step[4], s0)
    with pytest.raises(ValueError):
        seq.delta_step(*step, make(b, hv, dv, dk))


@pytest.mark.gpu
def test_norm_statistics_in_another_order(seq):
    import torch
    x = torch.randn(3, 5, 16, device="cuda")
    y, mean, rstd = seq.layernorm(x)
    dx, _, _ = seq.layernorm_bwd(y, x, mean, rstd)
    for same in ((mean.flatten(), rstd.flatten()), (mean.view(3, 5, 1), rstd.view(3, 5, 1))):
        assert torch.equal(seq.layernorm_bwd(y, x, *same)[0], dx)
    for bad in ((mean.T.contiguous(), rstd), (mean, rstd.T.contiguous())):
        with pytest.raises(ValueError):
            seq.layernorm_bwd(y, x, *bad)
