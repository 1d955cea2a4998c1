"""The sequence-layer operators under autograd: loss.backward() gives the gradients of the operators' own
backward calls, and what carries none says so."""
import pytest

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


@pytest.fixture(scope="module")
def seq():
    import mixed_precision_refinement_gb300 as zs
    with zs.Seq() as s:
        yield s


def _randn(gen, *shape, dtype="bfloat16", scale=1.0):
    torch = _torch()
    return (scale * torch.randn(*shape, generator=gen, device="cuda")).to(getattr(torch, dtype))


def _leaves(*ts):
    return [None if t is None else t.clone().requires_grad_() for t in ts]


@pytest.mark.parametrize("wtype,bias", [("bfloat16", True), ("float32", True), ("float32", False)])
def test_layernorm(seq, wtype, bias):
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(1)
    x, w, dy = _randn(gen, 3, 20, 64), _randn(gen, 64, dtype=wtype), _randn(gen, 3, 20, 64)
    b = _randn(gen, 64, dtype=wtype) if bias else None
    y0, mean, rstd = seq.layernorm(x, w, b)
    X, W, B = _leaves(x, w, b)
    y, mean2, _ = seq.layernorm(X, W, B)
    assert torch.equal(y, y0) and y.requires_grad
    y.backward(dy)
    dx, dw, db = seq.layernorm_bwd(dy, x, mean, rstd, w)
    assert torch.equal(X.grad, dx) and torch.equal(W.grad, dw)
    assert not bias or torch.equal(B.grad, db)
    with pytest.raises(RuntimeError, match="mean and rstd"):
        mean2.sum().backward()
    # one of them alone, and the gradient of a sum, which has no memory of its own
    W, = _leaves(w)
    seq.layernorm(x, W, b)[0].float().sum().backward()
    assert torch.equal(W.grad, seq.layernorm_bwd(torch.ones_like(x), x, mean, rstd, w)[1])


def test_layernorm_without_weights(seq):
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(2)
    x, b, dy = _randn(gen, 9, 33), _randn(gen, 33, dtype="float32"), _randn(gen, 9, 33)
    X, B = _leaves(x, b)
    seq.layernorm(X, None, B)[0].backward(dy)
    _, mean, rstd = seq.layernorm(x)
    assert torch.equal(X.grad, seq.layernorm_bwd(dy, x, mean, rstd)[0])
    assert float((B.grad - dy.float().sum(0)).abs().max()) <= 32 * 2.0 ** -24 * float(dy.float().abs().sum(0).max())


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("keep", [False, True])
def test_linear(seq, act, keep):
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(3)
    x, w, b, r, dy = (_randn(gen, *s) for s in ((2, 30, 40), (24, 40), (24,), (2, 30, 24), (2, 30, 24)))
    y0, z = seq.linear(x, w, b, act=act, r=r, keep=True)
    X, W, B, R = _leaves(x, w, b, r)
    out = seq.linear(X, W, B, act=act, r=R, keep=keep)
    y = out[0] if keep else out
    assert torch.equal(y, y0)
    y.backward(dy)
    dx, dw, db = seq.linear_bwd(dy, x, w, z, act=act)
    for got, ref in ((X.grad, dx), (W.grad, dw), (B.grad, db), (R.grad, dy)):
        assert torch.equal(got, ref)
    if keep:
        assert torch.equal(out[1], z)
        with pytest.raises(RuntimeError, match="z"):
            seq.linear(*_leaves(x, w, b), act=act, keep=True)[1].sum().backward()
    W, = _leaves(w)  # the weight alone
    seq.linear(x, W, b, act=act).backward(dy)
    assert torch.equal(W.grad, dw)
    R, = _leaves(r)  # the residual alone
    seq.linear(x, w, r=R, act=act).backward(dy)
    assert torch.equal(R.grad, dy)


@pytest.mark.parametrize("state", [False, True])
def test_delta(seq, state):
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(4)
    n, hk, hv, dk, dv = 90, 2, 4, 32, 24
    q, k, v, do = (_randn(gen, n, h, d, scale=0.2) for h, d in ((hk, dk), (hk, dk), (hv, dv), (hv, dv)))
    g, beta = -_randn(gen, n, hv, dtype="float32").abs(), _randn(gen, n, hv, dtype="float32").sigmoid()
    offsets = torch.tensor([0, 50, 90], device="cuda")
    s0 = _randn(gen, 2, hv, dk, dv, dtype="float32") if state else None
    ds = _randn(gen, 2, hv, dk, dv, dtype="float32")
    ins = (q, k, v, g, beta, s0)
    leaves = _leaves(*ins)
    o, s = seq.delta(*leaves, offsets=offsets)
    o0, s1 = seq.delta(*ins, offsets=offsets)
    assert torch.equal(o, o0) and torch.equal(s, s1)
    torch.autograd.backward([o, s], [do, ds])
    ref = seq.delta_bwd(do, *ins, ds=ds, offsets=offsets)
    for leaf, want in zip(leaves, ref):
        assert leaf is None or torch.equal(leaf.grad, want)
    leaves = _leaves(*ins)  # the outputs alone, and the last states alone
    seq.delta(*leaves, offsets=offsets)[0].backward(do)
    assert torch.equal(leaves[0].grad, seq.delta_bwd(do, *ins, offsets=offsets)[0])
    leaves = _leaves(*ins)
    seq.delta(*leaves, offsets=offsets)[1].backward(ds)
    assert torch.equal(leaves[2].grad, seq.delta_bwd(torch.zeros_like(do), *ins, ds=ds, offsets=offsets)[2])


def test_step_says_that_it_has_none(seq):
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(5)
    q, k, v = (_randn(gen, 3, 2, 16) for _ in range(3))
    g, beta = -torch.rand(3, 2, device="cuda"), torch.rand(3, 2, device="cuda")
    s = torch.zeros(3, 2, 16, 16, device="cuda")
    ref = s.clone()
    o0, _ = seq.delta_step(q, k, v, g, beta, ref)
    o, s2 = seq.delta_step(*_leaves(q, k, v), g, beta, s)
    assert torch.equal(o, o0) and torch.equal(s2, ref) and torch.equal(s, ref)
    with pytest.raises(RuntimeError, match="delta_step"):
        o.sum().backward()
    with torch.no_grad():
        o, s3 = seq.delta_step(*_leaves(q, k, v), g, beta, ref)
    assert not o.requires_grad and s3 is ref


def test_a_layer_and_a_closed_handle():
    """A layer's loss.backward() on another stream and in two leading dimensions; a handle that is closed is an error."""
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(6)
    x, w, wi = _randn(gen, 2, 70, 48, scale=0.5), _randn(gen, 48), _randn(gen, 96, 48, scale=0.1)
    g, beta = -_randn(gen, 2, 70, 1, dtype="float32").abs(), _randn(gen, 2, 70, 1, dtype="float32").sigmoid()
    dy = _randn(gen, 2, 70, 1, 32)

    def run(s, x, w, wi):
        h = s.layernorm(x, w)[0]
        q, k, v = s.linear(h, wi, act="silu").split(32, dim=-1)
        return s.delta(*(t.unflatten(-1, (1, 32)) for t in (q, k, v)), g, beta)[0]

    with zs.Seq() as s:
        ref = _leaves(x, w, wi)
        run(s, *ref).backward(dy)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            leaves = _leaves(x, w, wi)
            run(s, *leaves).backward(dy)
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(ref, leaves):
            assert torch.equal(a.grad, b.grad) and bool(torch.isfinite(a.grad).all()) and bool(a.grad.any())
        late = run(s, *_leaves(x, w, wi))
    with pytest.raises(zs.ZsolveError):
        late.backward(dy)
