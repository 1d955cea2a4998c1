"""Gradients of linear attention with a decay for each head against float64 (limits: test_seq_decay.py)."""
import pytest

from test_seq_decay import LAYOUTS, OUTSIDE, SPANS, U, _all_pairs, _inputs, _limit, _near, _outside, _sizes

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "g", "s0")


@pytest.fixture(scope="module")
def seq():
    import mixed_precision_refinement_gb300 as zs
    s = zs.Seq()
    yield s
    zs.zsolve_seq_check(s.seq)
    s.close()


def _case(lens, hk, hv, dk, dv, dtype, seed, **kw):
    import torch
    x = _inputs(lens, hk, hv, dk, dv, dtype, seed, **kw)
    gen = torch.Generator("cuda").manual_seed(seed + 1)
    dout = torch.randn(x["v"].shape, generator=gen, device="cuda").to(x["v"].dtype)
    return x, dout, torch.randn(x["s0"].shape, generator=gen, device="cuda")


def _grads(x, dout, ds, scale, weight=None):
    import torch
    y = {n: t if n == "offsets" else t.double().requires_grad_() for n, t in x.items()}
    o, s = _all_pairs(y, scale, weight)
    total = (s * ds.double()).sum() if ds is not None else 0.0
    ((o * dout.double()).sum() + total).backward()
    return {n: torch.zeros_like(x[n], dtype=torch.float64) if y[n].grad is None else y[n].grad for n in NAMES}


def _limits(x, dout, ds, scale):
    """The limits of the gradients but for their own rounding.  dg is a sum over its span and head, at most the sequence, of
    terms q_i . dq_i and k_j . dk_j, and a state's product with its gradient, which is at most as large."""
    import torch
    size, of16 = _sizes(x), x["q"].dtype != torch.float32
    a = dout.abs(), None if ds is None else ds.abs()
    tol = _grads(size, *a, scale, _limit(x, of16))
    full = _grads(size, *a, scale, _limit(x))
    tol["s0"] = full["s0"]
    group = x["v"].shape[1] // x["k"].shape[1]
    # by value head: of each of them alone
    head = {n: t.repeat_interleave(group, 1) if n in ("q", "k") else t for n, t in size.items()}
    own = _grads(head, *a, scale, _limit(x))
    terms = (own["q"] * head["q"]).sum(-1) + (own["k"] * head["k"]).sum(-1)
    off = x["offsets"].tolist()
    g = torch.zeros(x["v"].shape[:2], dtype=torch.float64, device="cuda")
    for i, (p, q) in enumerate(zip(off, off[1:])):
        g[p:q] = terms[p:q].sum(0) + (own["s0"][i] * size["s0"][i]).sum((-1, -2))
    tol["g"] = g.sum(0) if x["g"].dim() == 1 else g
    return tol


def _check(seq, lens, hk, hv, dk, dv, dtype, seed=0, s0=True, last=True, **kw):
    import torch
    x, dout, ds = _case(lens, hk, hv, dk, dv, dtype, seed, **kw)
    scale = 0.7
    if not s0:
        x["s0"] = torch.zeros_like(x["s0"])
    ds = ds if last else None
    got = seq.decay_bwd(dout, x["q"], x["k"], x["v"], x["g"], x["s0"] if s0 else None, ds, x["offsets"], scale)
    ref, tol = _grads(x, dout, ds, scale), _limits(x, dout, ds, scale)
    for n, t in zip(NAMES, got):
        _near(t, ref[n], tol[n], U[dtype] if n in "qkv" else U["float32"], n)


HEADS = [(128, 128), (64, 64), (32, 32), (96, 80), (100, 33), (1, 1), (17, 130), (40, 16), (128, 256), (33, 64)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("dk,dv", HEADS)
def test_head_sizes(seq, dk, dv, dtype):
    _check(seq, [70, 300], 2, 4, dk, dv, dtype, seed=dk + dv)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("lens", [[1], [9], [64], [65], [127], [128], [129], [256], [257], [512], [513], [700], [1, 0, 2, 64, 0, 130, 63, 257]],
                         ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("per", ["token", "head"])
def test_lengths(seq, lens, dtype, per):
    _check(seq, lens, 1, 3, 48, 40, dtype, seed=sum(lens), per=per)


@pytest.mark.parametrize("hk,hv", [(1, 1), (1, 6), (5, 5), (3, 12)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_head_layouts(seq, hk, hv, dtype):
    _check(seq, [300, 31], hk, hv, 64, 32, dtype, seed=hk * hv)


@pytest.mark.parametrize("s0,last", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_without_states(seq, s0, last, dtype):
    _check(seq, [130, 270], 2, 2, 64, 48, dtype, seed=6, s0=s0, last=last)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_nonfinite_gradients_stay_in_their_heads(seq, dtype):
    """More rows of blocks than the GPU holds at a time: a gradient that is not finite changes no bit of later tokens, nor of other heads."""
    import torch
    x, dout, ds = _case([1100], 16, 64, 64, 64, dtype, 12)
    call = lambda d: seq.decay_bwd(d, x["q"], x["k"], x["v"], x["g"], x["s0"], ds, x["offsets"], 0.7)  # noqa: E731
    clean = call(dout)
    for token, head in ((700, 5), (0, 40), (1099, 63)):
        d = dout.clone()
        d[token, head, 7] = float("nan")
        got = call(d)
        assert bool(got[2][:token + 1, head, 7].isnan().all()) and bool(got[0][token, head // 4].isnan().all())
        for i, (a, b) in enumerate(zip(got[:4], clean)):
            own = head // 4 if i < 2 else head
            others = [h for h in range(a.shape[1]) if h != own]
            assert torch.equal(a[:, others], b[:, others])
            assert torch.equal(a[token + 1:, own], b[token + 1:, own])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("lens,hk,hv,dk,dv", SPANS)
def test_many_rows(seq, lens, hk, hv, dk, dv, dtype):
    _check(seq, lens, hk, hv, dk, dv, dtype, seed=11)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_positive_decays_grow(seq, dtype):
    _check(seq, [600, 3, 130], 1, 2, 64, 64, dtype, seed=10, decay=-0.2)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_strong_and_infinite_decays(seq, dtype):
    import torch
    x, dout, ds = _case([400], 1, 2, 64, 32, dtype, 8)
    x["g"][200, 0] = -float("inf")
    x["g"][133, 1] = -1e30
    x["g"][40:60:2] = -300.0
    got = seq.decay_bwd(dout, x["q"], x["k"], x["v"], x["g"], x["s0"], ds, x["offsets"], 0.7)
    y = dict(x, g=x["g"].clamp(min=-1e4))
    ref, tol = _grads(y, dout, ds, 0.7), _limits(y, dout, ds, 0.7)
    for n, t in zip(NAMES, got):
        _near(t, ref[n], tol[n], U[dtype] if n in "qkv" else U["float32"], n)
    assert bool(torch.isfinite(got[3]).all())


FACTOR, U32 = 32, 2.0 ** -24


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("n,hk,hv,dk,dv", [(200, 2, 2, 128, 128), (600, 2, 4, 64, 64), (130, 1, 2, 32, 32), (300, 1, 2, 96, 80),
                                           (64, 1, 1, 17, 33), (1500, 1, 1, 128, 64)])
def test_float32_accuracy(seq, n, hk, hv, dk, dv, dtype):
    """What is float32 (states, the decays' gradients, and everything where the inputs are) has float32's accuracy, by its
    root-mean-square error next to that of the same sums in plain float32.  Split operands keep 22 bits (four times float32's
    rounding), the tensor cores cut their sums (2^-23 an addition, always towards zero) in chains of at most sixteen before a float32
    addition; twice their sum, rounded down to a power of two, is 32.  One tf32 rounding alone is 8192 times float32's."""
    import torch
    x, dout, ds = _case([n], hk, hv, dk, dv, dtype, n + dk)
    x["s0"] *= 0.2
    exact, (oe, se) = _grads(x, dout, ds, 0.6), (t.detach() for t in _all_pairs(x, 0.6))
    group = hv // hk
    y = {i: t if i == "offsets" else t.float().clone().requires_grad_() for i, t in x.items()}
    q, k = (y[i].repeat_interleave(group, 1).transpose(0, 1) for i in ("q", "k"))
    v, b = y["v"].transpose(0, 1), y["g"].T.cumsum(1)
    d = (b[:, :, None] - b[:, None, :]).masked_fill(torch.ones(n, n, device="cuda", dtype=torch.bool).triu(1), -float("inf"))
    o = 0.6 * (torch.exp(b)[..., None] * (q @ y["s0"][0]) + (torch.exp(d) * (q @ k.mT)) @ v).transpose(0, 1)
    s = (torch.exp(b[:, -1])[:, None, None] * y["s0"][0] + (torch.exp(b[:, -1:] - b)[..., None] * k).mT @ v)[None]
    ((o * dout.float()).sum() + (s * ds).sum()).backward()
    plain = dict({i: y[i].grad for i in NAMES}, o=o.detach(), s=s.detach())
    exact = dict(exact, o=oe, s=se)
    args = [x[i] for i in NAMES]
    o, s = seq.decay(*args, x["offsets"], 0.6)
    got = {n: t.detach() for n, t in zip(NAMES, seq.decay_bwd(dout, *args, ds, x["offsets"], 0.6))}
    got.update(o=o, s=s)
    for name in ("s", "g", "s0") + (("o", "q", "k", "v") if dtype == "float32" else ()):
        limit = FACTOR * max(float((plain[name].double() - exact[name]).norm()), U32 * float(exact[name].norm()))
        assert float((got[name].double() - exact[name]).norm()) <= limit, name
    for name in ("o", "q", "k", "v"):  # what has 16 bits is off by little more than its own rounding
        err = float((got[name].double() - exact[name]).norm())
        assert err <= (1.1 * U[dtype] / 3 ** 0.5 + 32 * U32) * float(exact[name].norm()), name


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("dk,dv", [(64, 48), (128, 33), (24, 64)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nonfinite_gradients_reach_no_later_token(seq, dk, dv, dtype, value):
    import torch
    n, scale, col = 300, 0.6, 7
    x, dout, ds = _case([n], 2, 2, dk, dv, dtype, 18)
    args = [x[i] for i in NAMES]
    ref, tol = _grads(x, dout, ds, scale), _limits(x, dout, ds, scale)
    base = seq.decay_bwd(dout, *args, ds, x["offsets"], scale)
    for tok in (0, 5, 63, 64, 130, 255, 256, 299):
        d = dout.clone()
        d[tok, 0, col] = value
        got = seq.decay_bwd(d, *args, ds, x["offsets"], scale)
        for name, a, b in zip(NAMES[:4], got, base):
            # the tokens after it: the same gradients, in another order of summation at most
            u = U[dtype] if name in "qkv" else U["float32"]
            _near(a[tok + 1:], ref[name][tok + 1:], tol[name][tok + 1:], u, (name, tok))
            assert torch.equal(a[:, 1], b[:, 1]), (name, tok)  # the other head
        others = [c for c in range(dv) if c != col]
        _near(got[2][:, 0, others], ref["v"][:, 0, others], tol["v"][:, 0, others], U[dtype], tok)
        assert not torch.isfinite(got[2][:tok + 1, 0, col]).any() and not torch.isfinite(got[0][tok, 0]).any()
        assert not torch.isfinite(got[4][0, 0, :, col]).any() and torch.equal(got[4][0, 1], base[4][0, 1])


@pytest.mark.parametrize("before,lens,after", OUTSIDE)
@pytest.mark.parametrize("hk,hv,dk,dv,dtype", LAYOUTS)
@pytest.mark.parametrize("per", ["token", "head"])
def test_tokens_of_no_sequence(seq, before, lens, after, hk, hv, dk, dv, dtype, per):
    import torch

    import mixed_precision_refinement_gb300 as zs
    x, inner = _outside(before, lens, after, hk, hv, dk, dv, dtype)
    if per == "head":
        x["g"] = inner["g"] = -torch.rand(hv, device="cuda") / 4
    gen = torch.Generator("cuda").manual_seed(3)
    dout = torch.randn(x["v"].shape, generator=gen, device="cuda").to(x["v"].dtype)
    ds = torch.randn(x["s0"].shape, generator=gen, device="cuda")
    at = slice(before, before + sum(lens))
    clean = dout[at].clone()
    dout[:before] = dout[at.stop:] = float("nan")
    # the workspace holds something else before: the gradients of all tokens as one sequence, NaN
    everything = torch.full_like(x["offsets"], dout.shape[0])
    everything[0] = 0
    seq.decay_bwd(dout, *(x[n] for n in NAMES), ds, everything)

    def grads(y, d):
        out = [torch.full_like(y[n], 7.0) for n in NAMES]
        zs.zsolve_decay_bwd(seq.seq, d, *(y[n] for n in "qkvg"), *out, s0=y["s0"], ds=ds, offsets=y["offsets"])
        return out

    got, ref = grads(x, dout), grads(inner, clean)
    assert torch.equal(got[4], ref[4])
    for n, a, b in zip(NAMES[:4], got, ref):
        if a.dim() == 1:
            assert torch.equal(a, b), n
            continue
        assert torch.equal(a[at], b), n
        assert not a[:before].any() and not a[at.stop:].any(), n


@pytest.mark.parametrize("per", ["token", "head"])
def test_against_differences(seq, per):
    """Derivatives of (o, dout) + (s, ds) along a direction from forward values at +- h and +- 2 h (Richardson): off by the values'
    errors over h and by at most the difference of the two estimates."""
    import torch
    x, dout, ds = _case([90], 1, 2, 16, 24, "float32", 5, per=per)
    scale = 0.5
    got = dict(zip(NAMES, seq.decay_bwd(dout, *(x[n] for n in NAMES), ds, x["offsets"], scale)))
    tol = [t.abs() for t in _all_pairs(_sizes(x), scale, _limit(x))]
    value_tol = float((tol[0] * dout.abs()).sum() + (tol[1] * ds.abs()).sum())
    own = _limits(x, dout, ds, scale)
    for name in NAMES:
        along = torch.randn(x[name].shape, generator=torch.Generator("cuda").manual_seed(2), device="cuda") / 4
        h = 2.0 ** -4 if name != "g" else 2.0 ** -7

        def value(t):
            o, s = seq.decay(*({**x, name: x[name] + t * along}[n] for n in NAMES), x["offsets"], scale)
            return float((o.double() * dout.double()).sum() + (s.double() * ds.double()).sum())

        val = {t: value(t * h) for t in (-2, -1, 1, 2)}
        d1, d2 = (val[1] - val[-1]) / (2 * h), (val[2] - val[-2]) / (4 * h)
        terms = got[name].double() * along.double()
        # the values' errors do not all have one sign: a quarter of their sum is still far above what happens
        assert abs((4 * d1 - d2) / 3 - float(terms.sum())) <= 1.5 / h * value_tol + abs(d1 - d2) + float((own[name] * along.abs()).sum()), name


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_strides_and_the_same_twice(seq, dtype):
    import torch
    dt = getattr(torch, dtype)
    b, n, hk, hv, dk, dv = 2, 290, 2, 4, 32, 24
    x, dout, ds = _case([n] * b, hk, hv, dk, dv, dtype, 10)
    args = [x[i] for i in NAMES]
    ref = seq.decay_bwd(dout, *args, ds, x["offsets"])
    for p, q in zip(seq.decay_bwd(dout, *args, ds, x["offsets"]), ref):
        assert torch.equal(p, q)
    for pad in (0, 3):
        wide = torch.empty(b, n, pad + 2 * hk * dk + 2 * hv * dv, device="cuda", dtype=dt)
        at, views = pad, []
        for h, d, src in ((hk, dk, x["q"]), (hk, dk, x["k"]), (hv, dv, x["v"]), (hv, dv, dout)):
            views.append(wide[..., at:at + h * d].unflatten(-1, (h, d)))
            views[-1].copy_(src.view(b, n, h, d))
            at += h * d
        q, k, v, do = views
        got = seq.decay_bwd(do, q, k, v, x["g"].view(b, n, hv), x["s0"], ds)
        for p, w in zip(got, ref):
            assert torch.equal(p.reshape(w.shape), w)


@pytest.mark.parametrize("per", ["token", "head"])
@pytest.mark.parametrize("state", [False, True])
def test_autograd(seq, state, per):
    import torch
    x, dout, ds = _case([50, 40], 2, 4, 32, 24, "bfloat16", 4, per=per)
    ins = [x[n] if n != "s0" or state else None for n in NAMES]

    def leaves():
        return [None if t is None else t.clone().requires_grad_() for t in ins]

    a = leaves()
    o, s = seq.decay(*a, offsets=x["offsets"])
    o0, s1 = seq.decay(*ins, offsets=x["offsets"])
    assert torch.equal(o, o0) and torch.equal(s, s1)
    torch.autograd.backward([o, s], [dout, ds])
    for leaf, want in zip(a, seq.decay_bwd(dout, *ins, ds=ds, offsets=x["offsets"])):
        assert leaf is None or torch.equal(leaf.grad, want)
    a = leaves()  # the outputs alone, and the last states alone
    seq.decay(*a, offsets=x["offsets"])[0].backward(dout)
    assert torch.equal(a[3].grad, seq.decay_bwd(dout, *ins, offsets=x["offsets"])[3])
    a = leaves()
    seq.decay(*a, offsets=x["offsets"])[1].backward(ds)
    assert torch.equal(a[2].grad, seq.decay_bwd(torch.zeros_like(dout), *ins, ds=ds, offsets=x["offsets"])[2])
    one = [t[:2].clone().requires_grad_() for t in ins[:3]]
    g = ins[3][:2] if per == "token" else ins[3]
    st = torch.zeros(2, 4, 32, 24, device="cuda")
    with pytest.raises(RuntimeError, match="decay_step"):
        seq.decay_step(*one, g, st)[0].sum().backward()
