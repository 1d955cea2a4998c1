"""A block of a sequence model from the operators together: layer norm, projections, attention with decays, the norm around it with
its gate and residual scale, the gated feed-forward projections and the norm around those; forward, backward, token by token and in
graphs.

Tolerance.  Each operator's own tests hold it to its arithmetic; here its results count as exact but for a rounding to 16 bits,
half a step of it, u = eps / 2 relative, forwards and, of the gradients, backwards; the float32 statistics and decays count for nothing
beside it.  What such errors do to the block's results is measured on the float64 block itself: every value and every gradient
between two operators times 1 + u r, r uniform in [-1, 1].  Rounding errors have that size at most; eight draws' largest
distance is exceeded by another draw's one time in nine, by twice as much hardly ever (a distance of a hundred thousand values
varies by a few hundredths of itself), and twice as much again is for the roundings within an operator (a residual sum's terms, a
gradient's two shares): four times the largest.
"""
import pytest

gpu = pytest.mark.gpu
D, HK, HV, DK, DV, F = 128, 2, 4, 32, 48, 160
LENS = [1, 0, 130, 300, 17]


def _torch():
    import torch
    return torch


def _params(dtype, seed=0):
    torch = _torch()
    gen = torch.Generator("cuda").manual_seed(seed)

    def randn(*shape, by=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * by).to(dtype)

    def around(value, n):
        return (value + 0.2 * torch.randn(n, generator=gen, device="cuda")).to(dtype)

    t = sum(LENS)
    p = dict(x=randn(t, D), n1=around(1, D), m1=around(0, D), wq=randn(HK * DK, D, by=D ** -0.5), wk=randn(HK * DK, D, by=D ** -0.5),
             wv=randn(HV * DV, D, by=D ** -0.5), wo=randn(D, HV * DV, by=(HV * DV) ** -0.5), wz=randn(D, D, by=D ** -0.5), w1=around(1, D),
             b1=around(0, D), c1=around(0.5, D), w2=around(1, D), b2=around(0, D), wg=randn(F, D, by=D ** -0.5), wu=randn(F, D, by=D ** -0.5),
             bg=around(0, F), bu=around(0, F), wd=randn(D, F, by=F ** -0.5), c2=around(0.5, D), w3=around(1, D))
    p["g"] = -0.2 * torch.rand(t, HV, generator=gen, device="cuda")
    return p, randn(t, D), randn(t, D), gen


def _offsets():
    torch = _torch()
    return torch.tensor([sum(LENS[:i]) for i in range(len(LENS) + 1)], device="cuda")


def _block(s, p, offsets=None, step=None):
    """The block on handle s: over whole sequences, or (step: the states) for one token of each."""
    h = s.layernorm(p["x"], p["n1"], p["m1"])[0]
    q, k, v = (s.linear(h, p[w]).unflatten(1, n) for w, n in (("wq", (HK, DK)), ("wk", (HK, DK)), ("wv", (HV, DV))))
    o, state = s.decay(q, k, v, p["g"], offsets=offsets) if step is None else s.decay_step(q, k, v, p["g"], step)
    o = s.linear(o.flatten(1), p["wo"])
    y, h, _ = s.resnorm(p["x"], o, p["w1"], p["b1"], z=s.linear(h, p["wz"]), c=p["c1"], w2=p["w2"], b2=p["b2"])
    o = s.linear(s.glu(h, p["wg"], p["wu"], p["bg"], p["bu"]), p["wd"])
    y, h, _ = s.resnorm(y, o, c=p["c2"], w2=p["w3"], kind="rms", after=False)
    return y, h, state


def _off(u, gen):
    """A value and its gradient, off by up to u."""
    torch = _torch()

    class Off(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return x * (1 + u * (2 * torch.rand(x.shape, generator=gen, device="cuda", dtype=x.dtype) - 1))

        @staticmethod
        def backward(ctx, d):
            return d * (1 + u * (2 * torch.rand(d.shape, generator=gen, device="cuda", dtype=d.dtype) - 1))

    return Off.apply


def _block64(p, off):
    """The block's y and h from its formulas, in the type of p (float64)."""
    torch = _torch()
    fn = torch.nn.functional
    h = off(fn.layer_norm(p["x"], (D,), p["n1"], p["m1"]))
    q, k, v = (off(h @ p[w].T).unflatten(1, n) for w, n in (("wq", (HK, DK)), ("wk", (HK, DK)), ("wv", (HV, DV))))
    q, k = (t.repeat_interleave(HV // HK, 1) for t in (q, k))
    outs, at = [], 0
    for n in LENS:
        b = p["g"][at:at + n].cumsum(0).T  # heads x tokens
        w = (b[:, :, None] - b[:, None, :]).masked_fill(torch.ones(n, n, device="cuda", dtype=torch.bool).triu(1), float("-inf")).exp()
        Q, K, V = (t[at:at + n].transpose(0, 1) for t in (q, k, v))
        outs.append(((w * (Q @ K.mT) * DK ** -0.5) @ V).transpose(0, 1))
        at += n
    o = off(off(torch.cat(outs).flatten(1)) @ p["wo"].T)
    t = fn.layer_norm(o, (D,), p["w1"], p["b1"])
    y = off(p["x"] + p["c1"] * fn.silu(off(h @ p["wz"].T)) * t)
    h = off(fn.layer_norm(y, (D,), p["w2"], p["b2"]))
    f = off(fn.silu(off(h @ p["wg"].T + p["bg"])) * off(h @ p["wu"].T + p["bu"]))
    y = off(y + p["c2"] * off(f @ p["wd"].T))
    return y, off(y * (y.square().mean(1, keepdim=True) + 1e-5).rsqrt() * p["w3"])


def _all64(p, dy, dh, off):
    p = {n: t.detach().double().requires_grad_() for n, t in p.items()}
    out = _block64(p, off)
    _torch().autograd.backward(out, (dy.double(), dh.double()))
    return {"y": out[0].detach(), "h": out[1].detach(), **{"d" + n: t.grad for n, t in p.items()}}


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_block_and_its_gradients(dtype):
    torch = _torch()
    import mixed_precision_refinement_gb300 as zs
    dt = getattr(torch, dtype)
    p, dy, dh, gen = _params(dt)
    ref = _all64(p, dy, dh, lambda t: t)
    draws = [_all64(p, dy, dh, _off(torch.finfo(dt).eps / 2, gen)) for _ in range(8)]
    leaves = {n: t.clone().requires_grad_() for n, t in p.items()}
    with zs.Seq() as s:
        y, h, _ = _block(s, leaves, _offsets())
        torch.autograd.backward((y, h), (dy, dh))
        s.check()
    got = {"y": y.detach(), "h": h.detach(), **{"d" + n: t.grad for n, t in leaves.items()}}
    for n, r in ref.items():
        limit = 4 * max(float((d[n] - r).norm()) for d in draws)
        # the result's own rounding, where no draw has it (the gradients of the block's inputs)
        limit += torch.finfo(got[n].dtype).eps / 2 * float(r.norm())
        assert float((got[n].double() - r).norm()) <= limit, (n, float((got[n].double() - r).norm()), limit)


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_token_by_token_is_the_block(dtype):
    """One token of each of 5 sequences after the other gives what whole sequences give, to the same limit (rows' results do not
    depend on how many rows a call has, but for the attention's two forms)."""
    torch = _torch()
    import mixed_precision_refinement_gb300 as zs
    dt = getattr(torch, dtype)
    p, dy, dh, gen = _params(dt, 1)
    n, seqs = 12, 5
    cut = {k: t[:n * seqs] if k in ("x", "g") else t for k, t in p.items()}
    with zs.Seq() as s:
        y, h, last = _block(s, cut, torch.arange(0, n * seqs + 1, n, device="cuda"))
        state = torch.zeros_like(last)
        ys, hs = zip(*(_block(s, {**cut, "x": cut["x"][i::n].contiguous(), "g": cut["g"][i::n].contiguous()}, step=state)[:2] for i in range(n)))
        s.check()
    u = torch.finfo(dt).eps / 2
    global LENS
    lens, LENS = LENS, [n] * seqs
    try:
        ref = _all64(cut, dy[:n * seqs], dh[:n * seqs], lambda t: t)
        draws = [_all64(cut, dy[:n * seqs], dh[:n * seqs], _off(u, gen)) for _ in range(8)]
    finally:
        LENS = lens
    for name, whole, steps in (("y", y, ys), ("h", h, hs)):
        limit = 4 * max(float((d[name] - ref[name]).norm()) for d in draws)
        steps = torch.stack(steps, 1).flatten(0, 1).double()
        assert float((whole.double() - ref[name]).norm()) <= limit
        assert float((steps - ref[name]).norm()) <= limit


def _direct(s, p, dy, dh, offsets):
    """Forward and backward by the operators' own calls, as a program without autograd makes them."""
    h0, mean, rstd = s.layernorm(p["x"], p["n1"], p["m1"])
    q, k, v = (s.linear(h0, p[w]).unflatten(1, n) for w, n in (("wq", (HK, DK)), ("wk", (HK, DK)), ("wv", (HV, DV))))
    a, state = s.decay(q, k, v, p["g"], offsets=offsets)
    a = a.flatten(1)
    o, z = s.linear(a, p["wo"]), s.linear(h0, p["wz"])
    y1, h1, st1 = s.resnorm(p["x"], o, p["w1"], p["b1"], z=z, c=p["c1"], w2=p["w2"], b2=p["b2"])
    f, zg, zu = s.glu(h1, p["wg"], p["wu"], p["bg"], p["bu"], keep=True)
    o2 = s.linear(f, p["wd"])
    y2, h2, st2 = s.resnorm(y1, o2, c=p["c2"], w2=p["w3"], kind="rms", after=False)
    back = s.resnorm_bwd(dh, y2, o2, st2, c=p["c2"], w2=p["w3"], dy=dy, kind="rms", after=False)
    df, dwd, _ = s.linear_bwd(back[1], f, p["wd"])
    dh1, *dglu = s.glu_bwd(df, h1, p["wg"], p["wu"], zg, zu)
    dx, do, dz, *sums = s.resnorm_bwd(dh1, y1, o, st1, p["w1"], p["b1"], z=z, c=p["c1"], w2=p["w2"], b2=p["b2"], dy=back[0])
    da, dwo, _ = s.linear_bwd(do, a, p["wo"])
    grads = s.decay_bwd(da.unflatten(1, (HV, DV)), q, k, v, p["g"], offsets=offsets)
    parts = [s.linear_bwd(d.flatten(1), h0, p[w])[:2] for d, w in zip(grads[:3], ("wq", "wk", "wv"))] + [s.linear_bwd(dz, h0, p["wz"])[:2]]
    dh0 = parts[0][0] + parts[1][0] + parts[2][0] + parts[3][0]
    norm = s.layernorm_bwd(dh0, p["x"], mean, rstd, p["n1"])
    return [t for t in (y2, h2, state, *back, dwd, *dglu, dx, *sums, dwo, *grads, *(w for _, w in parts), *norm) if t is not None]


@gpu
def test_block_in_graphs_on_one_handle():
    """Two graphs of one handle (they share its workspace) on new inputs, replayed one after the other: the bits of eager calls."""
    torch = _torch()
    import mixed_precision_refinement_gb300 as zs
    dt = torch.bfloat16
    sets = [_params(dt, seed) for seed in (2, 3)]
    offsets = _offsets()
    with zs.Seq() as s:
        for p, dy, dh, _ in sets:
            _direct(s, p, dy, dh, offsets)  # the workspace grows here
        torch.cuda.synchronize()
        graphs, outs = [], []
        for p, dy, dh, _ in sets:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                outs.append(_direct(s, p, dy, dh, offsets))
        for seed in (4, 5):
            for i, (p, dy, dh, _) in enumerate(sets):
                new = _params(dt, seed + 10 * i)
                for n, t in p.items():
                    t.copy_(new[0][n])
                dy.copy_(new[1]), dh.copy_(new[2])
            for graph in graphs + graphs[:1]:
                graph.replay()
            torch.cuda.synchronize()
            for (p, dy, dh, _), out in zip(sets, outs):
                for a, b in zip(out, _direct(s, p, dy, dh, offsets)):
                    assert torch.equal(a, b)
        s.check()


@gpu
def test_block_twice_on_two_streams_and_handles():
    """The same bits from one handle twice, and from two handles at work on two streams at once."""
    torch = _torch()
    import mixed_precision_refinement_gb300 as zs
    p, dy, dh, _ = _params(torch.bfloat16, 6)
    offsets = _offsets()
    with zs.Seq() as s, zs.Seq() as t:
        first = [x.clone() for x in _direct(s, p, dy, dh, offsets)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        for stream in streams:
            stream.wait_stream(torch.cuda.current_stream())
        both = []
        for _ in range(3):
            for handle, stream in zip((s, t), streams):
                with torch.cuda.stream(stream):
                    both.append(_direct(handle, p, dy, dh, offsets))
        torch.cuda.synchronize()
        for out in both:
            for a, b in zip(first, out):
                assert torch.equal(a, b)
        s.check(), t.check()


@gpu
def test_training_step_in_a_graph():
    """Forward and backward under autograd, captured: the warm-up's graph is gone by then, as torch's capture of a backward pass
    needs it to be."""
    torch = _torch()
    import mixed_precision_refinement_gb300 as zs
    p, dy, dh, _ = _params(torch.bfloat16, 7)
    leaves = {n: t.clone().requires_grad_() for n, t in p.items()}
    offsets = _offsets()

    def step():
        for t in leaves.values():
            t.grad = None
        y, h, _ = _block(s, leaves, offsets)
        torch.autograd.backward((y, h), (dy, dh))

    with zs.Seq() as s:
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            for _ in range(2):
                step()
        torch.cuda.current_stream().wait_stream(stream)
        want = {n: t.grad.clone() for n, t in leaves.items()}
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        for n, t in leaves.items():
            assert torch.equal(t.grad, want[n]), n
        s.check()
