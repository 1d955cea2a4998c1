"""The gated delta rule through the C-ABI against the recurrence in float64.

Tolerances.  With keys of norm at most 1, steps in 0 .. 1 and decays at most 1, the map of a state to
the next is not expansive, so the errors of the chunks add up at most.  One chunk's products carry
float32-class errors (2^-21 of their terms for the split products), and its 64 x 64 solve magnifies
them at most 64 times; the state and u are held to (chunks + 1) 64 2^-21 of the largest column norm
that a state, a value or u has.  o is that, plus its own rounding, plus, where it has 16 bits, tf32
operands (2^-11 each of two or three) on its terms |q| |S| + sum over a chunk |P| |u|.
"""
import ctypes

import pytest

pytestmark = pytest.mark.gpu

U = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
E32 = 64 * 2.0 ** -21


def _torch():
    import torch
    return torch


@pytest.fixture(scope="module")
def seq():
    import mixed_precision_refinement_gb300 as zs
    s = zs.Seq()
    yield s
    s.close()


def _inputs(lens, hk, hv, dk, dv, dtype, seed=0, decay=0.3, positive=False):
    torch = _torch()
    dt = getattr(torch, dtype)
    gen = torch.Generator("cuda").manual_seed(seed)
    t = sum(lens)

    def randn(*shape):
        x = torch.randn(*shape, generator=gen, device="cuda")
        return x.abs() if positive else x

    def unit(x):  # norm 0.99, so that it is below 1 after rounding
        return (0.99 * x / x.norm(dim=-1, keepdim=True).clamp(min=1e-9)).to(dt)

    q, k = unit(randn(t, hk, dk)), unit(randn(t, hk, dk))
    v = torch.randn(t, hv, dv, generator=gen, device="cuda").to(dt)
    g = -decay * torch.rand(t, hv, generator=gen, device="cuda") ** 2
    beta = torch.rand(t, hv, generator=gen, device="cuda")
    s0 = torch.randn(len(lens), hv, dk, dv, generator=gen, device="cuda")
    offsets = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], device="cuda")
    return dict(q=q, k=k, v=v, g=g, beta=beta, s0=s0, offsets=offsets)


def reference(q, k, v, g, beta, s0, offsets, scale):
    """o, the last states, u, and the largest column norm along the way."""
    torch = _torch()
    group = v.shape[1] // k.shape[1]
    q, k = (x.double().repeat_interleave(group, 1) for x in (q, k))
    v, a, beta = v.double(), torch.exp(g.double()), beta.double()
    o, u_all, last, size = torch.zeros_like(v), torch.zeros_like(v), [], 0.0
    off = offsets.tolist()
    for i in range(len(off) - 1):
        s = s0[i].double()
        for t in range(off[i], off[i + 1]):
            s = s * a[t][:, None, None]
            u = beta[t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", s, k[t]))
            s = s + k[t][..., None] * u[:, None, :]
            o[t] = scale * torch.einsum("hkv,hk->hv", s, q[t])
            u_all[t] = u
            size = torch.maximum(torch.as_tensor(size, device=s.device), s.norm(dim=1).max())
        last.append(s)
    size = max(float(size), float(s0.double().norm(dim=2).max()) if s0.numel() else 0.0,
               float(v.abs().max()) * 8 if v.numel() else 0.0)
    return o, torch.stack(last), u_all, size


def _tol(chunks, size):
    return (chunks + 1) * E32 * size


def _o_tol(ref, u_all, offsets, dtype, chunks, size, scale):
    torch = _torch()
    tol = scale * _tol(chunks, size) + U[dtype] * ref.abs()
    if dtype != "float32":
        window = torch.zeros_like(u_all)
        off = offsets.tolist()
        for a, b in zip(off, off[1:]):
            for c in range(a, b, 64):
                window[c:min(c + 64, b)] = u_all[c:min(c + 64, b)].abs().sum(0)
        tol = tol + 3 * 2.0 ** -11 * scale * (size + window)
    return tol


def _check(seq, lens, hk, hv, dk, dv, dtype, seed=0, form="delta", s0=True, **kw):
    torch = _torch()
    x = _inputs(lens, hk, hv, dk, dv, dtype, seed, **kw)
    scale = 0.7
    ref, last, u_all, size = reference(**x, scale=scale)
    if not s0:
        x["s0"] = torch.zeros_like(x["s0"])
        ref, last, u_all, size = reference(**x, scale=scale)
        x["s0"] = None
    import mixed_precision_refinement_gb300 as zs
    o, s = torch.full_like(x["v"], 7.0), torch.full(last.shape, 7.0, device="cuda")
    call = zs.zsolve_delta if form == "delta" else zs.zsolve_delta_step
    call(seq.seq, x["q"], x["k"], x["v"], x["g"], x["beta"], o, s, x["s0"], x["offsets"], scale)
    chunks = max(-(-n // 64) for n in lens)
    assert float((s.double() - last).abs().max()) <= _tol(chunks, size)
    tol = _o_tol(ref, u_all, x["offsets"], dtype, chunks, size, scale)
    assert bool(((o.double() - ref).abs() <= tol).all()), float(((o.double() - ref).abs() / tol).max())
    return x, o, s


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (32, 32), (96, 80), (100, 33), (1, 1), (17, 130), (40, 16)])
def test_head_sizes(seq, dk, dv, dtype):
    _check(seq, [70, 200], 2, 4, dk, dv, dtype, seed=dk + dv)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("lens", [[1], [9], [63], [64], [65], [128], [129], [400], [1, 0, 2, 64, 0, 130, 63]],
                         ids=lambda x: "-".join(map(str, x)))
def test_lengths(seq, lens, dtype):
    _check(seq, lens, 1, 3, 48, 40, dtype, seed=sum(lens))


@pytest.mark.parametrize("hk,hv", [(1, 1), (1, 6), (5, 5), (3, 12)])
def test_head_layouts(seq, hk, hv):
    _check(seq, [100, 31], hk, hv, 64, 32, "bfloat16", seed=hk * hv)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (96, 80), (100, 33), (1, 1), (128, 31)])
def test_token_by_token(seq, dk, dv, dtype):
    _check(seq, [1, 1, 1], 2, 4, dk, dv, dtype, form="step", seed=1)
    _check(seq, [5, 0, 2], 2, 4, dk, dv, dtype, form="step", seed=2)
    _check(seq, [3, 4], 1, 2, dk, dv, dtype, form="step", seed=3, s0=False)


def test_long_memory(seq):
    """No decay at all and correlated keys: every token stays, and the chunk's solve is at its worst."""
    _check(seq, [1000], 1, 2, 128, 64, "float32", seed=4, decay=0.0, positive=True)
    _check(seq, [1000], 1, 2, 128, 64, "bfloat16", seed=5, decay=0.0, positive=True)


def test_no_first_state(seq):
    _check(seq, [130, 5], 2, 2, 64, 48, "bfloat16", seed=6, s0=False)


@pytest.mark.parametrize("form", ["delta", "step"])
def test_empty_state_at_infinite_decay_and_idle_tokens(seq, form):
    """g = -infinity and very negative decays empty the state; beta = 0 leaves it as it was."""
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    n = 200 if form == "delta" else 7
    x = _inputs([n], 1, 2, 64, 64, "float32", seed=8)
    x["g"][n // 2, 0] = -float("inf")
    x["g"][n // 3, 1] = -1e30
    x["g"][n - 2] = -300.0
    x["beta"][n // 4] = 0.0
    ref, last, u_all, size = reference(**x, scale=1.0)
    o, s = torch.empty_like(x["v"]), torch.empty_like(last, dtype=torch.float32)
    (zs.zsolve_delta if form == "delta" else zs.zsolve_delta_step)(
        seq.seq, x["q"], x["k"], x["v"], x["g"], x["beta"], o, s, x["s0"], x["offsets"], 1.0)
    assert float((s.double() - last).abs().max()) <= _tol(4, size)
    assert float((o.double() - ref).abs().max()) <= _tol(4, size)


def test_strong_decays_keep_the_digits_after_them(seq):
    """Slow decays after strong ones in the same chunk: e_ij comes from sums near -6000, whose float32
    steps alone would spoil it in the fourth digit."""
    torch = _torch()
    import mixed_precision_refinement_gb300 as zs
    x = _inputs([64], 1, 1, 32, 32, "float32", seed=9, decay=0.05)
    x["g"][:40:2] = -300.0
    ref, last, _, size = reference(**x, scale=1.0)
    o, s = torch.empty_like(x["v"]), torch.empty_like(last, dtype=torch.float32)
    zs.zsolve_delta(seq.seq, x["q"], x["k"], x["v"], x["g"], x["beta"], o, s, x["s0"], x["offsets"], 1.0)
    assert float((s.double() - last).abs().max()) <= _tol(1, size)
    assert float((o.double() - ref).abs().max()) <= _tol(1, size)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_strides_batches_and_states_in_place(seq, dtype):
    """q, k and v as slices of one projection's output, equal lengths in two leading dimensions, s over s0:
    the same as the packed call."""
    torch = _torch()
    dt = getattr(torch, dtype)
    b, n, hk, hv, dk, dv = 3, 90, 2, 4, 32, 24
    x = _inputs([n] * b, hk, hv, dk, dv, dtype, seed=10)
    o, s = seq.delta(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], x["offsets"])
    for pad in (0, 3):  # 3: neither pointers nor strides are multiples of 16 bytes
        wide = torch.empty(b, n, pad + 2 * hk * dk + hv * dv, device="cuda", dtype=dt)
        q, k, v = (wide[..., pad + i:pad + j] for i, j in ((0, hk * dk), (hk * dk, 2 * hk * dk),
                                                           (2 * hk * dk, 2 * hk * dk + hv * dv)))
        q, k, v = q.unflatten(-1, (hk, dk)), k.unflatten(-1, (hk, dk)), v.unflatten(-1, (hv, dv))
        for d, src in ((q, "q"), (k, "k"), (v, "v")):
            d.copy_(x[src].view(d.shape))
        g, beta = x["g"].view(b, n, hv), x["beta"].view(b, n, hv)
        o2, s2 = seq.delta(q, k, v, g, beta, x["s0"])
        assert torch.equal(o2.view(o.shape), o) and torch.equal(s2, s)
    import mixed_precision_refinement_gb300 as zs
    state = x["s0"].clone()
    zs.zsolve_delta(seq.seq, x["q"], x["k"], x["v"], x["g"], x["beta"], o, state, state, x["offsets"])
    assert torch.equal(state, s)


def test_prefill_then_steps_equals_one_call(seq):
    torch = _torch()
    x = _inputs([75, 75], 1, 2, 64, 64, "float32", seed=11)
    qq, kk, vv = (x[n].view(2, 75, *x[n].shape[1:]) for n in "qkv")
    gg, bb = (x[n].view(2, 75, 2) for n in ("g", "beta"))
    ref, s_ref = seq.delta(qq, kk, vv, gg, bb, x["s0"])
    first = [t[:, :70].contiguous() for t in (qq, kk, vv, gg, bb)]
    o, s = seq.delta(*first, x["s0"])
    outs = [o]
    for t in range(70, 75):
        o, s2 = seq.delta_step(*(z[:, t].contiguous() for z in (qq, kk, vv, gg, bb)), s)
        assert s2 is s
        outs.append(o.unsqueeze(1))
    size = float(s_ref.norm(dim=2).max())
    assert float((torch.cat(outs, 1) - ref).abs().max()) <= _tol(3, size)
    assert float((s - s_ref).abs().max()) <= _tol(3, size)
    few, s3 = seq.delta_step(*(z[:, 70:75].contiguous() for z in (qq, kk, vv, gg, bb)), seq.delta(*first, x["s0"])[1])
    assert float((few - ref[:, 70:75]).abs().max()) <= _tol(3, size)


def test_no_tokens(seq):
    torch = _torch()
    x = _inputs([0, 0], 1, 2, 8, 8, "float32", seed=12)
    o, s = seq.delta(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], x["offsets"])
    assert o.shape == (0, 2, 8) and torch.equal(s, x["s0"])
    o, s = seq.delta(x["q"], x["k"], x["v"], x["g"], x["beta"], None, x["offsets"])
    assert not s.any()


def test_nonfinite_stays_in_its_sequence_and_head(seq):
    torch = _torch()
    x = _inputs([100, 100], 2, 2, 32, 32, "bfloat16", seed=13)
    o, s = seq.delta(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], x["offsets"])
    x["v"][130, 1, 3] = float("nan")
    o2, s2 = seq.delta(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], x["offsets"])
    assert torch.equal(o2[:100], o[:100]) and torch.equal(o2[:, 0], o[:, 0])
    assert torch.isnan(s2[1, 1, :, 3]).all() and torch.equal(s2[1, 1, :, :3], s[1, 1, :, :3])
    x["g"][130, 1] = float("nan")
    _, s3 = seq.delta(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], x["offsets"])
    assert torch.isnan(s3[1, 1]).all() and torch.equal(s3[0], s[0])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nonfinite_values_reach_no_earlier_token(seq, dtype, value):
    """A token's infinity or NaN is in what follows it alone, also within its chunk.  (The chunk may be
    computed in another order because of it: both results lie within the tolerance of the exact one.)"""
    torch = _torch()
    x = _inputs([150], 1, 2, 64, 48, dtype, seed=18)
    names = ("q", "k", "v", "g", "beta", "s0", "offsets")
    scale = 0.125  # the call's own, 64 ** -0.5
    ref, _, u_all, size = reference(**x, scale=scale)
    tol = 2 * _o_tol(ref, u_all, x["offsets"], dtype, 3, size, scale)
    o, _ = seq.delta(*(x[n] for n in names))

    def same(a, where):
        return bool(((a.double() - o.double()).abs() <= tol)[where].all())

    for name in ("v", "k", "q", "g", "beta"):
        for tok in (0, 5, 68, 80, 101, 149):
            y = {n: t.clone() for n, t in x.items()}
            if name in "vkq":
                y[name][tok, 0, 7] = value
            else:
                y[name][tok, 0] = float("nan")
            o2, s2 = seq.delta(*(y[n] for n in names))
            assert same(o2, slice(0, tok)), (name, tok)
            if name != "k" and name != "q":  # the other head
                assert torch.equal(o2[:, 1], o[:, 1]), (name, tok)
            if name == "v":  # column 7 from there on
                others = [c for c in range(48) if c != 7]
                assert not torch.isfinite(o2[tok, 0, 7]) and not torch.isfinite(s2[0, 0, :, 7]).any()
                assert bool(((o2.double() - o.double()).abs() <= tol)[:, 0, others].all())
            elif name == "q":
                assert torch.equal(o2[tok + 1:], o[tok + 1:]) and not torch.isfinite(o2[tok]).any()
            else:
                assert not torch.isfinite(s2[0, 0]).any()


def test_offsets_out_of_range_are_kept_within_the_tensors(seq):
    """Offsets that do not ascend or leave 0 .. tokens: what is written stays inside the outputs."""
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    x = _inputs([100], 1, 1, 32, 32, "float32", seed=14)
    buf = torch.full((140, 1, 32), 9.0, device="cuda")
    s = torch.zeros(4, 1, 32, 32, device="cuda")
    off = torch.tensor([-5, 40, 20, 1 << 40, 70], device="cuda")
    for call in (zs.zsolve_delta, zs.zsolve_delta_step):
        call(seq.seq, x["q"], x["k"], x["v"], x["g"], x["beta"], buf[20:120], s, None, off)
        torch.cuda.synchronize()
        assert bool((buf[:20] == 9.0).all()) and bool((buf[120:] == 9.0).all()) and bool(torch.isfinite(s).all())


def test_same_result_twice_and_on_another_stream(seq):
    torch = _torch()
    x = _inputs([300, 20], 2, 4, 128, 64, "bfloat16", seed=15)
    args = (x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], x["offsets"])
    o, s = seq.delta(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, s2 = seq.delta(*args)
    o3, s3 = seq.delta(*args)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(s, s2) and torch.equal(o, o3) and torch.equal(s, s3)


def test_refusals(seq):
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    x = _inputs([10], 2, 4, 16, 8, "float32", seed=16)
    good = [x[n] for n in ("q", "k", "v", "g", "beta")]

    def bad(i, t, error):
        args = list(good)
        args[i] = t
        with pytest.raises(error):
            seq.delta(*args)

    bad(1, x["k"].half(), TypeError)
    bad(1, x["k"][:9], ValueError)
    bad(2, x["v"][:9], ValueError)
    bad(3, x["g"].double(), TypeError)
    bad(3, x["g"][:, :3], ValueError)
    bad(0, x["q"].double(), TypeError)
    bad(0, x["q"].cpu(), ValueError)
    bad(0, x["q"].transpose(1, 2), ValueError)
    bad(2, x["v"][:, :3].contiguous(), ValueError)  # g has four heads
    with pytest.raises(ValueError):
        seq.delta(*good, s0=torch.zeros(1, 4, 16, 7, device="cuda"))
    with pytest.raises(TypeError):
        seq.delta(*good, offsets=torch.tensor([0, 10], device="cuda", dtype=torch.int32))
    wide = _inputs([10], 1, 1, 129, 8, "float32", seed=17)
    with pytest.raises(zs.ZsolveError) as e:
        seq.delta(*(wide[n] for n in ("q", "k", "v", "g", "beta")))
    assert e.value.status == zs.ZSOLVE_EINVAL and "dk" in str(e.value)
    with pytest.raises(zs.ZsolveError):
        seq.delta(*good, scale=float("nan"))
    lib = zs.raw_lib()
    p = x["q"].data_ptr()

    def call(o=p, **kw):
        a = zs.zsolve_delta_args(type=0, hk=2, hv=4, dk=16, dv=8, nseq=1, tokens=10, offsets=None, q=p, k=p, v=p,
                                 ldq=32, ldk=32, ldv=32, g=p, beta=p, s0=None, scale=1.0)
        for n, v in kw.items():
            setattr(a, n, v)
        return lib.zsolve_delta(seq.seq, ctypes.byref(a), o, 32, None)

    for kw in (dict(type=5), dict(hk=3), dict(hk=0), dict(dk=0), dict(dv=0), dict(nseq=-1), dict(nseq=0),
               dict(nseq=3), dict(tokens=-1), dict(ldq=31), dict(ldv=31), dict(q=None), dict(g=None), dict(o=None)):
        assert call(**kw) == zs.ZSOLVE_EINVAL, kw
    assert lib.zsolve_delta(seq.seq, None, p, 32, None) == zs.ZSOLVE_EINVAL
    assert lib.zsolve_delta(None, None, p, 32, None) == zs.ZSOLVE_EINVAL
