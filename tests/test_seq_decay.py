"""Linear attention with a decay for each head, through the C-ABI against sums over all pairs of tokens in float64.

Tolerances.  Every result is a sum of products of inputs and a weight exp(x), x a sum of log decays.  The kernels' products
have float32-class errors: split operands keep 22 bits, the tensor cores cut their short sums, and at most one
float32 addition for eight terms and one a span follow, so that a result of n tokens and heads of dk and dv values is off
by at most (n / 8 + dk / 8 + dv / 8 + 64) 2^-23 of the sum of its terms' sizes.  A weight's own error is that of x, |x| / ln 2
times 2^-23 at most, and a few units of exp.  Both are summed here as the results are, with absolute values for
inputs.  Results of 16 bits are also off by their rounding, and by 2^-16 of the terms' sizes, where their operands have 16 bits.
"""
import ctypes
import math

import pytest

U = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
gpu = pytest.mark.gpu


def _torch():
    import torch
    return torch


@pytest.fixture(scope="module")
def seq():
    import mixed_precision_refinement_gb300 as zs
    s = zs.Seq()
    yield s
    zs.zsolve_seq_check(s.seq)
    s.close()


def _inputs(lens, hk, hv, dk, dv, dtype, seed=0, decay=0.3, per="token"):
    torch = _torch()
    dt = getattr(torch, dtype)
    gen = torch.Generator("cuda").manual_seed(seed)
    t = sum(lens)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    g = -decay * torch.rand(*((hv,) if per == "head" else (t, hv)), generator=gen, device="cuda") ** 2
    return dict(q=randn(t, hk, dk).to(dt), k=randn(t, hk, dk).to(dt), v=randn(t, hv, dv).to(dt), g=g, s0=randn(len(lens), hv, dk, dv),
                offsets=torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], device="cuda"))


def _all_pairs(x, scale, weight=None):
    """o and the last states of all sequences in float64; weight(d): a factor for each weight exp(d)."""
    torch = _torch()
    group = x["v"].shape[1] // x["k"].shape[1]
    q, k = (x[n].double().repeat_interleave(group, 1).transpose(0, 1) for n in ("q", "k"))
    v = x["v"].double().transpose(0, 1)
    g = x["g"].double().clamp(min=-1e4).expand(v.shape[1], v.shape[0]).T
    off = x["offsets"].tolist()
    o, last = [v.new_zeros(v.shape[0], 0, v.shape[2])], []

    def e(d):
        return torch.exp(d) if weight is None else torch.exp(d) * weight(d)

    for i, (a, z) in enumerate(zip(off, off[1:])):
        s0 = x["s0"][i].double()
        b = g[:, a:z].cumsum(1)
        n = z - a
        if n == 0:
            last.append(s0 if weight is None else s0 * weight(torch.zeros((), device="cuda", dtype=torch.float64)))
            continue
        Q, K, V = q[:, a:z], k[:, a:z], v[:, a:z]
        d = (b[:, :, None] - b[:, None, :]).masked_fill(torch.ones(n, n, device="cuda", dtype=torch.bool).triu(1), -math.inf)
        pairs = torch.where(d == -math.inf, torch.zeros_like(d), e(torch.where(d == -math.inf, torch.zeros_like(d), d)))
        o.append(scale * (e(b)[..., None] * (Q @ s0) + (pairs * (Q @ K.mT)) @ V))
        last.append(e(b[:, -1])[:, None, None] * s0 + (e(b[:, -1:] - b)[..., None] * K).mT @ V)
    return torch.cat(o, 1).transpose(0, 1), torch.stack(last)


def _limit(x, of16=False):
    """weight(d) of the errors' sums (and, of16, of the results whose operands have 16 bits)."""
    n = int((x["offsets"][1:] - x["offsets"][:-1]).max()) if x["offsets"].numel() > 1 else 0
    c = (n / 8 + x["q"].shape[-1] / 8 + x["v"].shape[-1] / 8 + 64) * 2.0 ** -23 + (2.0 ** -16 if of16 else 0.0)
    return lambda d: c + 2.0 ** -22 * d.abs()


def _sizes(x):
    return {n: t if n in ("g", "offsets") else t.abs() for n, t in x.items()}


def _near(got, ref, tol, u, what):
    tol = tol + u * (ref.abs() + tol) + (2.0 ** -25 if u == U["float16"] else 1e-30)
    off = (got.double() - ref).abs() / tol
    assert bool((off <= 1).all()), (what, float(off.max()), int((off > 1).sum()))


def _check(seq, lens, hk, hv, dk, dv, dtype, seed=0, form="decay", s0=True, **kw):
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    x = _inputs(lens, hk, hv, dk, dv, dtype, seed, **kw)
    scale = 0.7
    if not s0:
        x["s0"] = torch.zeros_like(x["s0"])
    o, s = torch.full_like(x["v"], 7.0), torch.full(x["s0"].shape, 7.0, device="cuda")
    call = zs.zsolve_decay if form == "decay" else zs.zsolve_decay_step
    call(seq.seq, x["q"], x["k"], x["v"], x["g"], o, s, x["s0"] if s0 else None, x["offsets"], scale)
    _verify(x, scale, o, s, dtype)
    return x, o, s


def _verify(x, scale, o, s, dtype):
    ref, last = _all_pairs(x, scale)
    otol, stol = (_all_pairs(_sizes(x), scale, _limit(x, f))[i] for i, f in enumerate((dtype != "float32", False)))
    _near(s, last, stol, U["float32"], "s")
    _near(o, ref, otol, U[dtype], "o")


HEADS = [(128, 128), (64, 64), (32, 32), (96, 80), (100, 33), (1, 1), (17, 130), (40, 16), (128, 256), (33, 64)]


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("dk,dv", HEADS)
def test_head_sizes(seq, dk, dv, dtype):
    _check(seq, [70, 300], 2, 4, dk, dv, dtype, seed=dk + dv)


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("lens", [[1], [9], [63], [64], [65], [127], [128], [129], [255], [256], [257], [400], [512], [513], [900],
                                  [1, 0, 2, 64, 0, 130, 63, 257]], ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("per", ["token", "head"])
def test_lengths(seq, lens, dtype, per):
    _check(seq, lens, 1, 3, 48, 40, dtype, seed=sum(lens), per=per)


@gpu
@pytest.mark.parametrize("hk,hv", [(1, 1), (1, 6), (5, 5), (3, 12)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_head_layouts(seq, hk, hv, dtype):
    _check(seq, [300, 31], hk, hv, 64, 32, dtype, seed=hk * hv)


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (96, 80), (100, 33), (1, 1), (128, 31)])
@pytest.mark.parametrize("per", ["token", "head"])
def test_token_by_token(seq, dk, dv, dtype, per):
    _check(seq, [1, 1, 1], 2, 4, dk, dv, dtype, form="step", seed=1, per=per)
    _check(seq, [5, 0, 2], 2, 4, dk, dv, dtype, form="step", seed=2, per=per)
    _check(seq, [3, 4], 1, 2, dk, dv, dtype, form="step", seed=3, s0=False, per=per)


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_long_memory_and_no_first_state(seq, dtype):
    _check(seq, [1000], 1, 2, 128, 64, dtype, seed=4, decay=0.0)
    _check(seq, [130, 5], 2, 2, 64, 48, dtype, seed=6, s0=False)


@gpu
@pytest.mark.parametrize("form", ["decay", "step"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_empty_state_at_infinite_decay(seq, form, dtype):
    """g = -infinity and very negative decays empty the state."""
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    n = 400 if form == "decay" else 7
    x = _inputs([n], 1, 2, 64, 64, dtype, seed=8)
    x["g"][n // 2, 0] = -float("inf")
    x["g"][n // 3, 1] = -1e30
    x["g"][n - 2] = -300.0
    o, s = torch.empty_like(x["v"]), torch.empty_like(x["s0"])
    (zs.zsolve_decay if form == "decay" else zs.zsolve_decay_step)(seq.seq, x["q"], x["k"], x["v"], x["g"], o, s, x["s0"], x["offsets"], 1.0)
    _verify(x, 1.0, o, s, dtype)


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_strong_decays_keep_the_digits_after_them(seq, dtype):
    """Slow decays after strong ones in the same span: their weights come from sums near -6000, whose float32
    steps alone would spoil them in the fourth digit (differences of their sizes are what the limit counts)."""
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    x = _inputs([200], 1, 1, 32, 32, dtype, seed=9, decay=0.05)
    x["g"][:40:2] = -300.0
    o, s = torch.empty_like(x["v"]), torch.empty_like(x["s0"])
    zs.zsolve_decay(seq.seq, x["q"], x["k"], x["v"], x["g"], o, s, x["s0"], x["offsets"], 1.0)
    _verify(x, 1.0, o, s, dtype)


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_nonfinite_values_stay_in_their_head(seq, dtype):
    """More rows of blocks than the GPU holds at a time: what is not finite in one head's diagonal tiles changes no bit elsewhere."""
    torch = _torch()
    x = _inputs([1100], 16, 64, 64, 64, dtype, seed=12)
    clean = seq.decay(x["q"], x["k"], x["v"], x["g"], x["s0"], x["offsets"], 0.7)
    for token, head, column in ((700, 5, 3), (0, 40, 63), (1099, 63, 0)):
        v = x["v"].clone()
        v[token, head, column] = float("nan")
        o, s = seq.decay(x["q"], x["k"], v, x["g"], x["s0"], x["offsets"], 0.7)
        assert bool(o[token:, head, column].isnan().all()) and bool(s[0, head, :, column].isnan().all())
        o[token:, head, column], s[0, head, :, column] = clean[0][token:, head, column], clean[1][0, head, :, column]
        assert torch.equal(o, clean[0]) and torch.equal(s, clean[1])


# tokens x heads that each length of a span is taken for
SPANS = [([600, 3, 130], 8, 24, 32, 48), ([1030, 70, 0, 1], 16, 64, 32, 32), ([700, 3], 32, 64, 64, 32)]


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("lens,hk,hv,dk,dv", SPANS)
def test_many_rows(seq, lens, hk, hv, dk, dv, dtype):
    _check(seq, lens, hk, hv, dk, dv, dtype, seed=11)


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_positive_decays_grow(seq, dtype):
    """g above zero: states that grow, up to e^40 over two spans and a part."""
    _check(seq, [600, 3, 130], 1, 2, 64, 64, dtype, seed=10, decay=-0.2)


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_strides_batches_and_states_in_place(seq, dtype):
    """q, k and v as slices of one projection's output, equal lengths in two leading dimensions, s over s0:
    the same as the packed call."""
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    dt = getattr(torch, dtype)
    b, n, hk, hv, dk, dv = 3, 290, 2, 4, 32, 24
    x = _inputs([n] * b, hk, hv, dk, dv, dtype, seed=10)
    o, s = seq.decay(x["q"], x["k"], x["v"], x["g"], x["s0"], x["offsets"])
    for pad in (0, 3):  # 3: neither pointers nor strides are multiples of 16 bytes
        wide = torch.empty(b, n, pad + 2 * hk * dk + hv * dv, device="cuda", dtype=dt)
        q, k, v = (wide[..., pad + i:pad + j] for i, j in ((0, hk * dk), (hk * dk, 2 * hk * dk), (2 * hk * dk, 2 * hk * dk + hv * dv)))
        q, k, v = q.unflatten(-1, (hk, dk)), k.unflatten(-1, (hk, dk)), v.unflatten(-1, (hv, dv))
        for d, src in ((q, "q"), (k, "k"), (v, "v")):
            d.copy_(x[src].view(d.shape))
        o2, s2 = seq.decay(q, k, v, x["g"].view(b, n, hv), x["s0"])
        assert torch.equal(o2.view(o.shape), o) and torch.equal(s2, s)
    state, apart = x["s0"].clone(), torch.full((n * b, hv * dv + 5), 7.0, device="cuda", dtype=dt)
    zs.zsolve_decay(seq.seq, x["q"], x["k"], x["v"], x["g"], apart[:, :hv * dv].unflatten(-1, (hv, dv)), state, state, x["offsets"])
    assert torch.equal(state, s) and torch.equal(apart[:, :hv * dv], o.flatten(1)) and bool((apart[:, hv * dv:] == 7).all())


@gpu
def test_one_decay_a_head_is_that_decay_for_every_token(seq):
    torch = _torch()
    for n in (300, 5):
        x = _inputs([n], 2, 4, 64, 48, "bfloat16", seed=3, per="head")
        o, s = seq.decay(x["q"], x["k"], x["v"], x["g"], x["s0"])
        o2, s2 = seq.decay(x["q"], x["k"], x["v"], x["g"].expand(n, 4).contiguous(), x["s0"])
        assert torch.equal(o, o2) and torch.equal(s, s2)


@gpu
def test_prefill_then_steps_equals_one_call(seq):
    torch = _torch()
    x = _inputs([275, 275], 1, 2, 64, 64, "float32", seed=11)
    qq, kk, vv = (x[n].view(2, 275, *x[n].shape[1:]) for n in "qkv")
    gg = x["g"].view(2, 275, 2)
    first = [t[:, :270].contiguous() for t in (qq, kk, vv, gg)]
    o, s = seq.decay(*first, x["s0"])
    outs = [o]
    kept = s.clone()
    for t in range(270, 275):
        o, s2 = seq.decay_step(*(z[:, t].contiguous() for z in (qq, kk, vv, gg)), s)
        assert s2 is s
        outs.append(o.unsqueeze(1))
    scale = 64 ** -0.5
    _verify(x, scale, torch.cat(outs, 1).flatten(0, 1), s, "float32")
    beside = torch.zeros_like(kept)
    few, s3 = seq.decay_step(*(z[:, 270:275].contiguous() for z in (qq, kk, vv, gg)), kept, s_out=beside)
    assert s3 is beside and torch.equal(beside, s) and torch.equal(few, torch.cat(outs[1:], 1))


@gpu
def test_no_tokens(seq):
    torch = _torch()
    x = _inputs([0, 0], 1, 2, 8, 8, "float32", seed=12)
    o, s = seq.decay(x["q"], x["k"], x["v"], x["g"], x["s0"], x["offsets"])
    assert o.shape == (0, 2, 8) and torch.equal(s, x["s0"])
    o, s = seq.decay(x["q"], x["k"], x["v"], x["g"], None, x["offsets"])
    assert not s.any()
    ds = torch.randn(2, 2, 8, 8, device="cuda")
    for g in (x["g"], torch.zeros(2, device="cuda")):
        *_, dg, ds0 = seq.decay_bwd(o, x["q"], x["k"], x["v"], g, x["s0"], ds, x["offsets"])
        assert dg.shape == g.shape and not dg.any() and torch.equal(ds0, ds)
    assert not seq.decay_bwd(o, x["q"], x["k"], x["v"], x["g"], x["s0"], None, x["offsets"])[4].any()
    none = torch.zeros(1, device="cuda", dtype=torch.int64)  # no sequences at all
    o, s = seq.decay(x["q"], x["k"], x["v"], x["g"], None, none)
    assert s.shape == (0, 2, 8, 8)


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nonfinite_values_reach_no_earlier_token(seq, dtype, value):
    """A token's infinity or NaN is in what follows it alone, also within its span.  (The span may be
    computed in another order because of it: both results lie within the tolerance of the exact one.)"""
    torch = _torch()
    x = _inputs([300, 40], 2, 2, 64, 48, dtype, seed=18)
    names = ("q", "k", "v", "g", "s0", "offsets")
    scale = 0.125  # the call's own, 64 ** -0.5
    otol = 2 * (_all_pairs(_sizes(x), scale, _limit(x, dtype != "float32"))[0] + U[dtype] * _all_pairs(x, scale)[0].abs() + 2.0 ** -25)
    o, s = seq.decay(*(x[n] for n in names))

    def same(a, where):
        return bool(((a.double() - o.double()).abs() <= otol)[where].all())

    for name in ("v", "k", "q", "g"):
        for tok in (0, 5, 68, 80, 130, 255, 256, 299):
            y = {n: t.clone() for n, t in x.items()}
            if name == "g":
                y[name][tok, 0] = float("nan")
            else:
                y[name][tok, 0, 7] = value
            o2, s2 = seq.decay(*(y[n] for n in names))
            assert same(o2, slice(0, tok)) and same(o2, slice(300, 340)) and torch.equal(s2[1], s[1]), (name, tok)
            assert torch.equal(o2[:, 1], o[:, 1]) and torch.equal(s2[:, 1], s[:, 1]), (name, tok)  # the other head
            if name == "v":  # column 7 from there on
                others = [c for c in range(48) if c != 7]
                assert not torch.isfinite(o2[tok:300, 0, 7]).any() and not torch.isfinite(s2[0, 0, :, 7]).any()
                assert bool(((o2.double() - o.double()).abs() <= otol)[:, 0, others].all())
            elif name == "q":
                assert same(o2, slice(tok + 1, 340)) and not torch.isfinite(o2[tok, 0]).any() and torch.equal(s2, s)
            elif name == "k":
                assert not torch.isfinite(s2[0, 0, 7]).any() and torch.equal(s2[0, 0, :7], s[0, 0, :7])
            else:
                assert torch.isnan(s2[0, 0]).all() and torch.isnan(o2[tok + 1:300, 0]).all()


# tokens before, the sequences' lengths, tokens after; the small ones go token by token
OUTSIDE = [(5, [35, 0, 30], 30), (0, [64], 1), (300, [270], 0), (130, [0], 70), (1, [0, 1, 0], 1), (2, [3], 3), (4, [0], 4)]
LAYOUTS = [(2, 2, 32, 40, "float32"), (1, 3, 128, 64, "bfloat16"), (2, 4, 17, 33, "float16")]


def _outside(before, lens, after, hk, hv, dk, dv, dtype):
    torch = _torch()
    x = _inputs([before + sum(lens) + after], hk, hv, dk, dv, dtype, seed=before + after)
    x["s0"] = torch.randn(len(lens), hv, dk, dv, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    x["offsets"] = torch.tensor([before + sum(lens[:i]) for i in range(len(lens) + 1)], device="cuda")
    inner = dict(x, offsets=x["offsets"] - before)
    for n in "qkvg":  # what lies outside is not read
        inner[n] = x[n][before:before + sum(lens)].clone()
        x[n][:before] = x[n][before + sum(lens):] = float("nan")
    return x, inner


@gpu
@pytest.mark.parametrize("before,lens,after", OUTSIDE)
@pytest.mark.parametrize("hk,hv,dk,dv,dtype", LAYOUTS)
@pytest.mark.parametrize("form", ["decay", "step"])
def test_tokens_of_no_sequence(seq, before, lens, after, hk, hv, dk, dv, dtype, form):
    """Offsets that leave tokens to no sequence: the sequences' results are those of the tokens alone, the others' are zero."""
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    x, inner = _outside(before, lens, after, hk, hv, dk, dv, dtype)
    call = zs.zsolve_decay_step if form == "step" else zs.zsolve_decay
    o, s = torch.full_like(x["v"], 7.0), torch.full_like(x["s0"], 7.0)
    call(seq.seq, *(x[n] for n in "qkvg"), o, s, x["s0"], x["offsets"], 0.7)
    at = slice(before, before + sum(lens))
    _verify(inner, 0.7, o[at], s, dtype)
    assert not o[:before].any() and not o[at.stop:].any()
    if form == "step" or (sum(lens) <= 8) == (before + sum(lens) + after <= 8):  # zsolve_decay takes up to 8 tokens one by one
        oi, si = torch.full_like(inner["v"], 7.0), torch.full_like(x["s0"], 7.0)
        call(seq.seq, *(inner[n] for n in "qkvg"), oi, si, x["s0"], inner["offsets"], 0.7)
        assert torch.equal(o[at], oi) and torch.equal(s, si)


@gpu
def test_offsets_out_of_range_are_kept_within_the_tensors(seq):
    """Offsets that do not ascend or leave 0 .. tokens: what is written stays inside the outputs."""
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    x = _inputs([300], 1, 1, 32, 32, "float32", seed=14)
    buf = torch.full((340, 1, 32), 9.0, device="cuda")
    s = torch.zeros(4, 1, 32, 32, device="cuda")
    off = torch.tensor([-5, 40, 20, 1 << 40, 70], device="cuda")
    for call in (zs.zsolve_decay, zs.zsolve_decay_step):
        call(seq.seq, x["q"], x["k"], x["v"], x["g"], buf[20:320], s, None, off)
        torch.cuda.synchronize()
        assert bool((buf[:20] == 9.0).all()) and bool((buf[320:] == 9.0).all()) and bool(torch.isfinite(s).all())


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_same_result_twice_and_on_another_stream(seq, dtype):
    torch = _torch()
    x = _inputs([700, 20], 2, 4, 128, 64, dtype, seed=15)
    args = (x["q"], x["k"], x["v"], x["g"], x["s0"], x["offsets"])
    o, s = seq.decay(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, s2 = seq.decay(*args)
    o3, s3 = seq.decay(*args)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(s, s2) and torch.equal(o, o3) and torch.equal(s, s3)


@gpu
def test_shapes_that_are_refused(seq):
    import mixed_precision_refinement_gb300 as zs
    torch = _torch()
    b, t, hk, hv, dk, dv = 2, 6, 1, 3, 8, 4

    def make(*shape):
        return torch.rand(*shape, device="cuda")

    good = dict(q=make(b, t, hk, dk), k=make(b, t, hk, dk), v=make(b, t, hv, dv), g=-make(b, t, hv), s0=make(b, hv, dk, dv))
    o, _ = seq.decay(**good)
    for same in (dict(g=good["g"].view(b * t, hv)), dict(g=good["g"].flatten()), dict(s0=good["s0"].flatten())):
        assert torch.equal(seq.decay(**{**good, **same})[0], o)
    for bad in (dict(g=make(b, hv, t)), dict(g=make(hv, b * t)), dict(g=make(hv + 1)), dict(g=make(1, hv)), dict(s0=make(b, hv, dv, dk)),
                dict(s0=make(hv, b, dk, dv)), dict(k=make(t, b, hk, dk)), dict(v=make(t, b, hv, dv)), dict(k=make(b, t, hk, dk + 1)),
                dict(q=make(b, t, dk)[:, :, None].transpose(2, 3)), dict(offsets=torch.zeros(0, device="cuda", dtype=torch.int64))):
        with pytest.raises(ValueError):
            seq.decay(**{**good, **bad})
        if "offsets" not in bad:
            with pytest.raises(ValueError):
                seq.decay_bwd(o, **{**good, **bad})
    for bad in (dict(k=good["k"].half()), dict(v=good["v"].double()), dict(g=good["g"].half()), dict(s0=good["s0"].half()),
                dict(offsets=torch.zeros(3, device="cuda", dtype=torch.int32))):
        with pytest.raises(TypeError):
            seq.decay(**{**good, **bad})
    with pytest.raises(zs.ZsolveError) as e:
        seq.decay(make(9, 2, 8), make(9, 2, 8), make(9, 3, 4), -make(9, 3))  # 3 value heads, 2 key heads
    assert e.value.status == zs.ZSOLVE_EINVAL
    with pytest.raises(zs.ZsolveError):
        seq.decay(make(9, 1, 129), make(9, 1, 129), make(9, 1, 4), -make(9, 1))
    with pytest.raises(ValueError):
        seq.decay_step(*(good[n][:, 0].contiguous() for n in "qkv"), make(hv, b), good["s0"])


def _calls(lib, handle):
    from mixed_precision_refinement_gb300 import seq as binding
    p = 64  # never read: every call below is refused before the device is touched
    good = dict(type=1, hk=2, hv=4, dk=16, dv=8, nseq=1, tokens=20, offsets=p, q=p, k=p, v=p, ldq=32, ldk=32, ldv=32, g=p, ldg=4, s0=None,
                scale=1.0)

    def args(over):
        a = {**good, **over}
        return binding.zsolve_decay_args(*(a[n] for n, _ in binding.zsolve_decay_args._fields_))

    def fwd(call=lib.zsolve_decay, o=p, ldo=32, a=None, **over):
        return call(handle, ctypes.byref(args(over)) if a is None else None, o, ldo, None)

    def step(**over):
        return fwd(call=lib.zsolve_decay_step, **over)

    def bwd(o=p, ldo=32, dq=p, dk_=p, dv_=p, dg=p, a=None, **over):
        return lib.zsolve_decay_bwd(handle, ctypes.byref(args(over)) if a is None else None, o, ldo, None, dq, dk_, dv_, dg, None)

    both = [dict(a=0), dict(type=3), dict(type=-1), dict(hk=0), dict(hk=3), dict(hv=0), dict(hv=65536, hk=1), dict(dk=0), dict(dk=129), dict(dv=0),
            dict(dv=65537), dict(nseq=-1), dict(nseq=0), dict(tokens=-1), dict(tokens=1 << 31), dict(offsets=None, nseq=3), dict(q=None),
            dict(k=None), dict(v=None), dict(g=None), dict(o=None), dict(ldq=31), dict(ldk=31), dict(ldv=31), dict(ldo=31), dict(ldg=3),
            dict(scale=float("nan")), dict(scale=float("inf"))]
    return (fwd, both), (step, both), (bwd, both + [dict(dq=None), dict(dk_=None), dict(dv_=None), dict(dg=None),
                                                    dict(dg=None, tokens=0, ldg=0)])


@gpu
def test_refusals_of_the_library(seq):
    import mixed_precision_refinement_gb300 as zs
    for call, bad in _calls(zs.raw_lib(), seq.seq):
        for args in bad:
            assert call(**args) == zs.ZSOLVE_EINVAL, args


def test_null_handle_is_refused_without_a_device():
    import mixed_precision_refinement_gb300 as zs
    for call, _ in _calls(zs.raw_lib(), None):
        assert call() == zs.ZSOLVE_EINVAL
