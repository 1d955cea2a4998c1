"""More operators of a sequence layer, as cases that can be timed and compared: linear attention with a decay for each
head (whole sequences, gradients, single tokens), the gated feed-forward projections (forward, backward), and the norms
around a block fused with its gate and residual scale (forward, backward).

`run` computes a case in its plain form (elementary torch operations in float32, rounded once), or,
where `own` is true, through the package's entry points.  `exact` gives the same outputs in float64.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 256  # tokens the plain decayed attention takes together
EPS = 1e-5


def listed():
    return [
        # one decoded token of a batch of 64 sequences: reads and writes every state
        dict(name="decay step", op="decay_step", b=64, hk=16, hv=32, dk=128, dv=128, dt="bf16", per="token"),
        # ragged prompts that continue from states, in float32, odd head sizes, a fixed decay for each head
        dict(name="decay ragged", op="decay", lens="1,700,63,1289,64,0,333,17", hk=4, hv=8, dk=96, dv=80, dt="f32", per="head"),
        # prefill of one long sequence
        dict(name="decay long", op="decay", lens="32768", hk=16, hv=32, dk=128, dv=128, dt="bf16", per="token"),
        # training step: gradients of all inputs and of the first states
        dict(name="decay backward", op="decay_bwd", lens="4096,4096", hk=16, hv=32, dk=128, dv=128, dt="bf16", per="token"),
        # the feed-forward projections of one decoded token: reads both weights once
        dict(name="glu one token", op="glu", m=1, n=4096, k=2048, dt="bf16", act="silu"),
        # ragged number of tokens, odd widths, float16
        dict(name="glu odd", op="glu", m=801, n=1001, k=2157, dt="f16", act="gelu"),
        # a long packed batch
        dict(name="glu forward", op="glu", m=16384, n=8192, k=4096, dt="bf16", act="silu"),
        # gradients in training
        dict(name="glu backward", op="glu_bwd", m=8192, n=4096, k=2048, dt="bf16", act="silu"),
        # one decoding step of a small batch: latency alone
        dict(name="resnorm few rows", op="resnorm", rows=8, d=2048, dt="bf16", kind="layer", after=True, gate="silu", scaled=True),
        # forward over a packed batch of ragged prompts
        dict(name="resnorm forward", op="resnorm", rows=16384, d=4096, dt="bf16", kind="rms", after=True, gate="silu", scaled=True),
        # training step in float32 at an odd width (the sweep's 2157 unknowns as features), no norm of the block's output
        dict(name="resnorm backward odd", op="resnorm_bwd", rows=6614, d=2157, dt="f32", kind="layer", after=False, gate="none", scaled=True),
        # training step of a large batch
        dict(name="resnorm backward", op="resnorm_bwd", rows=32768, d=4096, dt="bf16", kind="layer", after=True, gate="silu", scaled=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decay_step", "decay", "decay_bwd", "glu", "glu_bwd", "resnorm", "resnorm_bwd"])
    if op in ("resnorm", "resnorm_bwd"):
        return dict(op=op, rows=_log(rng, 1, 32768), d=_log(rng, 32, 4096), dt=rng.choice(["f32", "bf16", "f16"]),
                    kind=rng.choice(["layer", "rms"]), after=rng.random() < 0.7, gate=rng.choice(["", "none", "silu", "gelu"]), scaled=rng.random() < 0.7)
    if op in ("glu", "glu_bwd"):
        c = dict(op=op, m=_log(rng, 1, 16384 if op == "glu" else 8192), n=_log(rng, 64, 8192), k=_log(rng, 64, 4096), dt=rng.choice(["bf16", "f16"]),
                 act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]))
        if rng.random() < 0.5:  # half of them at widths that are multiples of 64, as most layers have
            c["n"], c["k"] = -(-c["n"] // 64) * 64, -(-c["k"] // 64) * 64
        return c
    hk = rng.choice([1, 2, 4, 8, 16])
    c = dict(op=op, hk=hk, hv=hk * rng.choice([1, 2]), dk=rng.choice([32, 48, 64, 96, 128]), dv=rng.choice([32, 64, 80, 128]),
             dt=rng.choice(["f32", "bf16", "f16"]), per=rng.choice(["token", "head"]))
    if op == "decay_step":
        return dict(c, b=_log(rng, 1, 128))
    total = _log(rng, 1, 16384 if op == "decay" else 6144)
    seqs = min(total, rng.choice([1, 1, 2, 3, 5]))
    cuts = sorted(rng.randint(0, total) for _ in range(seqs - 1))
    return dict(c, lens=",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total])))


def _lens(case):
    return [1] * case["b"] if case["op"] == "decay_step" else [int(t) for t in case["lens"].split(",")]


def _offsets(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dt = DT[case["dt"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    op = case["op"]
    s = {"case": case}
    if op in ("resnorm", "resnorm_bwd"):
        rows, d = case["rows"], case["d"]
        # a residual stream: an offset a row, some channels larger than the others
        s["x"] = (randn(rows, d) * (0.5 + randn(d).abs()) + 0.3 * randn(rows, 1)).to(dt)
        s["o"] = (randn(rows, d) * (0.2 + randn(rows, 1).abs()) + 0.1 * randn(rows, 1)).to(dt)
        s["z"] = randn(rows, d).to(dt) if case["gate"] else None
        s["c"] = (0.5 + 0.1 * randn(d)).to(dt) if case["scaled"] else None
        bias = case["kind"] == "layer"
        s["w2"], s["b2"] = (1 + 0.2 * randn(d)).to(dt), (0.1 * randn(d)).to(dt) if bias else None
        s["w1"], s["b1"] = (1 + 0.2 * randn(d)).to(dt) if case["after"] else None, (0.1 * randn(d)).to(dt) if case["after"] and bias else None
        if op == "resnorm_bwd":
            # what the forward pass leaves: the sum and both norms' statistics
            y, _, stats = _resnorm(s)
            s["y"], s["stats"] = y, stats
            s["dy"], s["dh"] = randn(rows, d).to(dt), randn(rows, d).to(dt)
    elif op in ("glu", "glu_bwd"):
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = randn(m, k).to(dt)
        s["wg"], s["wu"] = ((randn(n, k) / math.sqrt(k)).to(dt) for _ in range(2))
        s["bg"], s["bu"] = ((0.1 * randn(n)).to(dt) for _ in range(2))
        if op == "glu_bwd":
            s["dy"] = randn(m, n).to(dt)
            s["zg"], s["zu"] = ((s["x"].float() @ s[w].float().T + s[b].float()).to(dt) for w, b in (("wg", "bg"), ("wu", "bu")))
    else:
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        lens = _lens(case)
        t = sum(lens)
        s["q"], s["k"] = (randn(t, h, dk).to(dt) for h in (hk, hk))
        s["v"] = randn(t, hv, dv).to(dt)
        # log decays: a rate a head, between long memory and nearly none
        rate = torch.exp(torch.rand(hv, generator=gen, device="cuda") * 6 - 5.5)
        s["g"] = -rate if case["per"] == "head" else -rate * 2 * torch.rand(t, hv, generator=gen, device="cuda")
        s["s0"] = randn(len(lens), hv, dk, dv)
        s["offsets"] = torch.tensor(_offsets(lens), device="cuda")
        if op == "decay_step":
            s["s"] = s["s0"].clone()
        if op == "decay_bwd":
            s["do"] = randn(t, hv, dv).to(dt)
            s["ds"] = 0.1 * randn(len(lens), hv, dk, dv)
    return s


# ---------------------------------------------------------------- plain forms


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _f(t):
    return None if t is None else t.float()


def _scaled(t, w, b=None):
    t = t if w is None else t * w
    return t if b is None else t + b


def _standard(x, kind):
    """x with the norm's mean and scale taken out, and both."""
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    c = x - mean
    rstd = ((c * c).mean(1, keepdim=True) + EPS).rsqrt()
    return c * rstd, mean, rstd


def _resnorm(s):
    case, dt = s["case"], s["x"].dtype
    t, one = s["o"].float(), torch.ones_like(s["o"][:, :1], dtype=torch.float32)
    mean1, rstd1 = 0 * one, one
    if case["after"]:
        t, mean1, rstd1 = _standard(t, case["kind"])
    t = _scaled(t, _f(s["w1"]), _f(s["b1"]))
    if s["z"] is not None:
        t = t * _act(s["z"].float(), case["gate"])
    y = s["x"].float() + _scaled(t, _f(s["c"]))
    h, mean2, rstd2 = _standard(y, case["kind"])
    return y.to(dt), _scaled(h, _f(s["w2"]), _f(s["b2"])).to(dt), torch.cat([mean1, rstd1, mean2, rstd2], 1)


def _norm_slope(a, h, rstd, kind):
    """The gradient of a norm's input from that of its standardised values h."""
    d = a - h * (a * h).mean(1, keepdim=True)
    return rstd * (d - a.mean(1, keepdim=True) if kind == "layer" else d)


def _resnorm_bwd(s):
    case, dt = s["case"], s["x"].dtype
    mean1, rstd1, mean2, rstd2 = s["stats"].split(1, dim=1)
    dh = s["dh"].float()
    h2 = (s["y"].float() - mean2) * rstd2
    dx = s["dy"].float() + _norm_slope(_scaled(dh, _f(s["w2"])), h2, rstd2, case["kind"])
    h1 = (s["o"].float() - mean1) * rstd1
    t = _scaled(h1, _f(s["w1"]), _f(s["b1"]))
    dt_, dz, gated = _scaled(dx, _f(s["c"])), None, t
    if s["z"] is not None:
        z = s["z"].float()
        a = _act(z, case["gate"])
        dz, gated, dt_ = (dt_ * t * _act_slope(z, case["gate"])).to(dt), t * a, dt_ * a
    dh1 = _scaled(dt_, _f(s["w1"]))
    do = _norm_slope(dh1, h1, rstd1, case["kind"]) if case["after"] else dh1
    sums = {"w1": (dt_ * h1).sum(0), "b1": dt_.sum(0), "c": (dx * gated).sum(0), "w2": (dh * h2).sum(0), "b2": dh.sum(0)}
    return (dx.to(dt), do.to(dt), dz) + tuple(v.to(dt) if s[n] is not None else None for n, v in sums.items())


def _glu(s):
    x = s["x"].float()
    g, u = (x @ s[w].float().T + s[b].float() for w, b in (("wg", "bg"), ("wu", "bu")))
    return (_act(g, s["case"]["act"]) * u).to(s["x"].dtype)


def _glu_bwd(s):
    dt, act, x = s["x"].dtype, s["case"]["act"], s["x"].float()
    dy, zg, zu = s["dy"].float(), s["zg"].float(), s["zu"].float()
    dg, du = dy * zu * _act_slope(zg, act), dy * _act(zg, act)
    return tuple(t.to(dt) for t in (dg @ s["wg"].float() + du @ s["wu"].float(), dg.T @ x, du.T @ x, dg.sum(0), du.sum(0)))


def _places(s, blocks):
    """Where token i of the packed tensors lies among sequences of `blocks` whole blocks."""
    off = s["offsets"]
    lens = off[1:] - off[:-1]
    first = torch.arange(len(lens), device="cuda") * blocks * BLOCK - off[:-1]
    return torch.arange(int(off[-1]), device="cuda") + torch.repeat_interleave(first, lens)


def _padded(x, at, seqs, blocks):
    """Packed tokens (t, h, ...) as (sequence, head, block, token of the block, ...), zeros beyond each sequence's end: a
    token with k = v = 0 and g = 0 leaves the state as it is."""
    out = x.new_zeros((seqs * blocks * BLOCK,) + x.shape[1:], dtype=torch.float64 if x.dtype == torch.float64 else torch.float32)
    out[at] = x.to(out.dtype)
    return out.unflatten(0, (seqs, blocks * BLOCK)).transpose(1, 2).unflatten(2, (blocks, BLOCK))


def _packed(x, at, dtype):
    return x.flatten(2, 3).transpose(1, 2).flatten(0, 1)[at].to(dtype)


def _scale(case):
    return 1 / math.sqrt(case["dk"])


def _decay_terms(s):
    """Padded inputs, decays within and between the blocks, and the states in front of every block and after the last."""
    case, lens = s["case"], _lens(s["case"])
    blocks = max(1, -(-max(lens) // BLOCK))
    at, seqs, group = _places(s, blocks), len(lens), case["hv"] // case["hk"]
    q, k = (_padded(s[n], at, seqs, blocks).repeat_interleave(group, 1) for n in ("q", "k"))
    v, g = _padded(s["v"], at, seqs, blocks), _padded(s["g"].double().expand(len(at), case["hv"]), at, seqs, blocks)
    b = g.cumsum(-1)  # in 64 bits: differences of long sums
    low = torch.ones(BLOCK, BLOCK, device="cuda", dtype=torch.bool).tril()
    e = torch.exp((b[..., :, None] - b[..., None, :]).float().masked_fill(~low, -math.inf))
    c, end = torch.exp(b).float(), torch.exp((b[..., -1:] - b).float())
    u = (k * end[..., None]).mT @ v
    total = torch.nn.functional.pad(b[..., -1].cumsum(-1), (1, 0))  # log decay up to each block
    early = torch.ones(blocks + 1, blocks, device="cuda", dtype=torch.bool).tril(-1)
    between = torch.exp((total[..., :, None] - total[..., None, 1:]).masked_fill(~early, -math.inf)).float()
    states = (between @ u.flatten(3)).unflatten(3, u.shape[3:]) + torch.exp(total).float()[..., None, None] * s["s0"][:, :, None]
    return at, q, k, v, b, e, c, end, total, states


def _decay(s):
    at, q, k, v, b, e, c, end, total, states = _decay_terms(s)
    o = _scale(s["case"]) * (c[..., None] * (q @ states[:, :, :-1]) + ((q @ k.mT) * e) @ v)
    return _packed(o, at, s["v"].dtype), states[:, :, -1]


def _decay_bwd(s):
    at, q, k, v, b, e, c, end, total, states = _decay_terms(s)
    case, dt = s["case"], s["v"].dtype
    group, blocks = case["hv"] // case["hk"], q.shape[2]
    do = _scale(case) * _padded(s["do"], at, len(s["offsets"]) - 1, blocks)
    w = (q * c[..., None]).mT @ do
    # the gradients of the states in front of every block and after the last
    late = torch.ones(blocks + 1, blocks, device="cuda", dtype=torch.bool).triu()
    between = torch.exp((total[..., None, :-1] - total[..., :, None]).masked_fill(~late, -math.inf)).float()
    d = (between @ w.flatten(3)).unflatten(3, w.shape[3:]) + torch.exp(total[..., -1:] - total).float()[..., None, None] * s["ds"][:, :, None]
    before, after = states[:, :, :-1], d[:, :, 1:]
    p, dp = (q @ k.mT) * e, (do @ v.mT) * e
    q_state, k_state = c[..., None] * (do @ before.mT), end[..., None] * (v @ after.mT)
    dq, dk = q_state + dp @ k, k_state + dp.mT @ q
    dv = p.mT @ do + end[..., None] * (k @ after)
    # d b of each token as a query and as a key, without the pairs of a token with itself
    pair = ((do @ v.mT) * p).tril(-1)
    from_q, from_k = (q * q_state).sum(-1), (k * k_state).sum(-1)
    within = from_q + pair.sum(-1) - pair.sum(-2)
    dg = within.flip(-1).cumsum(-1).flip(-1) + from_k.cumsum(-1) - from_k + torch.exp(b[..., -1:]).float() * (before * after).sum((-1, -2))[..., None]
    dq, dk = (_packed(x.unflatten(1, (-1, group)).sum(2), at, dt) for x in (dq, dk))
    dg = _packed(dg, at, torch.float32)
    return dq, dk, _packed(dv, at, dt), dg.sum(0) if case["per"] == "head" else dg, d[:, :, 0]


def _decay_step(s):
    group = s["v"].shape[1] // s["k"].shape[1]
    q, k = (s[n].float().repeat_interleave(group, 1) for n in ("q", "k"))
    state = s["s0"] * torch.exp(s["g"])[..., None, None] + k[..., None] * s["v"].float()[..., None, :]
    o = _scale(s["case"]) * (state * q[..., None]).sum(2)
    return o.to(s["v"].dtype), state


# ---------------------------------------------------------------- the package's operators

_handle = None


def _seq():
    """The handle a program keeps for as long as it runs."""
    global _handle
    if _handle is None:
        import mixed_precision_refinement_gb300 as zs

        _handle = zs.Seq()
    return _handle


def _own(s):
    h, case = _seq(), s["case"]
    op = case["op"]
    if op == "resnorm":
        return h.resnorm(s["x"], s["o"], s["w1"], s["b1"], z=s["z"], act=case["gate"] or "none", c=s["c"], w2=s["w2"], b2=s["b2"], kind=case["kind"],
                         after=case["after"], eps=EPS)
    if op == "resnorm_bwd":
        return h.resnorm_bwd(s["dh"], s["y"], s["o"], s["stats"], s["w1"], s["b1"], z=s["z"], act=case["gate"] or "none", c=s["c"], w2=s["w2"], b2=s["b2"],
                             dy=s["dy"], kind=case["kind"], after=case["after"])
    if op == "glu":
        return h.glu(s["x"], s["wg"], s["wu"], s["bg"], s["bu"], act=case["act"])
    if op == "glu_bwd":
        return h.glu_bwd(s["dy"], s["x"], s["wg"], s["wu"], s["zg"], s["zu"], act=case["act"])
    if op == "decay_step":
        # the new states go beside the old ones, so that a pass can be repeated
        return h.decay_step(s["q"], s["k"], s["v"], s["g"], s["s0"], s_out=s["s"])
    if op == "decay":
        return h.decay(s["q"], s["k"], s["v"], s["g"], s0=s["s0"], offsets=s["offsets"])
    return h.decay_bwd(s["do"], s["q"], s["k"], s["v"], s["g"], s0=s["s0"], ds=s["ds"], offsets=s["offsets"])


def run(state):
    if own:
        return _own(state)
    return {"decay": _decay, "decay_bwd": _decay_bwd, "decay_step": _decay_step, "glu": _glu, "glu_bwd": _glu_bwd, "resnorm": _resnorm,
            "resnorm_bwd": _resnorm_bwd}[state["case"]["op"]](state)


# ---------------------------------------------------------------- work


def work(case):
    op, e = case["op"], BYTES[case["dt"]]
    if op in ("resnorm", "resnorm_bwd"):
        rows, d = case["rows"], case["d"]
        gate = bool(case["gate"])
        bias = case["kind"] == "layer"
        weights = 1 + bias + (1 + bias) * case["after"] + case["scaled"]
        if op == "resnorm":  # x, o and the gate; the sum and its norm
            return {"bytes": rows * d * (4 + gate) * e + weights * d * e + 16 * rows, "flops": rows * d * 20}
        # dy, dh, y, o and the gate; dx, do and the gate's gradient
        return {"bytes": rows * d * (6 + 2 * gate) * e + 2 * weights * d * e + 16 * rows, "flops": rows * d * 40}
    if op in ("glu", "glu_bwd"):
        m, n, k = case["m"], case["n"], case["k"]
        if op == "glu":
            return {"bytes": (m * k + 2 * n * k + m * n + 2 * n) * e, "flops": 4 * m * n * k}
        return {"bytes": (2 * m * k + 4 * n * k + 3 * m * n + 2 * n) * e, "flops": 8 * m * n * k}
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    lens = _lens(case)
    t, states = sum(lens), 4 * len(lens) * hv * dk * dv
    inputs = t * (2 * hk * dk + hv * dv) * e + 4 * hv * (t if case["per"] == "token" else 1)
    # a token's product with and update of the state, in the recurrence: k v^T, S^T q
    flops = 4 * t * hv * dk * dv
    if op == "decay_bwd":
        # the states again, and for each of the two products two more
        return {"bytes": 2 * inputs + t * hv * dv * e + 3 * states, "flops": 3 * flops}
    return {"bytes": inputs + t * hv * dv * e + 2 * states, "flops": flops}


# ---------------------------------------------------------------- the same in float64


def _exact_norm(x, kind, w, b):
    if kind == "layer":
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    else:
        var, mean = torch.square(x).mean(1, keepdim=True), x.new_zeros(x.shape[0], 1)
    rstd = 1 / torch.sqrt(var + EPS)
    h = (x - mean) / torch.sqrt(var + EPS)
    h = h if w is None else torch.einsum("ij,j->ij", h, w)
    return h if b is None else h + b, mean, rstd


def _exact_act(z, act):
    return {"none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
            "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[act](z)


def _exact_resnorm(s):
    case = s["case"]
    s = {n: t.double() if isinstance(t, torch.Tensor) else t for n, t in s.items()}
    if case["after"]:
        t, mean1, rstd1 = _exact_norm(s["o"], case["kind"], s["w1"], s["b1"])
    else:
        t, mean1, rstd1 = s["o"], s["o"].new_zeros(case["rows"], 1), s["o"].new_ones(case["rows"], 1)
    if case["gate"]:
        t = t * _exact_act(s["z"], case["gate"])
    y = s["x"] + (t * s["c"] if case["scaled"] else t)
    h, mean2, rstd2 = _exact_norm(y, case["kind"], s["w2"], s["b2"])
    return y, h, torch.cat([mean1, rstd1, mean2, rstd2], 1)


def _exact_norm_bwd(dh, x, mean, rstd, w, kind):
    """(gradient of x, of w) of a norm whose statistics are given."""
    d = x.shape[1]
    h = (x - mean) * rstd
    a = dh if w is None else dh * w
    inner = torch.einsum("ij,ij->i", a, h)[:, None]
    dx = rstd / d * (d * a - h * inner - (a.sum(1, keepdim=True) if kind == "layer" else 0))
    return dx, torch.einsum("ij,ij->j", dh, h)


def _exact_resnorm_bwd(s):
    case = s["case"]
    none = {n: s[n] is None for n in ("w1", "b1", "c", "w2", "b2")}
    s = {n: t.double() if isinstance(t, torch.Tensor) else t for n, t in s.items()}
    m1, r1, m2, r2 = s["stats"].split(1, dim=1)
    dx, dw2 = _exact_norm_bwd(s["dh"], s["y"], m2, r2, s["w2"], case["kind"])
    dx = dx + s["dy"]
    h = (s["o"] - m1) * r1
    t = h * s["w1"] if s["w1"] is not None else h
    t = t + s["b1"] if s["b1"] is not None else t
    z = s["z"].requires_grad_() if case["gate"] else None
    branch = dx * s["c"] if case["scaled"] else dx
    a = _exact_act(z, case["gate"]) if case["gate"] else torch.ones_like(t)
    dz = torch.autograd.grad(a, z, branch * t)[0] if case["gate"] else None
    a = a.detach()
    dt = branch * a
    if case["after"]:
        do, dw1 = _exact_norm_bwd(dt, s["o"], m1, r1, s["w1"], case["kind"])
    else:
        do, dw1 = dt, None
    grads = (dw1, torch.einsum("ij->j", dt), torch.einsum("ij,ij->j", dx, t * a), dw2, torch.einsum("ij->j", s["dh"]))
    return (dx, do, dz) + tuple(None if none[n] else g for n, g in zip(("w1", "b1", "c", "w2", "b2"), grads))


def _exact_decay(s, lens, scale):
    """The recurrence, token by token."""
    group = s["v"].shape[1] // s["k"].shape[1]
    q, k = (s[n].double().repeat_interleave(group, 1) for n in ("q", "k"))
    v, state = s["v"].double(), s["s0"].double().clone()
    a = torch.exp(s["g"].double()).expand(v.shape[:2])
    o, starts = torch.zeros_like(v), _offsets(lens)
    for i in range(max(lens)):
        live = [j for j, n in enumerate(lens) if n > i]
        seqs, at = torch.tensor(live, device="cuda"), torch.tensor([starts[j] + i for j in live], device="cuda")
        new = state[seqs] * a[at][..., None, None] + k[at][..., None] * v[at][..., None, :]
        o[at] = scale * torch.einsum("bhkv,bhk->bhv", new, q[at])
        state[seqs] = new
    return o, state


def _exact_decay_bwd(s, lens, scale):
    """Derivatives of all pairs of a sequence's tokens, head by head."""
    leaves = {n: s[n].double().requires_grad_() for n in ("q", "k", "v", "g", "s0")}
    group, starts, hv = s["v"].shape[1] // s["k"].shape[1], _offsets(lens), s["v"].shape[1]
    g = leaves["g"].expand(s["v"].shape[:2])
    for i, n in enumerate(lens):
        rows = slice(starts[i], starts[i] + n)
        later = torch.ones(n, n, device="cuda", dtype=torch.bool).triu(1)
        for h in range(hv):
            q, k, v = leaves["q"][rows, h // group], leaves["k"][rows, h // group], leaves["v"][rows, h]
            b, s0 = torch.cumsum(g[rows, h], 0), leaves["s0"][i, h]
            pairs = torch.exp((b[:, None] - b[None, :]).masked_fill(later, -math.inf))
            o = scale * (torch.exp(b)[:, None] * (q @ s0) + (pairs * (q @ k.T)) @ v)
            last = b[-1] if n else b.sum()
            state = torch.exp(last) * s0 + (torch.exp(last - b)[:, None] * k).T @ v
            ((o * s["do"][rows, h].double()).sum() + (state * s["ds"][i, h].double()).sum()).backward()
    return tuple(leaves[n].grad for n in ("q", "k", "v", "g", "s0"))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "resnorm":
        return _exact_resnorm(s)
    if op == "resnorm_bwd":
        return _exact_resnorm_bwd(s)
    if op == "glu":
        x = s["x"].double()
        g, u = (torch.addmm(s[b].double(), x, s[w].double().T) for w, b in (("wg", "bg"), ("wu", "bu")))
        return _exact_act(g, case["act"]) * u
    if op == "glu_bwd":
        x, wg, wu = (s[n].double() for n in ("x", "wg", "wu"))
        zg, zu = (s[n].double().requires_grad_() for n in ("zg", "zu"))
        dg, du = torch.autograd.grad(_exact_act(zg, case["act"]) * zu, (zg, zu), s["dy"].double())
        return torch.addmm(dg @ wg, du, wu), torch.mm(dg.T, x), torch.mm(du.T, x), torch.einsum("ij->j", dg), torch.einsum("ij->j", du)
    lens = _lens(case)
    return _exact_decay_bwd(s, lens, _scale(case)) if op == "decay_bwd" else _exact_decay(s, lens, _scale(case))
