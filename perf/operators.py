"""The operators of a token-mixing layer, as cases that can be timed and compared: layer norm, the
matrix product with its epilogue, and the gated delta rule; forward, backward and for few tokens.

`run` computes a case in its plain form (elementary torch operations in float32, rounded once), or,
where `own` is true, through the package's entry points.  `exact` gives the same outputs in float64.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
CHUNK = 64  # tokens the plain delta rule takes together


def listed():
    return [
        # layer norm of the tokens of one decoding step of a small batch: latency alone
        dict(name="norm few rows", op="norm", rows=8, d=2048, dt="bf16"),
        # forward over a packed batch of ragged prompts
        dict(name="norm forward", op="norm", rows=6614, d=4096, dt="bf16"),
        # training step in float32 at an odd width (the sweep's 2157 unknowns as features)
        dict(name="norm backward odd", op="norm_bwd", rows=6614, d=2157, dt="f32"),
        # training step of a large batch: 32768 tokens
        dict(name="norm backward", op="norm_bwd", rows=32768, d=4096, dt="bf16"),
        # the projection of one decoded token: reads the weight once
        dict(name="linear one token", op="linear", m=1, n=4096, k=2048, dt="bf16", act="silu"),
        # ragged number of tokens, odd input width, float16
        dict(name="linear odd", op="linear", m=801, n=1000, k=2157, dt="f16", act="gelu"),
        # the wide projection over a long packed batch
        dict(name="linear forward", op="linear", m=16384, n=8192, k=4096, dt="bf16", act="silu"),
        # gradients of a projection in training
        dict(name="linear backward", op="linear_bwd", m=8192, n=4096, k=2048, dt="bf16", act="silu"),
        # one decoded token of a batch of 64 sequences: reads and writes every state
        dict(name="delta step", op="delta_step", b=64, hk=16, hv=32, dk=128, dv=128, dt="bf16"),
        # prefill of ragged prompts continuing from states, in float32, odd head sizes
        dict(name="delta ragged", op="delta", lens="1,700,63,1289,64,0,333,17", hk=4, hv=8, dk=96, dv=80, dt="f32"),
        # prefill of one long sequence
        dict(name="delta long", op="delta", lens="32768", hk=16, hv=32, dk=128, dv=128, dt="bf16"),
        # training step: gradients of all inputs and of the first state
        dict(name="delta backward", op="delta_bwd", lens="4096,4096", hk=16, hv=32, dk=128, dv=128, dt="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "linear", "linear_bwd", "delta_step", "delta", "delta_bwd"])
    if op in ("norm", "norm_bwd"):
        return dict(op=op, rows=_log(rng, 1, 32768), d=_log(rng, 32, 4096), dt=rng.choice(["f32", "bf16", "f16"]))
    if op in ("linear", "linear_bwd"):
        c = dict(op=op, m=_log(rng, 1, 16384), n=_log(rng, 64, 8192), k=_log(rng, 64, 4096), dt=rng.choice(["bf16", "f16"]),
                 act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]))
        if rng.random() < 0.5:  # half of them at widths that are multiples of 64, as most layers have
            c["n"], c["k"] = -(-c["n"] // 64) * 64, -(-c["k"] // 64) * 64
        return c
    hk = rng.choice([1, 2, 4, 8, 16])
    c = dict(op=op, hk=hk, hv=hk * rng.choice([1, 2]), dk=rng.choice([32, 48, 64, 96, 128]), dv=rng.choice([32, 64, 80, 128]),
             dt=rng.choice(["f32", "bf16", "f16"]))
    if op == "delta_step":
        return dict(c, b=_log(rng, 1, 128))
    total = _log(rng, 1, 16384 if op == "delta" else 6144)
    seqs = min(total, rng.choice([1, 1, 2, 3, 5]))
    cuts = sorted(rng.randint(0, total) for _ in range(seqs - 1))
    return dict(c, lens=",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total])))


def _lens(case):
    return [int(t) for t in case["lens"].split(",")]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dt = DT[case["dt"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    op = case["op"]
    s = {"case": case}
    if op in ("norm", "norm_bwd"):
        rows, d = case["rows"], case["d"]
        # a residual stream: an offset a row, some channels larger than the others
        s["x"] = (randn(rows, d) * (0.5 + randn(d).abs()) + 0.3 * randn(rows, 1)).to(dt)
        s["w"], s["b"] = (1 + 0.2 * randn(d)).to(dt), (0.1 * randn(d)).to(dt)
        if op == "norm_bwd":
            s["dy"] = randn(rows, d).to(dt)
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = (x.var(1, unbiased=False) + 1e-5).rsqrt()
    elif op in ("linear", "linear_bwd"):
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = randn(m, k).to(dt)
        s["w"] = (randn(n, k) / math.sqrt(k)).to(dt)
        s["b"] = (0.1 * randn(n)).to(dt)
        if op == "linear":
            s["r"] = randn(m, n).to(dt)
        else:
            s["dy"] = randn(m, n).to(dt)
            s["z"] = (s["x"].float() @ s["w"].float().T + s["b"].float()).to(dt)
    else:
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        if op == "delta_step":
            lens = [1] * case["b"]
        else:
            lens = _lens(case)
        t = sum(lens)
        silu, unit = torch.nn.functional.silu, torch.nn.functional.normalize
        s["q"], s["k"] = (unit(silu(randn(t, hk, dk)), dim=-1).to(dt) for _ in range(2))
        s["v"] = silu(randn(t, hv, dv)).to(dt)
        s["beta"] = torch.sigmoid(randn(t, hv))
        # log decays: a rate a head, between long memory and nearly none
        rate = torch.exp(torch.rand(hv, generator=gen, device="cuda") * 6 - 4.5)
        s["g"] = -rate * torch.nn.functional.softplus(randn(t, hv) - 1)
        s["s0"] = 0.1 * randn(len(lens), hv, dk, dv)
        s["offsets"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], device="cuda")
        if op == "delta_step":
            s["s"] = s["s0"].clone()
        if op == "delta_bwd":
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


def _norm(s):
    x = s["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = ((c * c).mean(1) + 1e-5).rsqrt()
    y = c * rstd[:, None] * s["w"].float() + s["b"].float()
    return y.to(s["x"].dtype), mean, rstd


def _norm_bwd(s):
    dt = s["x"].dtype
    h = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    a = dy * s["w"].float()
    dx = (a - a.mean(1, keepdim=True) - h * (a * h).mean(1, keepdim=True)) * s["rstd"][:, None]
    return dx.to(dt), (dy * h).sum(0).to(dt), dy.sum(0).to(dt)


def _linear(s):
    z = s["x"].float() @ s["w"].float().T + s["b"].float()
    return (_act(z, s["case"]["act"]) + s["r"].float()).to(s["x"].dtype)


def _linear_bwd(s):
    dt = s["x"].dtype
    dz = s["dy"].float() * _act_slope(s["z"].float(), s["case"]["act"])
    return (dz @ s["w"].float()).to(dt), (dz.T @ s["x"].float()).to(dt), dz.sum(0).to(dt)


def _padded(x, lens, chunks):
    """Packed tokens (t, h, ...) as (sequence, head, chunk, token of the chunk, ...), zeros beyond each
    sequence's end: a token with k = v = 0 and g = beta = 0 leaves the state as it is."""
    out = x.new_zeros((len(lens), chunks * CHUNK) + x.shape[1:], dtype=torch.float32)
    at = 0
    for i, n in enumerate(lens):
        out[i, :n] = x[at:at + n]
        at += n
    return out.transpose(1, 2).unflatten(2, (chunks, CHUNK))


def _packed(x, lens, dtype):
    x = x.flatten(2, 3).transpose(1, 2)
    return torch.cat([x[i, :n] for i, n in enumerate(lens)]).to(dtype)


def _chunk_terms(s, lens):
    """What the chunks need that does not depend on the state, for all of them at once."""
    group = s["v"].shape[1] // s["k"].shape[1]
    chunks = max(1, -(-max(lens) // CHUNK))
    q, k = (_padded(s[n], lens, chunks).repeat_interleave(group, 1) for n in ("q", "k"))
    v, g, beta = (_padded(s[n], lens, chunks) for n in ("v", "g", "beta"))
    b = g.cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, device=b.device, dtype=torch.bool).tril()
    e = torch.exp((b[..., :, None] - b[..., None, :]).masked_fill(~low, -math.inf))
    kk = k @ k.mT
    a = (beta[..., None] * kk * e).tril(-1)
    t = torch.eye(CHUNK, device=b.device).expand_as(a).clone()
    for i in range(1, CHUNK):  # (I + a)^-1, row by row
        t[..., i, :i] = -(a[..., i:i + 1, :i] @ t[..., :i, :i])[..., 0, :]
    p = (q @ k.mT) * e
    return q, k, v, b, beta, e, kk, a, t, p


def _delta_states(s, lens):
    q, k, v, b, beta, e, kk, a, t, p = terms = _chunk_terms(s, lens)
    c = torch.exp(b)
    state, states, us = s["s0"], [], []
    for i in range(k.shape[2]):  # the recurrence over the chunks
        x = beta[:, :, i, :, None] * (v[:, :, i] - c[:, :, i, :, None] * (k[:, :, i] @ state))
        u = t[:, :, i] @ x
        states.append(state)
        us.append(u)
        state = c[:, :, i, -1, None, None] * state + (k[:, :, i] * e[:, :, i, -1, :, None]).mT @ u
    return terms, torch.stack(states, 2), torch.stack(us, 2), state


def _scale(case):
    return 1 / math.sqrt(case["dk"])


def _delta(s, lens):
    (q, k, v, b, beta, e, kk, a, t, p), states, u, last = _delta_states(s, lens)
    o = _scale(s["case"]) * (torch.exp(b)[..., None] * (q @ states) + p @ u)
    return _packed(o, lens, s["v"].dtype), last


def _delta_bwd(s, lens):
    (q, k, v, b, beta, e, kk, a, t, p), states, u, _ = _delta_states(s, lens)
    group, dt = s["v"].shape[1] // s["k"].shape[1], s["v"].dtype
    do = _scale(s["case"]) * _padded(s["do"], lens, k.shape[2])
    c = torch.exp(b)[..., None]
    kend = k * e[..., -1, :, None]
    du0, ds0 = p.mT @ do, (c * q).mT @ do
    d_state, d_states, dxs = s["ds"], [], []
    for i in reversed(range(k.shape[2])):  # the recurrence backwards
        dx = t[:, :, i].mT @ (du0[:, :, i] + kend[:, :, i] @ d_state)
        d_states.append(d_state)
        dxs.append(dx)
        d_state = c[:, :, i, -1, :, None] * d_state + ds0[:, :, i] - (beta[:, :, i, :, None] * c[:, :, i] * k[:, :, i]).mT @ dx
    d_end, dx = torch.stack(d_states[::-1], 2), torch.stack(dxs[::-1], 2)
    low = torch.ones(CHUNK, CHUNK, device=b.device, dtype=torch.bool).tril()
    dp = (do @ u.mT).masked_fill(~low, 0)
    da = -(dx @ u.mT).tril(-1)
    dkend, ex, f = u @ d_end.mT, dx @ states.mT, do @ states.mT
    dpe, dae = dp * e, da * e * beta[..., None]
    dq = c * f + dpe @ k
    kex = (k * ex).sum(-1)
    dk = dpe.mT @ q + e[..., -1, :, None] * dkend - beta[..., None] * c * ex + dae @ k + dae.mT @ k
    dbeta = (dx * v).sum(-1) - c[..., 0] * kex + (da * kk * e).sum(-1)
    through_end = (kend * dkend).sum(-1)
    pair = dp * p + da * a
    db = c[..., 0] * (q * f).sum(-1) + pair.sum(-1) - pair.sum(-2) - through_end - beta * c[..., 0] * kex
    db[..., -1] += through_end.sum(-1) + c[..., -1, 0] * (states * d_end).sum((-1, -2))
    dg = db.flip(-1).cumsum(-1).flip(-1)
    dq, dk = (_packed(x.unflatten(1, (-1, group)).sum(2), lens, dt) for x in (dq, dk))
    dv = _packed(beta[..., None] * dx, lens, dt)
    return dq, dk, dv, _packed(dg, lens, torch.float32), _packed(dbeta, lens, torch.float32), d_state


def _delta_step(s):
    group = s["v"].shape[1] // s["k"].shape[1]
    q, k = (s[n].float().repeat_interleave(group, 1) for n in ("q", "k"))
    state = s["s0"] * torch.exp(s["g"])[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (state * k[..., None]).sum(2))
    state = state + k[..., None] * u[..., None, :]
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
    if op == "norm":
        return h.layernorm(s["x"], s["w"], s["b"], eps=1e-5)
    if op == "norm_bwd":
        return h.layernorm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
    if op == "linear":
        return h.linear(s["x"], s["w"], s["b"], act=case["act"], r=s["r"])
    if op == "linear_bwd":
        return h.linear_bwd(s["dy"], s["x"], s["w"], s["z"], act=case["act"])
    if op == "delta_step":
        # the new states go beside the old ones, so that a pass can be repeated
        return h.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["s0"], s_out=s["s"])
    if op == "delta":
        return h.delta(s["q"], s["k"], s["v"], s["g"], s["beta"], s0=s["s0"], offsets=s["offsets"])
    return h.delta_bwd(s["do"], s["q"], s["k"], s["v"], s["g"], s["beta"], s0=s["s0"], ds=s["ds"], offsets=s["offsets"])


def run(state):
    if own:
        return tuple(_own(state)) if state["case"]["op"] != "linear" else _own(state)
    op = state["case"]["op"]
    if op in ("delta", "delta_bwd"):
        return (_delta if op == "delta" else _delta_bwd)(state, _lens(state["case"]))
    return {"norm": _norm, "norm_bwd": _norm_bwd, "linear": _linear, "linear_bwd": _linear_bwd, "delta_step": _delta_step}[op](state)


# ---------------------------------------------------------------- work


def work(case):
    op, e = case["op"], BYTES[case["dt"]]
    if op == "norm":
        n = case["rows"] * case["d"]
        return {"bytes": 2 * n * e + 2 * case["d"] * e + 8 * case["rows"], "flops": 7 * n}
    if op == "norm_bwd":
        n = case["rows"] * case["d"]
        return {"bytes": 3 * n * e + 3 * case["d"] * e + 8 * case["rows"], "flops": 12 * n}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m * k + n * k + 2 * m * n + n) * e, "flops": 2 * m * n * k}
    if op == "linear_bwd":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (2 * m * k + 2 * n * k + 2 * m * n + n) * e, "flops": 4 * m * n * k}
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    lens = [1] * case["b"] if op == "delta_step" else _lens(case)
    t, states = sum(lens), 4 * len(lens) * hv * dk * dv
    inputs = t * ((2 * hk * dk + hv * dv) * e + 8 * hv)
    # a token's products with and update of the state, in the recurrence: S^T k, k u^T, S^T q
    flops = 6 * t * hv * dk * dv
    if op == "delta_bwd":
        # the states again, and for each of the three products two more
        return {"bytes": 2 * inputs + t * hv * dv * e + 3 * states, "flops": 3 * flops}
    return {"bytes": inputs + t * hv * dv * e + 2 * states, "flops": flops}


# ---------------------------------------------------------------- the same in float64


def _exact_tokens(s, lens):
    """Token i of every sequence that has one: which sequences, and their places in the packed tensors."""
    starts = [sum(lens[:i]) for i in range(len(lens))]
    for i in range(max(lens)):
        live = [j for j, n in enumerate(lens) if n > i]
        yield (slice(None) if len(live) == len(lens) else torch.tensor(live, device="cuda"),
               torch.tensor([starts[j] + i for j in live], device="cuda"))


def _exact_delta(s, lens, scale):
    """The recurrence, token by token."""
    group = s["v"].shape[1] // s["k"].shape[1]
    q, k = (s[n].double().repeat_interleave(group, 1) for n in ("q", "k"))
    v, a, beta = s["v"].double(), torch.exp(s["g"].double()), s["beta"].double()
    state, o = s["s0"].double(), torch.zeros_like(v)
    for seqs, at in _exact_tokens(s, lens):
        decayed = state[seqs] * a[at][..., None, None]
        u = beta[at][..., None] * (v[at] - torch.einsum("bhkv,bhk->bhv", decayed, k[at]))
        new = decayed + k[at][..., None] * u[..., None, :]
        o[at] = scale * torch.einsum("bhkv,bhk->bhv", new, q[at])
        state = state.clone() if not isinstance(seqs, slice) else state
        state[seqs] = new
    return o, state


def _exact_delta_bwd(s, lens, scale):
    """The derivative of the recurrence, token by token, with its states kept every 128 tokens."""
    group = s["v"].shape[1] // s["k"].shape[1]
    q, k = (s[n].double().repeat_interleave(group, 1) for n in ("q", "k"))
    v, a, beta, do = s["v"].double(), torch.exp(s["g"].double()), s["beta"].double(), scale * s["do"].double()
    dq, dk, dv = torch.zeros_like(k), torch.zeros_like(k), torch.zeros_like(v)
    dg, dbeta = torch.zeros_like(beta), torch.zeros_like(beta)
    tokens, every = list(_exact_tokens(s, lens)), 128

    def step(state, seqs, at):
        decayed = state[seqs] * a[at][..., None, None]
        w = v[at] - torch.einsum("bhkv,bhk->bhv", decayed, k[at])
        new = decayed + k[at][..., None] * (beta[at][..., None] * w)[..., None, :]
        return decayed, w, new

    state, kept = s["s0"].double().clone(), []
    for i, (seqs, at) in enumerate(tokens):
        if i % every == 0:
            kept.append(state.clone())
        state[seqs] = step(state, seqs, at)[2]
    d = s["ds"].double().clone()
    for first in reversed(range(0, len(tokens), every)):
        state, saved = kept.pop(), []
        for seqs, at in tokens[first:first + every]:
            saved.append(step(state, seqs, at))
            state[seqs] = saved[-1][2]
        for (seqs, at), (decayed, w, new) in reversed(list(zip(tokens[first:first + every], saved))):
            dn = d[seqs] + q[at][..., None] * do[at][..., None, :]
            dq[at] = torch.einsum("bhkv,bhv->bhk", new, do[at])
            u = beta[at][..., None] * w
            du = torch.einsum("bhkv,bhk->bhv", dn, k[at])
            dbeta[at] = (du * w).sum(-1)
            dw = beta[at][..., None] * du
            dv[at] = dw
            dk[at] = torch.einsum("bhkv,bhv->bhk", dn, u) - torch.einsum("bhkv,bhv->bhk", decayed, dw)
            dd = dn - k[at][..., None] * dw[..., None, :]
            dg[at] = (dd * decayed).sum((-1, -2))
            d[seqs] = dd * a[at][..., None, None]
    dq, dk = (x.unflatten(1, (-1, group)).sum(2) for x in (dq, dk))
    return dq, dk, dv, dg, dbeta, d


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = 1 / torch.sqrt(var + 1e-5)
        return torch.addcmul(s["b"].double(), (x - mean[:, None]) * rstd[:, None], s["w"].double()), mean, rstd
    if op == "norm_bwd":
        x, dy, w = s["x"].double(), s["dy"].double(), s["w"].double()
        d, rstd = case["d"], s["rstd"].double()[:, None]
        h = (x - s["mean"].double()[:, None]) * rstd
        wdy = w * dy
        dx = rstd / d * (d * wdy - wdy.sum(1, keepdim=True) - h * torch.einsum("ij,ij->i", wdy, h)[:, None])
        return dx, torch.einsum("ij,ij->j", dy, h), torch.einsum("ij->j", dy)
    if op in ("linear", "linear_bwd"):
        act = {"none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
               "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[case["act"]]
        x, w = s["x"].double(), s["w"].double()
        if op == "linear":
            return act(torch.addmm(s["b"].double(), x, w.T)) + s["r"].double()
        z = s["z"].double().requires_grad_()
        dz, = torch.autograd.grad(act(z), z, s["dy"].double())
        return dz @ w, torch.mm(dz.T, x), torch.einsum("ij->j", dz)
    scale = _scale(case)
    if op == "delta_step":
        return _exact_delta(s, [1] * case["b"], scale)
    lens = _lens(case)
    return _exact_delta(s, lens, scale) if op == "delta" else _exact_delta_bwd(s, lens, scale)
