"""A sequence layer trained on a frequency sweep, and applied one frequency at a time.

The sweep (zsolve_sweep) gives, for every right-hand side, the solution at each frequency: a sequence
with one token a frequency.  A pre-norm token-mixing layer

    h = norm(x),  a = silu(h Wi^T + bi) = [q | k | v],  q, k normalised per head,
    o = gated delta rule (q, k, v, g(h), beta(h)),  y = o Wo^T + bo + x

learns to give the next frequency's features from those so far.  Norms, projections and the delta rule run on
the sequence-layer operators of the library, the gates' two small projections in float32 in torch; training
takes whole sequences, answering takes one token at a time and keeps only the states.

    python examples/sweep_sequence.py
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import mixed_precision_refinement_gb300 as zs
import workload

HK, HV, DK, DV = 2, 4, 32, 32  # two value heads share a key head
EPS = 1e-6


class Layer:
    """The layer's float32 weights and its passes in bfloat16 on the operators of a `Seq`."""

    def __init__(self, seq, d, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=gen, device="cuda")

        width = 2 * HK * DK + HV * DV
        self.seq, self.d = seq, d
        self.p = dict(norm_w=torch.ones(d, device="cuda"), norm_b=torch.zeros(d, device="cuda"),
                      wi=randn(width, d) / d ** 0.5, bi=torch.zeros(width, device="cuda"),
                      wo=0.2 * randn(d, HV * DV) / (HV * DV) ** 0.5, bo=torch.zeros(d, device="cuda"),
                      # log decay -softplus, step sigmoid; small decays at the start
                      wg=randn(HV, d) / d ** 0.5, bg=torch.full((HV,), -3.0, device="cuda"),
                      wb=randn(HV, d) / d ** 0.5, bb=torch.zeros(HV, device="cuda"))
        # layer norm with this weight gives rows of norm 1
        self.unit = torch.full((DK,), DK ** -0.5, device="cuda", dtype=torch.bfloat16)

    def _before(self, x):
        """Everything in front of the delta rule, for tokens x (tokens, d); what backward needs is kept."""
        s, p, b16 = self.seq, self.p, torch.bfloat16
        h, mean, rstd = s.layernorm(x, p["norm_w"], p["norm_b"], eps=EPS)
        a, z = s.linear(h, p["wi"].to(b16), p["bi"].to(b16), act="silu", keep=True)
        q0, k0, v = a.split([HK * DK, HK * DK, HV * DV], dim=1)
        q0, k0 = (t.unflatten(1, (HK, DK)).contiguous() for t in (q0, k0))
        q, mq, rq = s.layernorm(q0, self.unit, eps=EPS)
        k, mk, rk = s.layernorm(k0, self.unit, eps=EPS)
        hf = h.float()
        zg, zb = torch.addmm(p["bg"], hf, p["wg"].T), torch.addmm(p["bb"], hf, p["wb"].T)
        g, beta = -torch.nn.functional.softplus(zg), torch.sigmoid(zb)
        v = v.unflatten(1, (HV, DV))
        return dict(x=x, h=h, mean=mean, rstd=rstd, z=z, q0=q0, k0=k0, mq=mq, rq=rq, mk=mk, rk=rk, zg=zg, q=q, k=k, v=v, g=g,
                    beta=beta)

    def _after(self, o, x):
        b16 = torch.bfloat16
        return self.seq.linear(o, self.p["wo"].to(b16), self.p["bo"].to(b16), r=x)

    def forward(self, x, offsets, s0=None):
        """y, the states after the sequences, and what backward needs; x: bfloat16 (tokens, d), packed sequences."""
        c = self._before(x)
        o, state = self.seq.delta(c["q"], c["k"], c["v"], c["g"], c["beta"], s0, offsets)
        c["o"], c["offsets"] = o.flatten(1), offsets
        return self._after(c["o"], x), state, c

    def step(self, x, state):
        """y of the next token of every sequence, x: (sequences, d); the states are updated in place."""
        c = self._before(x)
        o, _ = self.seq.delta_step(c["q"], c["k"], c["v"], c["g"], c["beta"], state)
        return self._after(o.flatten(1), x)

    def backward(self, dy, c):
        """The gradients of the weights (float32) and of x."""
        s, p, b16, grad = self.seq, self.p, torch.bfloat16, {}
        do, grad["wo"], grad["bo"] = s.linear_bwd(dy, c["o"], p["wo"].to(b16))
        dq, dk, dv, dg, dbeta, _ = s.delta_bwd(do.unflatten(1, (HV, DV)), c["q"], c["k"], c["v"], c["g"], c["beta"],
                                               offsets=c["offsets"])
        dq0 = s.layernorm_bwd(dq, c["q0"], c["mq"], c["rq"], self.unit)[0]
        dk0 = s.layernorm_bwd(dk, c["k0"], c["mk"], c["rk"], self.unit)[0]
        da = torch.cat([dq0.flatten(1), dk0.flatten(1), dv.flatten(1)], dim=1)
        dh, grad["wi"], grad["bi"] = s.linear_bwd(da, c["h"], p["wi"].to(b16), c["z"], act="silu")
        dzg, dzb = -dg * torch.sigmoid(c["zg"]), dbeta * c["beta"] * (1 - c["beta"])
        hf = c["h"].float()
        grad["wg"], grad["bg"], grad["wb"], grad["bb"] = dzg.T @ hf, dzg.sum(0), dzb.T @ hf, dzb.sum(0)
        dh = dh.float() + dzg @ p["wg"] + dzb @ p["wb"]
        dx, grad["norm_w"], grad["norm_b"] = s.layernorm_bwd(dh.to(b16), c["x"], c["mean"], c["rstd"], p["norm_w"])
        return {n: t.float() for n, t in grad.items()}, dx + dy


def sequences(d, n=96, frequencies=200, nrhs=6, seed=3):
    """Features of a sweep's solutions: bfloat16 (nrhs, frequencies, d), a projection of Re and Im scaled to one."""
    wl = workload.make_resonant_small(n, seed, frequencies, nrhs=nrhs)
    x = torch.empty((frequencies, nrhs, n), dtype=torch.complex128, device="cuda")
    with zs.Solver(n, nrhs, batch=8) as solver:
        zs.zsolve_sweep(solver.ctx, *(torch.from_numpy(m).cuda() for m in (wl.L, wl.Psi, wl.G)), wl.omega, wl.zs,
                        torch.from_numpy(wl.B).cuda(), x)
    parts = torch.view_as_real(x.transpose(0, 1)).flatten(2)
    parts = parts / parts.norm(dim=-1, keepdim=True).mean(dim=1, keepdim=True)
    gen = torch.Generator("cuda").manual_seed(seed)
    return (parts.float() @ torch.randn(2 * n, d, generator=gen, device="cuda")).to(torch.bfloat16)


def main(steps=40, d=128, rate=3e-3):
    """Trains the layer; returns the losses and the largest difference of whole sequences and single tokens."""
    data = sequences(d)
    nseq, t = data.shape[0], data.shape[1] - 1
    x, target = data[:, :-1].reshape(-1, d), data[:, 1:].reshape(-1, d).float()
    offsets = torch.arange(nseq + 1, device="cuda") * t
    with zs.Seq() as seq:
        layer = Layer(seq, d)
        adam = torch.optim.Adam(list(layer.p.values()), lr=rate)
        losses = []
        for _ in range(steps):
            y, _, kept = layer.forward(x, offsets)
            off = y.float() - target
            losses.append(off.square().mean())
            grads, _ = layer.backward((off * (2 / off.numel()) * 1024).to(torch.bfloat16), kept)
            for name, w in layer.p.items():
                w.grad = grads[name] / 1024  # the loss was scaled so that its gradients keep their bits
            adam.step()
        whole, last, _ = layer.forward(x, offsets)
        # the same one frequency at a time, as the sweep goes on
        state = torch.zeros_like(last)
        singles = torch.stack([layer.step(data[:, i].contiguous(), state) for i in range(t)], dim=1)
        zs.zsolve_seq_check(seq.seq)
        apart = float((singles.reshape(-1, d).float() - whole.float()).abs().max() / whole.float().abs().max())
        states_apart = float((state - last).abs().max() / last.abs().max())
    return [float(v) for v in losses], apart, states_apart


if __name__ == "__main__":
    losses, apart, states_apart = main()
    print(f"loss {losses[0]:.2e} -> {losses[-1]:.2e} in {len(losses)} steps; one frequency at a time: outputs within "
          f"{apart:.1e}, states within {states_apart:.1e} of the whole sequences'")
