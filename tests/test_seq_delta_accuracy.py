"""The delta rule's float32 results (states, float32 outputs, gradients) have float32 accuracy, not that of one
tensor-core product in tf32: root-mean-square errors against float64, next to those of the chunked form computed
here in plain float32 and with every product's operands rounded once to tf32.

Limit.  Plain float32 rounds each operand and sum to 2^-24.  A product from split operands keeps 22 bits of each
(2^-22, four times that), and the tensor cores cut their sums, 2^-23 an addition and always towards zero, in chains
of at most eight before a float32 addition (2^-20, sixteen times).  Twice their sum, rounded down to a power of two,
is 32: the kernels are held to 32 times the plain form's error, and at least to 32 times one rounding of the result.
One tf32 rounding is 2^-11, 8192 times a float32 one, and has to exceed the limit.
"""
import pytest

from test_seq_delta import _inputs

pytestmark = pytest.mark.gpu

FACTOR, U32 = 32, 2.0 ** -24
NAMES = ("q", "k", "v", "g", "beta", "s0")


@pytest.fixture(scope="module")
def seq():
    import mixed_precision_refinement_gb300 as zs
    with zs.Seq() as s:
        yield s


def _tf32(x):
    """float64 values rounded to 11 significant bits."""
    import torch
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 2.0 ** 11) / 2.0 ** 11, e)


def _tf32_product():
    import torch

    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a, b):
            ctx.save_for_backward(a, b)
            return _tf32(a) @ _tf32(b)

        @staticmethod
        def backward(ctx, g):
            a, b = ctx.saved_tensors
            return _tf32(g) @ _tf32(b).mT, _tf32(a).mT @ _tf32(g)

    return Product.apply


def _chunked(x, scale, dtype, mm):
    """o and the last state of one sequence in chunks of 64, in `dtype` with products by mm; from x's tensors, which
    may require gradients."""
    import torch
    group = x["v"].shape[1] // x["k"].shape[1]
    q, k = (x[n].to(dtype).repeat_interleave(group, 1).transpose(0, 1) for n in ("q", "k"))
    v, beta = x["v"].to(dtype).transpose(0, 1), x["beta"].to(dtype).T
    g, state, o = x["g"].double().T, x["s0"][0].to(dtype), []
    for at in range(0, q.shape[1], 64):
        Q, K, V, bt = (t[:, at:at + 64] for t in (q, k, v, beta))
        b = g[:, at:at + 64].cumsum(1)
        n = b.shape[1]
        low = torch.ones(n, n, dtype=torch.bool, device=b.device).tril()
        e = torch.exp((b[:, :, None] - b[:, None, :]).masked_fill(~low, -float("inf"))).to(dtype)
        c, end = torch.exp(b).to(dtype)[..., None], torch.exp(b[:, -1:] - b).to(dtype)[..., None]
        a = (bt[..., None] * mm(K, K.mT) * e).tril(-1)
        t = torch.linalg.solve_triangular(a + torch.eye(n, dtype=dtype, device=b.device),
                                          torch.eye(n, dtype=dtype, device=b.device).expand_as(a), upper=False, unitriangular=True)
        u = mm(t, bt[..., None] * (V - c * mm(K, state)))
        o.append(scale * (c * mm(Q, state) + mm(mm(Q, K.mT) * e, u)))
        state = c[:, -1:] * state + mm((end * K).mT, u)
    return torch.cat(o, 1).transpose(0, 1), state[None]


def _recurrence(x, scale):
    import torch
    group = x["v"].shape[1] // x["k"].shape[1]
    q, k = (x[n].double().repeat_interleave(group, 1) for n in ("q", "k"))
    v, a, beta, s, o = x["v"].double(), torch.exp(x["g"].double()), x["beta"].double(), x["s0"][0].double(), []
    for t in range(q.shape[0]):
        s = s * a[t][:, None, None]
        s = s + k[t][..., None] * (beta[t][:, None] * (v[t] - (s * k[t][..., None]).sum(1)))[:, None, :]
        o.append(scale * (s * q[t][..., None]).sum(1))
    return torch.stack(o), s[None]


def _with_gradients(form, x, dout, ds):
    """o, s and the gradients of all inputs, as float64."""
    import torch
    y = {n: t if n == "offsets" else t.double().requires_grad_() for n, t in x.items()}
    o, s = form(y)
    ((o * dout.to(o.dtype)).sum() + (s * ds.to(s.dtype)).sum()).backward()
    return {"o": o.detach().double(), "s": s.detach().double(), **{n: y[n].grad.double() for n in NAMES}}


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("n,hk,hv,dk,dv", [(200, 2, 2, 128, 128), (200, 2, 4, 64, 64), (130, 1, 2, 32, 32), (200, 1, 2, 96, 80),
                                           (64, 1, 1, 17, 33), (700, 1, 1, 128, 64)])
def test_float32_accuracy(seq, n, hk, hv, dk, dv, dtype):
    import torch
    scale = 0.6
    x = _inputs([n], hk, hv, dk, dv, dtype, seed=n + dk)
    x["s0"] *= 0.2
    gen = torch.Generator("cuda").manual_seed(1)
    dout = torch.randn(x["v"].shape, generator=gen, device="cuda").to(x["v"].dtype)
    ds = 0.2 * torch.randn(x["s0"].shape, generator=gen, device="cuda")
    exact = _with_gradients(lambda y: _recurrence(y, scale), x, dout, ds)
    plain = _with_gradients(lambda y: _chunked(y, scale, torch.float32, torch.matmul), x, dout, ds)
    tf32 = _with_gradients(lambda y: _chunked(y, scale, torch.float64, _tf32_product()), x, dout, ds)
    args = [x[i] for i in NAMES]
    o, s = seq.delta(*args, offsets=x["offsets"], scale=scale)
    got = dict(zip(NAMES, seq.delta_bwd(dout, *args, ds, x["offsets"], scale)), o=o, s=s)
    # what has 16 bits is off by its own rounding
    for name in ("s", "g", "beta", "s0") + (("o", "q", "k", "v") if dtype == "float32" else ()):
        limit = FACTOR * max(float((plain[name] - exact[name]).norm()), U32 * float(exact[name].norm()))
        err = float((got[name].double() - exact[name]).norm())
        assert err <= limit, (name, err / float(exact[name].norm()), limit / float(exact[name].norm()))
        assert float((tf32[name] - exact[name]).norm()) > limit, name  # products in tf32 alone would be found out
