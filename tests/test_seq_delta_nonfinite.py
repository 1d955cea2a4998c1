"""An infinity or NaN in the gradient of a token's output: it is in the gradients of that token and those
before it alone, also within a chunk, as the recurrence has it."""
import pytest

from test_seq_delta_bwd import NAMES, _case, _reference, _tolerances
from test_seq_delta import U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def seq():
    import mixed_precision_refinement_gb300 as zs
    s = zs.Seq()
    yield s
    zs.zsolve_seq_check(s.seq)
    s.close()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("dk,dv", [(64, 48), (128, 33), (24, 64)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nonfinite_gradients_reach_no_later_token(seq, dk, dv, dtype, value):
    import torch
    n, scale, col = 150, 0.6, 7
    x, dout, ds = _case([n], 2, 2, dk, dv, dtype, 18)
    args = [x[i] for i in ("q", "k", "v", "g", "beta", "s0")]
    ref, sizes = _reference(x, dout, ds, scale)
    tol = _tolerances(x, dout, sizes, scale, 3)
    base = seq.delta_bwd(dout, *args, ds, x["offsets"], scale)
    for tok in (0, 5, 63, 64, 68, 80, 101, 146, 149):
        d = dout.clone()
        d[tok, 0, col] = value
        got = seq.delta_bwd(d, *args, ds, x["offsets"], scale)
        for name, a, b in zip(NAMES[:5], got, base):
            # the tokens after it: the same gradients, in another order of summation at most
            u = U[dtype] if name in "qkv" else U["float32"]
            err = (a.double() - ref[name]).abs()[tok + 1:]
            assert bool((err <= u * ref[name].abs()[tok + 1:] + tol[name]).all()), (name, tok)
            assert torch.equal(a[:, 1], b[:, 1]), (name, tok)  # the other head
        dv_ = got[2]
        others = [c for c in range(dv) if c != col]
        assert torch.equal(dv_[:, 0, others], base[2][:, 0, others]), tok
        assert not torch.isfinite(dv_[tok, 0, col]) and not torch.isfinite(got[0][tok, 0]).any()
        assert not torch.isfinite(got[5][0, 0, :, col]).any() and torch.equal(got[5][0, 1], base[5][0, 1])
