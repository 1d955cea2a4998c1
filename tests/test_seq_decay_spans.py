"""Decayed attention in spans of several blocks of 128 tokens whose last block is a part of one (limits: test_seq_decay.py).

Such a block's tokens behind the span are another sequence's.  It is the second, third or fourth of its span, so that its tile takes the
place of one that the products before it need."""
import pytest

from test_seq_decay import _inputs, _verify
from test_seq_decay_bwd import _check as _check_bwd

pytestmark = pytest.mark.gpu
# 512 tokens a span above 65536 rows (tokens x heads), 256 above 16384: parts of a block behind one, two or three whole ones
LENS = [300, 400, 130, 511, 897, 260, 513]
MANY = {256: (4, 16), 512: (8, 32)}
LAYOUTS = [(128, 128), (64, 128), (128, 200), (96, 40)]


@pytest.fixture(scope="module")
def seq():
    import mixed_precision_refinement_gb300 as zs
    s = zs.Seq()
    yield s
    zs.zsolve_seq_check(s.seq)
    s.close()


def _call(seq, x):
    return seq.decay(*(x[n] for n in ("q", "k", "v", "g", "s0", "offsets")), 0.7)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("span", MANY)
@pytest.mark.parametrize("dk,dv", LAYOUTS)
def test_last_blocks_in_part(seq, span, dk, dv, dtype):
    """Against float64, and the same bits from call to call."""
    import torch
    x = _inputs(LENS, *MANY[span], dk, dv, dtype, seed=span + dk)
    o, s = _call(seq, x)
    _verify(x, 0.7, o, s, dtype)
    for _ in range(20):
        o2, s2 = _call(seq, x)
        assert torch.equal(o, o2) and torch.equal(s, s2)


@pytest.mark.parametrize("span", MANY)
@pytest.mark.parametrize("dk,dv", LAYOUTS)
def test_what_lies_behind_a_span_is_not_read(seq, span, dk, dv):
    """Every other sequence is not finite at all: the ones before and after it keep their bits."""
    import torch
    x = _inputs(LENS, *MANY[span], dk, dv, "bfloat16", seed=span + dv)
    o, s = _call(seq, x)
    off = x["offsets"].tolist()
    y = {n: t.clone() for n, t in x.items()}
    for i in range(1, len(LENS), 2):
        for n in "qkvg":
            y[n][off[i]:off[i + 1]] = float("nan")
    for _ in range(5):
        o2, s2 = _call(seq, y)
        for i, (a, b) in enumerate(zip(off, off[1:])):
            if i % 2:
                assert bool(o2[a:b].isnan().all()) and bool(s2[i].isnan().all())
            else:
                assert torch.equal(o2[a:b], o[a:b]) and torch.equal(s2[i], s[i])


@pytest.mark.parametrize("span", MANY)
def test_a_diagonal_block_that_is_not_finite(seq, span):
    """Values of all heads' later tokens in a block: the tokens before them keep their bits, those after them are not finite."""
    import torch
    hk, hv = MANY[span]
    x = _inputs(LENS, hk, hv, 128, 128, "bfloat16", seed=span)
    o, s = _call(seq, x)
    off = x["offsets"].tolist()
    for at in (1, 40, 127, 129, 250):  # tokens from the end of each sequence
        y = dict(x, v=x["v"].clone())
        for b in off[1:]:
            y["v"][b - at, :, 5] = float("inf") if at % 2 else float("nan")
        o2, s2 = _call(seq, y)
        for i, (a, b) in enumerate(zip(off, off[1:])):
            if at > b - a:
                continue
            assert torch.equal(o2[a:b - at], o[a:b - at])
            assert not torch.isfinite(o2[b - at:b, :, 5]).any() and not torch.isfinite(s2[i, :, :, 5]).any()
            others = [c for c in range(128) if c != 5]
            assert torch.equal(o2[b - at:b, :, others], o[b - at:b, :, others]) and torch.equal(s2[i][..., others], s[i][..., others])


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 40)])
def test_gradients_of_last_blocks_in_part(seq, dk, dv, dtype):
    _check_bwd(seq, [300, 400, 130, 511, 260], 8, 16, dk, dv, dtype, seed=dk)
