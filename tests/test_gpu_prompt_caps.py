"""Capped scores of the prompt attention: what a row does not see leaves its bits alone, and caps of any size."""
import math

import pytest
import torch

from tests import _prompt as P

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FORMS = [(BF, 128, (4, 2)), (BF, 128, (3, 3)), (BF, 64, (4, 1)), (BF, 16, (3, 1)), (F32, 64, (4, 2))]


def results(cuda, tensors, lengths, **kw):
    q, k, v, d_out = tensors
    return P.run(cuda, q, k, v, P.cu(lengths), max(lengths), d_out, out_type=F32, grad_type=F32, **kw)


@pytest.mark.parametrize("dtype,d,heads", FORMS, ids=str)
@pytest.mark.parametrize("softcap,size", [(30.0, 1.0), (30.0, 3.0), (2.0, 1.0)])
@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("other", [9.0, 0.01, math.nan])
def test_later_tokens_leave_a_row_alone(cuda, dtype, d, heads, softcap, size, window, other):
    """Other queries, keys and values from some position on (much larger, much smaller, no numbers at all): rows before it keep every
    bit of out and lse, and of dq where the others are numbers."""
    lengths, cut = [700, 41], 600
    tensors = P.inputs(741, *heads, d, dtype, 40, size=size)
    tensors[3][cut:700] = 0  # (a later row's gradient does not come into an earlier one's dq in any case)
    want = results(cuda, tensors, lengths, softcap=softcap, window=window)
    for x in tensors[:3]:
        x[cut:700] *= other
    got = results(cuda, tensors, lengths, softcap=softcap, window=window)
    rows = torch.ones(741, dtype=torch.bool, device="cuda")
    rows[cut:700] = False
    for n in ("out", "lse") + (() if math.isnan(other) else ("dq",)):
        assert torch.equal(got[n][rows], want[n][rows]), n


@pytest.mark.parametrize("dtype,d,heads", FORMS, ids=str)
@pytest.mark.parametrize("softcap", [30.0, 2.0])
@pytest.mark.parametrize("other", [9.0, 0.01, math.nan])
def test_neighbours_in_the_pack_leave_a_sequence_alone(cuda, dtype, d, heads, softcap, other):
    lengths, at = [150, 300, 70], slice(150, 450)
    tensors = P.inputs(520, *heads, d, dtype, 41)
    want = results(cuda, tensors, lengths, softcap=softcap)
    for x in tensors:
        x[:150] *= other
        x[450:] *= other
    got = results(cuda, tensors, lengths, softcap=softcap)
    for n in got:
        assert torch.equal(got[n][at], want[n][at]), n


@pytest.mark.parametrize("d,heads", [f[1:] for f in FORMS if f[0] == BF], ids=str)
@pytest.mark.parametrize("softcap", [30.0, 2.0])
def test_a_sequence_alone_and_in_a_batch(cuda, d, heads, softcap):
    """bf16 inputs: the batch may split sums of dk and dv, and nothing else."""
    lengths, at = [500, 333, 90], slice(500, 833)
    tensors = P.inputs(923, *heads, d, BF, 42)
    for x in tensors[:2]:
        x[:500] *= 5
        x[833:] *= 5
    got = results(cuda, tensors, lengths, softcap=softcap)
    alone = results(cuda, [x[at] for x in tensors], [333], softcap=softcap)
    for n in ("out", "lse", "dq"):
        assert torch.equal(got[n][at], alone[n]), n


@pytest.mark.parametrize("dtype,d,heads", FORMS, ids=str)
@pytest.mark.parametrize("softcap,size", [(30.0, 2.5), (30.0, 4.0), (8.0, 2.0)])
@pytest.mark.parametrize("window", [0, 200])
def test_scores_of_every_part_of_the_cap(cuda, dtype, d, heads, softcap, size, window):
    # products from far below the cap to far above it within a tile
    P.compare(cuda, [600, 131], *heads, d, dtype, seed=43, softcap=softcap, size=size, window=window)
    P.compare(cuda, [300], *heads, d, dtype, seed=44, softcap=softcap, size=size, window=window, scale=-0.3)


@pytest.mark.parametrize("dtype,d,heads", FORMS, ids=str)
@pytest.mark.parametrize("softcap", [1e-30, 1e-20, 1e-12, 1e-8, 1e-4, 1.0])
def test_products_of_zero_are_scores_of_zero(cuda, dtype, d, heads, softcap):
    """Padded queries or keys: every key weighs the same, whatever the cap."""
    q, k, v, d_out = P.inputs(500, *heads, d, dtype, 45)
    q[100:], k[:50] = 0, 0
    got = P.run(cuda, q, k, v, P.cu([500]), 500, d_out, softcap=softcap)
    want = P.attention(q, k, v, d_out, [500], softcap=softcap)
    rows = torch.arange(500, device="cuda") >= 100
    # a product of zero has no error, so neither have these rows' scores: p = 1 / n and lse = log n to what sums, exponentials and logarithms round
    for n in ("out", "lse"):
        value, bound = want[n]
        assert P.worst(got[n], value, bound, rows) <= 1, n
    assert all(torch.isfinite(x).all() for x in got.values())


@pytest.mark.parametrize("dtype,d,heads", FORMS, ids=str)
@pytest.mark.parametrize("softcap", [1.0, 30.0])
def test_products_whose_squares_overflow(cuda, dtype, d, heads, softcap):
    # products of 1e20 and more, scores of 1
    P.compare(cuda, [400], *heads, d, dtype, seed=46, size=1e10, scale=1e-20 * d ** -0.5, softcap=softcap)


@pytest.mark.parametrize("dtype,d,heads", FORMS, ids=str)
@pytest.mark.parametrize("softcap", [0.0, 1e-20, 5.0])
@pytest.mark.parametrize("scale", [3e38, -3e38])
def test_products_of_zero_under_the_largest_scale(cuda, dtype, d, heads, softcap, scale):
    q, k, v, _ = P.inputs(300, *heads, d, dtype, 48)
    q[:] = 0
    got = P.run(cuda, q, k, v, P.cu([300]), 300, softcap=softcap, scale=scale)
    want = P.attention(q, k, v, None, [300])
    for n, (value, bound) in want.items():
        assert P.worst(got[n], value, bound, slice(None)) <= 1, n
