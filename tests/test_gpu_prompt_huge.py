"""Scores up to 2^28, where fp32's last place is 16: the largest takes all."""
import math

import pytest
import torch

from tests import _prompt as P

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FORMS = [(BF, 128, (4, 2)), (BF, 128, (3, 3)), (BF, 64, (4, 1)), (BF, 16, (3, 1)), (F32, 64, (4, 2))]


@pytest.mark.parametrize("dtype,d,heads", FORMS, ids=str)
@pytest.mark.parametrize("size", [30.0, 300.0, 1000.0])
@pytest.mark.parametrize("softcap,scale", [(0.0, 1.0), (0.0, -0.3), (1e30, 1.0), (1e30, -1.0), (1e10, 1.0)])
@pytest.mark.parametrize("window", [0, 150])
def test_the_largest_of_huge_scores_takes_all(cuda, dtype, d, heads, size, softcap, scale, window):
    """Wherever a row's largest score leads by more than the products', the scale's and the cap's rounding (2^-12 of a product's terms,
    and 30: an exponential of 1e-13), its value is the row's result, to the roundings of its probability (bf16 inputs: to 2^-8, and
    the sum is taken before) and of the result."""
    q, k, v, _ = P.inputs(400, *heads, d, dtype, 46, size=size)
    v = P.inputs(400, *heads, d, dtype, 47)[2]
    got = P.run(cuda, q, k, v, P.cu([400]), 400, softcap=softcap, scale=scale, window=window)
    keys, values = k.double().repeat_interleave(heads[0] // heads[1], 1), v.repeat_interleave(heads[0] // heads[1], 1)
    x = torch.einsum("ihc,jhc->hij", q.double(), keys) * scale
    terms = torch.einsum("ihc,jhc->hij", q.double().abs(), keys.abs()) * abs(scale)
    i = torch.arange(400, device="cuda")
    unseen = i[None] > i[:, None]
    if window:
        unseen |= i[None] <= i[:, None] - window
    x = x.masked_fill(unseen, -math.inf)
    top = x.topk(2).values
    clear = (top[..., 0] - top[..., 1]) > 2.0 ** -12 * terms.amax(2) + 30
    best = torch.stack([values[x[h].argmax(1), h] for h in range(heads[0])], 1)
    assert clear.float().mean() > 0.5 and x.masked_fill(unseen, 0).abs().max() < 2 ** 28
    u = 2 * P.U[dtype] + (2.0 ** -16 if dtype == BF else 2.0 ** -21)  # fp32: sums and quotient
    assert ((got["out"].double() - best.double()).abs() <= u * best.double().abs())[clear.T].all()
    lse = top[..., 0].T[clear.T]
    assert ((got["lse"][clear.T].double() - lse).abs() <= 2.0 ** -12 * terms.amax(2).T[clear.T] + 1e-4).all()
