"""The 64-bit form that the prompt attention's tests compare with, against autograd and by hand (no GPU needed)."""
import math

import pytest
import torch

from tests import _prompt as P


@pytest.mark.parametrize("softcap,window,scale", [(0.0, 0, None), (3.0, 0, None), (0.0, 4, 0.3), (2.0, 3, -0.5)])
def test_values_and_gradients_match_autograd(softcap, window, scale):
    g = torch.Generator().manual_seed(1)
    lengths, Hq, Hkv, d = [5, 0, 9, 1], 4, 2, 8
    T = sum(lengths)
    q, k, v, do = (torch.randn(T, h, d, generator=g) for h in (Hq, Hkv, Hkv, Hq))
    got = P.attention(q, k, v, do, lengths, softcap=softcap, window=window, scale=scale)
    x = [t.double().requires_grad_() for t in (q, k, v)]
    seq = torch.cat([torch.full((n,), i) for i, n in enumerate(lengths)])
    at = torch.arange(T)
    seen = (seq[:, None] == seq[None]) & (at[None] <= at[:, None])
    if window:
        seen &= at[None] > at[:, None] - window
    s = torch.einsum("ihc,jhc->hij", x[0], x[1].repeat_interleave(Hq // Hkv, 1)) * (d ** -0.5 if scale is None else scale)
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    s = s.masked_fill(~seen, -math.inf)
    out = torch.einsum("hij,jhc->ihc", torch.softmax(s, -1), x[2].repeat_interleave(Hq // Hkv, 1))
    (out * do.double()).sum().backward()
    for name, want in (("out", out), ("lse", torch.logsumexp(s, -1).T), *zip(("dq", "dk", "dv"), (t.grad for t in x))):
        value, bound = got[name]
        assert (value - want).abs().max() <= 1e-12 and (bound > 0).all() and torch.isfinite(bound).all(), name


def test_a_wrong_rounding_would_show():
    """fp32 results rounded to bf16, and a window one key short, lie outside the bounds."""
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(64, 1, 16, generator=g).bfloat16() for _ in range(3))
    rows = torch.ones(64, dtype=torch.bool)
    value, bound = P.attention(q, k, v, None, [64], window=1)["out"]  # each row is its own value: exact
    assert P.worst(value.bfloat16(), value, bound, rows) <= 1
    value, bound = P.attention(q.float(), k.float(), v.float(), None, [64])["out"]
    assert P.worst(value.bfloat16(), value, bound, rows) > 1
    full, bound = P.attention(q, k, v, None, [64], window=3)["out"]
    less = P.attention(q, k, v, None, [64], window=2)["out"][0]
    assert P.worst(less, full, bound, rows) > 1
