"""The plain 64-bit forms used by the attention operators' tests, against independent evaluations (no GPU needed)."""
import math

import pytest
import torch

from tests import _attention as ref

NPOS = 300


@pytest.mark.parametrize("d,rot,il", [(16, 16, False), (64, 32, True), (128, 0, False)])
def test_formula_matches_differences(d, rot, il):
    """The fp64 gradient formula against central differences of the fp64 forward (step 1e-6: truncation about 1e-12
    relative, rounding about 1e-10)."""
    g = torch.Generator().manual_seed(d)
    T, H = 3, 2
    x, dy = torch.randn(T, H, d, generator=g).double(), torch.randn(T, H, d, generator=g).double()
    w = 1 + 0.3 * torch.randn(d, generator=g).double()
    cos, sin = ref.angles(NPOS, rot)
    R = ref.rotations(cos, sin, torch.tensor([1, 17, 200]), d, rot, il)
    dx, dw = ref.norm_rope_grad(dy, x, w, R, 1e-5)
    f = lambda x, w: float((ref.norm_rope(x, w, R, 1e-5) * dy).sum())  # noqa: E731
    h = 1e-6
    for t, hh, c in ((0, 0, 0), (1, 1, d // 2), (2, 0, d - 1), (1, 0, min(d - 1, rot // 2 + 1))):
        e = torch.zeros_like(x)
        e[t, hh, c] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - float(dx[t, hh, c])) <= 1e-7
    for c in (0, d // 2, d - 1):
        e = torch.zeros_like(w)
        e[c] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - float(dw[c])) <= 1e-7


def test_e4m3_grid():
    """The 253 finite e4m3 values are fixed points; midpoints go to the even neighbour."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    finite = codes[codes.isfinite()]
    assert finite.numel() == 254 and torch.equal(ref.e4m3(finite), finite)
    pos = finite[finite >= 0].unique()
    mid = (pos[:-1] + pos[1:]) / 2
    even = torch.where(torch.arange(len(mid)) % 2 == 0, pos[:-1], pos[1:])  # consecutive codes alternate in parity
    assert torch.equal(ref.e4m3(mid), even)
    assert ref.e4m3(torch.tensor([1e9], dtype=torch.float64)).item() == 448


def test_quantised_rows():
    x = torch.tensor([[448.0, 1.0], [449.0, 1.0], [0.0, 0.0], [1e-30, 0.0], [3e38, 1.0], [2.0 ** -70, 0.0]],
                     dtype=torch.float64)
    c, s = ref.quantise(x)
    assert s.tolist() == [1.0, 2.0, 1.0, 2.0 ** -63, 2.0 ** 63, 2.0 ** -63]
    assert torch.all(c.abs() <= 448)


def test_attention_of_equal_scores_is_the_mean():
    g = torch.Generator().manual_seed(1)
    v = torch.randn(6, 2, 4, generator=g).double()
    out, lse, _, _ = ref.attend(torch.zeros(2, 4, 4).double(), torch.randn(6, 2, 4, generator=g).double(), v, 6, 1.0,
                                window=3)
    for w in range(2):
        for h in range(4):
            assert torch.allclose(out[w, h], v[2 + w:5 + w, h // 2].mean(0))
            assert lse[w, h] == pytest.approx(math.log(3))
