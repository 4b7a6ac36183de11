"""The softmax references of the attention over the paged cache, in all its forms: references that move at every chance, rows
without a value, scales at both ends of their range, scores at the ends of fp32.  Bounds as in test_gpu_paged_attention.py.
"""
import pytest
import torch

from tests._attention_rows import put
from tests.test_gpu_paged_attention import BF, E4, Problem

pytestmark = pytest.mark.gpu
kinds = pytest.mark.parametrize("kind", [BF, E4], ids=["bf16", "e4m3"])


def rising_keys(n, Hkv, d, step, by, g):
    """Keys whose first channel rises by `by` every `step` tokens, the others small."""
    k = 0.1 * torch.randn(n, Hkv, d, generator=g).double()
    k[:, :, 0] = (by * (torch.arange(n) // step).double())[:, None]
    return k


@kinds
@pytest.mark.parametrize("step", [32, 64, 128])
def test_many_rows_move_in_every_pass(cuda, kind, step):
    """The many-rows form takes 32 tokens of a tile at a time: scores rise by 8 (bf16) or 23 (e4m3) powers of two
    from one such pass to the next, so the reference moves in both passes of every tile, over the probabilities and
    accumulators that the pass before it stored.
    With a bf16 cache the values fall as the scores rise, so that every token counts for as much as every other."""
    n, W, d = 12 * step, 2, 128
    g = torch.Generator().manual_seed(step)
    p = Problem([n], W, 24, 1, d, 16, kind)
    by = 0.7 if kind == BF else 2.0  # times the query's 8: nats
    put(p, "k", 0, rising_keys(n, 1, d, step, by, g))
    p.q[..., 0] = 8.0
    if kind == BF:
        v = 1 + torch.rand(n, 1, d, generator=g).double()
        put(p, "v", 0, v * torch.exp2(48 - 8.0 * (torch.arange(n) // step).double())[:, None, None])
    first = p.run(cuda, scale=1.0).out.clone()
    p.check(scale=1.0)
    for _ in range(5):
        assert torch.equal(p.run(cuda, scale=1.0).out, first)
