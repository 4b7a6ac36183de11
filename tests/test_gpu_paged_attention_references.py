"""The softmax references of the attention over the paged cache, in all its forms: references that move at every chance, rows
without a value, scales at both ends of their range, scores at the ends of fp32.  Bounds as in test_gpu_paged_attention.py.
"""
import pytest
import torch

from tests import _attention as ref
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


F32 = torch.float32
# Hq, Hkv, W, d, type: the register form with 8 and with 16 or more columns, with fp32, and the many-rows form
E4_FORMS = [(4, 1, 1, 128, BF), (12, 1, 1, 64, BF), (6, 2, 2, 32, F32), (12, 1, 2, 128, BF), (130, 1, 1, 128, BF)]
e4_forms = pytest.mark.parametrize("Hq,Hkv,W,d,dt", E4_FORMS)


def many_times(p, times, g):
    """The problem's one request `times` over, each with queries of its own: enough that a worker's share is whole requests."""
    p.lens, p.table_cpu = p.lens * times, p.table_cpu.expand(times, -1)
    p.table = p.table.expand(times, -1).contiguous()
    p.q = (1.5 * torch.randn(times, *p.q.shape[1:], generator=g)).to(p.q.dtype).cuda()


@e4_forms
@pytest.mark.parametrize("n,times", [(600, 1), (320, 1500), (5000, 1)])
@pytest.mark.parametrize("first,second", [(-63, 63), (63, -63)])
def test_value_scales_of_both_ends_one_after_the_other(cuda, Hq, Hkv, W, d, dt, n, times, first, second):
    """Half of a request's values with scale 2^-63, the other half with 2^63: all count alike in the sum of the softmax.  Within one
    worker's share and across shares, in either order."""
    g = torch.Generator().manual_seed(n)
    p = Problem([n], W, Hq, Hkv, d, 64, E4, dt, dt)
    scale = torch.exp2(torch.where(torch.arange(n) < n // 2, first, second).double())[:, None].expand(n, Hkv)
    put(p, "v", 0, 100 * torch.randn(n, Hkv, d, generator=g).double() * scale[..., None], scale=scale)
    if times > 1:
        many_times(p, times, g)
    p.run(cuda)
    p.check(only=range(0, times, 499))


@e4_forms
def test_value_scales_that_alternate_by_tiles(cuda, Hq, Hkv, W, d, dt):
    """Scales from one end to the other and back, in runs of 16 to 256 tokens."""
    n = 1500
    g = torch.Generator().manual_seed(d)
    for run in (16, 32, 64, 128, 256):
        p = Problem([n], W, Hq, Hkv, d, 16, E4, dt, dt)
        scale = torch.exp2(torch.where((torch.arange(n) // run) % 2 == 0, -63, 63).double())[:, None].expand(n, Hkv)
        put(p, "v", 0, 100 * torch.randn(n, Hkv, d, generator=g).double() * scale[..., None], scale=scale)
        p.run(cuda).check()


@e4_forms
@pytest.mark.parametrize("above", [0.0, 5.0, 8.0, 12.0, 15.0, 40.0])
@pytest.mark.parametrize("where", [[0], [77], [199], list(range(64, 128)), list(range(0, 200, 3))], ids=len)
def test_values_of_zeros_far_above_the_others(cuda, Hq, Hkv, W, d, dt, above, where):
    """A row of zeros has scale 1 in the cache, other rows one after their size: such a token may score `above` nats more than all
    that add something, and leaves the others' 11 (21) bits."""
    n = 200
    g = torch.Generator().manual_seed(len(where))
    p = Problem([n, 300], W, Hq, Hkv, d, 16, E4, dt, dt)
    k, v = 0.3 * torch.randn(2, n, Hkv, d, generator=g).double()
    k[:, :, 0] = 0
    k[where] = 0
    k[where, :, 0] = (above + 3.0) * d ** 0.5 / 4.0
    v[where] = 0
    put(p, "k", 0, k)
    put(p, "v", 0, v)
    p.q[0, ..., 0] = 4.0
    p.run(cuda).check()


@e4_forms
def test_nothing_but_values_of_zeros(cuda, Hq, Hkv, W, d, dt):
    """All of a request's values are zeros, of scale 1 or any other."""
    n = 150
    g = torch.Generator().manual_seed(d)
    for e in (0, -63, 63):
        p = Problem([n], W, Hq, Hkv, d, 16, E4, dt, dt)
        put(p, "v", 0, torch.zeros(n, Hkv, d).double(), scale=torch.full((n, Hkv), 2.0 ** e).double())
        put(p, "k", 0, 30 * torch.randn(n, Hkv, d, generator=g).double())
        p.run(cuda).check()
        assert not p.out.any()


@e4_forms
@pytest.mark.parametrize("above", [6.0, 9.0, 12.0, 14.5])
@pytest.mark.parametrize("at", [0, 199])
def test_channels_of_unlikely_tokens_only(cuda, Hq, Hkv, W, d, dt, above, at):
    """A token that scores `above` nats (up to 21 powers of two) more than all others has a value in channel 0 alone: the other
    channels are sums of small probabilities, which have their 11 (21) bits all the same."""
    n = 200
    g = torch.Generator().manual_seed(at)
    p = Problem([n, 300], W, Hq, Hkv, d, 16, E4, dt, dt)
    k, v = 0.1 * torch.randn(2, n, Hkv, d, generator=g).double()
    v *= 10
    k[:, :, 0] = 0
    k[at] = 0
    k[at, :, 0] = above * d ** 0.5 / 4.0
    v[at] = 0
    v[at, :, 0] = 3.0
    put(p, "k", 0, k)
    put(p, "v", 0, v)
    p.q[0, ..., 0] = 4.0
    p.run(cuda).check()


ALL_FORMS = [(BF, 4, 1, 1, 128, BF), (BF, 16, 1, 1, 128, BF), (BF, 12, 1, 2, 128, BF), (BF, 4, 2, 1, 64, BF),
             (BF, 6, 2, 2, 32, F32)] + [(E4, *f) for f in E4_FORMS]
all_forms = pytest.mark.parametrize("kind,Hq,Hkv,W,d,dt", ALL_FORMS)


@all_forms
@pytest.mark.parametrize("size", [1e16, 1e18])
def test_scores_far_below_zero(cuda, kind, Hq, Hkv, W, d, dt, size):
    """Equal scores of about -1e32 and -1e36: the result is the values' mean (bf16's and fp16's rounding of it at most), and its
    log-sum-exp the score."""
    n = 300
    p = Problem([n, 5], W, Hq, Hkv, d, 16, kind, dt, dt)
    for i, m in enumerate(p.lens):
        k = torch.zeros(m, Hkv, d).double()
        k[:, :, 0] = -size
        put(p, "k", i, k)
    p.q.zero_()
    p.q[..., 0] = size
    p.run(cuda, scale=1.0)
    for i, m in enumerate(p.lens):
        v = p.rows(p.vd, i)
        score = float(p.q[0, 0, 0, 0]) * float(p.rows(p.kd, i)[0, 0, 0])
        for w in range(W):
            want = v[:m - W + 1 + w].mean(0).repeat_interleave(Hq // Hkv, 0)
            got = p.out[i, w].cpu().double()
            assert torch.all((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * v.abs().mean(0).repeat_interleave(Hq // Hkv, 0))
        assert torch.all((p.lse[i].cpu().double() / score - 1).abs() <= 2.0 ** -20)


@all_forms
@pytest.mark.parametrize("qscale,kscale", [(1e36, 1e-18), (4e37, 1e-16), (1e-30, 1e17)])
def test_queries_at_the_ends_of_fp32(cuda, kind, Hq, Hkv, W, d, dt, qscale, kscale):
    """Ordinary scores of very large or very small queries and keys of the opposite size."""
    scale = d ** -0.5 / (qscale * kscale)
    p = Problem([70, 257], W, Hq, Hkv, d, 16, kind, dt, dt, qscale=qscale, kscale=kscale).run(cuda, scale=scale)
    p.check(scale=scale)


# types, and Hq, Hkv, W: fp32 in the register form, then each form with bf16
CAPPED = [(F32, 32, 4, 1), (BF, 32, 4, 1), (BF, 128, 128, 1), (BF, 24, 1, 1), (BF, 12, 1, 2)]


@kinds
@pytest.mark.parametrize("dt,Hq,Hkv,W", CAPPED)
@pytest.mark.parametrize("softcap", [1.0, 10.0, 30.0, 64.0, 65.0, 1000.0])
@pytest.mark.parametrize("size", [0.01, 0.5, 3.0])
def test_small_scores_under_a_cap(cuda, kind, dt, Hq, Hkv, W, softcap, size):
    """Scores well below the cap have fp32's precision: their products have one term each, so the bound (of the log-sum-exp, with
    bf16 types) leaves little to anything else."""
    lens = [1, 2, 3, 40]
    d = 16 if dt == F32 else 128
    g = torch.Generator().manual_seed(int(softcap))
    p = Problem(lens, W, Hq, Hkv, d, 16, kind, dt, dt)
    for i, n in enumerate(lens):
        k = torch.zeros(n, Hkv, d).double()
        k[:, :, 0] = 1 + torch.rand(n, Hkv, generator=g).double()
        put(p, "k", i, k)
    p.q[..., 0] = (size * torch.randn(len(lens), W, Hq, generator=g)).to(dt).cuda()
    p.q[..., 1:] = 0
    p.run(cuda, scale=1.0, softcap=softcap).check(scale=1.0, softcap=softcap)


@e4_forms
def test_log_sum_exp_with_values_of_zeros(cuda, Hq, Hkv, W, d, dt):
    """Values of zeros of scale 1 put the references 62 powers of two below the scores.  Scores of one term each: the bound on the
    log-sum-exp leaves 2^-20 to the exponentials, and here 2^-19 more to the rounding of exponents up to 64."""
    lens = [1, 2, 3, 9]
    g = torch.Generator().manual_seed(d)
    p = Problem(lens, W, Hq, Hkv, d, 16, E4, dt, dt)
    for i, n in enumerate(lens):
        k = torch.zeros(n, Hkv, d).double()
        k[:, :, 0] = 1 + torch.rand(n, Hkv, generator=g).double()
        put(p, "k", i, k)
        put(p, "v", i, torch.zeros(n, Hkv, d).double(), scale=torch.ones(n, Hkv).double())
    p.q[..., 0] = 0.3 * torch.randn(len(lens), W, Hq, generator=g).to(dt).cuda()
    p.q[..., 1:] = 0
    p.run(cuda, scale=1.0)
    lse = p.lse.cpu().double()
    for i, n in enumerate(lens):
        want = ref.attend(p.q[i].cpu().double(), p.rows(p.kd, i), p.rows(p.vd, i), n, 1.0)
        none = want[1] == -float("inf")
        _, tol = ref.attend_bound(*want, d, n, dt == BF, 11)
        assert torch.all((lse[i] - want[1])[~none].abs() <= tol[~none] + 2.0 ** -19)
