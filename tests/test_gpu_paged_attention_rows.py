"""The many-rows form of the attention (d = 128, bf16 queries and outputs, more than 16 query rows per cached row; both
caches), against the fp64 softmax: blocks of 128 rows that are full, partly full and several, rings that wrap, scores near
the cap, references that move in the second half of a tile's 64 tokens, pages smaller and larger than its tiles,
and everything that must not reach a query's result.  Bounds as in test_gpu_paged_attention.py.
"""
import math

import pytest
import torch

from tests import _attention as ref
from tests._gpu import status
from tests.test_gpu_paged_attention import BF, E4, Problem

pytestmark = pytest.mark.gpu
NAN = float("nan")
# (Hq, Hkv, W): 17, 24, 32, 33, 96, 128, 130 and 260 query rows per key/value head
ROWS = [(17, 1, 1), (24, 2, 2), (8, 1, 4), (11, 1, 3), (12, 1, 8), (16, 1, 8), (26, 2, 10), (26, 1, 10)]
kinds = pytest.mark.parametrize("kind", [BF, E4], ids=["bf16", "e4m3"])


@kinds
@pytest.mark.parametrize("Hq,Hkv,W", ROWS)
@pytest.mark.parametrize("page", [16, 48, 128])
def test_ragged_lengths(cuda, Hq, Hkv, W, page, kind):
    lens = [0, 1, 5, 127, 128, 129, 300, 513]
    p = Problem(lens, W, Hq, Hkv, 128, page, kind).run(cuda)
    assert status(p.st) == (0, len(lens) * W * Hq)
    p.check()


@kinds
@pytest.mark.parametrize("Hq,Hkv,W", [(12, 1, 2), (26, 1, 10)])
@pytest.mark.parametrize("n", [4097, 20011])
def test_long_requests_wrap_the_rings(cuda, Hq, Hkv, W, n, kind):
    """Over a hundred tiles: every slot and buffer is used many times, and the request is split over the CTAs."""
    p = Problem([n], W, Hq, Hkv, 128, 256, kind).run(cuda)
    p.check()
    first = p.out.clone()
    for _ in range(3):
        assert torch.equal(p.run(cuda).out, first)


@kinds
def test_a_share_of_many_units(cuda, kind):
    """More units than CTAs, each of one to three tiles."""
    lens = [40 + (i * 37) % 300 for i in range(300)]
    p = Problem(lens, 8, 12, 1, 128, 32, kind).run(cuda)
    assert status(p.st) == (0, 300 * 8 * 12)
    p.check(only=range(0, 300, 17))


@kinds
@pytest.mark.parametrize("softcap,window,scale", [(20.0, 0, None), (1.0, 0, None), (3.0, 70, 0.2), (500.0, 0, None),
                                                  (0.0, 100, None), (8.0, 300, 0.2), (0.0, 1, None), (0.0, 0, -0.1),
                                                  (0.0, 0, 0.0)])
def test_caps_windows_and_scales(cuda, softcap, window, scale, kind):
    p = Problem([9, 400, 777], 8, 12, 1, 128, 64, kind).run(cuda, softcap=softcap, window=window, scale=scale)
    p.check(softcap=softcap, window=window, scale=scale)


@kinds
@pytest.mark.parametrize("qscale,kscale", [(60.0, 1.0), (1.0, 1e4), (1e-6, 1e6), (1e18, 1e-17)])
def test_large_scores(cuda, qscale, kscale, kind):
    Problem([70, 257], 8, 12, 1, 128, 16, kind, qscale=qscale, kscale=kscale).run(cuda).check()


@pytest.mark.parametrize("step", [16, 32, 48, 100])
def test_rising_scores_move_the_reference(cuda, step):
    """Scores that double every `step` tokens: in the first and second half of a group's 64, and between tiles."""
    n = 12 * step
    p = Problem([n], 2, 24, 1, 128, 16, BF)
    at = torch.arange(n)
    grow = torch.ones(p.pages, 1, p.page, 1, dtype=torch.float64)
    grow[p.table_cpu[0][at // p.page], 0, at % p.page, 0] = torch.exp2((at // step).double())
    p.k *= grow.to(BF).cuda()
    p.kd = p.kd * grow
    p.run(cuda).check()


@pytest.mark.parametrize("down", [0, 1])
def test_scales_at_both_ends_of_their_range(cuda, down):
    """Value scales 2^-63 and 2^63 next to one another: the few rows with the large one are all of the result, whatever
    the score; and keys' scales with queries of the opposite size."""
    p = Problem([200], 2, 12, 1, 128, 16, E4)
    e = torch.full((p.pages, 1, 16), -40, dtype=torch.int32)
    for t in (3, 70, 150):
        e[p.table_cpu[0][t // 16], 0, t % 16] = 40
    if down:
        e -= 23
    s = torch.exp2(e.double())
    p.vd = p.vd / p.vs.cpu().double()[..., None] * s[..., None]
    p.vs.copy_(s.float())
    p.run(cuda).check()


@kinds
def test_nan_in_a_draft_token_reaches_only_the_queries_that_see_it(cuda, kind):
    lens, W = [140, 300, 64], 8
    for which in ("k", "v"):
        p = Problem(lens, W, 24, 2, 128, 16, kind)
        for i, n in enumerate(lens):
            t = n - 3  # window tokens 5, 6, 7 see it
            getattr(p, which).view(torch.uint8)[p.table_cpu[i][t // 16], 1, t % 16] = 0xff
        p.run(cuda)
        assert p.out[:, 5:, 12:].isnan().all() and p.out[:, :5].isfinite().all() and p.out[:, :, :12].isfinite().all()
        p.out, p.lse = p.out[:, :5], p.lse[:, :5]  # the others as without it: the window's first five queries
        for i, n in enumerate(lens):
            want = ref.attend(p.q[i, :5].cpu().double(), p.rows(p.kd, i)[:n - 3], p.rows(p.vd, i)[:n - 3], n - 3,
                              128 ** -0.5)
            tol, tol_l = ref.attend_bound(*want, 128, n, True, 16 if kind == BF else 11)
            assert torch.all((p.out[i].cpu().double() - want[0]).abs() <= tol)
            assert torch.all((p.lse[i].cpu().double() - want[1]).abs() <= tol_l)


@kinds
def test_nan_behind_the_window(cuda, kind):
    p = Problem([330], 3, 12, 1, 128, 16, kind)
    for t in range(330 - 3 - 20 + 1):
        for x in (p.k, p.v):
            x.view(torch.uint8)[p.table_cpu[0][t // 16], :, t % 16] = 0xff
    p.run(cuda, window=20).check(window=20)


def test_infinite_values_and_nan_queries(cuda):
    p = Problem([20, 20], 1, 40, 2, 128, 16, BF)
    p.v[p.table_cpu[0][0], 0, 3, 5] = float("inf")
    p.q[1, 0, 1] = NAN
    p.run(cuda)
    assert p.out[0, 0, :20, 5].isinf().all() and p.out[0, 0, :20, 6].isfinite().all() and p.out[0, 0, 20:].isfinite().all()
    assert p.out[1, 0, 1].isnan().all() and p.lse[1, 0, 1].isnan() and p.out[1, 0, 0].isfinite().all()
    assert p.out[1, 0, 2:].isfinite().all()


@kinds
def test_bad_pages_and_lengths(cuda, kind):
    lens = [290, 290, 290, 33]
    p = Problem(lens, 2, 12, 1, 128, 32, kind)
    p.table[0, 2], p.table[1, 0] = p.pages, -1
    p.lens = [290, 290, p.table.shape[1] * 32 + 1, -4]
    p.run(cuda)
    assert status(p.st)[0] == cuda.KDA_DEV_PAGE_OOB | cuda.KDA_DEV_SEQ_OOB
    assert not p.out[2:].any() and (p.lse[2:] == -math.inf).all()
    p.lens = lens
    p.table_cpu = p.table.cpu().long().clamp(0, p.pages - 1)
    p.check(hidden=set(range(64, 96)), only=[0])
    p.check(hidden=set(range(32)), only=[1])


@kinds
def test_captured_and_on_another_stream(cuda, kind):
    p = Problem([700, 90], 2, 12, 1, 128, 64, kind).run(cuda)
    want = p.out.clone()
    lens = torch.tensor(p.lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(cuda.kda_paged_attention_workspace_size(2, 2, 12, 1, 128), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cuda.kda_paged_attention(p.q, p.k, p.v, p.table, lens, out, ws, k_scales=p.ks, v_scales=p.vs)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda.kda_paged_attention(p.q, p.k, p.v, p.table, lens, out, ws, k_scales=p.ks, v_scales=p.vs)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)


@kinds
@pytest.mark.parametrize("Hq,Hkv,W", [(12, 1, 8), (4, 1, 1), (200, 100, 1)])
def test_caps_at_the_ends_of_fp32(cuda, Hq, Hkv, W, kind):
    """The same in all three forms: a cap that no score feels, and one that leaves nothing of any score."""
    p = Problem([9, 257], W, Hq, Hkv, 128, 16, kind)
    want = p.run(cuda).out.clone()
    for cap in (1e31, 1e37, 3e38):
        assert torch.equal(p.run(cuda, softcap=cap).out, want)
    for cap in (1e-18, 1e-30, 1e-38):
        p.run(cuda, softcap=cap).check(softcap=cap)
