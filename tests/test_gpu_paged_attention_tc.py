"""The tensor-memory form of the attention (d = 128, bf16 cache, bf16 queries and outputs; many query rows or few units),
against the fp64 softmax: rings that wrap, units that begin and end in every place, pages smaller and larger than its
tiles of 128 tokens, and everything that must not reach a query's result.  Bounds as in test_gpu_paged_attention.py.
"""
import math

import pytest
import torch

from tests import _attention as ref
from tests._gpu import status
from tests.test_gpu_paged_attention import BF, Problem

pytestmark = pytest.mark.gpu
NAN = float("nan")
# (Hq, Hkv, W): 1, 4, 8, 12, 16, 24, 33 and 96 query rows per key/value head
ROWS = [(1, 1, 1), (8, 2, 1), (8, 1, 1), (12, 1, 1), (16, 1, 1), (12, 1, 2), (11, 1, 3), (12, 1, 8)]


@pytest.mark.parametrize("Hq,Hkv,W", ROWS)
@pytest.mark.parametrize("page", [16, 48, 128])
def test_ragged_lengths(cuda, Hq, Hkv, W, page):
    lens = [0, 1, 5, 127, 128, 129, 300, 513]
    p = Problem(lens, W, Hq, Hkv, 128, page, BF).run(cuda)
    assert status(p.st) == (0, len(lens) * W * Hq)
    p.check()


@pytest.mark.parametrize("Hq,Hkv,W", [(4, 1, 1), (12, 1, 2), (12, 1, 8)])
@pytest.mark.parametrize("n", [4097, 20011])
def test_long_requests_wrap_the_rings(cuda, Hq, Hkv, W, n):
    """Over a hundred tiles: every slot and buffer is used many times, and the request is split over the CTAs."""
    p = Problem([n], W, Hq, Hkv, 128, 256, BF).run(cuda)
    p.check()
    first = p.out.clone()
    for _ in range(3):
        assert torch.equal(p.run(cuda).out, first)


def test_a_share_of_many_units(cuda):
    """More units than CTAs, most of a tile or two: 3 row blocks of 300 requests of 40 .. 339 tokens."""
    lens = [40 + (i * 37) % 300 for i in range(300)]
    p = Problem(lens, 8, 12, 1, 128, 32, BF).run(cuda)
    assert status(p.st) == (0, 300 * 8 * 12)
    p.check(only=range(0, 300, 17))


@pytest.mark.parametrize("softcap,window,scale", [(20.0, 0, None), (500.0, 0, None), (0.0, 100, None), (8.0, 300, 0.2),
                                                  (0.0, 1, None), (0.0, 0, -0.1), (0.0, 0, 0.0)])
def test_caps_windows_and_scales(cuda, softcap, window, scale):
    p = Problem([9, 400, 777], 8, 12, 1, 128, 64, BF).run(cuda, softcap=softcap, window=window, scale=scale)
    p.check(softcap=softcap, window=window, scale=scale)


@pytest.mark.parametrize("qscale,kscale", [(60.0, 1.0), (1.0, 1e4), (1e-6, 1e6)])
def test_large_scores(cuda, qscale, kscale):
    Problem([70, 257], 8, 12, 1, 128, 16, BF, qscale=qscale, kscale=kscale).run(cuda).check()


def test_rising_scores_move_the_reference(cuda):
    p = Problem([1200], 2, 24, 1, 128, 16, BF)
    at = torch.arange(1200)
    grow = torch.ones(p.pages, 1, p.page, 1, dtype=torch.float64)
    grow[p.table_cpu[0][at // p.page], 0, at % p.page, 0] = torch.exp2((at // 100).double())
    p.k *= grow.to(BF).cuda()
    p.kd = p.kd * grow
    p.run(cuda).check()


def test_nan_in_a_draft_token_reaches_only_the_queries_that_see_it(cuda):
    lens, W = [140, 300, 64], 8
    for which in ("k", "v"):
        p = Problem(lens, W, 24, 2, 128, 16, BF)
        for i, n in enumerate(lens):
            t = n - 3  # window tokens 5, 6, 7 see it
            getattr(p, which).view(torch.uint8)[p.table_cpu[i][t // 16], 1, t % 16] = 0xff
        p.run(cuda)
        assert p.out[:, 5:, 12:].isnan().all() and p.out[:, :5].isfinite().all() and p.out[:, :, :12].isfinite().all()
        p.out, p.lse = p.out[:, :5], p.lse[:, :5]  # the others as without it: the window's first five queries
        for i, n in enumerate(lens):
            want = ref.attend(p.q[i, :5].cpu().double(), p.rows(p.kd, i)[:n - 3], p.rows(p.vd, i)[:n - 3], n - 3,
                              128 ** -0.5)
            tol, tol_l = ref.attend_bound(*want, 128, n, True, 16)
            assert torch.all((p.out[i].cpu().double() - want[0]).abs() <= tol)
            assert torch.all((p.lse[i].cpu().double() - want[1]).abs() <= tol_l)


def test_nan_behind_the_window_and_infinite_values(cuda):
    p = Problem([330], 3, 12, 1, 128, 16, BF)
    for t in range(330 - 3 - 20 + 1):
        for x in (p.k, p.v):
            x.view(torch.uint8)[p.table_cpu[0][t // 16], :, t % 16] = 0xff
    p.run(cuda, window=20).check(window=20)
    p = Problem([20, 20], 1, 4, 2, 128, 16, BF)
    p.v[p.table_cpu[0][0], 0, 3, 5] = float("inf")
    p.q[1, 0, 1] = NAN
    p.run(cuda)
    assert p.out[0, 0, :2, 5].isinf().all() and p.out[0, 0, :2, 6].isfinite().all() and p.out[0, 0, 2:].isfinite().all()
    assert p.out[1, 0, 1].isnan().all() and p.lse[1, 0, 1].isnan() and p.out[1, 0, 0].isfinite().all()


def test_bad_pages_and_lengths(cuda):
    lens = [290, 290, 290, 33]
    p = Problem(lens, 2, 12, 1, 128, 32, BF)
    p.table[0, 2], p.table[1, 0] = p.pages, -1
    p.lens = [290, 290, p.table.shape[1] * 32 + 1, -4]
    p.run(cuda)
    assert status(p.st)[0] == cuda.KDA_DEV_PAGE_OOB | cuda.KDA_DEV_SEQ_OOB
    assert not p.out[2:].any() and (p.lse[2:] == -math.inf).all()
    p.lens = lens
    p.table_cpu = p.table.cpu().long().clamp(0, p.pages - 1)
    p.check(hidden=set(range(64, 96)), only=[0])
    p.check(hidden=set(range(32)), only=[1])


def test_captured_and_on_another_stream(cuda):
    p = Problem([700, 90], 2, 12, 1, 128, 64, BF).run(cuda)
    want = p.out.clone()
    lens = torch.tensor(p.lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(cuda.kda_paged_attention_workspace_size(2, 2, 12, 1, 128), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cuda.kda_paged_attention(p.q, p.k, p.v, p.table, lens, out, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda.kda_paged_attention(p.q, p.k, p.v, p.table, lens, out, ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
