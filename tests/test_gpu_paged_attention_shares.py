"""The two tensor-memory forms of the attention with many tiles and several units in each worker's share, so that every ring,
buffer and double buffer is used again and again: against the fp64 softmax, under windows, caps, scales, bad pages, NaN and
infinities.  Bounds as in test_gpu_paged_attention.py.

Which form a call takes goes by its query rows per key/value head (W Hq / Hkv), types and units: with d = 128 and bf16 queries and
outputs, up to 16 rows, a bf16 cache and at most 64 units (requests times key/value heads) take the form for few rows, more
than 16 rows the many-rows form.  A share is a CTA's, of 152: a request of 152 x 20 tiles of 128 tokens beside 60 short ones gives
each CTA some 20 tiles, and some of them the ends of several units.
"""
import math

import pytest
import torch

from tests import _attention as ref
from tests._attention_rows import put
from tests._gpu import status
from tests.test_gpu_paged_attention import BF, E4, Problem

pytestmark = pytest.mark.gpu
# cache, Hq, W for one key/value head: 1, 4, 6, 8, 12 and 16 rows (one and two softmax groups, full and partly full), then
# 24 and 130 rows in both caches
FEW = [(BF, 1, 1), (BF, 4, 1), (BF, 3, 2), (BF, 4, 2), (BF, 12, 1), (BF, 4, 4)]
MANY = [(BF, 12, 2), (BF, 13, 10), (E4, 12, 2), (E4, 13, 10)]
forms = pytest.mark.parametrize("kind,Hq,W", FEW + MANY)
LONG = 9000


def shared(kind, Hq, W, page, lens, seed=0):
    """Requests of the given lengths over the same pages (one after another in a shuffled order), with queries of their own."""
    p = Problem([max(lens)], W, Hq, 1, 128, page, kind, seed=seed)
    B = len(lens)
    p.lens, p.table_cpu = list(lens), p.table_cpu.expand(B, -1)
    p.table = p.table.expand(B, -1).contiguous()
    g = torch.Generator().manual_seed(seed + 1)
    p.q = (1.5 * torch.randn(B, W, Hq, 128, generator=g)).to(BF).cuda()
    return p


def many_lengths(B=64, most=LONG):
    """B lengths, half of them near the most, the others from nothing up."""
    return [most - 37 * i if i % 2 else (i * i * 7) % 1500 for i in range(B)]


CHECKED = [1, 6, 10, 31, 34, 62]


@forms
@pytest.mark.parametrize("page", [16, 48, 256])
def test_many_tiles(cuda, kind, Hq, W, page):
    lens = many_lengths()
    p = shared(kind, Hq, W, page, lens).run(cuda)
    assert status(p.st) == (0, len(lens) * W * Hq)
    p.check(only=CHECKED)
    first, lse = p.out.clone(), p.lse.clone()
    for _ in range(3):
        p.run(cuda)
        assert torch.equal(p.out, first) and torch.equal(p.lse, lse)


@forms
def test_short_units_beside_a_long_one(cuda, kind, Hq, W):
    """60 units of a tile or two, four or five to a CTA, and one that all CTAs have a part of."""
    lens = [1 + (i * 53) % 200 for i in range(60)] + [250000]
    p = shared(kind, Hq, W, 128, lens).run(cuda)
    assert status(p.st) == (0, len(lens) * W * Hq)
    p.check(only=list(range(0, 60, 7)) + ([60] if W * Hq <= 24 else []))


@forms
@pytest.mark.parametrize("softcap,window,scale", [(20.0, 0, None), (1.0, 0, None), (3.0, 70, 0.2), (500.0, 0, None), (0.0, 100, None),
                                                  (8.0, 2500, 0.2), (0.0, 1, None), (0.0, 3000, -0.1), (0.0, 0, 0.0)])
def test_caps_windows_and_scales(cuda, kind, Hq, W, softcap, window, scale):
    p = shared(kind, Hq, W, 64, many_lengths(), seed=2).run(cuda, softcap=softcap, window=window, scale=scale)
    p.check(softcap=softcap, window=window, scale=scale, only=CHECKED[1:5])


@forms
@pytest.mark.parametrize("qscale,kscale", [(60.0, 1.0), (1.0, 1e4), (1e-6, 1e6)])
def test_large_scores(cuda, kind, Hq, W, qscale, kscale):
    Problem([70, 257, 1500], W, Hq, 1, 128, 16, kind, qscale=qscale, kscale=kscale).run(cuda).check()


@forms
@pytest.mark.parametrize("step", [48, 128, 300])
def test_rising_scores(cuda, kind, Hq, W, step):
    """Scores that rise by 3 nats every `step` tokens over many tiles of a share; with a bf16 cache, values fall with them, so that the
    parts of all moves count."""
    lens = many_lengths(most=3000)
    p = shared(kind, Hq, W, 16, lens, seed=step)
    g = torch.Generator().manual_seed(step)
    rise = (torch.arange(max(lens)) // step % 20).double()
    k = 0.1 * torch.randn(max(lens), 1, 128, generator=g).double()
    k[:, :, 0] = 0.375 * rise[:, None]
    put(p, "k", 0, k)
    p.q[..., 0] = 8.0
    if kind == BF:
        put(p, "v", 0, (1 + torch.rand(max(lens), 1, 128, generator=g).double()) * torch.exp(-3.0 * rise)[:, None, None])
    p.run(cuda, scale=1.0).check(scale=1.0, only=CHECKED)


@forms
def test_nan_in_a_draft_token_reaches_only_the_queries_that_see_it(cuda, kind, Hq, W):
    lens = [140, 2000, 64, 257]
    for which in ("k", "v"):
        p = Problem(lens, W, Hq, 1, 128, 16, kind)
        for i, n in enumerate(lens):
            t = n - 1  # the window's last token sees it
            getattr(p, which).view(torch.uint8)[p.table_cpu[i][t // 16], 0, t % 16] = 0xff
        p.run(cuda)
        assert p.out[:, W - 1].isnan().all() and p.out[:, :W - 1].isfinite().all()
        for i, n in enumerate(lens) if W > 1 else ():
            want = ref.attend(p.q[i, :W - 1].cpu().double(), p.rows(p.kd, i)[:n - 1], p.rows(p.vd, i)[:n - 1], n - 1, 128 ** -0.5)
            tol, tol_l = ref.attend_bound(*want, 128, n, True, 16 if kind == BF else 11)
            assert torch.all((p.out[i, :W - 1].cpu().double() - want[0]).abs() <= tol)
            assert torch.all((p.lse[i, :W - 1].cpu().double() - want[1]).abs() <= tol_l)


@forms
@pytest.mark.parametrize("window", [20, 300])
def test_nan_behind_the_window(cuda, kind, Hq, W, window):
    n = 2330
    p = Problem([n, n], W, Hq, 1, 128, 16, kind)
    for i in range(2):
        at = torch.arange(n - W - window + 1)  # before the first query's window
        for x in (p.k, p.v):
            x.view(torch.uint8)[p.table_cpu[i][at // 16], :, at % 16] = 0xff
    p.run(cuda, window=window).check(window=window)


@pytest.mark.parametrize("kind,Hq,W", [f for f in FEW + MANY if f[0] == BF])
def test_infinite_values(cuda, kind, Hq, W):
    p = Problem([2000, 20], W, Hq, 1, 128, 16, kind)
    p.v[p.table_cpu[0][70], 0, 3, 5] = float("inf")
    p.v[p.table_cpu[1][0], 0, 1, 77] = -float("inf")
    p.run(cuda)
    assert (p.out[0, :, :, 5] == float("inf")).all() and (p.out[1, :, :, 77] == -float("inf")).all()
    p.out[0, :, :, 5], p.out[1, :, :, 77] = 0, 0
    p.vd[p.table_cpu[0][:125], :, :, 5], p.vd[p.table_cpu[1][:2], :, :, 77] = 0, 0
    p.check()


@forms
@pytest.mark.parametrize("bad", [-1, -2, 2 ** 31 - 1])
def test_bad_pages_and_lengths(cuda, kind, Hq, W, bad):
    """Pages outside the cache in the first, a middle and the last place, alone and side by side, and lengths that are none."""
    lens = [1500, 1500, 1500, 290, 290]
    p = Problem(lens, W, Hq, 1, 128, 32, kind)
    hidden = {0: [0], 1: [7, 8, 9, 10, 20], 2: [46]}
    for i, pages in hidden.items():
        p.table[i, pages] = bad
    p.lens = lens[:3] + [p.table.shape[1] * 32 + 1, -4]
    p.run(cuda)
    assert status(p.st)[0] == cuda.KDA_DEV_PAGE_OOB | cuda.KDA_DEV_SEQ_OOB
    assert not p.out[3:].any() and (p.lse[3:] == -math.inf).all()
    p.lens, p.table_cpu = lens, p.table.cpu().long().clamp(0, p.pages - 1)
    for i, pages in hidden.items():
        p.check(hidden={t for x in pages for t in range(32 * x, 32 * x + 32)}, only=[i])


@forms
def test_captured_and_on_another_stream(cuda, kind, Hq, W):
    p = shared(kind, Hq, W, 64, many_lengths(B=20), seed=3).run(cuda)
    want = p.out.clone()
    lens = torch.tensor(p.lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(cuda.kda_paged_attention_workspace_size(20, W, Hq, 1, 128), dtype=torch.uint8, device="cuda")
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
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
