"""Attention over the paged cache against the fp64 softmax, at the lengths, masks and shapes where it can go wrong.

Tolerances are tests/_attention.py's attend_bound, from the kernel's roundings; p_bits, the bits of a probability in the
second product: 16 (bf16 cache: a sum of two bf16), 11 (e4m3 cache: fp16), 21 with fp32 queries or outputs.
"""
import math

import pytest
import torch

from tests import _attention as ref
from tests._gpu import status

pytestmark = pytest.mark.gpu
F32, BF, E4 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
NAN = float("nan")


class Problem:
    """Requests of the given lengths in a shuffled paged cache; every cache row no request owns holds NaN, and table
    entries past a request's pages hold garbage."""

    def __init__(self, lens, W, Hq, Hkv, d, page, kind, qdt=BF, odt=BF, seed=0, qscale=1.5, kscale=1.0):
        g = torch.Generator().manual_seed(seed + 17 * d + Hq)
        self.lens, self.W, self.Hq, self.Hkv, self.d, self.page, self.kind, self.odt = lens, W, Hq, Hkv, d, page, kind, odt
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g)
        table = torch.randint(-5, pages + 5, (len(lens), max(max(need), 1) + 1), generator=g)
        rows = lambda s: (torch.randn(pages, Hkv, page, d, generator=g) * s).to(BF)  # noqa: E731
        k, v = rows(kscale), rows(1.0)
        own = torch.zeros(pages, page, dtype=torch.bool)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            for j in range(n):
                own[order[at + j], :min(page, lens[i] - j * page)] = True
            at += n
        hole = ~own[:, None, :].expand(pages, Hkv, page)
        self.ks = self.vs = None
        if kind == E4:
            (kc, ks), (vc, vs) = ref.quantise(k.double()), ref.quantise(v.double())
            self.kd, self.vd = kc * ks[..., None], vc * vs[..., None]
            kc[hole], vc[hole], ks[hole], vs[hole] = NAN, NAN, NAN, NAN
            k, v = kc.float().to(E4), vc.float().to(E4)
            self.ks, self.vs = ks.float().cuda(), vs.float().cuda()
        else:
            self.kd, self.vd = k.double(), v.double()
            k[hole], v[hole] = NAN, NAN
        self.k, self.v, self.table_cpu = k.cuda(), v.cuda(), table
        self.table = table.to(torch.int32).cuda()
        self.q = (torch.randn(len(lens), W, Hq, d, generator=g) * qscale).to(qdt).cuda()
        self.pages = pages

    def run(self, cuda, **kw):
        B = len(self.lens)
        self.out = torch.full((B, self.W, self.Hq, self.d), 7.0, dtype=self.odt, device="cuda")
        self.lse = torch.full((B, self.W, self.Hq), 7.0, device="cuda")
        ws = torch.full((cuda.kda_paged_attention_workspace_size(B, self.W, self.Hq, self.Hkv, self.d),), 255,
                        dtype=torch.uint8, device="cuda")
        self.st = torch.zeros(2, dtype=torch.int32, device="cuda")
        lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        cuda.kda_paged_attention(self.q, self.k, self.v, self.table, lens, self.out, ws, k_scales=self.ks,
                                 v_scales=self.vs, lse=self.lse, dev_status=self.st, **kw)
        return self

    def rows(self, x, i):
        at = torch.arange(self.lens[i])
        return x[self.table_cpu[i][at // self.page], :, at % self.page]

    def check(self, scale=None, softcap=0.0, window=0, hidden=None, only=None):
        out, lse = self.out.cpu().double(), self.lse.cpu().double()
        bits = 21 if F32 in (self.odt, self.q.dtype) else 16 if self.kind == BF else 11
        for i, n in enumerate(self.lens):
            if only is not None and i not in only:
                continue
            want = ref.attend(self.q[i].cpu().double(), self.rows(self.kd, i), self.rows(self.vd, i), n,
                              self.d ** -0.5 if scale is None else scale, softcap, window, hidden)
            tol, tol_l = ref.attend_bound(*want, self.d, max(n, 1), self.odt == BF, bits)
            assert torch.all((out[i] - want[0]).abs() <= tol), (i, n, ((out[i] - want[0]).abs() / tol).max())
            none = want[1] == -math.inf
            assert torch.equal(lse[i] == -math.inf, none)
            assert torch.all((lse[i] - want[1])[~none].abs() <= tol_l[~none]), (i, n)
            assert not out[i][none].any()


SHAPES = [  # Hq, Hkv, d, page, cache, q, out, W, softcap, window
    (32, 8, 128, 16, BF, BF, BF, 1, 0.0, 0),
    (12, 4, 128, 64, E4, BF, BF, 1, 0.0, 0),
    (12, 1, 128, 48, E4, BF, BF, 3, 20.0, 40),
    (12, 1, 128, 32, BF, BF, BF, 8, 0.0, 50),
    (6, 6, 64, 16, BF, F32, F32, 2, 0.0, 0),
    (6, 2, 64, 16, E4, F32, F32, 4, 5.0, 0),
    (7, 7, 64, 80, E4, BF, F32, 1, 0.0, 17),
    (4, 2, 32, 16, BF, BF, BF, 5, 30.0, 0),
    (9, 1, 32, 16, E4, BF, BF, 1, 0.0, 0),
    (3, 1, 16, 16, BF, F32, BF, 7, 0.0, 1),
    (2, 1, 16, 112, E4, BF, BF, 9, 0.0, 33),
    (40, 1, 128, 16, BF, F32, F32, 1, 0.0, 0),
    (33, 1, 64, 16, E4, BF, BF, 1, 0.0, 0),
]
LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 333]


@pytest.mark.parametrize("Hq,Hkv,d,page,kind,qdt,odt,W,softcap,window", SHAPES)
def test_ragged_batch(cuda, Hq, Hkv, d, page, kind, qdt, odt, W, softcap, window):
    p = Problem(LENS, W, Hq, Hkv, d, page, kind, qdt, odt).run(cuda, softcap=softcap, window=window)
    assert status(p.st) == (0, len(LENS) * W * Hq)
    p.check(softcap=softcap, window=window)


@pytest.mark.parametrize("kind", [BF, E4])
@pytest.mark.parametrize("n", [1, 31, 4097, 20011])
def test_one_long_request_is_split_and_joined(cuda, kind, n):
    p = Problem([n], 1, 8, 2, 64, 32, kind).run(cuda)
    p.check()
    first = p.out.clone()
    assert torch.equal(p.run(cuda).out, first)  # the join's order is fixed


@pytest.mark.parametrize("kind", [BF, E4])
def test_more_requests_than_ctas(cuda, kind):
    lens = [(i * 37) % 90 for i in range(700)]
    p = Problem(lens, 1, 4, 2, 32, 16, kind).run(cuda)
    assert status(p.st) == (0, 700 * 4)
    p.check(only=range(0, 700, 23))
    # and the rest against the same requests on their own
    for i in range(0, 700, 61):
        one = Problem.__new__(Problem)
        one.__dict__.update(p.__dict__)
        one.lens, one.table, one.q = [lens[i]], p.table[i:i + 1].contiguous(), p.q[i:i + 1].contiguous()
        one.run(cuda)
        assert torch.allclose(one.out.float(), p.out[i:i + 1].float(), rtol=2 ** -7, atol=1e-3)


@pytest.mark.parametrize("kind", [BF, E4])
@pytest.mark.parametrize("scale,qscale,kscale", [(None, 60.0, 1.0), (-0.3, 1.5, 1.0), (0.0, 1.5, 1.0), (None, 1.0, 1e4),
                                                 (1e-3, 1e-6, 1e6)])
def test_scales_and_large_scores(cuda, kind, scale, qscale, kscale):
    """Scores up to about 1e5 apart (one key takes everything), negative and zero scales."""
    p = Problem([70, 257], 2, 4, 2, 64, 16, kind, qscale=qscale, kscale=kscale).run(cuda, scale=scale)
    p.check(scale=scale)


@pytest.mark.parametrize("kind", [BF, E4])
def test_rising_scores_move_the_reference(cuda, kind):
    """Keys that grow along the sequence: every tile has a new maximum."""
    p = Problem([600], 1, 8, 1, 32, 16, kind)
    at = torch.arange(600)
    grow = torch.zeros(p.pages, 1, p.page, 1, dtype=torch.float64)
    grow[p.table_cpu[0][at // p.page], 0, at % p.page, 0] = torch.exp2((at // 40).double())
    if kind == E4:
        p.ks *= grow[..., 0].float().cuda()
    else:
        p.k *= grow.to(BF).cuda()
    p.kd = p.kd * grow
    p.run(cuda).check()


def test_value_scales_far_apart(cuda):
    """Value scales from 2^-63 to 2^63 within a request, with the heavy tokens unlikely and likely."""
    p = Problem([150], 1, 4, 1, 32, 16, E4)
    at = torch.arange(150)
    e = ((at * 29) % 127 - 63).double()
    s = torch.ones(p.pages, 1, p.page, dtype=torch.float64)
    s[p.table_cpu[0][at // p.page], 0, at % p.page] = torch.exp2(e)
    old = p.vs.cpu().double()
    codes = p.vd / torch.where(old.isnan(), torch.ones_like(old), old)[..., None]
    p.vs = torch.where(old.isnan(), old, s).float().cuda()
    p.vd = codes * s[..., None]
    p.run(cuda).check()


@pytest.mark.parametrize("kind", [BF, E4])
def test_nan_in_a_draft_token_reaches_only_the_queries_that_see_it(cuda, kind):
    lens, W = [40, 100, 64], 5
    p = Problem(lens, W, 6, 2, 64, 16, kind).run(cuda)
    clean = p.out.clone()
    for which in ("k", "v"):
        p2 = Problem(lens, W, 6, 2, 64, 16, kind)
        for i, n in enumerate(lens):
            t = n - 3  # seen by window tokens 2, 3, 4
            x = getattr(p2, which)
            y = x.view(torch.uint8)
            y[p2.table_cpu[i][t // 16], 1, t % 16] = 0x7f if kind == E4 else 0xff
        p2.run(cuda)
        assert torch.equal(p2.out[:, :2], clean[:, :2]) or torch.allclose(p2.out[:, :2].float(), clean[:, :2].float(),
                                                                          rtol=2 ** -8, atol=1e-6)
        assert torch.equal(p2.out[:, :, :3], clean[:, :, :3])
        assert p2.out[:, 2:, 3:].isnan().all()


@pytest.mark.parametrize("kind", [BF, E4])
def test_nan_behind_the_sliding_window(cuda, kind):
    p = Problem([130], 3, 4, 2, 64, 16, kind)
    for t in range(130 - 3 - 20 + 1):  # before the first query's window of 20
        for x in (p.k, p.v):
            x.view(torch.uint8)[p.table_cpu[0][t // 16], :, t % 16] = 0x7f if kind == E4 else 0xff
    p.run(cuda, window=20).check(window=20)


@pytest.mark.parametrize("kind", [BF, E4])
def test_infinite_values_and_all_nan_scores(cuda, kind):
    p = Problem([20, 20], 1, 2, 1, 32, 16, BF)
    p.v[p.table_cpu[0][0], 0, 3, 5] = float("inf")
    p.q[1, 0, 1] = NAN
    p.run(cuda)
    assert p.out[0, 0, :, 5].isinf().all() and p.out[0, 0, :, 6].isfinite().all()
    assert p.out[1, 0, 1].isnan().all() and p.lse[1, 0, 1].isnan() and p.out[1, 0, 0].isfinite().all()


def test_bad_page_and_bad_length(cuda):
    lens = [90, 90, 90, 33]
    p = Problem(lens, 2, 4, 2, 64, 16, BF)
    p.table[0, 2], p.table[1, 1] = p.pages, -1
    p.lens = [90, 90, p.table.shape[1] * 16 + 1, -4]
    p.run(cuda)
    assert status(p.st)[0] == cuda.KDA_DEV_PAGE_OOB | cuda.KDA_DEV_SEQ_OOB
    assert not p.out[2:].any() and (p.lse[2:] == -math.inf).all()
    p.lens = lens
    p.table_cpu = p.table.cpu().long().clamp(0, p.pages - 1)
    p.check(hidden=set(range(32, 48)), only=[0])
    p.check(hidden=set(range(16, 32)), only=[1])


def test_no_pages_and_no_lse(cuda):
    B, W, Hq, d = 2, 1, 4, 64
    q = torch.randn(B, W, Hq, d, device="cuda").to(BF)
    out = torch.full_like(q, 3)
    pages = torch.empty(0, 2, 16, d, dtype=BF, device="cuda")
    ws = torch.empty(cuda.kda_paged_attention_workspace_size(B, W, Hq, 2, d), dtype=torch.uint8, device="cuda")
    z = torch.zeros(B, dtype=torch.int32, device="cuda")
    cuda.kda_paged_attention(q, pages, pages, torch.empty(B, 0, dtype=torch.int32, device="cuda"), z, out, ws)
    assert not out.any()
    p = Problem([40, 77], 1, 4, 2, 64, 16, E4).run(cuda)
    with_lse = p.out.clone()
    out = torch.empty_like(p.out)
    cuda.kda_paged_attention(p.q, p.k, p.v, p.table, torch.tensor(p.lens, dtype=torch.int32, device="cuda"), out, ws,
                             k_scales=p.ks, v_scales=p.vs)
    assert torch.equal(out, with_lse)
    cuda.kda_paged_attention(p.q[:0], p.k, p.v, p.table[:0], z[:0], out[:0], ws, k_scales=p.ks, v_scales=p.vs)


def test_other_stream_and_graph(cuda):
    """A decode step of norm, write and attention captured once and replayed on new inputs, bit for bit the eager
    calls' results; the eager calls run on a stream of their own."""
    B, Hq, Hkv, d, page, n = 3, 8, 2, 128, 16, 50
    g = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    p = Problem([n] * B, 1, Hq, Hkv, d, page, E4)
    ones = torch.ones(d, device="cuda")
    cos, sin = (x.cuda() for x in ref.angles(64, d))
    pos = torch.full((B,), n - 1, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    slots = p.table_cpu[:, (n - 1) // page].cuda() * page + (n - 1) % page
    x = torch.empty(B, Hq + 2 * Hkv, d, dtype=BF, device="cuda")
    q, k = torch.empty(B, 1, Hq, d, dtype=BF, device="cuda"), torch.empty(B, Hkv, d, dtype=BF, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(cuda.kda_paged_attention_workspace_size(B, 1, Hq, Hkv, d), dtype=torch.uint8, device="cuda")

    def step():
        cuda.kda_qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], ones, ones, q[:, 0], k, cos=cos, sin=sin, positions=pos)
        cuda.kda_kv_write(k, x[:, Hq + Hkv:], p.k, p.v, slots, k_scales=p.ks, v_scales=p.vs)
        cuda.kda_paged_attention(q, p.k, p.v, p.table, lens, out, ws, k_scales=p.ks, v_scales=p.vs)

    inputs, want = [rnd(*x.shape) for _ in range(3)], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i in inputs:
            x.copy_(i)
            step()
            want.append(out.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, w in zip(inputs, want):
        x.copy_(i)
        out.zero_()
        graph.replay()
        assert torch.equal(out, w)
    assert not torch.equal(want[0], want[1])
