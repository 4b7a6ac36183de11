"""Per-head query/key norm with rotation and its gradient against the fp64 formulas.

Bounds.  A row's sum of d squares runs over at most 8 sequential and 4 tree additions, so r and the products with
it are within 24 fp32 roundings; the rotation adds three on two channels.  An fp32 output is then within 32 U32 of
the pair's magnitude |a| + |b|, at most 2 max|y| of the row; a bf16 output one bf16 rounding more.  A weight's gradient is
a sum over N rows, within (N + 40) U32 of the sum of magnitudes.  dx is within 64 U32 of r (max|g w| + max|u| max|g w u|).
"""
import pytest
import torch

from tests import _attention as ref
from tests._attention import U16, U32
from tests._gpu import status

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
NPOS = 300


def make(T, Hq, Hkv, d, dt, seed, packed):
    g = torch.Generator().manual_seed(seed)
    rows = (torch.randn(T, Hq + 2 * Hkv, d, generator=g) * torch.exp(torch.randn(T, Hq + 2 * Hkv, 1, generator=g))).to(dt)
    if packed:
        r = rows.cuda()
        q, k = r[:, :Hq], r[:, Hq:Hq + Hkv]
    else:
        q, k = rows[:, :Hq].contiguous().cuda(), rows[:, Hq:Hq + Hkv].contiguous().cuda()
    wq, wk = (1 + 0.3 * torch.randn(2, d, generator=g)).cuda()
    pos = torch.randint(0, NPOS, (T,), generator=g, dtype=torch.int32)
    return q, k, wq, wk, pos


def rope_kw(d, rot, interleaved, pos):
    if not rot:
        return {}, None, None
    cos, sin = ref.angles(NPOS, rot)
    return dict(cos=cos.cuda(), sin=sin.cuda(), positions=pos.cuda(), interleaved=interleaved), cos, sin


CASES = [  # T, Hq, Hkv, d, rot, interleaved, in, out, packed
    (1, 32, 8, 128, 128, False, BF, BF, True),
    (7, 3, 1, 128, 64, True, BF, F32, False),
    (65, 12, 4, 128, 0, False, F32, F32, True),
    (33, 2, 2, 64, 64, False, F32, BF, True),
    (200, 5, 5, 64, 32, True, BF, BF, True),
    (19, 1, 1, 32, 16, False, BF, BF, False),
    (70, 6, 3, 32, 32, True, F32, F32, True),
    (13, 4, 2, 16, 16, False, BF, F32, True),
    (600, 7, 1, 16, 16, True, F32, BF, False),
    (513, 9, 2, 128, 48, False, BF, BF, True),
]


@pytest.mark.parametrize("T,Hq,Hkv,d,rot,il,idt,odt,packed", CASES)
def test_forward(cuda, T, Hq, Hkv, d, rot, il, idt, odt, packed):
    q, k, wq, wk, pos = make(T, Hq, Hkv, d, idt, T + d, packed)
    kw, cos, sin = rope_kw(d, rot, il, pos)
    out = torch.full((T, Hq + Hkv + 1, d), 7.0, dtype=odt, device="cuda")  # outputs side by side, one column block spare
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    cuda.kda_qk_norm_rope(q, k, wq, wk, out[:, :Hq], out[:, Hq:Hq + Hkv], eps=1e-5, dev_status=st, **kw)
    torch.cuda.synchronize()
    assert status(st) == (0, T * (Hq + Hkv))
    assert torch.all(out[:, -1] == 7.0)
    R = ref.rotations(cos, sin, pos, d, rot, il)
    for x, w, y in ((q, wq, out[:, :Hq]), (k, wk, out[:, Hq:Hq + Hkv])):
        want = ref.norm_rope(x.cpu().double(), w.cpu().double(), R, 1e-5)
        tol = 64 * U32 * want.abs().amax(-1, keepdim=True) + (U16 * want.abs() * 1.01 if odt == BF else 0)
        assert torch.all((y.cpu().double() - want).abs() <= tol)


@pytest.mark.parametrize("dt", [BF, F32])
def test_in_place_gives_the_same_bits(cuda, dt):
    q, k, wq, wk, pos = make(77, 6, 2, 128, dt, 5, True)
    kw, _, _ = rope_kw(128, 128, False, pos)
    yq, yk = torch.empty(77, 6, 128, dtype=dt, device="cuda"), torch.empty(77, 2, 128, dtype=dt, device="cuda")
    cuda.kda_qk_norm_rope(q, k, wq, wk, yq, yk, **kw)
    cuda.kda_qk_norm_rope(q, k, wq, wk, q, k, **kw)
    assert torch.equal(q, yq) and torch.equal(k, yk)


def test_unit_length_norm_of_the_kda_layers(cuda):
    """w = 1 / sqrt(d), eps = 1e-6 / d is x / sqrt(|x|^2 + 1e-6)."""
    d = 128
    q, k, _, _, _ = make(50, 12, 12, d, F32, 6, False)
    q[0] = 0
    w = torch.full((d,), d ** -0.5, device="cuda")
    yq, yk = torch.empty_like(q), torch.empty_like(k)
    cuda.kda_qk_norm_rope(q, k, w, w, yq, yk, eps=1e-6 / d)
    for x, y in ((q, yq), (k, yk)):
        x = x.cpu().double()
        want = x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()
        assert torch.all((y.cpu().double() - want).abs() <= 64 * U32 * want.abs().amax(-1, keepdim=True))


def test_rows_are_independent_of_nan_and_infinity_elsewhere(cuda):
    q, k, wq, wk, pos = make(9, 4, 2, 64, BF, 7, False)
    kw, _, _ = rope_kw(64, 64, False, pos)
    y0, y1 = torch.empty_like(q), torch.empty_like(k)
    cuda.kda_qk_norm_rope(q, k, wq, wk, y0, y1, **kw)
    q2 = q.clone()
    q2[4, 1, 3], q2[5, 2, 9] = float("nan"), float("inf")
    z0, z1 = torch.empty_like(q), torch.empty_like(k)
    cuda.kda_qk_norm_rope(q2, k, wq, wk, z0, z1, **kw)
    same = torch.ones(9, 4, dtype=torch.bool, device="cuda")
    same[4, 1] = same[5, 2] = False
    assert torch.equal(y0[same], z0[same]) and torch.equal(y1, z1) and z0[4, 1].isnan().all()


def test_bad_position_is_flagged_and_skipped(cuda):
    q, k, wq, wk, pos = make(40, 3, 1, 128, BF, 8, False)
    pos[3], pos[17] = NPOS, -1
    kw, _, _ = rope_kw(128, 128, False, pos)
    yq, yk = torch.full_like(q, 5), torch.full_like(k, 5)
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    cuda.kda_qk_norm_rope(q, k, wq, wk, yq, yk, dev_status=st, **kw)
    assert status(st) == (cuda.KDA_DEV_POS_OOB, 38 * 4)
    for t in range(40):
        assert bool((yq[t] == 5).all()) == (t in (3, 17))
    # the backward leaves such a token out of everything
    ws = torch.empty(cuda.kda_qk_norm_rope_backward_workspace_size(40, 3, 1, 128), dtype=torch.uint8, device="cuda")
    res = []
    for keep in (None, [t for t in range(40) if t not in (3, 17)]):
        sel = slice(None) if keep is None else torch.tensor(keep).cuda()
        a = [x[sel].contiguous() for x in (yq, yk, q, k)]
        dq, dk, dw = torch.full_like(a[2], 5), torch.full_like(a[3], 5), torch.empty(2, 128, device="cuda")
        kw2 = dict(kw, positions=kw["positions"][sel].contiguous())
        st.zero_()
        cuda.kda_qk_norm_rope_backward(*a[:2], *a[2:], wq, wk, dq, dk, dw[0], dw[1], ws, dev_status=st, **kw2)
        res.append((status(st), dq, dw))
    assert res[0][0] == (cuda.KDA_DEV_POS_OOB, 38 * 4) and res[1][0] == (0, 38 * 4)
    assert (res[0][1][3] == 5).all() and torch.isfinite(res[0][2]).all()
    assert torch.allclose(res[0][2], res[1][2], rtol=1e-4, atol=1e-3)


@pytest.mark.parametrize("T,Hq,Hkv,d,rot,il,idt,odt,packed", CASES)
def test_backward_matches_the_formula(cuda, T, Hq, Hkv, d, rot, il, idt, odt, packed):
    q, k, wq, wk, pos = make(T, Hq, Hkv, d, idt, T + d, packed)
    kw, cos, sin = rope_kw(d, rot, il, pos)
    gdt = F32 if T % 2 else BF
    g = torch.Generator().manual_seed(T)
    dyq, dyk = (torch.randn(T, h, d, generator=g).to(gdt).cuda() for h in (Hq, Hkv))
    grads = torch.empty(T, Hq + Hkv, d, dtype=odt, device="cuda")
    dw = torch.full((2, d), 9.0, device="cuda")
    ws = torch.empty(cuda.kda_qk_norm_rope_backward_workspace_size(T, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    args = (dyq, dyk, q, k, wq, wk, grads[:, :Hq], grads[:, Hq:], dw[0], dw[1], ws)
    cuda.kda_qk_norm_rope_backward(*args, eps=1e-5, dev_status=st, **kw)
    assert status(st) == (0, T * (Hq + Hkv))
    R = ref.rotations(cos, sin, pos, d, rot, il)
    for x, w, dy, dx, got in ((q, wq, dyq, grads[:, :Hq], dw[0]), (k, wk, dyk, grads[:, Hq:], dw[1])):
        x, w, dy = x.cpu().double(), w.cpu().double(), dy.cpu().double()
        want, dwant = ref.norm_rope_grad(dy, x, w, R, 1e-5)
        r = (x.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
        gr = torch.einsum("tji,thj->thi", R, dy)
        big = lambda z: z.abs().amax(-1, keepdim=True)  # noqa: E731
        tol = 64 * U32 * r * (big(gr * w) + big(x * r) * big(gr * w) * big(x * r)) + (
            U16 * want.abs() * 1.01 if odt == BF else 0)
        assert torch.all((dx.cpu().double() - want).abs() <= tol)
        n = T * x.shape[1]
        per_term = 2 * gr.abs().amax() * (x * r).abs().amax()  # the rotation mixes two channels of dy
        assert torch.all((got.cpu().double() - dwant).abs() <= (n + 40) * U32 * (gr * x * r).abs().sum((0, 1))
                         + 40 * U32 * per_term * n ** 0.5)
    again, dw2 = torch.empty_like(grads), torch.empty_like(dw)
    cuda.kda_qk_norm_rope_backward(dyq, dyk, q, k, wq, wk, again[:, :Hq], again[:, Hq:], dw2[0], dw2[1], ws, eps=1e-5,
                                   **kw)
    assert torch.equal(grads, again) and torch.equal(dw, dw2)


def test_no_tokens(cuda):
    q, k, wq, wk, pos = make(0, 4, 2, 64, BF, 1, False)
    cuda.kda_qk_norm_rope(q, k, wq, wk, torch.empty_like(q), torch.empty_like(k))
    dw = torch.full((2, 64), 3.0, device="cuda")
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    cuda.kda_qk_norm_rope_backward(q, k, q, k, wq, wk, torch.empty_like(q), torch.empty_like(k), dw[0], dw[1], ws)
    assert not dw.any()


def test_gradients_over_the_incoming_ones(cuda):
    q, k, wq, wk, pos = make(31, 4, 2, 128, BF, 2, False)
    kw, _, _ = rope_kw(128, 128, True, pos)
    g = torch.Generator(device="cuda").manual_seed(3)
    dyq, dyk = (torch.randn(x.shape, generator=g, device="cuda").to(BF) for x in (q, k))
    ws = torch.empty(cuda.kda_qk_norm_rope_backward_workspace_size(31, 4, 2, 128), dtype=torch.uint8, device="cuda")
    dq, dk, dw = torch.empty_like(q), torch.empty_like(k), torch.empty(2, 128, device="cuda")
    cuda.kda_qk_norm_rope_backward(dyq, dyk, q, k, wq, wk, dq, dk, dw[0], dw[1], ws, **kw)
    dw2 = torch.empty_like(dw)
    cuda.kda_qk_norm_rope_backward(dyq, dyk, q, k, wq, wk, dyq, dyk, dw2[0], dw2[1], ws, **kw)
    assert torch.equal(dq, dyq) and torch.equal(dk, dyk) and torch.equal(dw, dw2)
