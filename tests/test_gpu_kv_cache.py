"""Paged cache rows written and read back, against the format's definition in fp64.

Scales are powers of two, so the only rounding is the one to e4m3 (or to bf16): codes, scales and values read back are
compared bit for bit.
"""
import pytest
import torch

from tests import _attention as ref
from tests._gpu import status

pytestmark = pytest.mark.gpu
F32, BF, E4 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def pool(pages, Hkv, page, d, kind):
    """A cache filled with a mark; returns (k, v, k_scales, v_scales)."""
    k = torch.full((pages, Hkv, page, d), 3.0, device="cuda", dtype=BF).to(kind)
    s = (lambda: torch.full((pages, Hkv, page), 5.0, device="cuda") if kind == E4 else None)  # noqa: E731
    return k, k.clone(), s(), s()


def rows_of(x, slots, page):
    """x [pages, Hkv, page, ...] -> [T, Hkv, ...]"""
    return x[slots // page, :, slots % page]


def values(T, H, d, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, d, generator=g) * torch.exp2(torch.randint(-20, 20, (T, H, 1), generator=g))).to(dt)


CASES = [  # T, Hkv, d, page, in, cache, out
    (1, 8, 128, 16, BF, E4, BF), (50, 1, 128, 48, BF, E4, F32), (301, 4, 64, 64, F32, E4, F32),
    (33, 3, 32, 16, BF, E4, BF), (700, 5, 16, 32, F32, E4, BF), (900, 8, 128, 128, F32, E4, F32),
    (40, 2, 128, 16, BF, BF, BF), (301, 12, 64, 80, F32, BF, F32), (5, 1, 16, 16, BF, BF, F32), (77, 3, 32, 16, F32, BF, BF),
]


@pytest.mark.parametrize("T,Hkv,d,page,idt,kind,odt", CASES)
def test_write_and_read(cuda, T, Hkv, d, page, idt, kind, odt):
    pages = -(-T // page) + 2
    k, v, ks, vs = pool(pages, Hkv, page, d, kind)
    marks = [None if x is None else x.clone() for x in (k, v, ks, vs)]
    rows = torch.empty(T, 3 * Hkv, d, dtype=idt)  # keys and values as column blocks of a wider array
    rows[:, Hkv:2 * Hkv], rows[:, 2 * Hkv:] = values(T, Hkv, d, idt, 1), values(T, Hkv, d, idt, 2)
    rows = rows.cuda()
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(T))[:T].cuda()
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    cuda.kda_kv_write(rows[:, Hkv:2 * Hkv], rows[:, 2 * Hkv:], k, v, slots, k_scales=ks, v_scales=vs, dev_status=st)
    assert status(st) == (0, T * Hkv)
    ko, vo = torch.empty(2, T, Hkv, d, dtype=odt, device="cuda")
    cuda.kda_kv_read(k, v, slots, ko, vo, k_scales=ks, v_scales=vs, dev_status=st)
    assert status(st)[0] == 0
    taken = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    taken[slots // page, slots % page] = True
    for x, p, s, mark, smark, back in ((rows[:, Hkv:2 * Hkv], k, ks, marks[0], marks[2], ko),
                                       (rows[:, 2 * Hkv:], v, vs, marks[1], marks[3], vo)):
        x = x.cpu().double()
        if kind == E4:
            c, scale = ref.quantise(x)
            assert torch.equal(rows_of(p.float(), slots, page).cpu().double(), c)
            assert torch.equal(rows_of(s, slots, page).cpu().double(), scale)
            want = c * scale[..., None]
            assert torch.all(s.transpose(1, 2)[~taken] == 5.0)
        else:
            want = x.to(BF).double()
            assert torch.equal(rows_of(p, slots, page).cpu().double(), want)
        bits = lambda z: z.view(torch.uint8).view(pages, Hkv, page, -1).transpose(1, 2)  # noqa: E731
        assert torch.equal(bits(p)[~taken], bits(mark)[~taken])
        assert torch.equal(back.cpu().double(), want.to(odt).double())
    # what was read back, written again, keeps its values
    k2, v2, ks2, vs2 = pool(pages, Hkv, page, d, kind)
    ko, vo = torch.empty(2, T, Hkv, d, device="cuda")
    cuda.kda_kv_read(k, v, slots, ko, vo, k_scales=ks, v_scales=vs)
    cuda.kda_kv_write(ko, vo, k2, v2, slots, k_scales=ks2, v_scales=vs2)
    ko2, vo2 = torch.empty(2, T, Hkv, d, device="cuda")
    cuda.kda_kv_read(k2, v2, slots, ko2, vo2, k_scales=ks2, v_scales=vs2)
    assert torch.equal(ko, ko2) and torch.equal(vo, vo2)


def test_edges_of_the_8_bit_format(cuda):
    """Rows at the scale's steps, at its limits, of zeros, subnormals, infinities and NaN."""
    d, inf, nan = 16, float("inf"), float("nan")
    tops = [448.0, 448.0 * (1 + 2.0 ** -23), 447.9, 1.75, 1.7500001, 1.0, 0.0, 1e-45, 2.0 ** -126, 448 * 2.0 ** 63,
            448 * 2.0 ** 63 * (1 + 2.0 ** -23), 3.4e38, 448 * 2.0 ** -63, 2.0 ** -73, 1.5 * 2.0 ** -73, 2.0 ** -72]
    x = torch.zeros(len(tops) + 3, 1, d)
    for i, t in enumerate(tops):
        x[i, 0] = t * torch.linspace(-1, 1, d)
        x[i, 0, 3] = t
    x[-3, 0, 2], x[-3, 0, 5] = inf, 1.0
    x[-2, 0, 1], x[-2, 0, 4], x[-2, 0, 6] = nan, -3.0, 448.0
    x[-1] = nan
    T = len(x)
    k, v, ks, vs = pool(2, 1, 32, d, E4)
    slots = torch.arange(T, device="cuda")
    cuda.kda_kv_write(x.cuda(), (-x).cuda(), k, v, slots, k_scales=ks, v_scales=vs)
    ordinary = x[:len(tops)].double()
    c, s = ref.quantise(ordinary)
    got = rows_of(k.float(), slots, 32).cpu().double()
    assert torch.equal(rows_of(ks, slots, 32).cpu().double()[:len(tops)], s)
    assert torch.equal(got[:len(tops)], c)
    assert torch.equal(rows_of(v.float(), slots, 32).cpu().double()[:len(tops)], -c)
    gs = rows_of(ks, slots, 32).cpu()[:, 0]
    assert gs[-3] == 2.0 ** 63 and got[-3, 0, 2] == 448 and got[-3, 0, 5] == 0
    assert gs[-2] == 1 and got[-2, 0, 1].isnan() and got[-2, 0, 4] == -3 and got[-2, 0, 6] == 448
    assert gs[-1] == 1 and got[-1].isnan().all()


@pytest.mark.parametrize("kind", [E4, BF])
def test_skipped_and_bad_slots(cuda, kind):
    T, Hkv, d, page, pages = 6, 2, 64, 16, 3
    k, v, ks, vs = pool(pages, Hkv, page, d, kind)
    was = [x.clone() for x in (k.view(torch.uint8), v.view(torch.uint8))]
    x = torch.randn(T, Hkv, d, device="cuda").to(BF)
    slots = torch.tensor([-1, 5, pages * page, 7, -2 ** 62, 2 ** 62], device="cuda")
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    cuda.kda_kv_write(x, x, k, v, slots, k_scales=ks, v_scales=vs, dev_status=st)
    assert status(st) == (cuda.KDA_DEV_PAGE_OOB, 2 * Hkv)
    for now, then in zip((k, v), was):
        diff = (now.view(torch.uint8) != then).flatten(3).any(-1).any(1)  # [pages, page]
        assert diff.flatten().nonzero().flatten().tolist() == [5, 7]
    st.zero_()
    ko, vo = torch.full((2, T, Hkv, d), 9.0, device="cuda", dtype=BF)
    cuda.kda_kv_read(k, v, slots, ko, vo, k_scales=ks, v_scales=vs, dev_status=st)
    assert status(st)[0] == cuda.KDA_DEV_PAGE_OOB
    for t in range(T):
        assert bool(ko[t].any()) == bool(vo[t].any()) == (t in (1, 3))
    # repeats may be read
    cuda.kda_kv_read(k, v, slots[[1, 1, 3]], ko[:3], vo[:3], k_scales=ks, v_scales=vs)
    assert torch.equal(ko[0], ko[1])


def test_debug_checks_see_repeated_slots(cuda):
    k, v, _, _ = pool(2, 1, 16, 16, BF)
    x = torch.randn(3, 1, 16, device="cuda").to(BF)
    was = cuda.kda_debug_checks()
    try:
        cuda.kda_set_debug_checks(True)
        cuda.kda_kv_write(x, x, k, v, torch.tensor([1, -1, -1], device="cuda"))
        with pytest.raises(cuda.KdaError):
            cuda.kda_kv_write(x, x, k, v, torch.tensor([1, 2, 1], device="cuda"))
    finally:
        cuda.kda_set_debug_checks(was)


def test_offsets_past_32_bits(cuda):
    """A bf16 pool of 2^32 + elements (8.6 GB each for keys and values): the last page's rows, written and read."""
    Hkv, page, d = 8, 128, 128
    pages = 2 ** 32 // (Hkv * page * d) + 2
    k = torch.empty(pages, Hkv, page, d, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    k[0], v[0] = 1.0, 2.0
    x = torch.randn(page, Hkv, d, device="cuda").to(BF)
    slots = torch.arange(page, device="cuda") + (pages - 1) * page
    cuda.kda_kv_write(x, -x, k, v, slots)
    assert torch.equal(k[-1].transpose(0, 1), x) and torch.equal(v[-1].transpose(0, 1), -x)
    assert torch.all(k[0] == 1) and torch.all(v[0] == 2)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    cuda.kda_kv_read(k, v, slots, ko, vo)
    assert torch.equal(ko, x) and torch.equal(vo, -x)
    # attention over the far page: one request of exactly that page
    q = torch.randn(1, 1, 8, d, device="cuda").to(BF)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(1, 1, 8, device="cuda")
    ws = torch.empty(cuda.kda_paged_attention_workspace_size(1, 1, 8, 8, d), dtype=torch.uint8, device="cuda")
    cuda.kda_paged_attention(q, k, v, table, torch.tensor([page], dtype=torch.int32, device="cuda"), out, ws, lse=lse)
    c = lambda z: z.cpu().double()  # noqa: E731
    want = ref.attend(c(q)[0], c(x), -c(x), page, d ** -0.5)
    tol, tol_l = ref.attend_bound(*want, d, page, True, 16)
    assert torch.all((c(out)[0] - want[0]).abs() <= tol) and torch.all((c(lse)[0] - want[1]).abs() <= tol_l)


def test_no_tokens(cuda):
    k, v, _, _ = pool(2, 1, 16, 16, BF)
    x = torch.empty(0, 1, 16, device="cuda", dtype=BF)
    s = torch.empty(0, dtype=torch.int64, device="cuda")
    cuda.kda_kv_write(x, x, k, v, s)
    cuda.kda_kv_read(k, v, s, x, x.clone())
