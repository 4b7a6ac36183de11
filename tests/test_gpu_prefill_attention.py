"""Prompt attention and its gradients against the definitions in fp64, at the lengths, heads, types and masks where the kernels
change course; the bounds are derived in _prompt.py."""
import math

import pytest
import torch

from tests import _prompt as P

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

LENGTHS = [[1], [2], [63, 1, 64], [65, 0, 127, 5], [128, 129], [255, 256, 257], [300, 3, 511]]


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", [(2, 2), (4, 1)], ids=str)
def test_lengths(cuda, lengths, dtype, heads):
    P.compare(cuda, lengths, *heads, 128, dtype, seed=sum(lengths))


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", [(1, 1), (6, 2), (12, 1), (5, 5)], ids=str)
def test_heads_and_sizes(cuda, d, dtype, heads):
    P.compare(cuda, [70, 200, 13], *heads, d, dtype, seed=d, packed=True)


@pytest.mark.parametrize("window", [1, 2, 64, 100, 128, 129, 300, 10000])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)], ids=["bf16-128", "bf16-64", "f32-64"])
def test_windows(cuda, window, dtype, d):
    P.compare(cuda, [400, 37, 129], 4, 2, d, dtype, seed=window, window=window)


@pytest.mark.parametrize("softcap,size", [(30.0, 1.0), (2.0, 1.5), (0.5, 1.0), (50.0, 4.0)])
@pytest.mark.parametrize("dtype,d,window", [(BF, 128, 0), (BF, 64, 90), (F32, 32, 0)])
def test_capped_scores(cuda, softcap, size, dtype, d, window):
    P.compare(cuda, [260, 41], 4, 2, d, dtype, seed=5, softcap=softcap, size=size, window=window)


@pytest.mark.parametrize("scale", [1.0, -0.2, 0.0, 0.01])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("softcap,window", [(0.0, 0), (4.0, 70)])
def test_scales(cuda, scale, dtype, softcap, window):
    P.compare(cuda, [200], 2, 1, 64, dtype, seed=2, scale=scale, softcap=softcap, window=window)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,heads", [(128, (8, 8)), (64, (6, 2)), (16, (12, 1))], ids=str)
@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_a_query_that_sees_one_key_has_no_gradient(cuda, dtype, d, heads, softcap):
    """A softmax over one key is 1 whatever the scores are: dq and what dk has of such a query are zero, exactly."""
    for lengths, window in (([1], 0), ([1, 0, 1, 1], 0), ([1], 1000), ([300, 41, 1], 1)):
        q, k, v, d_out = P.inputs(sum(lengths), *heads, d, dtype, 51, size=3.0)
        got = P.run(cuda, q, k, v, P.cu(lengths), max(lengths), d_out, softcap=softcap, window=window)
        assert not got["dq"].any() and not got["dk"].any(), (lengths, window)
    lengths = [200, 130]
    q, k, v, d_out = P.inputs(330, *heads, d, dtype, 52)
    got = P.run(cuda, q, k, v, P.cu(lengths), 200, d_out, softcap=softcap)
    assert not got["dq"][[0, 200]].any() and got["dq"][[1, 201]].any()


@pytest.mark.parametrize("d,heads", [(128, (8, 8)), (64, (12, 1)), (32, (6, 2))], ids=str)
@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("lengths", [[2], [1, 2], [39], [128], [127, 300, 5]], ids=str)
def test_gradients_of_short_sequences_keep_their_bits(cuda, d, heads, softcap, lengths):
    """Sequences of up to 128 tokens, bf16: p and dx as two bf16 are off by 2^-16, the scores' fp32 products by d 2^-24 of their magnitudes (a few,
    so 2^-14): 2^-12 of the results' size, where one bf16 would leave 2^-9.  Gradients in fp32, so that no rounding of theirs covers it."""
    q, k, v, d_out = P.inputs(sum(lengths), *heads, d, BF, 53)
    got = P.run(cuda, q, k, v, P.cu(lengths), max(lengths), d_out, out_type=F32, grad_type=F32, softcap=softcap)
    want = P.attention(q, k, v, d_out, lengths, softcap=softcap)
    at = 0
    for n in lengths:
        rows = slice(at, at + n)
        at += n
        for name in ("dq", "dk", "dv") if n > 1 else ("dv",):
            value = want[name][0][rows]
            if n <= 128 or name == "dq":
                ratio = ((got[name][rows].double() - value).norm() / value.norm()).item()
                assert ratio <= 2.0 ** -12, (name, n, ratio)


@pytest.mark.parametrize("tokens,heads", [(7700, (12, 1)), (4100, (13, 1)), (1000, (34, 2)), (9900, (10, 2))], ids=str)
def test_shared_heads_dealt_to_several_blocks(cuda, tokens, heads):
    # 5 of 12 heads' parts, 9 of 13, 16 of 17, 1 of 5: uneven shares too
    lengths = [tokens // 30 + (i % 3) * 7 - 7 for i in range(30)]
    P.compare(cuda, lengths, *heads, 32, BF, seed=tokens)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 16), (F32, 32)])
def test_results_and_gradients_in_columns_of_larger_buffers(cuda, dtype, d):
    T, Hq, Hkv = 190, 4, 2
    q, k, v, d_out = P.inputs(T, Hq, Hkv, d, dtype, 24)
    offsets = P.cu([150, 40])
    want = P.run(cuda, q, k, v, offsets, 150, d_out)
    wide = torch.full((T, 3 * Hq + 2 * Hkv + 1, d), 7.0, device="cuda").to(dtype)
    out, dq, dk, dv = wide[:, 1:1 + Hq], wide[:, 5:5 + Hq], wide[:, 10:10 + Hkv], wide[:, 12:12 + Hkv]
    grad = torch.full((T, Hq + 3, d), 9.0, device="cuda").to(dtype)
    grad[:, 2:2 + Hq] = d_out
    lse = torch.empty(T, Hq, device="cuda")
    ws = torch.empty(cuda.kda_prefill_attention_backward_workspace_size(T, 2, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    cuda.kda_prefill_attention(q, k, v, offsets, 150, out, lse=lse)
    cuda.kda_prefill_attention_backward(grad[:, 2:2 + Hq], q, k, v, out, lse, offsets, 150, dq, dk, dv, ws)
    for n, x in zip(("out", "dq", "dk", "dv"), (out, dq, dk, dv)):
        assert torch.equal(x, want[n]), n
    assert (wide[:, [0, 9, 14, 15, 16]] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_offsets_beyond_32_bits(cuda, dtype):
    """The last sequence of a batch whose elements number more than 2^31 gives what it gives alone."""
    T, Hq, Hkv, d, n = 700001, 16, 4, 128, 300
    rows = torch.empty(T, Hq + 2 * Hkv, d, dtype=dtype, device="cuda")
    rows[:2 * n].normal_()
    rows[-2 * n:].normal_()
    assert rows.numel() > 2 ** 31
    d_out, out, dq = (torch.empty(T, Hq, d, dtype=dtype, device="cuda") for _ in range(3))
    d_out[-n:].normal_()
    dk, dv = (torch.empty(T, Hkv, d, dtype=dtype, device="cuda") for _ in range(2))
    lse = torch.empty(T, Hq, device="cuda")
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    offsets = P.cu([n], T - n)
    ws = torch.empty(cuda.kda_prefill_attention_backward_workspace_size(T, 1, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    cuda.kda_prefill_attention(q, k, v, offsets, n, out, lse=lse)
    cuda.kda_prefill_attention_backward(d_out, q, k, v, out, lse, offsets, n, dq, dk, dv, ws)
    at = slice(T - n, T)
    # the alone call is of so few rows that its sums come in parts: all in fp32, dk and dv in bf16
    alone = P.run(cuda, q[at], k[at], v[at], P.cu([n]), n, d_out[at])
    for name, x in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, dq, dk, dv)):
        if dtype == F32 or name in ("dk", "dv"):
            ratio = ((x[at].double() - alone[name].double()).norm() / alone[name].double().norm()).item()
            assert ratio <= (2 ** -8 if dtype == BF else 2 ** -20), name
        else:
            assert torch.equal(x[at], alone[name]), name


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_calls_on_two_streams_at_once(cuda, dtype, d):
    sets = [P.inputs(900, 8, 2, d, dtype, 30 + i) for i in range(2)]
    offsets = P.cu([500, 400])
    want = [P.run(cuda, *s[:3], offsets, 500, s[3]) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, (s, stream) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(stream):
                got[i].append(P.run(cuda, *s[:3], offsets, 500, s[3]))
    torch.cuda.synchronize()
    for i in range(2):
        for res in got[i]:
            for n in res:
                assert torch.equal(res[n], want[i][n]), n


@pytest.mark.parametrize("dtype,out_type,grad_type", [(BF, F32, F32), (BF, BF, F32), (F32, BF, BF), (BF, F32, BF)])
@pytest.mark.parametrize("d", [32, 128])
def test_types_of_the_results(cuda, dtype, out_type, grad_type, d):
    P.compare(cuda, [130, 61], 4, 2, d, dtype, seed=3, out_type=out_type, grad_type=grad_type)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("start,tail", [(1, 0), (0, 1), (130, 77), (5, 300)])
def test_rows_outside_the_sequences_are_left_alone(cuda, dtype, start, tail):
    # they hold NaN in every input and are not written
    P.compare(cuda, [129, 0, 64], 4, 2, 128, dtype, start=start, tail=tail, packed=True)
    P.compare(cuda, [3], 2, 2, 64, dtype, start=start, tail=tail)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_large_scores(cuda, dtype):
    # one key takes nearly everything, references move by hundreds of powers of two
    P.compare(cuda, [300, 150], 2, 1, 128, dtype, seed=9, size=5.0)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_many_sequences(cuda, dtype, d):
    lengths = [(7 * i * i + 3) % 97 for i in range(200)] + [0, 0, 900] + [1] * 40
    P.compare(cuda, lengths, 2, 1, d, dtype, seed=4)


@pytest.mark.parametrize("dtype,d,heads", [(BF, 128, (2, 1)), (BF, 64, (3, 3)), (F32, 64, (2, 1))])
@pytest.mark.parametrize("n", [256, 257, 1500])
def test_more_sequences_than_a_warp_keeps(cuda, dtype, d, heads, n):
    lengths = [(5 * i * i + 1) % 23 for i in range(n - 2)] + [200, 131]
    P.compare(cuda, lengths, *heads, d, dtype, seed=n, start=3, tail=9)


@pytest.mark.parametrize("softcap", [1e-25, 1e-12, 1e12, 1e35])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 32), (F32, 64)])
def test_caps_of_any_size(cuda, softcap, dtype, d):
    """A tiny cap leaves equal scores and no gradient of them; a huge one is none."""
    q, k, v, d_out = P.inputs(150, 2, 1, d, dtype, 22)
    got = P.run(cuda, q, k, v, P.cu([150]), 150, d_out, softcap=softcap)
    if softcap > 1:
        want = P.attention(q, k, v, d_out, [150])
    else:
        want = P.attention(q, k, v, d_out, [150], scale=0.0)
    for n, (value, bound) in want.items():
        # |x| is at most 1e-12 of a score's 1 here, and the slope's: both far below the bounds' 2^-21 of P's
        slack = 1e-9 * (d_out.abs().sum().double() if n in ("dq", "dk") else 1)
        assert ((got[n].double() - value).abs() <= bound + slack).all(), n


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_offsets_out_of_order_are_flagged(cuda, dtype, d):
    # which rows are written is not defined, that the call returns and says so is
    q, k, v, d_out = P.inputs(340, 4, 2, d, dtype, 23)
    for offsets in ([0, 200, 100, 340], [340, 0], [0, 50, 20, 20, 300, 299, 340] + [5, 340] * 200):
        status = torch.zeros(2, dtype=torch.int32, device="cuda")
        P.run(cuda, q, k, v, torch.tensor(offsets, dtype=torch.int32, device="cuda"), 340, d_out, dev_status=status)
        assert status[0].item() == cuda.KDA_DEV_SEQ_OOB


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_offsets_out_of_order_write_only_the_batch(cuda, dtype, d):
    T, Hq, Hkv, guard = 340, 4, 2, 512
    q, k, v, d_out = P.inputs(T, Hq, Hkv, d, dtype, 24)
    at = slice(guard, guard + T)

    def inside(x):  # a copy between rows of ones
        y = torch.ones(T + 2 * guard, *x.shape[1:], dtype=x.dtype, device="cuda")
        y[at] = x
        return y[at]
    q, k, v, d_out = map(inside, (q, k, v, d_out))
    rng = torch.Generator().manual_seed(25)
    for offsets in ([0, 50, 20, 20, 300, 299, 340] + [5, 340] * 200, torch.randint(-3, 345, (300,), generator=rng).tolist(),
                    torch.randint(-3, 345, (200,), generator=rng).tolist()):
        N = len(offsets) - 1
        bufs = [torch.full((T + 2 * guard, h, d), 7.0, dtype=dtype, device="cuda") for h in (Hq, Hq, Hkv, Hkv)]
        lse = torch.full((T + 2 * guard, Hq), 7.0, device="cuda")
        out, dq, dk, dv = (b[at] for b in bufs)
        size = cuda.kda_prefill_attention_backward_workspace_size(T, N, Hq, Hkv, d)
        ws = torch.full((size + 2 * (1 << 20),), 7, dtype=torch.uint8, device="cuda")
        cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        cuda.kda_prefill_attention(q, k, v, cu, T, out, lse=lse[at])
        cuda.kda_prefill_attention_backward(d_out, q, k, v, out, lse[at], cu, T, dq, dk, dv, ws[1 << 20:(1 << 20) + size])
        for b in (*bufs, lse):
            assert (b[:guard] == 7.0).all() and (b[guard + T:] == 7.0).all()
        assert (ws[:1 << 20] == 7).all() and (ws[(1 << 20) + size:] == 7).all()


@pytest.mark.parametrize("dtype,d,heads", [(BF, 128, (4, 1)), (BF, 64, (3, 3)), (F32, 32, (2, 2))])
@pytest.mark.parametrize("window", [0, 700])
def test_longer_prompts(cuda, dtype, d, heads, window):
    P.compare(cuda, [2500, 1100], *heads, d, dtype, seed=6, window=window)


@pytest.mark.parametrize("dtype,d,heads,softcap,window", [(BF, 128, (2, 1), 0.0, 0), (BF, 128, (1, 1), 30.0, 3000), (BF, 64, (3, 3), 30.0, 0),
                                                          (BF, 16, (2, 1), 0.0, 1000), (F32, 64, (2, 1), 0.0, 0), (F32, 128, (1, 1), 30.0, 3000)])
def test_prompts_of_thousands_of_tokens(cuda, dtype, d, heads, softcap, window):
    P.compare(cuda, [9001, 5000], *heads, d, dtype, seed=50, softcap=softcap, window=window)


@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("window", [0, 100])
def test_many_heads_in_fp32(cuda, d, window):
    """So many rows' blocks that each has one CTA, and so few keys' that each has several."""
    P.compare(cuda, [300, 200], 64, 8, d, F32, seed=8, window=window)


def test_nothing_to_do(cuda):
    e = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    cuda.kda_prefill_attention(e(0, 2, 16), e(0, 1, 16), e(0, 1, 16), P.cu([0, 0]), 0, e(0, 2, 16))
    out = torch.full((4, 2, 16), 7.0, device="cuda")
    cuda.kda_prefill_attention(e(4, 2, 16), e(4, 1, 16), e(4, 1, 16), P.cu([]), 4, out)
    cuda.kda_prefill_attention(e(4, 2, 16), e(4, 1, 16), e(4, 1, 16), P.cu([0, 0, 0]), 4, out)
    assert (out == 7.0).all()


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("window", [0, 50])
def test_what_a_row_does_not_see_does_not_matter(cuda, dtype, d, value, window):
    """Values that are no numbers at some tokens: rows that do not see them are as without, the others are no numbers
    in those channels alone (values), or anywhere (keys)."""
    lengths, where = [150, 200], [40, 149, 150 + 60, 150 + 129]
    T = sum(lengths)
    q, k, v, _ = P.inputs(T, 4, 2, d, dtype, 8)
    seq = torch.tensor([0] * 150 + [1] * 200, device="cuda")
    pos = torch.cat([torch.arange(n, device="cuda") for n in lengths])
    sees = torch.zeros(T, dtype=torch.bool, device="cuda")
    for w in where:
        hit = (seq == seq[w]) & (pos >= pos[w])
        if window:
            hit &= pos < pos[w] + window
        sees |= hit
    args = (P.cu(lengths), 200)
    clean = P.run(cuda, q, k, v, *args, window=window)
    v2 = v.clone()
    v2[where, :, 3] = value
    got = P.run(cuda, q, k, v2, *args, window=window)
    assert torch.equal(got["out"][~sees], clean["out"][~sees]) and torch.equal(got["lse"], clean["lse"])
    others = [c for c in range(d) if c != 3]
    assert torch.equal(got["out"][..., others], clean["out"][..., others])
    assert not torch.isfinite(got["out"][sees][..., 3]).any()
    k2 = k.clone()
    k2[where] = math.nan
    got = P.run(cuda, q, k2, v, *args, window=window)
    assert torch.equal(got["out"][~sees], clean["out"][~sees]) and torch.equal(got["lse"][~sees], clean["lse"][~sees])
    assert torch.isnan(got["out"][sees]).all() and torch.isnan(got["lse"][sees]).all()


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_a_gradient_stays_within_its_sequence(cuda, dtype, d):
    lengths = [70, 130, 90]
    q, k, v, d_out = P.inputs(290, 4, 2, d, dtype, 11)
    clean = P.run(cuda, q, k, v, P.cu(lengths), 130, d_out)
    for x in (q, k, v, d_out):
        x[100] = math.nan
    got = P.run(cuda, q, k, v, P.cu(lengths), 130, d_out)
    others = torch.ones(290, dtype=torch.bool, device="cuda")
    others[70:200] = False
    for n in got:
        assert torch.equal(got[n][others], clean[n][others]), n


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 32), (F32, 64)])
def test_the_same_call_gives_the_same_bits(cuda, dtype, d):
    lengths = [777, 5, 300]
    q, k, v, d_out = P.inputs(sum(lengths), 6, 2, d, dtype, 12)
    a = P.run(cuda, q, k, v, P.cu(lengths), 777, d_out)
    b = P.run(cuda, q, k, v, P.cu(lengths), 777, d_out)
    # and the batch around a sequence changes nothing
    at = slice(777, 782)
    alone = P.run(cuda, q[at], k[at], v[at], P.cu([5]), 5, d_out[at])
    for n in a:
        assert torch.equal(a[n], b[n]), n
        assert torch.equal(a[n][at], alone[n]), n


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_captured_and_on_another_stream(cuda, dtype, d):
    lengths = [140, 33]
    q, k, v, d_out = P.inputs(173, 4, 2, d, dtype, 13)
    want = P.run(cuda, q, k, v, P.cu(lengths), 140, d_out)
    offsets = P.cu(lengths)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = P.run(cuda, q, k, v, offsets, 140, d_out)
    torch.cuda.current_stream().wait_stream(side)
    for n in want:
        assert torch.equal(want[n], got[n]), n
    out, lse = torch.zeros_like(want["out"]), torch.zeros_like(want["lse"])
    grads = [torch.zeros_like(want[n]) for n in ("dq", "dk", "dv")]
    ws = torch.empty(cuda.kda_prefill_attention_backward_workspace_size(173, 2, 4, 2, d), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda.kda_prefill_attention(q, k, v, offsets, 140, out, lse=lse)
        cuda.kda_prefill_attention_backward(d_out, q, k, v, out, lse, offsets, 140, *grads, ws)
    for fresh in range(2):
        if fresh:  # other tokens, cut elsewhere
            new = P.inputs(173, 4, 2, d, dtype, 14)
            for x, y in zip((q, k, v, d_out), new):
                x.copy_(y)
            offsets.copy_(P.cu([20, 140]))
            want = P.run(cuda, q, k, v, offsets, 140, d_out)
        ws.fill_(255)
        graph.replay()
        rows = slice(0, 160 if fresh else 173)
        for n, x in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
            assert torch.equal(want[n][rows], x[rows]), n


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("offsets,longest,written", [([0, 100, 300, 340], 150, [(0, 100), (300, 340)]),
                                                     ([0, 100, 341], 400, [(0, 100)]),
                                                     ([-1, 100, 340], 400, [(100, 340)])])
def test_offsets_out_of_range_are_flagged(cuda, dtype, d, offsets, longest, written):
    q, k, v, d_out = P.inputs(340, 4, 2, d, dtype, 15)
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    at = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    got = P.run(cuda, q, k, v, at, longest, d_out, dev_status=status)
    assert status[0].item() == cuda.KDA_DEV_SEQ_OOB
    rows = torch.zeros(340, dtype=torch.bool, device="cuda")
    for a, b in written:
        rows[a:b] = True
        alone = P.run(cuda, q[a:b], k[a:b], v[a:b], P.cu([b - a]), b - a, d_out[a:b])
        for n in got:
            assert torch.equal(got[n][a:b], alone[n]), n
    for n in got:
        assert (got[n][~rows] == 7.0).all(), n


def test_work_is_counted(cuda):
    for dtype in (BF, F32):
        q, k, v, d_out = P.inputs(200, 6, 2, 64, dtype, 16)
        status = torch.zeros(2, dtype=torch.int32, device="cuda")
        P.run(cuda, q, k, v, P.cu([120, 50]), 120, dev_status=status)
        assert status.tolist() == [0, 170 * 6]
        P.run(cuda, q, k, v, P.cu([120, 50]), 120, d_out, dev_status=status)
        assert status.tolist() == [0, 3 * 170 * 6]


@pytest.mark.parametrize("softcap,window", [(0.0, 0), (3.0, 0), (0.0, 17)])
def test_gradients_against_differences(cuda, softcap, window):
    """Along a random direction: the fp32 loss's central difference and the gradient's product with the direction.  The
    loss sums 50 x 3 x 32 outputs of size 1 in fp64 from fp32 rows (2^-22 relative each), the step is 2^-7: noise
    sqrt(4800) 2^-22 / 2^-7 < 0.003 and a third-order term of 2^-14 times the third derivative (within 50 here)."""
    lengths = [40, 10]
    q, k, v, d_out = P.inputs(50, 3, 1, 32, F32, 17)
    got = P.run(cuda, q, k, v, P.cu(lengths), 40, d_out, softcap=softcap, window=window)

    def loss(*x):
        return (P.run(cuda, *x, P.cu(lengths), 40, softcap=softcap, window=window)["out"].double() * d_out.double()).sum().item()

    g = torch.Generator(device="cuda").manual_seed(18)
    for i, name in enumerate(("dq", "dk", "dv")):
        x = [q, k, v]
        step = torch.randn(x[i].shape, generator=g, device="cuda")
        step /= step.norm()
        h = 2.0 ** -7
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + h * step, x[i] - h * step
        slope = (loss(*up) - loss(*down)) / (2 * h)
        want = (got[name].double() * step.double()).sum().item()
        assert abs(slope - want) <= 0.01, (name, slope, want)


def test_a_layer_trained(cuda):
    """The norm with rotation, the attention and both gradients in one chain over a fused projection's columns, fp32: the chain's
    gradient along a random direction of the projection and of the norm's weights against the loss's central difference.  Noise and
    third-order term as in the test above, with the norm's curvature (rows of length near sqrt(32), steps of 2^-7)."""
    T, Hq, Hkv, d, eps = 60, 4, 2, 32, 1e-6
    lengths = [45, 15]
    offsets = P.cu(lengths)
    g = torch.Generator(device="cuda").manual_seed(21)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rows, d_out, wq, wk = r(T, Hq + 2 * Hkv, d), r(T, Hq, d), 1 + 0.1 * r(d), 1 + 0.1 * r(d)
    angle = torch.arange(45, device="cuda")[:, None] * 100.0 ** (-torch.arange(d // 2, device="cuda") / (d // 2))
    pos = torch.cat([torch.arange(n, device="cuda") for n in lengths]).int()
    rope = dict(cos=angle.cos().contiguous(), sin=angle.sin().contiguous(), positions=pos, eps=eps)
    cut = lambda x: (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:])  # noqa: E731

    def forward(rows, wq, wk):
        q, k, v = cut(rows)
        yq, yk = torch.empty(T, Hq, d, device="cuda"), torch.empty(T, Hkv, d, device="cuda")
        cuda.kda_qk_norm_rope(q, k, wq, wk, yq, yk, **rope)
        out, lse = torch.empty(T, Hq, d, device="cuda"), torch.empty(T, Hq, device="cuda")
        cuda.kda_prefill_attention(yq, yk, v, offsets, 45, out, lse=lse)
        return yq, yk, out, lse

    yq, yk, out, lse = forward(rows, wq, wk)
    grads = torch.empty_like(rows)
    dq, dk, dv = cut(grads)
    gq, gk = torch.empty_like(yq), torch.empty_like(yk)
    ws = torch.empty(cuda.kda_prefill_attention_backward_workspace_size(T, 2, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    cuda.kda_prefill_attention_backward(d_out, yq, yk, cut(rows)[2], out, lse, offsets, 45, gq, gk, dv, ws)
    dw = torch.empty(2, d, device="cuda")
    ws = torch.empty(cuda.kda_qk_norm_rope_backward_workspace_size(T, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    cuda.kda_qk_norm_rope_backward(gq, gk, *cut(rows)[:2], wq, wk, dq, dk, dw[0], dw[1], ws, **rope)
    loss = lambda *x: (forward(*x)[2].double() * d_out.double()).sum().item()  # noqa: E731
    for i, grad in enumerate((grads, dw[0], dw[1])):
        x = [rows, wq, wk]
        step = r(*x[i].shape)
        step /= step.norm()
        h = 2.0 ** -7
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + h * step, x[i] - h * step
        slope, want = (loss(*up) - loss(*down)) / (2 * h), (grad.double() * step.double()).sum().item()
        assert abs(slope - want) <= 0.02, (i, slope, want)
