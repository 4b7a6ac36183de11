"""Acceptance of drafts against the definition in exact arithmetic (Python's fractions for the sums that decide, fp64 where they
cannot tie)."""
from fractions import Fraction

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def make(B, W, V, dtype, proposal, seed, spread=2.0, near=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = spread * torch.randn(B, W, V, generator=g, device="cuda")
    target = torch.softmax(logits, -1).to(dtype)
    guess = torch.softmax(logits[:, :W - 1] + near * torch.randn(B, W - 1, V, generator=g, device="cuda"), -1).to(dtype)
    source = (guess if proposal else target[:, :W - 1]).float().reshape(-1, V)
    drafts = torch.multinomial(source, 1, generator=g).view(B, W - 1).to(I32) if W > 1 else torch.zeros(B, 0, dtype=I32, device="cuda")
    uniform = torch.rand(B, W, generator=g, device="cuda")
    return target, guess if proposal else None, drafts, uniform


def call(kda, target, guess, drafts, uniform, num=None, status=None):
    B, W, _ = target.shape
    accepted, tokens = torch.full((B,), 77, dtype=I32, device="cuda"), torch.full((B, W), 77, dtype=I32, device="cuda")
    kda.kda_verify_accept(target, drafts, uniform, accepted, tokens, draft_probs=guess, num_drafts=num, dev_status=status)
    return accepted.tolist(), tokens.tolist()


def expected(target, guess, drafts, uniform, num=None):
    """By the definition, in rational numbers."""
    B, W, V = target.shape
    p, q = target.cpu().double().tolist(), guess.cpu().double().tolist() if guess is not None else None
    u, x = uniform.cpu().double().tolist(), drafts.tolist()
    accepted, tokens = [], []
    for b in range(B):
        have = W - 1 if num is None else num[b]
        n = 0
        while n < have and Fraction(u[b][n]) * Fraction(q[b][n][x[b][n]] if q else 1) < Fraction(p[b][n][x[b][n]]):
            n += 1
        full = [Fraction(c) for c in p[b][n]]
        w = full
        if n < have:
            w = [max(c - Fraction(e), Fraction(0)) for c, e in zip(full, q[b][n])] if q else \
                [c if v != x[b][n] else Fraction(0) for v, c in enumerate(full)]
            if not any(w):
                w = full
        limit, upto = Fraction(u[b][W - 1]) * sum(w), Fraction(0)
        for v, c in enumerate(w):
            upto += c
            if upto > limit:
                break
        accepted.append(n + 1)
        tokens.append(x[b][:n] + [v] + [-1] * (W - 1 - n))
    return accepted, tokens


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("proposal", [True, False], ids=["drawn", "certain"])
@pytest.mark.parametrize("B,W,V", [(1, 1, 1), (3, 2, 1), (5, 4, 2), (2, 5, 31), (40, 3, 129), (3, 9, 513), (2, 35, 64), (1, 2, 8191),
                                   (200, 2, 33), (700, 2, 17)])
def test_small_vocabularies_exactly(cuda, B, W, V, dtype, proposal):
    data = make(B, W, V, dtype, proposal, seed=B + W + V)
    assert call(cuda, *data) == expected(*data)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,W,V", [(1, 4, 32768), (70, 3, 50001), (3, 2, 262144), (330, 2, 4097)])
def test_large_vocabularies(cuda, B, W, V, dtype):
    """fp64 sums: the threshold is nearer than 1e-9 to a token's border in none of these draws."""
    target, guess, drafts, uniform = make(B, W, V, dtype, True, seed=V)
    accepted, tokens = call(cuda, target, guess, drafts, uniform)
    for b in range(B):
        n = accepted[b] - 1
        p = target[b, :W - 1].gather(1, drafts[b, :, None].long())[:, 0].double()
        q = guess[b].gather(1, drafts[b, :, None].long())[:, 0].double()
        ok = (uniform[b, :W - 1].double() * q < p).tolist() + [False]
        assert n == ok.index(False)
        w = target[b, n].double()
        if n < W - 1:
            w = (w - guess[b, n].double()).clamp(min=0)
        upto = w.cumsum(0)
        limit = uniform[b, W - 1].double() * upto[-1]
        v = int((upto <= limit).sum())
        near = min(abs(float(upto[i] - limit)) for i in (max(v - 1, 0), v))
        assert near > 1e-9 * float(upto[-1]) and tokens[b] == drafts[b, :n].tolist() + [v] + [-1] * (W - 1 - n)


def test_certain_drafts_from_the_target_itself_are_accepted(cuda):
    target, _, drafts, uniform = make(6, 5, 300, F32, False, 1)
    accepted, tokens = call(cuda, target, target[:, :4].contiguous(), drafts, uniform)
    assert accepted == [5] * 6 and [t[:4] for t in tokens] == drafts.tolist()


def test_nothing_left_of_the_target(cuda):
    # p = 0 at the draft, and p <= q elsewhere: the draw is from p
    p = torch.tensor([[[0.0, 0.25, 0.25], [1.0, 0.0, 0.0]]], device="cuda")
    q = torch.tensor([[[0.25, 0.5, 0.25]]], device="cuda")
    x = torch.zeros(1, 1, dtype=I32, device="cuda")
    for r, v in ((0.0, 1), (0.49, 1), (0.5, 2), (0.99, 2)):
        assert call(cuda, p, q, x, torch.tensor([[0.3, r]], device="cuda")) == ([1], [[v, -1]])


@pytest.mark.parametrize("proposal", [True, False])
def test_fewer_drafts(cuda, proposal):
    target, guess, drafts, uniform = make(6, 4, 50, F32, proposal, 2, near=0.1)
    num = [0, 1, 2, 3, 1, 0]
    drafts[0] = -5  # not read
    drafts[1, 1:] = 1 << 30
    device_num = torch.tensor(num, dtype=I32, device="cuda")
    assert call(cuda, target, guess, drafts, uniform, device_num) == expected(target, guess, drafts, uniform, num)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [0.01, 3.0, 25.0])
def test_rows_that_are_not_normalised(cuda, dtype, size):
    target, guess, drafts, uniform = make(30, 3, 60, F32, True, 8, spread=4.0)
    target, guess = (size * target).to(dtype), (size * 0.9 * guess).to(dtype)
    assert call(cuda, target, guess, drafts, uniform) == expected(target, guess, drafts, uniform)


def test_flags(cuda):
    target, guess, drafts, uniform = make(8, 3, 40, F32, True, 3)
    uniform[:, :2] = 0.0  # every draft with weight is accepted
    num = torch.tensor([2, 2, -1, 3, 2, 2, 2, 2], dtype=I32, device="cuda")
    drafts[0, 0], drafts[1, 1] = 40, -1
    target[4, 2] = 0.0
    target[5, 2] = 2.0  # sums to 80
    target[6, 2, 7], target[6, 2, 8] = float("nan"), -1.0
    target[7, 2] = float("inf")
    status = torch.zeros(2, dtype=I32, device="cuda")
    accepted, tokens = call(cuda, target, guess, drafts, uniform, num, status)
    assert status[0].item() == cuda.KDA_DEV_TOKEN_OOB | cuda.KDA_DEV_ACCEPT_OOB | cuda.KDA_DEV_PROB_OOB
    assert accepted == [1, 2, 1, 1, 3, 3, 3, 3] and status[1].item() == sum(accepted)
    x = drafts.tolist()

    def draw(b, n):
        w = target[b, n].double().nan_to_num(0.0).clamp(min=0)
        return int((w.cumsum(0) <= uniform[b, 2].double() * w.sum()).sum())

    assert tokens[0] == [draw(0, 0), -1, -1] and tokens[1] == [x[1][0], draw(1, 1), -1]
    assert tokens[2] == [draw(2, 0), -1, -1] and tokens[3] == [draw(3, 0), -1, -1]
    assert tokens[4] == x[4] + [-1] and tokens[5] == x[5] + [-1] and tokens[6] == x[6] + [draw(6, 2)]
    assert tokens[7] == x[7] + [-1]


@pytest.mark.parametrize("r,v", [(0.0, 3), (1.0, 7), (2.0, 7), (-1.0, 3), (float("nan"), 3)])
def test_random_numbers_outside_the_range(cuda, r, v):
    p = torch.zeros(1, 1, 9, device="cuda")
    p[0, 0, 3], p[0, 0, 7] = 0.5, 0.5
    assert call(cuda, p, None, torch.zeros(1, 0, dtype=I32, device="cuda"), torch.tensor([[r]], device="cuda")) == ([1], [[v]])


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("p,q,u,taken", [(0.0, -1.0, 0.5, False), (-0.25, -1.0, 0.5, False), (0.25, NAN, 0.5, True), (NAN, 0.25, 0.5, False),
                                         (NAN, NAN, 0.5, False), (-0.25, 0.25, -2.0, False), (0.0, 0.5, -0.5, False), (0.25, 0.5, -0.5, True),
                                         (0.25, 0.25, 1.0, True), (0.25, 0.5, 1.0, False), (0.25, 0.25, 2.0, True), (0.25, 0.5, 2.0, False),
                                         (0.25, 0.0, INF, True), (0.25, 0.5, NAN, True), (0.0, 0.5, NAN, False),
                                         (0.0, None, -1.0, False), (1.0, None, 1.0, True), (0.5, None, NAN, True), (0.0, None, NAN, False)])
def test_values_outside_their_range_at_a_draft(cuda, dtype, p, q, u, taken):
    """Probabilities that are negative or NaN count as zero and random numbers as the nearest in [0, 1), NaN as 0, in the
    test of a draft as in the draw."""
    W, V, at = 3, 600, 300
    target, guess = torch.full((2, W, V), 0.0625, device="cuda"), torch.full((2, W - 1, V), 0.0625, device="cuda")
    target[:, :, 10:] = 0.0
    target[:, 1, at], guess[:, 1, at] = p, 0.5 if q is None else q
    drafts = torch.tensor([[3, at]] * 2, dtype=I32, device="cuda")
    uniform = torch.tensor([[0.0, u, 0.0]] * 2, device="cuda")
    accepted, tokens = call(cuda, target.to(dtype), None if q is None else guess.to(dtype), drafts, uniform)
    assert accepted == [3 if taken else 2] * 2
    assert [t[:2] for t in tokens] == [[3, at] if taken else [3, tokens[0][1]]] * 2 and (taken or tokens[0][2] == -1)


def pieces(x):
    """Fractions that fp32 holds, with the sum x."""
    out = []
    while x:
        e = 0
        while x * 2 ** e < 2 ** 23:
            e += 1
        while x * Fraction(2) ** e >= 2 ** 24:
            e -= 1
        out.append(Fraction(int(x * Fraction(2) ** e)) / Fraction(2) ** e)
        x -= out[-1]
    return out


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("p,q", [(1.37 * 2.0 ** -20, 2.0 ** -34 + 2.0 ** -57), (1.37 * 2.0 ** -20, 2.0 ** -34 - 2.0 ** -58),
                                 (0.0624, 2.0 ** -34 + 2.0 ** -57), (0.137, 2.0 ** -34 + 2.0 ** -57), (0.137, 2.0 ** -34 - 2.0 ** -58),
                                 (0.9, 2.0 ** -33 - 2.0 ** -57), (2.5, 2.0 ** -34 + 2.0 ** -57), (1.1 * 2.0 ** -30, 2.0 ** -36 + 2.0 ** -59)])
def test_differences_keep_what_fp32_cannot_hold(cuda, p, q, first):
    """A token of weight p - q against others that weigh the same together, all multiples of 2^-59: half of the sum is exactly where
    the one ends and the others begin, so one unit more or less of any would move the token."""
    f32 = lambda x: Fraction(float(torch.tensor(x, dtype=F32)))  # noqa: E731
    p, q = f32(p), f32(q)
    rest = pieces(p - q)
    assert len(rest) > 1 and (p - q) * 2 ** 59 % 1 == 0
    row, guess = ([p] + rest, [q] + [0] * len(rest)) if first else (rest + [p], [0] * len(rest) + [q])
    target = torch.zeros(1, 2, 300, device="cuda")
    proposal = torch.zeros(1, 1, 300, device="cuda")
    target[0, 0, 7:7 + len(row)] = torch.tensor([float(x) for x in row], device="cuda")
    proposal[0, 0, 7:7 + len(row)] = torch.tensor([float(x) for x in guess], device="cuda")
    proposal[0, 0, 299] = 0.5  # the draft, refused
    target[0, 1, 0] = 1.0
    data = target, proposal, torch.tensor([[299]], dtype=I32, device="cuda"), torch.tensor([[0.5, 0.5]], device="cuda")
    want = expected(*data)
    assert want[1][0][0] == (8 if first else 7 + len(rest))
    assert call(cuda, *data) == want


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("q", [2.0, 31.5, 32.0, 40.0, 1e10, 3e38, INF])
@pytest.mark.parametrize("p", [0.5, 1.0, 3.0, 20.0])
def test_proposals_far_from_normalised(cuda, dtype, p, q):
    # whatever the proposal holds too much of, its tokens weigh nothing
    target, guess = torch.full((3, 2, 500), 0.0078125, device="cuda"), torch.full((3, 1, 500), 0.00390625, device="cuda")
    target[:, 0, [5, 70, 400]] = p if p < 10 else p / 4
    guess[:, 0, [5, 70, 400]] = q
    drafts = torch.tensor([[5]] * 3, dtype=I32, device="cuda")
    target[:, 0, 5] = 0.0  # refused
    uniform = torch.tensor([[0.5, 0.01], [0.5, 0.2], [0.5, 0.99]], device="cuda")
    target, guess = target.to(dtype), guess.to(dtype)
    assert call(cuda, target, guess, drafts, uniform) == expected(target, guess.clamp(max=1e30), drafts, uniform)


def test_the_draw_has_the_target_distribution(cuda):
    """Drafts from q, 40000 windows of one draft: token counts against p.  A count's standard deviation is at most
    sqrt(40000 / 4) = 100; five of them."""
    n, V = 40000, 6
    g = torch.Generator(device="cuda").manual_seed(4)
    p = torch.tensor([0.3, 0.05, 0.2, 0.25, 0.0, 0.2], device="cuda")
    q = torch.tensor([0.1, 0.4, 0.2, 0.1, 0.1, 0.1], device="cuda")
    drafts = torch.multinomial(q.expand(n, V), 1, generator=g).to(I32)
    uniform = torch.rand(n, 2, generator=g, device="cuda")
    _, tokens = call(cuda, p.expand(n, 2, V).contiguous(), q.expand(n, 1, V).contiguous(), drafts, uniform)
    counts = torch.bincount(torch.tensor(tokens)[:, 0], minlength=V)
    assert ((counts - n * p.cpu()).abs() <= 500).all() and counts[4] == 0


def test_captured_and_on_another_stream(cuda):
    data = make(9, 4, 1000, F32, True, 5)
    want = call(cuda, *data)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert call(cuda, *data) == want
    target, guess, drafts, uniform = data
    accepted, tokens = torch.zeros(9, dtype=I32, device="cuda"), torch.zeros(9, 4, dtype=I32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda.kda_verify_accept(target, drafts, uniform, accepted, tokens, draft_probs=guess)
    graph.replay()
    assert (accepted.tolist(), tokens.tolist()) == want
    for x, y in zip(data, make(9, 4, 1000, F32, True, 6)):
        x.copy_(y)
    graph.replay()
    assert (accepted.tolist(), tokens.tolist()) == call(cuda, *data)


@pytest.mark.parametrize("B,V", [(76, 3), (300, 40), (152, 2049)])
def test_clusters_with_little_to_read(cuda, B, V):
    """Most of a cluster's CTAs have no token of so small a vocabulary and come to the sums at once, in calls close behind one
    another: they store into CTAs that may have only just started."""
    sets = [make(B, 2, V, F32, i % 2 == 0, seed=20 + i) for i in range(4)]
    accepted, tokens = torch.full((200, B), 77, dtype=I32, device="cuda"), torch.full((200, B, 2), 77, dtype=I32, device="cuda")
    for i in range(200):
        target, guess, drafts, uniform = sets[i % 4]
        cuda.kda_verify_accept(target, drafts, uniform, accepted[i], tokens[i], draft_probs=guess)
    for i, data in enumerate(sets):
        a, t = expected(*data)
        assert (accepted[i::4].cpu() == torch.tensor(a, dtype=I32)).all() and (tokens[i::4].cpu() == torch.tensor(t, dtype=I32)).all()


def test_unaligned_rows(cuda):
    # probabilities and drafts one element into their storage
    target, guess, drafts, uniform = make(4, 3, 77, BF, True, 7)
    off = lambda t: torch.cat((t.new_zeros(1), t.flatten()))[1:].view(t.shape)  # noqa: E731
    assert call(cuda, off(target), off(guess), off(drafts), off(uniform)) == expected(target, guess, drafts, uniform)


def test_no_requests(cuda):
    e = torch.zeros
    cuda.kda_verify_accept(e(0, 2, 5, device="cuda"), e(0, 1, dtype=I32, device="cuda"), e(0, 2, device="cuda"),
                           e(0, dtype=I32, device="cuda"), e(0, 2, dtype=I32, device="cuda"))
