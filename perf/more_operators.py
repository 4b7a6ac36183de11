"""Workloads of the prompt attention and of the acceptance of drafted tokens.

Three calls, as a serving or training program makes them: causal attention over whole packed prompts with grouped heads
(`prompt`), the same with its gradients in a training step (`train`), and the acceptance of a window of drafted tokens
against the target's probabilities (`accept`).  With `own` set, `run` calls the library; otherwise it evaluates the
definitions with elementary torch operations, in fp32 for the attention and in fp64 for the acceptance, whose sums decide
whole numbers.  `exact` evaluates them in fp64.

A case is a dict of plain values:
  op          one of the names above
  sequences, tokens    packed sequences and their tokens together; the lengths follow from these two (`_lengths`)
  heads, kv_heads, d   query heads, key/value heads, head size
  dtype       "bf16" or "f32": type of the activations, or of the probabilities
  sliding, softcap     positions a query sees (0: all before it), tanh cap of the scores (0: none)
  packed      q, k, v are column blocks of one fused projection's output, their gradients of one buffer
  batch, window, vocab  requests, tokens of the draft window (the first was accepted before), vocabulary
  proposal    the drafts came from a distribution (else: each was certain, from a lookup)
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def _attention(name, op, sequences, tokens, heads, kv_heads, d, dtype="bf16", sliding=0, softcap=0.0, packed=True):
    return {"name": name, "op": op, "sequences": sequences, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "d": d,
            "dtype": dtype, "sliding": sliding, "softcap": softcap, "packed": packed}


def _accept(name, batch, window, vocab, dtype="f32", proposal=True):
    return {"name": name, "op": "accept", "batch": batch, "window": window, "vocab": vocab, "dtype": dtype,
            "proposal": proposal}


def listed():
    return [
        # one short question of a chat: latency
        _attention("prompt_short", "prompt", 1, 137, 32, 8, 128),
        # a prefill batch of prompts of many lengths, three query heads to a key/value head
        _attention("prompt_batch", "prompt", 16, 32771, 12, 4, 128),
        # one long document
        _attention("prompt_long", "prompt", 1, 16384, 32, 8, 128),
        # a layer with a sliding window and capped scores, heads of 64
        _attention("prompt_window", "prompt", 5, 24001, 16, 2, 64, sliding=1024, softcap=30.0),
        # a small model evaluated in fp32
        _attention("prompt_f32", "prompt", 3, 2047, 12, 12, 64, dtype="f32", packed=False),
        # a training step of a small fp32 model, an odd token count
        _attention("train_f32", "train", 2, 509, 12, 12, 64, dtype="f32", packed=False),
        # a micro-batch of documents packed to 8K tokens
        _attention("train_batch", "train", 8, 8192, 32, 8, 128),
        # long documents, as many key/value heads as query heads
        _attention("train_long", "train", 1, 8192, 12, 12, 128),
        # all query heads share one key/value head, within a window
        _attention("train_shared", "train", 3, 6001, 12, 1, 128, sliding=2048),
        # one request generating with four drafts: latency
        _accept("accept_one", 1, 5, 32768),
        # a batch of requests, a large vocabulary of odd size
        _accept("accept_batch", 64, 8, 150001),
        # drafts looked up in the prompt, probabilities kept in bf16
        _accept("accept_lookup", 192, 4, 65536, dtype="bf16", proposal=False),
    ]


_HEADS = ((12, 12), (12, 4), (12, 1), (32, 8), (16, 2), (8, 8))
_MOST = 16384 * 16384 * 32 * 128  # tokens squared x heads x head size of the largest prompt


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "train", "train", "accept"))
    if op == "accept":
        window = rng.choice((1, 2, 3, 5, 8))
        vocab = _log(rng, 500, 200000)
        batch = _log(rng, 1, max(1, min(512, 64 * 8 * 150001 // (window * vocab))))
        c = _accept("", batch, window, vocab, rng.choice(("f32", "bf16")), rng.random() < 0.6)
    else:
        heads, kv_heads = rng.choice(_HEADS)
        d = rng.choice((32, 64, 128, 128))
        dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
        most = _MOST / (heads * d) / (16 if dtype == "f32" else 1) / (4 if op == "train" else 1)
        tokens = _log(rng, 1, min(16384, int(math.sqrt(most))))
        c = _attention("", op, min(tokens, rng.choice((1, 1, 2, 5, 13))), tokens, heads, kv_heads, d, dtype,
                       rng.choice((0, 0, 100, 1000)), rng.choice((0.0, 0.0, 30.0)), rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """Even steps of the logarithm over a factor of 32, in a mixed order that depends on the case alone, filling `tokens`."""
    n, tokens = case["sequences"], case["tokens"]
    if n == 1:
        return [tokens]
    share = [32.0 ** (i / (n - 1)) for i in range(n)]
    random.Random(n * 1000003 + tokens).shuffle(share)
    ends, at, total = [], 0.0, sum(share)
    for s in share:
        at += s
        ends.append(round(tokens * at / total))
    return [b - a for a, b in zip([0] + ends[:-1], ends)]


def _rand(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _attention_inputs(case, gen):
    t, hq, hkv, d, dt = case["tokens"], case["heads"], case["kv_heads"], case["d"], _DT[case["dtype"]]
    channel = torch.exp(0.3 * torch.randn(d, generator=gen, device="cuda"))  # some channels larger, as projections have them
    if case["packed"]:
        rows = (_rand(gen, t, hq + 2 * hkv, d) * channel).to(dt)
        q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    else:
        q, k, v = ((_rand(gen, t, h, d) * channel).to(dt) for h in (hq, hkv, hkv))
    ends = [0]
    for n in _lengths(case):
        ends.append(ends[-1] + n)
    s = {"case": case, "q": q, "k": k, "v": v, "ends": ends, "longest": max(_lengths(case)),
         "cu": torch.tensor(ends, dtype=torch.int32, device="cuda")}
    if case["op"] == "train":
        s["d_out"] = _rand(gen, t, hq, d, dtype=dt)
        if own:
            import kda_gated_delta_rule_gb300 as kda
            size = kda.kda_prefill_attention_backward_workspace_size(t, case["sequences"], hq, hkv, d)
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


def _accept_inputs(case, gen):
    b, w, v, dt = case["batch"], case["window"], case["vocab"], _DT[case["dtype"]]
    logits = 2.5 * _rand(gen, b, w, v)
    target = torch.softmax(logits, -1).to(dt)
    s = {"case": case, "target": target, "proposal": None,
         "uniform": torch.rand(b, w, generator=gen, device="cuda", dtype=torch.float32)}
    if case["proposal"]:
        # a smaller model's view of the same text
        guess = torch.softmax(0.9 * logits[:, :w - 1] + 0.7 * _rand(gen, b, w - 1, v), -1).to(dt)
        s["proposal"] = guess
    else:
        guess = target[:, :w - 1]
    if w > 1:
        drafts = torch.multinomial(guess.float().reshape(b * (w - 1), v), 1, generator=gen)
    else:
        drafts = torch.zeros(0, device="cuda")
    s["drafts"] = drafts.view(b, w - 1).to(torch.int32)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return _accept_inputs(case, gen) if case["op"] == "accept" else _attention_inputs(case, gen)


# ------------------------------------------------------------------ one pass

def run(s):
    return (_RUN_OWN if own else _RUN_PLAIN)[s["case"]["op"]](s)


def _own_prompt(s):
    import kda_gated_delta_rule_gb300 as kda
    c, q = s["case"], s["q"]
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    kda.kda_prefill_attention(q, s["k"], s["v"], s["cu"], s["longest"], out, softcap=c["softcap"], window=c["sliding"],
                              lse=lse)
    return {"out": out, "lse": lse}


def _own_train(s):
    import kda_gated_delta_rule_gb300 as kda
    c, q, k = s["case"], s["q"], s["k"]
    done = _own_prompt(s)
    hq, hkv = c["heads"], c["kv_heads"]
    if c["packed"]:
        grads = torch.empty(c["tokens"], hq + 2 * hkv, c["d"], dtype=q.dtype, device=q.device)
        dq, dk, dv = grads[:, :hq], grads[:, hq:hq + hkv], grads[:, hq + hkv:]
    else:
        dq, dk, dv = (torch.empty(x.shape, dtype=q.dtype, device=q.device) for x in (q, k, k))
    kda.kda_prefill_attention_backward(s["d_out"], q, k, s["v"], done["out"], done["lse"], s["cu"], s["longest"], dq, dk, dv,
                                       s["workspace"], softcap=c["softcap"], window=c["sliding"])
    return {"out": done["out"], "dq": dq, "dk": dk, "dv": dv}


def _own_accept(s):
    import kda_gated_delta_rule_gb300 as kda
    b, w = s["uniform"].shape
    accepted = torch.empty(b, dtype=torch.int32, device="cuda")
    tokens = torch.empty(b, w, dtype=torch.int32, device="cuda")
    kda.kda_verify_accept(s["target"], s["drafts"], s["uniform"], accepted, tokens, draft_probs=s["proposal"])
    return {"accepted": accepted, "tokens": tokens}


def _blocks(case):
    """Rows per block: scores of a block stay within half a gigabyte."""
    return max(64, min(2048, (1 << 27) // (case["heads"] * max(1, max(_lengths(case))))))


def _block_scores(s, q, k, r0, r1):
    """Raw and final scores [kv_heads, group, rows, keys] of rows r0 .. r1 of one sequence's q, k [heads, tokens, d]."""
    c = s["case"]
    first = max(0, r0 - c["sliding"] + 1) if c["sliding"] else 0
    x = torch.matmul(q[:, :, r0:r1], k[:, None, first:r1].transpose(-1, -2)) * c["d"] ** -0.5
    y = c["softcap"] * torch.tanh(x / c["softcap"]) if c["softcap"] else x
    row = torch.arange(r0, r1, device=x.device)[:, None]
    key = torch.arange(first, r1, device=x.device)
    seen = key <= row
    if c["sliding"]:
        seen &= key > row - c["sliding"]
    return first, y.masked_fill(~seen, -math.inf)


def _heads_first(s, a, b):
    """fp32 q [kv_heads, group, tokens, d] and k, v [kv_heads, tokens, d] of the sequence at a .. b."""
    hkv = s["case"]["kv_heads"]
    q = s["q"][a:b].float().transpose(0, 1)
    return (q.reshape(hkv, -1, b - a, q.shape[-1]), s["k"][a:b].float().transpose(0, 1).contiguous(),
            s["v"][a:b].float().transpose(0, 1).contiguous())


def _plain_prompt(s):
    c = s["case"]
    out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    step = _blocks(c)
    for a, b in zip(s["ends"], s["ends"][1:]):
        if a == b:
            continue
        q, k, v = _heads_first(s, a, b)
        for r0 in range(0, b - a, step):
            r1 = min(b - a, r0 + step)
            first, y = _block_scores(s, q, k, r0, r1)
            top = y.amax(-1, keepdim=True)
            p = torch.exp(y - top)
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p, v[:, None, first:r1]) / total
            out[a + r0:a + r1] = o.flatten(0, 1).transpose(0, 1).to(out.dtype)
            lse[a + r0:a + r1] = (top + torch.log(total)).flatten(0, 1)[..., 0].transpose(0, 1)
    return {"out": out, "lse": lse}


def _plain_train(s):
    c, dt = s["case"], s["q"].dtype
    cap, scale = c["softcap"], c["d"] ** -0.5
    out, dq = (torch.empty(s["q"].shape, dtype=dt, device="cuda") for _ in range(2))
    dk, dv = (torch.empty(s["k"].shape, dtype=dt, device="cuda") for _ in range(2))
    step = _blocks(c)
    for a, b in zip(s["ends"], s["ends"][1:]):
        if a == b:
            continue
        q, k, v = _heads_first(s, a, b)
        do = s["d_out"][a:b].float().transpose(0, 1).reshape(q.shape)
        sum_k, sum_v = torch.zeros_like(k), torch.zeros_like(v)
        for r0 in range(0, b - a, step):
            r1 = min(b - a, r0 + step)
            first, y = _block_scores(s, q, k, r0, r1)
            p = torch.exp(y - y.amax(-1, keepdim=True))
            p = p / p.sum(-1, keepdim=True)
            keys, values, d_rows = k[:, None, first:r1], v[:, None, first:r1], do[:, :, r0:r1]
            o = torch.matmul(p, values)
            sum_v[:, first:r1] += torch.matmul(p.transpose(-1, -2), d_rows).sum(1)
            ds = p * (torch.matmul(d_rows, values.transpose(-1, -2)) - (d_rows * o).sum(-1, keepdim=True))
            if cap:
                ds = torch.where(p > 0, ds * (1 - (y / cap) ** 2), torch.zeros_like(ds))
            ds = ds * scale
            sum_k[:, first:r1] += torch.matmul(ds.transpose(-1, -2), q[:, :, r0:r1]).sum(1)
            out[a + r0:a + r1] = o.flatten(0, 1).transpose(0, 1).to(dt)
            dq[a + r0:a + r1] = torch.matmul(ds, keys).flatten(0, 1).transpose(0, 1).to(dt)
        dk[a:b], dv[a:b] = sum_k.transpose(0, 1).to(dt), sum_v.transpose(0, 1).to(dt)
    return {"out": out, "dq": dq, "dk": dk, "dv": dv}


def _plain_accept(s):
    target, drafts, u = s["target"], s["drafts"].long(), s["uniform"].double()
    b, w, v = target.shape
    rows = torch.arange(b, device="cuda")
    p = torch.gather(target[:, :w - 1], 2, drafts[..., None])[..., 0].double()
    q = torch.gather(s["proposal"], 2, drafts[..., None])[..., 0].double() if s["proposal"] is not None else 1.0
    taken = (u[:, :w - 1] * q < p).long().cumprod(1)
    n = taken.sum(1)  # accepted drafts
    weight = target[rows, n].double()
    if w > 1:
        at = n.clamp(max=w - 2)
        if s["proposal"] is not None:
            rest = (weight - s["proposal"][rows, at].double()).clamp(min=0)
        else:
            rest = weight.scatter(1, drafts[rows, at][:, None], 0.0)
        refused = (n < w - 1) & (rest.sum(1) > 0)
        weight = torch.where(refused[:, None], rest, weight)
    upto = weight.cumsum(1)
    token = (upto <= u[:, w - 1:] * upto[:, -1:]).sum(1).clamp(max=v - 1)
    tokens = torch.full((b, w), -1, dtype=torch.int32, device="cuda")
    tokens[:, :w - 1] = torch.where(taken > 0, drafts, -torch.ones_like(drafts)).int()
    tokens[rows, n] = token.int()
    return {"accepted": (n + 1).int(), "tokens": tokens}


_RUN_PLAIN = {"prompt": _plain_prompt, "train": _plain_train, "accept": _plain_accept}
_RUN_OWN = {"prompt": _own_prompt, "train": _own_train, "accept": _own_accept}


# ------------------------------------------------------------------ necessary work

def _pairs(case):
    """Query-key pairs that are seen, of one head."""
    n = 0
    for length in _lengths(case):
        seen = min(length, case["sliding"]) if case["sliding"] else length
        n += seen * (seen + 1) // 2 + (length - seen) * seen
    return n


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "accept":
        b, w, v = case["batch"], case["window"], case["vocab"]
        rows = 2 if case["proposal"] and w > 1 else 1  # one request's row of the target, and of the proposal
        return {"bytes": b * (rows * v * es + (w - 1) * (2 * es + 4) + 4 * w + 4 * w + 4), "flops": 3 * b * v}
    t, hq, hkv, d = case["tokens"], case["heads"], case["kv_heads"], case["d"]
    q, kv = t * hq * d * es, t * hkv * d * es
    if case["op"] == "prompt":
        return {"bytes": 2 * q + 2 * kv + 4 * t * hq, "flops": 4 * d * hq * _pairs(case)}
    return {"bytes": 4 * q + 4 * kv, "flops": 14 * d * hq * _pairs(case)}


# ------------------------------------------------------------------ fp64 definitions

_EXACT_MOST = 8e12  # operations in fp64 that take a few seconds


def _exact_attention(case, s):
    train = case["op"] == "train"
    if (14 if train else 4) * case["d"] * case["heads"] * sum(n * n for n in _lengths(case)) > _EXACT_MOST:
        return None
    t, hq, hkv, d = case["tokens"], case["heads"], case["kv_heads"], case["d"]
    new = lambda h: torch.zeros(t, h, d, dtype=torch.float64, device="cuda")  # noqa: E731
    out, dq, dk, dv = new(hq), new(hq), new(hkv), new(hkv)
    lse = torch.zeros(t, hq, dtype=torch.float64, device="cuda")
    at = 0
    for n in _lengths(case):
        here = slice(at, at + n)
        at += n
        distance = torch.arange(n, device="cuda")[:, None] - torch.arange(n, device="cuda")[None]
        unseen = (distance < 0) | (distance >= case["sliding"]) if case["sliding"] else distance < 0
        for h in range(hq):
            g = h // (hq // hkv)
            q, k, v = s["q"][here, h].double(), s["k"][here, g].double(), s["v"][here, g].double()
            x = torch.einsum("ic,jc->ij", q, k) / math.sqrt(d)
            slope = None
            if case["softcap"]:
                x = torch.tanh(x / case["softcap"])
                slope = 1 - x * x
                x = x * case["softcap"]
            x[unseen] = -math.inf
            size = torch.logsumexp(x, 1)
            a = torch.exp(x - size[:, None])
            del x
            o = torch.einsum("ij,jc->ic", a, v)
            out[here, h], lse[here, h] = o, size
            if not train:
                continue
            do = s["d_out"][here, h].double()
            dv[here, g] += torch.einsum("ij,ic->jc", a, do)
            da = torch.einsum("ic,jc->ij", do, v)
            dx = a * (da - torch.einsum("ij,ij->i", a, da)[:, None])
            if slope is not None:
                dx = dx * slope
            dx = dx / math.sqrt(d)
            dq[here, h] = torch.einsum("ij,jc->ic", dx, k)
            dk[here, g] += torch.einsum("ij,ic->jc", dx, q)
    return {"out": out, "dq": dq, "dk": dk, "dv": dv} if train else {"out": out, "lse": lse}


def _exact_accept(case, s):
    b, w, v = case["batch"], case["window"], case["vocab"]
    u, drafts = s["uniform"].double().tolist(), s["drafts"].tolist()
    accepted, tokens = [], []
    for i in range(b):
        row, weight = [], None
        for j in range(w - 1):
            x = drafts[i][j]
            p = s["target"][i, j].double()
            q = s["proposal"][i, j].double() if s["proposal"] is not None else torch.zeros_like(p).index_fill_(
                0, torch.tensor([x], device="cuda"), 1.0)
            if u[i][j] * q[x].item() < p[x].item():
                row.append(x)
                continue
            weight = torch.relu(p - q)
            if not weight.any():
                weight = p
            break
        if weight is None:
            weight = s["target"][i, w - 1].double()
        upto = torch.cumsum(weight, 0)
        token = int(torch.searchsorted(upto, upto[-1:] * u[i][w - 1], right=True).item())
        accepted.append(len(row) + 1)
        tokens.append(row + [min(token, v - 1)] + [-1] * (w - 1 - len(row)))
    return {"accepted": torch.tensor(accepted, dtype=torch.int32, device="cuda"),
            "tokens": torch.tensor(tokens, dtype=torch.int32, device="cuda").view(b, w)}


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_accept if case["op"] == "accept" else _exact_attention)(case, s)
