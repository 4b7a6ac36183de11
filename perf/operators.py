"""Workloads of the softmax-attention operators that stand beside the KDA layers of a hybrid model.

Four calls, as a serving or training program makes them: the per-head norm of queries and keys with the
position rotation (`norm`) and its gradient (`norm_grad`), writing (`write`) and reading back (`read`) a paged
key/value cache, and attention of the newest tokens over that cache (`attend`).  With `own` set, `run` calls
the library; otherwise it evaluates the definitions with elementary torch operations in fp32.  `exact`
evaluates them in fp64.

A case is a dict of plain values:
  op          one of the names above
  tokens      tokens of the call (norm, norm_grad, write, read)
  heads, kv_heads, d   query heads, key/value heads, head size
  dtype       "bf16" or "f32": type of the activations
  cache       "bf16" or "e4m3": type of the cached rows
  rot, interleaved     channels rotated, and how they pair up
  packed      the inputs are column blocks of one fused projection's output rather than tensors of their own
  batch, window_tokens, min_len, max_len, page, sliding, softcap   the attention's batch
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -63, 63  # range of a cached row's scale exponent

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def _norm(name, tokens, heads, kv_heads, d, rot, dtype="bf16", interleaved=False, packed=True, grad=False):
    return {"name": name, "op": "norm_grad" if grad else "norm", "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "d": d, "rot": rot, "dtype": dtype, "interleaved": interleaved, "packed": packed}


def _cache(name, op, tokens, kv_heads, d, page, dtype="bf16", cache="e4m3"):
    return {"name": name, "op": op, "tokens": tokens, "kv_heads": kv_heads, "d": d, "page": page, "dtype": dtype,
            "cache": cache}


def _attend(name, batch, window_tokens, heads, kv_heads, d, min_len, max_len, page, cache, sliding=0, softcap=0.0,
            dtype="bf16"):
    return {"name": name, "op": "attend", "batch": batch, "window_tokens": window_tokens, "heads": heads,
            "kv_heads": kv_heads, "d": d, "min_len": min_len, "max_len": max_len, "page": page, "cache": cache,
            "sliding": sliding, "softcap": softcap, "dtype": dtype}


def listed():
    return [
        # one request generating: a single token's heads, all launch latency
        _norm("norm_token", 1, 32, 8, 128, 128),
        # an 8K prompt out of a fused projection, whole heads rotated
        _norm("norm_prompt", 8192, 32, 8, 128, 128),
        # fp32 training of a small model without rotation: the unit-length keys of the KDA layers, an odd token count
        _norm("norm_grad_odd", 509, 12, 12, 64, 0, dtype="f32", packed=False, grad=True),
        # a training step's micro-batch, half of each head rotated in neighbouring pairs
        _norm("norm_grad_batch", 16384, 32, 8, 128, 64, interleaved=True, grad=True),
        # one decode step of 256 requests: a row per request scattered over the pool
        _cache("write_step", "write", 256, 4, 128, 64),
        # a packed prompt of 64K tokens going into the cache
        _cache("write_prompt", "write", 65536, 8, 128, 64),
        # a shared prefix of a thousand tokens brought back for a chunk of prefill
        _cache("read_prefix", "read", 1000, 8, 128, 16),
        # a long prefix brought back, odd length
        _cache("read_long", "read", 65535, 8, 128, 128),
        # one request, one new token, a short bf16 cache: latency
        _attend("attend_one", 1, 1, 32, 8, 128, 1000, 1000, 16, "bf16"),
        # a full decode batch with lengths spread over two orders of magnitude, 8-bit cache
        _attend("attend_batch", 256, 1, 12, 4, 128, 65, 8191, 64, "e4m3"),
        # one request with a quarter of a million cached tokens: the length is what there is to split
        _attend("attend_long", 1, 1, 32, 8, 128, 262144, 262144, 128, "bf16"),
        # an 8-token draft window checked against capped scores over a sliding window, one shared key/value head
        _attend("attend_draft", 64, 8, 12, 1, 128, 500, 6000, 64, "e4m3", sliding=4096, softcap=30.0),
    ]


_HEADS = ((12, 12), (12, 4), (12, 1), (32, 8), (16, 2), (8, 8))


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "write", "read", "attend", "attend"))
    heads, kv_heads = rng.choice(_HEADS)
    d = rng.choice((64, 128, 128))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op in ("norm", "norm_grad"):
        most = 16384 * 40 * 128 // ((heads + kv_heads) * d) // (2 if dtype == "f32" else 1)
        most //= 1 if op == "norm_grad" else 2
        c = _norm("", _log(rng, 1, most), heads, kv_heads, d, rng.choice((0, d // 2, d)), dtype, rng.random() < 0.5,
                  rng.random() < 0.5, op == "norm_grad")
    elif op in ("write", "read"):
        most = 65536 * 8 * 128 // (kv_heads * d) // (2 if dtype == "f32" else 1)
        c = _cache("", op, _log(rng, 1, min(most, 200000)), kv_heads, d, rng.choice((16, 32, 64, 128)), dtype,
                   rng.choice(("e4m3", "e4m3", "bf16")))
    else:
        cache = rng.choice(("bf16", "e4m3"))
        batch = _log(rng, 1, 256)
        # keys of the whole batch, at the longest length, within the longest listed cache
        most = min(262144, 262144 * 8 * 128 // (batch * kv_heads * d) // (2 if dtype == "f32" else 1))
        longest = _log(rng, 1, max(2, most))
        window_tokens = rng.choice((1, 1, 1, 2, 4, 8)) if batch * longest <= 262144 else 1
        c = _attend("", batch, window_tokens, heads, kv_heads, d, max(1, longest // rng.choice((1, 4, 64))), longest,
                    rng.choice((16, 32, 64, 128)), cache, rng.choice((0, 0, 100, 1024)),
                    rng.choice((0.0, 0.0, 30.0)), dtype)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """The batch's cache lengths: even steps of the logarithm from min_len to max_len, in a mixed order that
    depends on the case alone."""
    b, lo, hi = case["batch"], case["min_len"], case["max_len"]
    out = [round(lo * (hi / lo) ** (i / (b - 1))) if b > 1 else hi for i in range(b)]
    random.Random(b * 1000003 + hi).shuffle(out)
    return out


def _rand(gen, *shape, dtype=torch.float32, scale=1.0):
    x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x * scale if scale != 1.0 else x).to(dtype)


def _columns(gen, tokens, widths, d, dtype, packed):
    """Activations [tokens, heads, d] for each of `widths` heads: column blocks of one projection's output when
    packed, with some channels larger than others as projections have them."""
    channel = torch.exp(0.5 * torch.randn(d, generator=gen, device="cuda"))
    if not packed:
        return [(_rand(gen, tokens, h, d) * channel).to(dtype) for h in widths]
    rows = (_rand(gen, tokens, sum(widths), d) * channel).to(dtype)
    out, at = [], 0
    for h in widths:
        out.append(rows[:, at:at + h])
        at += h
    return out


def _pages_for(case):
    return [-(-n // case["page"]) for n in _lengths(case)]


def _quantised(x):
    """(e4m3 values, fp32 scale exponents) of rows x[..., d]."""
    amax = x.float().abs().amax(-1, keepdim=True).clamp(max=3.4e38)
    m, e = torch.frexp(amax)
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(MIN_EXP, MAX_EXP)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    power = lambda n: ((n.int() + 127) << 23).view(torch.float32)  # noqa: E731  2^n, exactly
    return (x.float() * power(-e)).to(torch.float8_e4m3fn), power(e)[..., 0]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    op, d, hkv, dt = case["op"], case["d"], case["kv_heads"], _DT[case["dtype"]]
    if op in ("norm", "norm_grad"):
        t, hq, rot = case["tokens"], case["heads"], case["rot"]
        q, k, _ = _columns(gen, t, (hq, hkv, hkv), d, dt, case["packed"])
        s.update(q=q, k=k, wq=1 + _rand(gen, d, scale=0.1), wk=1 + _rand(gen, d, scale=0.1), cos=None, sin=None,
                 positions=None)
        if rot:
            n = 16384
            angle = (torch.arange(n, dtype=torch.float64, device="cuda")[:, None]
                     * 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") / (rot // 2)))
            s.update(cos=angle.cos().float(), sin=angle.sin().float(),
                     positions=torch.randint(0, n, (t,), generator=gen, device="cuda", dtype=torch.int32))
        if op == "norm_grad":
            s.update(dyq=_rand(gen, t, hq, d, dtype=dt), dyk=_rand(gen, t, hkv, d, dtype=dt))
            if own:
                import kda_gated_delta_rule_gb300 as kda
                s["workspace"] = torch.empty(kda.kda_qk_norm_rope_backward_workspace_size(t, hq, hkv, d),
                                             dtype=torch.uint8, device="cuda")
    elif op in ("write", "read"):
        t, page = case["tokens"], case["page"]
        pages = -(-t // page) + 3
        # whole pages in a scattered order, the tokens of a page next to one another
        order = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(t, device="cuda")
        s["slots"] = order[at // page] * page + at % page
        shape = (pages, hkv, page, d)
        if op == "write":
            s["k"], s["v"] = _columns(gen, t, (hkv, hkv), d, dt, True)
            kind = torch.float8_e4m3fn if case["cache"] == "e4m3" else torch.bfloat16
            s.update(kp=torch.zeros(shape, device="cuda", dtype=torch.bfloat16).to(kind),
                     vp=torch.zeros(shape, device="cuda", dtype=torch.bfloat16).to(kind), ks=None, vs=None)
            if case["cache"] == "e4m3":
                s.update(ks=torch.ones(shape[:3], device="cuda"), vs=torch.ones(shape[:3], device="cuda"))
        else:
            _fill_pages(s, gen, shape, case["cache"])
    else:
        b, w, hq, page = case["batch"], case["window_tokens"], case["heads"], case["page"]
        need = _pages_for(case)
        total, widest = sum(need) + 5, max(need)
        _fill_pages(s, gen, (total, hkv, page, d), case["cache"])
        order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32).cpu()
        table, at = torch.zeros(b, widest, dtype=torch.int32), 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        s.update(table=table.cuda(), lens=torch.tensor(_lengths(case), dtype=torch.int32, device="cuda"),
                 q=_rand(gen, b, w, hq, d, dtype=dt, scale=1.5))
        if own:
            import kda_gated_delta_rule_gb300 as kda
            s["workspace"] = torch.empty(kda.kda_paged_attention_workspace_size(b, w, hq, hkv, d), dtype=torch.uint8,
                                         device="cuda")
    return s


def _fill_pages(s, gen, shape, cache):
    channel = torch.exp(0.5 * torch.randn(shape[-1], generator=gen, device="cuda"))
    for name, scale in (("k", "ks"), ("v", "vs")):
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
        if name == "k":
            x = (x * channel).to(torch.bfloat16)
        if cache == "e4m3":
            s[name + "p"], s[scale] = _quantised(x)
        else:
            s[name + "p"], s[scale] = x, None


# ------------------------------------------------------------------ one pass

def run(s):
    return (_RUN_OWN if own else _RUN_PLAIN)[s["case"]["op"]](s)


def _own_norm(s):
    import kda_gated_delta_rule_gb300 as kda
    q, k = s["q"], s["k"]
    yq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    yk = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    kda.kda_qk_norm_rope(q, k, s["wq"], s["wk"], yq, yk, cos=s["cos"], sin=s["sin"], positions=s["positions"], eps=EPS,
                         interleaved=s["case"]["interleaved"])
    return {"q": yq, "k": yk}


def _own_norm_grad(s):
    import kda_gated_delta_rule_gb300 as kda
    q, k = s["q"], s["k"]
    dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    dk = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    dw = torch.empty(2, q.shape[-1], dtype=torch.float32, device=q.device)
    kda.kda_qk_norm_rope_backward(s["dyq"], s["dyk"], q, k, s["wq"], s["wk"], dq, dk, dw[0], dw[1], s["workspace"],
                                  cos=s["cos"], sin=s["sin"], positions=s["positions"], eps=EPS,
                                  interleaved=s["case"]["interleaved"])
    return {"dq": dq, "dk": dk, "dwq": dw[0], "dwk": dw[1]}


def _own_write(s):
    import kda_gated_delta_rule_gb300 as kda
    kda.kda_kv_write(s["k"], s["v"], s["kp"], s["vp"], s["slots"], k_scales=s["ks"], v_scales=s["vs"])
    return _cached(s)


def _own_read(s):
    import kda_gated_delta_rule_gb300 as kda
    c, dt = s["case"], _DT[s["case"]["dtype"]]
    k = torch.empty(c["tokens"], c["kv_heads"], c["d"], dtype=dt, device="cuda")
    v = torch.empty_like(k)
    kda.kda_kv_read(s["kp"], s["vp"], s["slots"], k, v, k_scales=s["ks"], v_scales=s["vs"])
    return {"k": k, "v": v}


def _own_attend(s):
    import kda_gated_delta_rule_gb300 as kda
    c, q = s["case"], s["q"]
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    kda.kda_paged_attention(q, s["kp"], s["vp"], s["table"], s["lens"], out, s["workspace"], k_scales=s["ks"],
                            v_scales=s["vs"], softcap=c["softcap"], window=c["sliding"], lse=lse)
    return {"out": out, "lse": lse}


def _cached(s):
    return {n: s[n] for n in ("kp", "vp", "ks", "vs") if s[n] is not None}


def _rotated(x, s, inverse=False):
    """The first `rot` channels of x [T, H, d] turned by each token's angles."""
    rot = s["case"]["rot"]
    if not rot:
        return x
    cos, sin = s["cos"][s["positions"].long()][:, None], s["sin"][s["positions"].long()][:, None]
    if inverse:
        sin = -sin
    part, rest = x[..., :rot], x[..., rot:]
    if s["case"]["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, rest), -1)


def _normed(x, w, s):
    f = x.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w
    return _rotated(y, s).to(x.dtype)


def _plain_norm(s):
    return {"q": _normed(s["q"], s["wq"], s), "k": _normed(s["k"], s["wk"], s)}


def _normed_grad(dy, x, w, s):
    f = x.float()
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    g = _rotated(dy.float(), s, inverse=True)
    u, gw = f * r, g * w
    dx = r * (gw - u * (gw * u).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * u).sum((0, 1))


def _plain_norm_grad(s):
    dq, dwq = _normed_grad(s["dyq"], s["q"], s["wq"], s)
    dk, dwk = _normed_grad(s["dyk"], s["k"], s["wk"], s)
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _placed(s, x, pages, scales):
    page = s["case"]["page"]
    at, off = s["slots"] // page, s["slots"] % page
    if scales is None:
        pages[at, :, off] = x.to(torch.bfloat16)
        return
    c, scale = _quantised(x)
    pages.view(torch.uint8)[at, :, off] = c.view(torch.uint8)
    scales[at, :, off] = scale


def _plain_write(s):
    _placed(s, s["k"], s["kp"], s["ks"])
    _placed(s, s["v"], s["vp"], s["vs"])
    return _cached(s)


def _taken(s, pages, scales):
    page, dt = s["case"]["page"], _DT[s["case"]["dtype"]]
    at, off = s["slots"] // page, s["slots"] % page
    if scales is None:
        return pages[at, :, off].float().to(dt)
    x = pages.view(torch.uint8)[at, :, off].view(torch.float8_e4m3fn).float()
    return (x * scales[at, :, off][..., None]).to(dt)


def _plain_read(s):
    return {"k": _taken(s, s["kp"], s["ks"]), "v": _taken(s, s["vp"], s["vs"])}


def _gathered(pages, scales, table):
    """[B, kv_heads, tokens, d] fp32 rows of every page in the table, in order."""
    at = table.long()
    b, n = at.shape
    _, h, page, d = pages.shape
    if scales is None:
        x = pages[at].float()
    else:
        x = pages.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scales[at][..., None]
    return x.permute(0, 2, 1, 3, 4).reshape(b, h, n * page, d)


def _plain_attend(s):
    c, q = s["case"], s["q"].float()
    b, w, hq, d = q.shape
    hkv = c["kv_heads"]
    g = hq // hkv
    rows = q.view(b, w, hkv, g, d).transpose(1, 2).reshape(b, hkv, w * g, d)
    x = torch.matmul(rows, _gathered(s["kp"], s["ks"], s["table"]).transpose(-1, -2)) * d ** -0.5
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    at = torch.arange(x.shape[-1], device=x.device)
    newest = s["lens"][:, None] - w + torch.arange(w, device=x.device)  # [B, W]
    seen = at <= newest[..., None]
    if c["sliding"]:
        seen = seen & (at > newest[..., None] - c["sliding"])
    seen = seen[:, None, :, None].expand(b, hkv, w, g, -1).reshape(b, hkv, w * g, -1)
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _gathered(s["vp"], s["vs"], s["table"]))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.view(b, hkv, w, g, d).transpose(1, 2).reshape(b, w, hq, d)
    lse = (top + torch.log(total)).view(b, hkv, w, g).transpose(1, 2).reshape(b, w, hq)
    return {"out": o.to(s["q"].dtype), "lse": lse}


_RUN_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "write": _plain_write, "read": _plain_read,
              "attend": _plain_attend}
_RUN_OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "write": _own_write, "read": _own_read,
            "attend": _own_attend}


# ------------------------------------------------------------------ necessary work

def work(case):
    op, d, hkv = case["op"], case["d"], case["kv_heads"]
    es = 2 if case["dtype"] == "bf16" else 4
    if op in ("norm", "norm_grad"):
        t, n = case["tokens"], case["tokens"] * (case["heads"] + hkv) * d
        table = t * (4 + 4 * case["rot"]) if case["rot"] else 0
        if op == "norm":
            return {"bytes": 2 * n * es + table + 8 * d, "flops": 8 * n}
        return {"bytes": 3 * n * es + table + 16 * d, "flops": 18 * n}
    row = d * 2 if case["cache"] == "bf16" else d + 4
    if op in ("write", "read"):
        n = 2 * case["tokens"] * hkv
        return {"bytes": n * (d * es + row) + 8 * case["tokens"], "flops": 2 * n * d}
    w, sliding = case["window_tokens"], case["sliding"]
    rows = pairs = 0
    for length in _lengths(case):
        newest = [length - w + i for i in range(w)]
        first = [max(0, p - sliding + 1) if sliding else 0 for p in newest]
        pairs += sum(max(0, p + 1 - f) for p, f in zip(newest, first))
        rows += max(0, length - min(first))
    b, hq = case["batch"], case["heads"]
    return {"bytes": 2 * rows * hkv * row + b * w * hq * (2 * d * es + 4) + 4 * sum(_pages_for(case)) + 4 * b,
            "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ fp64 definitions

def _exact_rotation(rot, d, interleaved, cos, sin):
    """[T, d, d] is never formed: the partner channel and the sign of every channel, and per-channel angles."""
    partner, sign, cc, ss = np.arange(d), np.zeros(d), np.ones((len(cos), d)), np.zeros((len(cos), d))
    for i in range(rot // 2):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        partner[lo], partner[hi], sign[lo], sign[hi] = hi, lo, -1.0, 1.0
        cc[:, lo] = cc[:, hi] = cos[:, i]
        ss[:, lo] = ss[:, hi] = sin[:, i]
    return partner, sign, cc, ss


def _exact_angles(case, s):
    if not case["rot"]:
        return None
    at = s["positions"].long()
    cos, sin = (s[n][at].double().cpu().numpy() for n in ("cos", "sin"))
    partner, sign, cc, ss = _exact_rotation(case["rot"], case["d"], case["interleaved"], cos, sin)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return dev(partner), dev(sign), dev(cc)[:, None], dev(ss)[:, None]


def _exact_norm(case, s, grad):
    rotation = _exact_angles(case, s)
    out = {}
    for name, x, w, dy in (("q", s["q"], s["wq"], s.get("dyq")), ("k", s["k"], s["wk"], s.get("dyk"))):
        x, w = x.double(), w.double()
        size = torch.sqrt(torch.einsum("thc,thc->th", x, x) / case["d"] + EPS)[..., None]
        unit = x / size
        if not grad:
            y = unit * w
            if rotation:
                partner, sign, cc, ss = rotation
                y = y * cc + sign * ss * y[..., partner]
            out[name] = y
            continue
        g = dy.double()
        if rotation:  # the rotation's transpose: the opposite angle
            partner, sign, cc, ss = rotation
            g = g * cc - sign * ss * g[..., partner]
        out["dw" + name] = torch.einsum("thc,thc->c", g, unit)
        g = g * w
        out["d" + name] = (g - unit * torch.einsum("thc,thc->th", g, unit)[..., None] / case["d"]) / size
    return out


def _exact_e4m3(x):
    """x [.., d] fp64 -> (values on the e4m3 grid of the scaled row, scale), from the definition."""
    power = lambda n: ((n.long() + 1023) << 52).view(torch.float64)  # noqa: E731  2^n, exactly
    amax = x.abs().amax(-1, keepdim=True)
    e = torch.frexp(amax / E4M3_MAX)[1]  # amax / 448 is in [2^(e-1), 2^e)
    e = torch.where(amax <= E4M3_MAX * power(e - 1), e - 1, e).clamp(MIN_EXP, MAX_EXP)
    scale = power(torch.where(amax == 0, torch.zeros_like(e), e))
    y = x / scale
    step = power((torch.frexp(y)[1] - 1).clamp(min=-6) - 3)  # three bits below the leading one; a fixed step under 2^-6
    return torch.round(y / step) * step, scale[..., 0]


def _exact_write(case, s):
    page = case["page"]
    at, off = s["slots"] // page, s["slots"] % page
    out = {}
    for x, pages, scales in (("k", "kp", "ks"), ("v", "vp", "vs")):
        y = s[x].double()
        p = s[pages].to(torch.float32).double()
        if s[scales] is None:
            p[at, :, off] = y
        else:
            c, scale = _exact_e4m3(y)
            z = s[scales].double()
            p[at, :, off], z[at, :, off] = c, scale
            out[scales] = z
        out[pages] = p
    return out


def _exact_read(case, s):
    flat = (s["slots"] // case["page"] * case["kv_heads"] * case["page"] + s["slots"] % case["page"])[:, None]
    flat = flat + torch.arange(case["kv_heads"], device="cuda") * case["page"]
    out = {}
    for x, pages, scales in (("k", "kp", "ks"), ("v", "vp", "vs")):
        rows = s[pages].to(torch.float32).view(-1, case["d"])[flat].double()
        out[x] = rows if s[scales] is None else rows * s[scales].view(-1)[flat].double()[..., None]
    return out


def _exact_attend(case, s):
    b, w, hq, d, hkv, page = (case[n] for n in ("batch", "window_tokens", "heads", "d", "kv_heads", "page"))
    out = torch.zeros(b, w, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((b, w, hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, length in enumerate(_lengths(case)):
        at = torch.arange(length, device="cuda")
        pages, off = s["table"][i].long()[at // page], at % page
        rows = []
        for name, scale in (("kp", "ks"), ("vp", "vs")):
            x = s[name].view(torch.uint8 if s[scale] is not None else torch.bfloat16)[pages, :, off]
            x = x.view(torch.float8_e4m3fn).float().double() if s[scale] is not None else x.double()
            rows.append(x if s[scale] is None else x * s[scale][pages, :, off].double()[..., None])
        k, v = rows
        for j in range(w):
            newest = length - w + j
            first = max(0, newest + 1 - case["sliding"]) if case["sliding"] else 0
            if newest < 0:
                continue
            q = s["q"][i, j].double().view(hkv, hq // hkv, d)
            x = torch.einsum("hgc,thc->hgt", q, k[first:newest + 1]) / math.sqrt(d)
            if case["softcap"]:
                x = torch.tanh(x / case["softcap"]) * case["softcap"]
            lse[i, j] = torch.logsumexp(x, -1).view(hq)
            out[i, j] = torch.einsum("hgt,thc->hgc", torch.softmax(x, -1), v[first:newest + 1]).reshape(hq, d)
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        return _exact_norm(case, s, op == "norm_grad")
    return {"write": _exact_write, "read": _exact_read, "attend": _exact_attend}[op](case, s)
