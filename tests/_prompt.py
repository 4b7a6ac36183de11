"""The prompt attention and its gradients in fp64, with bounds on what a correct implementation's roundings may do.

The bounds count, with u the half step of the type that is rounded to (bf16 2^-8, fp32 2^-24):
  scores       each is a sum of d products in fp32, relative to the products' magnitudes (d + 8) 2^-23, tanh and the exponential
               add 2^-20 of the score's size and 2^-21; e_ij is the bound on a probability's relative error that follows (a
               score's error twice: in itself and in the log-sum-exp)
  p            rounded to bf16 for its product when the inputs are bf16 (u_p, else 0)
  D            the gradient's mean <d_out, out> from the rounded output, or (bf16, rows that see few keys) from p and d_out . v
  sums         over n rows in fp32: n 2^-24 of the terms' magnitudes, 2^-23 counted; rescaled sums stay within it
  results      rounded once to their type.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def attention(q, k, v, d_out, lengths, start=0, scale=None, softcap=0.0, window=0, out_type=None, grad_type=None):
    """dict of (value, bound) per result; q [T, Hq, d], k, v [T, Hkv, d] of bf16 or fp32; d_out None: no gradients."""
    dt = q.dtype
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    u_in = U[torch.bfloat16] if dt == torch.bfloat16 else 0.0
    u_out, u_grad = U[out_type or dt], U[grad_type or dt]
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device=q.device)  # noqa: E731
    names = {"out": (T, Hq, d), "lse": (T, Hq), "dq": (T, Hq, d), "dk": (T, Hkv, d), "dv": (T, Hkv, d)}
    val, bound = {n: z(*s) for n, s in names.items()}, {n: z(*s) for n, s in names.items()}
    at = start
    for n in lengths:
        s = slice(at, at + n)
        at += n
        if n == 0:
            continue
        i = torch.arange(n, device=q.device)
        seen = i[None] <= i[:, None]
        if window:
            seen &= i[None] > i[:, None] - window
        for h in range(Hq):
            g = h // G
            Q, K, V = q[s, h].double(), k[s, g].double(), v[s, g].double()
            raw = Q @ K.T * scale
            size = Q.abs() @ K.abs().T * abs(scale)
            x, slope = raw, torch.ones_like(raw)
            if softcap:
                x = softcap * torch.tanh(raw / softcap)
                slope = 1 - (x / softcap) ** 2
            e_score = (d + 8) * 2.0 ** -23 * size + 2.0 ** -20 * x.abs() + 2.0 ** -21
            x = x.masked_fill(~seen, -math.inf)
            e_score = e_score.masked_fill(~seen, 0.0)
            lse = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[:, None])
            e = 2 * e_score.amax(1, keepdim=True) + n * 2.0 ** -23
            e_lse = e_score.amax(1) + n * 2.0 ** -23 + 2.0 ** -22 * lse.abs() + 2.0 ** -22
            o = p @ V
            b_out = (u_in + e) * (p @ V.abs()) + u_out * o.abs()
            val["out"][s, h], bound["out"][s, h] = o, b_out * 1.01 + 1e-30
            val["lse"][s, h], bound["lse"][s, h] = lse, e_lse
            if d_out is None:
                continue
            dO = d_out[s, h].double()
            e = e + (e_lse + 2.0 ** -22 * lse.abs())[:, None]
            dp = dO @ V.T
            D = (dO * o).sum(1, keepdim=True)
            b_D = (dO.abs() * b_out).sum(1, keepdim=True) + d * 2.0 ** -23 * (dO.abs() * o.abs()).sum(1, keepdim=True)
            b_dp = d * 2.0 ** -23 * (dO.abs() @ V.abs().T)
            if dt == torch.bfloat16:  # rows whose block of 128 walks up to three tiles have it from their own p and dp
                own = ((e + n * 2.0 ** -23) * p * dp.abs() + p * b_dp).sum(1, keepdim=True)
                b_D = torch.where((i < 384)[:, None] | bool(window and window <= 257), own, b_D)
            e_slope = 4 * (e_score / softcap + 2.0 ** -20) if softcap else 0.0
            dx = p * (dp - D) * slope
            b_dx = (u_in + e) * dx.abs() + p * ((b_dp + b_D) * slope + (dp - D).abs() * e_slope)
            more = n * G * 2.0 ** -23
            val["dv"][s, g] += p.T @ dO
            bound["dv"][s, g] += ((u_in + e + more) * p).T @ dO.abs()
            val["dk"][s, g] += dx.T @ Q * scale
            bound["dk"][s, g] += (b_dx + more * dx.abs()).T @ Q.abs() * abs(scale)
            val["dq"][s, h] = dx @ K * scale
            bound["dq"][s, h] = (b_dx + more * dx.abs()) @ K.abs() * abs(scale)
    for name in ("dq", "dk", "dv"):
        bound[name] += u_grad * val[name].abs() + u_grad * bound[name] + 1e-30
    return {n: (val[n], bound[n]) for n in names if d_out is not None or n in ("out", "lse")}


def worst(got, value, bound, rows):
    """Largest excess of |got - value| over the bound, as a factor (at most 1 is right), over the given rows."""
    diff = (got[rows].double() - value[rows]).abs()
    factor = diff / bound[rows]
    return float(torch.nan_to_num(factor, nan=math.inf).max()) if factor.numel() else 0.0


def cu(lengths, start=0, device="cuda"):
    ends = [start]
    for n in lengths:
        ends.append(ends[-1] + n)
    return torch.tensor(ends, dtype=torch.int32, device=device)


def inputs(T, Hq, Hkv, d, dtype, seed, packed=False, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda") * size  # noqa: E731
    if packed:
        rows = r(T, Hq + 2 * Hkv, d).to(dtype)
        q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    else:
        q, k, v = (r(T, h, d).to(dtype) for h in (Hq, Hkv, Hkv))
    return q, k, v, r(T, Hq, d).to(dtype)


def run(kda, q, k, v, offsets, longest, d_out=None, out_type=None, grad_type=None, packed=False, fill=7.0, **kw):
    """The library's results in buffers that hold `fill` before the call."""
    T, Hq, d = q.shape
    Hkv, dt = k.shape[1], q.dtype
    res = {"out": torch.full((T, Hq, d), fill, dtype=out_type or dt, device="cuda"),
           "lse": torch.full((T, Hq), fill, device="cuda")}
    kda.kda_prefill_attention(q, k, v, offsets, longest, res["out"], lse=res["lse"], **kw)
    if d_out is not None:
        gt = grad_type or dt
        if packed:
            rows = torch.full((T, Hq + 2 * Hkv, d), fill, dtype=gt, device="cuda")
            res.update(dq=rows[:, :Hq], dk=rows[:, Hq:Hq + Hkv], dv=rows[:, Hq + Hkv:])
        else:
            res.update({n: torch.full((T, h, d), fill, dtype=gt, device="cuda") for n, h in (("dq", Hq), ("dk", Hkv), ("dv", Hkv))})
        N = offsets.numel() - 1
        ws = torch.full((kda.kda_prefill_attention_backward_workspace_size(T, N, Hq, Hkv, d),), 255, dtype=torch.uint8, device="cuda")
        kda.kda_prefill_attention_backward(d_out, q, k, v, res["out"], res["lse"], offsets, longest, res["dq"], res["dk"],
                                           res["dv"], ws, **kw)
    return res


def compare(kda, lengths, Hq, Hkv, d, dtype, seed=0, start=0, tail=0, packed=False, out_type=None, grad_type=None, size=1.0,
            grads=True, **kw):
    """Every result of a call within its bound, rows outside the sequences as they were."""
    T = start + sum(lengths) + tail
    q, k, v, d_out = inputs(T, Hq, Hkv, d, dtype, seed, packed, size)
    inside = torch.zeros(T, dtype=torch.bool, device="cuda")
    inside[start:T - tail] = True
    for x in (q, k, v, d_out):
        x[~inside] = math.nan
    if not grads:
        d_out = None
    got = run(kda, q, k, v, cu(lengths, start), max(lengths), d_out, out_type, grad_type, packed, **kw)
    want = attention(q, k, v, d_out, lengths, start, out_type=out_type, grad_type=grad_type, **kw)
    bad = {}
    for name, (value, bound) in want.items():
        f = worst(got[name], value, bound, inside)
        if not f <= 1:
            bad[name] = f
        assert (got[name][~inside] == 7.0).all(), name
    assert not bad, bad
