"""Plain 64-bit forms of the softmax-attention operators (norm and rotation, quantised cache rows, attention over a
paged cache), and the bounds their tests use.  Everything here runs on the CPU in fp64."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24  # unit roundoff of fp32
U16 = 2.0 ** -8   # of bf16 (8 significant bits)


# ---------------------------------------------------------------- norm and rotation

def angles(num, rot, seed=0):
    """cos, sin fp32 [num, rot / 2] of ordinary rotary angles."""
    a = torch.arange(num, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64)
                                                                      / max(rot // 2, 1))
    return a.cos().float(), a.sin().float()


def rotation_matrix(cos, sin, d, rot, interleaved):
    """[d, d] of one position's rotation: y = R x."""
    R = torch.eye(d, dtype=torch.float64)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = float(cos[i]), float(sin[i])
        R[a, a], R[a, b], R[b, a], R[b, b] = c, -s, s, c
    return R


def rotations(cos, sin, positions, d, rot, interleaved):
    if not rot:
        return torch.eye(d, dtype=torch.float64).expand(len(positions), d, d)
    return torch.stack([rotation_matrix(cos[p], sin[p], d, rot, interleaved) for p in positions.tolist()])


def norm_rope(x, w, R, eps):
    """x [T, H, d] fp64, R [T, d, d]."""
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    return torch.einsum("tij,thj->thi", R, x * r * w)


def norm_rope_grad(dy, x, w, R, eps):
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    g = torch.einsum("tji,thj->thi", R, dy)
    dx = r * (g * w - x * r * r * (g * w * x).mean(-1, keepdim=True))
    return dx, (g * x * r).sum((0, 1))


# ---------------------------------------------------------------- cache rows

def e4m3(x):
    """Nearest e4m3 value of x fp64, ties to even, saturating at 448."""
    e = torch.frexp(x)[1].double() - 1
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64), torch.clamp(e, min=-6) - 3)
    return torch.clamp(torch.round(x / step) * step, -448.0, 448.0)


def quantise(x):
    """x [..., d] fp64 -> (e4m3 values, scale [...]) as the cache format states them."""
    amax = torch.where(x.isnan(), torch.zeros_like(x), x.abs()).amax(-1)
    scale = torch.ones_like(amax)
    for i, a in enumerate(amax.flatten().tolist()):
        if a == 0:
            continue
        e = -63
        while e < 63 and a > 448.0 * 2.0 ** e:
            e += 1
        scale.view(-1)[i] = 2.0 ** e
    return e4m3(x / scale[..., None]), scale


# ---------------------------------------------------------------- attention

def attend(q, k, v, length, scale, softcap=0.0, window=0, hidden=None):
    """One request: q [W, Hq, d], k, v [L, Hkv, d] fp64 (rows of the cache in order).  hidden: positions no query sees.
    Returns out [W, Hq, d], lse [W, Hq], and per output the size its rounding errors are measured against: the
    probability-weighted |v|, and the largest sum |q||k| of a seen score."""
    W, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out, lse = torch.zeros(W, Hq, d, dtype=torch.float64), torch.full((W, Hq), -math.inf, dtype=torch.float64)
    mass, size = torch.zeros(W, Hq, d, dtype=torch.float64), torch.zeros(W, Hq, dtype=torch.float64)
    for w in range(W):
        p = length - W + w
        first = max(0, p - window + 1) if window else 0
        seen = [t for t in range(first, p + 1) if hidden is None or t not in hidden]
        if not seen:
            continue
        for h in range(Hq):
            kk, vv = k[seen, h // G], v[seen, h // G]
            s = kk @ q[w, h] * scale
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            lse[w, h] = torch.logsumexp(s, 0)
            pr = torch.exp(s - lse[w, h])
            out[w, h] = pr @ vv
            mass[w, h] = pr @ vv.abs()
            size[w, h] = (kk.abs() @ q[w, h].abs()).max() * abs(scale)
    return out, lse, mass, size


def attend_bound(out, lse, mass, size, d, n, bf16_out, p_bits):
    """Largest error of (out, lse) that the kernel's roundings allow.

    A score's products accumulate in fp32 (d terms, and a few roundings for scales, the change to powers of two and the
    cap): |ds| <= (d + 16) U32 size.  Relative to its softmax a probability is then off by at most 2 |ds|, by 2^-20 for
    the exponential, by n U32 for the sums over n tokens, and by 2^-p_bits for the part of it that enters the second
    product; out's error is that times the probability-weighted |v|, and one rounding to the output's type."""
    ds = (d + 16) * U32 * size
    rel = 2 * ds + 2.0 ** -20 + n * U32 + 2.0 ** -p_bits
    o = mass * rel[..., None] + (U16 if bf16_out else U32) * out.abs()
    return o * 1.01 + 1e-30, ds + 2.0 ** -20 + n * U32 + 4 * U32 * lse.abs().clamp(max=1e30)
