"""A small hybrid model served with the library: one KDA layer, one softmax-attention layer, tokens in and tokens out.

    python examples/hybrid_decode.py [--prompt 200] [--tokens 24] [--cache e4m3] [--drafts 4]

The weights are random; what it shows is which call does what to a token.  The prompt goes through in windows (the KDA
layer by kda_prefill_varlen, the attention layer by kda_paged_attention with that many queries per request), then every
request generates greedily, one token per step.  At the end the same tokens go through in windows of another size, and
the two runs' logits are compared: the cache and the states carry everything that a step needs.  With --drafts it also
generates by draft windows: the prompt at once (the attention layer by kda_prefill_attention), drafts looked up in the text, kda_verify
in the KDA layer, kda_verify_accept on the probabilities, and kda_verify_replay to commit what was accepted.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kda_gated_delta_rule_gb300 as kda  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
D, H, HKV, MODEL, VOCAB = 128, 4, 2, 256, 512  # head size, heads, key/value heads, model width, vocabulary


class Weights:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[0] ** -0.5).to(BF)  # noqa: E731
        self.embed = torch.randn(VOCAB, MODEL, generator=g, device="cuda").to(BF)
        self.kda_in, self.kda_gate, self.kda_out = w(MODEL, 3 * H * D), w(MODEL, H * D + H), w(H * D, MODEL)
        self.qkv, self.attn_out = w(MODEL, (H + 2 * HKV) * D), w(H * D, MODEL)
        self.head = w(MODEL, VOCAB)
        self.q_norm, self.k_norm = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
        self.unit = torch.full((D,), D ** -0.5, device="cuda")  # the norm with this weight gives unit length


class Model:
    """States and cache of B requests."""

    def __init__(self, weights, B, max_tokens, cache, page=32):
        self.w, self.B, self.page = weights, B, page
        pages = -(-max_tokens // page)
        kind = torch.float8_e4m3fn if cache == "e4m3" else BF
        shape = (B * pages, HKV, page, D)
        self.k, self.v = (torch.zeros(shape, device="cuda", dtype=BF).to(kind) for _ in range(2))
        self.scales = {}
        if cache == "e4m3":
            self.scales = dict(k_scales=torch.ones(shape[:3], device="cuda"), v_scales=torch.ones(shape[:3], device="cuda"))
        self.table = torch.randperm(B * pages, device="cuda").view(B, pages).to(torch.int32)  # pages in no order
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.pool = torch.zeros(B, H, D, D, device="cuda")  # the KDA layer's states, one slot per request
        self.slots = torch.arange(B, dtype=torch.int32, device="cuda")
        half = torch.arange(D // 2, device="cuda", dtype=torch.float64)
        angle = torch.arange(max_tokens, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-half / (D // 2))
        self.cos, self.sin = angle.cos().float(), angle.sin().float()

    def kda_layer(self, x, drafts=False):
        """x [B, W, MODEL]: the recurrence over W new tokens of every request; of drafts without a change of state."""
        B, W, w = x.shape[0], x.shape[1], self.w
        rows = (x.reshape(B * W, MODEL) @ w.kda_in).view(B * W, 3 * H, D)
        q, k = torch.empty(2, B * W, H, D, dtype=BF, device="cuda")
        kda.kda_qk_norm_rope(rows[:, :H], rows[:, H:2 * H], w.unit, w.unit, q, k, eps=1e-6 / D)
        v = rows[:, 2 * H:].contiguous()
        gates = (x.reshape(B * W, MODEL) @ w.kda_gate).float()
        g = -5.0 * torch.sigmoid(gates[:, :H * D] - 2.0).view(B * W, H, D)
        beta = torch.sigmoid(gates[:, H * D:]).contiguous()
        out = torch.empty(B * W, H, D, dtype=BF, device="cuda")
        if drafts:
            self.record = torch.empty(kda.kda_replay_bytes(B, W, H, D, D, kda.BF16), dtype=torch.uint8, device="cuda")
            kda.kda_verify(*(t.view(B, W, *t.shape[1:]) for t in (q, k, v, g, beta)), self.pool, self.slots,
                           out.view(B, W, H, D), self.record)
        elif W == 1:
            kda.kda_decode_step(q, k, v, g, beta, self.pool, self.slots, out)
        else:
            cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * W
            args = (q, k, v, g, beta, cu, W, self.pool, self.slots, out)
            ws = torch.empty(max(16, kda.kda_prefill_workspace_size(*args)), dtype=torch.uint8, device="cuda")
            kda.kda_prefill_varlen(*args, workspace=ws)
        return (out.view(B, W, H * D) @ w.kda_out).view(B, W, MODEL)

    def attention_layer(self, x, prompt=False):
        """x [B, W, MODEL]: W new tokens of every request written into the cache and attending over it; a whole prompt
        attends over itself."""
        B, W, w = x.shape[0], x.shape[1], self.w
        rows = (x.reshape(B * W, MODEL) @ w.qkv).view(B * W, H + 2 * HKV, D)
        at = self.lens[:, None] + torch.arange(W, device="cuda", dtype=torch.int32)  # positions of the new tokens
        q, k = torch.empty(B, W, H, D, dtype=BF, device="cuda"), torch.empty(B * W, HKV, D, dtype=BF, device="cuda")
        kda.kda_qk_norm_rope(rows[:, :H], rows[:, H:H + HKV], w.q_norm, w.k_norm, q.view(B * W, H, D), k, cos=self.cos,
                             sin=self.sin, positions=at.flatten())
        pages = torch.gather(self.table, 1, (at // self.page).long()).long()
        kda.kda_kv_write(k, rows[:, H + HKV:], self.k, self.v, (pages * self.page + at % self.page).flatten(),
                         **self.scales)
        self.lens += W
        out = torch.empty_like(q)
        if prompt:
            cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * W
            kda.kda_prefill_attention(q.view(B * W, H, D), k, rows[:, H + HKV:], cu, W, out.view(B * W, H, D))
            return (out.view(B, W, H * D) @ w.attn_out).view(B, W, MODEL)
        ws = torch.empty(kda.kda_paged_attention_workspace_size(B, W, H, HKV, D), dtype=torch.uint8, device="cuda")
        kda.kda_paged_attention(q, self.k, self.v, self.table, self.lens, out, ws, **self.scales)
        return (out.view(B, W, H * D) @ w.attn_out).view(B, W, MODEL)

    def __call__(self, tokens, prompt=False, drafts=False):
        """tokens [B, W] -> logits [B, W, VOCAB] fp32.  prompt: the requests' first tokens, all at once; drafts: a window of
        which `commit` keeps what was accepted."""
        x = self.w.embed[tokens]
        x = x + self.kda_layer(x, drafts)
        x = x + self.attention_layer(x, prompt)
        return x.float() @ self.w.head.float()

    def commit(self, accepted, window):
        """The first accepted[b] tokens of request b's window (int32) become part of its state; the cache's other rows are
        written over by the next."""
        kda.kda_verify_replay(self.pool, self.slots, self.record, accepted, window, H, D, D, kda.BF16)
        self.lens += accepted - window


def generate(prompt, tokens, cache, window):
    """Greedy tokens [B, prompt + tokens] and the logits of every position but the last."""
    m = Model(Weights(), prompt.shape[0], prompt.shape[1] + tokens, cache)
    logits = [m(prompt[:, i:i + window]) for i in range(0, prompt.shape[1], window)]
    out = prompt
    for _ in range(tokens):
        out = torch.cat((out, logits[-1][:, -1:].argmax(-1)), 1)
        logits.append(m(out[:, -1:]))
    return out, torch.cat(logits, 1)


def replay(sequence, cache, window):
    """Logits of a finished sequence taken in windows."""
    m = Model(Weights(), sequence.shape[0], sequence.shape[1], cache)
    return torch.cat([m(sequence[:, i:i + window]) for i in range(0, sequence.shape[1], window)], 1)


def looked_up(text, n):
    """The n tokens that followed the last token's latest earlier occurrence in the text (repeated where there are fewer)."""
    at = next((i for i in range(len(text) - 2, -1, -1) if text[i] == text[-1]), len(text) - 2)
    found = text[at + 1:at + 1 + n]
    return found + [found[-1]] * (n - len(found))


def speculate(prompt, tokens, cache, drafts, temperature=0.5):
    """At least `tokens` more tokens for each request of prompt [B, T], by windows with that many drafts: the texts, and the
    accepted drafts per window."""
    B, W = prompt.shape[0], drafts + 1
    # a request that is done goes on until the last is
    m = Model(Weights(), B, prompt.shape[1] + (tokens + 1) * W, cache)
    texts = prompt.tolist()
    logits = m(prompt, prompt=True)[:, -1:]
    accepted = torch.empty(B, dtype=torch.int32, device="cuda")
    got = torch.empty(B, 1, dtype=torch.int32, device="cuda")
    nothing = torch.empty(B, 0, dtype=torch.int32, device="cuda")
    kda.kda_verify_accept(torch.softmax(logits / temperature, -1), nothing, torch.rand(B, 1, device="cuda"), accepted, got)
    for text, row in zip(texts, got.tolist()):
        text.append(row[0])
    got, taken = torch.empty(B, W, dtype=torch.int32, device="cuda"), []
    while min(map(len, texts)) < prompt.shape[1] + tokens:
        window = torch.tensor([text[-1:] + looked_up(text, drafts) for text in texts], device="cuda")
        probs = torch.softmax(m(window, drafts=True) / temperature, -1)
        kda.kda_verify_accept(probs, window[:, 1:].int().contiguous(), torch.rand(B, W, device="cuda"), accepted, got)
        m.commit(accepted, W)
        for text, row, n in zip(texts, got.tolist(), accepted.tolist()):
            text += row[:n]
            taken.append(n - 1)
    return texts, taken


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=200)
    ap.add_argument("--tokens", type=int, default=24)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="e4m3")
    ap.add_argument("--drafts", type=int, default=0)
    a = ap.parse_args(argv)
    torch.manual_seed(1)
    prompt = torch.randint(0, VOCAB, (a.requests, a.prompt), device="cuda")
    sequence, stepped = generate(prompt, a.tokens, a.cache, window=32)
    at_once = replay(sequence, a.cache, window=48)
    torch.cuda.synchronize()
    difference = float((stepped - at_once).abs().max() / at_once.std())
    for row in sequence[:2, a.prompt:].tolist():
        print("generated:", *row[:16], "..." if len(row) > 16 else "")
    print(f"largest difference of a logit, step by step against windows: {difference:.2e} of the logits' spread")
    if a.drafts:
        texts, taken = speculate(prompt, a.tokens, a.cache, a.drafts)
        print("with drafts:", *texts[0][a.prompt:a.prompt + 16], "...")
        print(f"{sum(taken) / len(taken):.2f} of {a.drafts} drafts accepted a window")
    return difference


if __name__ == "__main__":
    main()
