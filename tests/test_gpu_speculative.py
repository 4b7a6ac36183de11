"""The prompt attention, the draft windows and the acceptance together, as a server of the example's hybrid model uses them."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("hybrid_decode", os.path.join(ROOT, "examples", "hybrid_decode.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def prompts(example, B, T, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, example.VOCAB, (B, T), generator=g, device="cuda")


@pytest.mark.parametrize("T", [1, 65, 300])
def test_a_prompt_at_once_and_in_windows(cuda, example, T):
    """As in the test of steps and windows: both round every layer's outputs to bf16 from sums in other orders."""
    prompt = prompts(example, 3, T, T)
    at_once = example.Model(example.Weights(), 3, T + 8, "bf16")
    windows = example.Model(example.Weights(), 3, T + 8, "bf16")
    a = at_once(prompt, prompt=True)
    b = torch.cat([windows(prompt[:, i:i + 32]) for i in range(0, T, 32)], 1)
    assert float((a - b).abs().max() / b.std()) <= 6 * 4 * 2 ** -8
    # and the cache and the states are left alike
    step = prompts(example, 3, 1, 1)
    a, b = at_once(step), windows(step)
    assert float((a - b).abs().max() / b.std()) <= 6 * 4 * 2 ** -8


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("drafts", [1, 3, 6])
def test_greedy_windows_give_the_greedy_text(cuda, example, cache, drafts):
    """The target is certain of its most likely token, the drafts are the text that single steps gave, wrong here and there: every
    window ends at the first wrong draft, and the text is the same."""
    B, T, n, W = 4, 50, 30, drafts + 1
    prompt = prompts(example, B, T, 7)
    certain = lambda logits: torch.nn.functional.one_hot(logits.argmax(-1), example.VOCAB).float()  # noqa: E731
    m = example.Model(example.Weights(), B, T + n + 2 * W, cache)
    step = m(prompt, prompt=True)[:, -1:].argmax(-1)
    steps = [step]
    for _ in range(n + W):
        step = m(step).argmax(-1)
        steps.append(step)
    want = torch.cat(steps, 1).tolist()
    m = example.Model(example.Weights(), B, T + n + 2 * W, cache)
    first = m(prompt, prompt=True)[:, -1:].argmax(-1)
    texts = first.tolist()
    accepted = torch.empty(B, dtype=torch.int32, device="cuda")
    got = torch.empty(B, W, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(drafts)
    windows = 0
    while min(map(len, texts)) < n:
        window, right = [], []
        for text, true in zip(texts, want):
            at = min(len(text), n)  # a request that is done repeats its end
            guess = true[at:at + drafts]
            ok = (torch.rand(drafts, generator=g) < 0.7).tolist() if len(text) <= n else [False] * drafts
            window.append([text[-1]] + [t if k else (t + 1) % example.VOCAB for t, k in zip(guess, ok)])
            right.append(ok.index(False) if False in ok else drafts)
        window = torch.tensor(window, device="cuda")
        uniform = torch.rand(B, W, generator=g).cuda()
        cuda.kda_verify_accept(certain(m(window, drafts=True)), window[:, 1:].int().contiguous(), uniform, accepted, got)
        m.commit(accepted, W)
        windows += 1
        for b, (row, k) in enumerate(zip(got.tolist(), accepted.tolist())):
            if len(texts[b]) <= n:
                assert k == right[b] + 1 and row[k:] == [-1] * (W - k), (windows, b)
            texts[b] += row[:k]
    for text, true in zip(texts, want):
        assert text[:n] == true[:n]
    assert windows < n


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_the_example_generates_by_windows(cuda, example, cache):
    torch.manual_seed(3)
    prompt = prompts(example, 3, 40, 9)
    texts, taken = example.speculate(prompt, 12, cache, 3)
    assert all(len(t) >= 52 and t[:40] == p for t, p in zip(texts, prompt.tolist()))
    assert all(0 <= x < example.VOCAB for t in texts for x in t) and all(0 <= n <= 3 for n in taken)
