"""Refusals of the prompt attention's calls and of the drafts' acceptance, none of which needs a GPU."""
import ctypes

import pytest
import torch

import kda_gated_delta_rule_gb300 as kda
from kda_gated_delta_rule_gb300 import _build

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
T, HQ, HKV, D, B, W, V = 6, 4, 2, 32, 3, 4, 11
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kda.load()


def z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


def prompt_kw():
    return dict(q=z(T, HQ, D, dtype=BF), k=z(T, HKV, D, dtype=BF), v=z(T, HKV, D, dtype=BF), cu_seqlens=z(3, dtype=I32),
                out=z(T, HQ, D), lse=z(T, HQ))


def grad_kw():
    return dict(prompt_kw(), d_out=z(T, HQ, D, dtype=BF), dq=z(T, HQ, D), dk=z(T, HKV, D), dv=z(T, HKV, D),
                workspace=z(16, dtype=torch.uint8))


def accept_kw():
    return dict(target_probs=z(B, W, V), draft_tokens=z(B, W - 1, dtype=I32), uniform=z(B, W), accepted=z(B, dtype=I32),
                tokens=z(B, W, dtype=I32), draft_probs=z(B, W - 1, V), num_drafts=z(B, dtype=I32))


CALLS = {"kda_prefill_attention": (prompt_kw, {"max_seqlen": 6}), "kda_prefill_attention_backward": (grad_kw, {"max_seqlen": 6}),
         "kda_verify_accept": (accept_kw, {})}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_matching_tensors_reach_the_device_check(name):
    tensors, more = CALLS[name]
    with pytest.raises(ValueError, match="expected contiguous CUDA tensors"):
        getattr(kda, name)(**tensors(), **more)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_each_mismatched_tensor_is_refused(name):
    make, more = CALLS[name]
    n = 0
    for arg, t in make().items():
        if arg == "workspace":
            continue
        wrong = [torch.zeros(*t.shape, 1, dtype=t.dtype)]  # rank
        if arg != "cu_seqlens":  # whose length is the caller's
            wrong.append(torch.zeros(t.shape[0] + 1, *t.shape[1:], dtype=t.dtype))
        for w in wrong:
            with pytest.raises(ValueError) as e:
                getattr(kda, name)(**dict(make(), **{arg: w}), **more)
            assert "contiguous CUDA" not in str(e.value), arg
            n += 1
        with pytest.raises((TypeError, ValueError)) as e:
            getattr(kda, name)(**dict(make(), **{arg: t.to(torch.float64)}), **more)
        assert "contiguous CUDA" not in str(e.value), arg
    assert n


def test_heads_and_empty_shapes_are_refused():
    for bad in (dict(k=z(T, 3, D, dtype=BF), v=z(T, 3, D, dtype=BF)), dict(k=z(T, 0, D, dtype=BF), v=z(T, 0, D, dtype=BF))):
        with pytest.raises(ValueError, match="multiple of the keys'"):
            kda.kda_prefill_attention(**dict(prompt_kw(), **bad), max_seqlen=6)
    with pytest.raises(ValueError, match="offsets"):
        kda.kda_prefill_attention(**dict(prompt_kw(), cu_seqlens=z(0, dtype=I32)), max_seqlen=6)
    with pytest.raises(ValueError, match="lse"):
        kda.kda_prefill_attention_backward(**dict(grad_kw(), lse=None), max_seqlen=6)
    with pytest.raises(ValueError, match="at least one"):
        kda.kda_verify_accept(z(B, 0, V), z(B, 0, dtype=I32), z(B, 0), z(B, dtype=I32), z(B, 0, dtype=I32))
    with pytest.raises(ValueError, match="dev_status"):
        kda.kda_verify_accept(**accept_kw(), dev_status=z(1, dtype=I32))


def prompt_args(**kw):
    a = kda.PrefillAttentionArgs()
    for n in ("q", "k", "v", "cu_seqlens", "out", "lse"):
        setattr(a, n, 1 << 20)
    a.q_stride, a.k_stride, a.v_stride, a.out_stride = HQ * D, HKV * D, HKV * D, HQ * D
    a.in_dtype = a.out_dtype = kda.BF16
    a.T, a.Hq, a.Hkv, a.d, a.N, a.max_seqlen, a.scale = T, HQ, HKV, D, 2, 6, 0.1
    for n, x in kw.items():
        setattr(a, n, x)
    return a


BAD_PROMPTS = [dict(in_dtype=7), dict(out_dtype=-1), dict(T=-1), dict(T=2 ** 31 - 1), dict(N=-1), dict(N=65536), dict(Hq=0), dict(Hkv=0),
               dict(Hq=5), dict(Hq=65536, Hkv=1), dict(max_seqlen=-1), dict(window=-1), dict(softcap=-1.0),
               dict(softcap=float("nan")), dict(softcap=float("inf")), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(q=0), dict(k=0), dict(v=0), dict(out=0), dict(cu_seqlens=0), dict(q=(1 << 20) + 8), dict(cu_seqlens=(1 << 20) + 2),
               dict(lse=(1 << 20) + 2), dict(q_stride=HQ * D - 8), dict(k_stride=HKV * D + 4), dict(out_stride=0),
               dict(T=2 ** 30, Hq=65535, Hkv=1), dict(N=65535, Hq=65534, Hkv=2, q_stride=65534 * D, out_stride=65534 * D)]


@pytest.mark.parametrize("bad", BAD_PROMPTS, ids=str)
def test_the_entry_point_refuses(lib, bad):
    a = prompt_args(**bad)
    assert lib.kda_prefill_attention(ctypes.byref(a), None) == INVALID
    g = kda.PrefillAttentionGrads()
    assert lib.kda_prefill_attention_backward(ctypes.byref(a), ctypes.byref(g), None) == INVALID


def grads(**kw):
    g = kda.PrefillAttentionGrads()
    for n in ("d_out", "dq", "dk", "dv", "workspace"):
        setattr(g, n, 1 << 20)
    g.d_out_stride, g.dq_stride, g.dk_stride, g.dv_stride = HQ * D, HQ * D, HKV * D, HKV * D
    g.grad_dtype, g.workspace_bytes = kda.BF16, 1 << 30
    for n, x in kw.items():
        setattr(g, n, x)
    return g


@pytest.mark.parametrize("bad", [dict(d_out=0), dict(dq=0), dict(dk=0), dict(dv=0), dict(grad_dtype=3), dict(dq_stride=8), dict(dk_stride=HKV * D + 1),
                                 dict(d_out=(1 << 20) + 4), dict(workspace=(1 << 20) + 8)], ids=str)
def test_the_gradient_refuses(lib, bad):
    assert lib.kda_prefill_attention_backward(ctypes.byref(prompt_args()), ctypes.byref(grads(**bad)), None) == INVALID


def test_head_sizes_workspaces_and_empty_calls(lib):
    assert lib.kda_prefill_attention(None, None) == INVALID
    assert lib.kda_prefill_attention(ctypes.byref(prompt_args(d=48)), None) == UNSUPPORTED
    assert lib.kda_prefill_attention_backward(ctypes.byref(prompt_args(d=48)), ctypes.byref(grads()), None) == UNSUPPORTED
    assert lib.kda_prefill_attention_backward(ctypes.byref(prompt_args()), None, None) == INVALID
    assert lib.kda_prefill_attention_backward(ctypes.byref(prompt_args(lse=0)), ctypes.byref(grads()), None) == INVALID
    size = kda.kda_prefill_attention_backward_workspace_size(T, 2, HQ, HKV, D)
    assert size >= T * HQ * 8
    for g in (grads(workspace=0), grads(workspace_bytes=size - 1)):
        assert lib.kda_prefill_attention_backward(ctypes.byref(prompt_args()), ctypes.byref(g), None) == WORKSPACE
    for bad in ((-1, 2, 4, 2, 32), (6, -1, 4, 2, 32), (6, 2, 0, 2, 32), (6, 2, 4, 3, 32), (6, 2, 4, 2, 48)):
        assert kda.kda_prefill_attention_backward_workspace_size(*bad) == 0
    for empty in (dict(T=0, q=0, out=0), dict(N=0, cu_seqlens=0)):
        assert lib.kda_prefill_attention(ctypes.byref(prompt_args(**empty)), None) == 0
        assert lib.kda_prefill_attention_backward(ctypes.byref(prompt_args(**empty)), ctypes.byref(grads(workspace=0)), None) == 0


def accept_args(**kw):
    a = kda.VerifyAcceptArgs()
    for n in ("target_probs", "draft_probs", "draft_tokens", "uniform", "accepted", "tokens"):
        setattr(a, n, 1 << 20)
    a.dtype, a.B, a.W, a.V = kda.F32, B, W, V
    for n, x in kw.items():
        setattr(a, n, x)
    return a


@pytest.mark.parametrize("bad", [dict(dtype=9), dict(B=-1), dict(W=0), dict(V=0), dict(V=2 ** 30 + 1), dict(B=2 ** 28), dict(target_probs=0),
                                 dict(draft_tokens=0), dict(uniform=0), dict(accepted=0), dict(tokens=0), dict(target_probs=(1 << 20) + 2),
                                 dict(draft_probs=(1 << 20) + 2), dict(num_drafts=(1 << 20) + 2), dict(tokens=(1 << 20) + 1)], ids=str)
def test_the_acceptance_refuses(lib, bad):
    assert lib.kda_verify_accept(ctypes.byref(accept_args(**bad)), None) == INVALID


def test_no_requests(lib):
    assert lib.kda_verify_accept(None, None) == INVALID
    assert lib.kda_verify_accept(ctypes.byref(accept_args(B=0, target_probs=0, tokens=0)), None) == 0
