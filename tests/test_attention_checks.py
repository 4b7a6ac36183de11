"""Refusals of the softmax-attention calls: the binding's shape, type and stride checks and the C entry points' own, none
of which needs a GPU."""
import ctypes

import pytest
import torch

import kda_gated_delta_rule_gb300 as kda
from kda_gated_delta_rule_gb300 import _build

BF, F32, I32, I64, E4 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.float8_e4m3fn
DEVICE_MSG = "expected contiguous CUDA tensors"
T, Hq, Hkv, D, P, PAGE, B, W = 5, 4, 2, 32, 3, 16, 2, 3
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kda.load()


def z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


def norm_kw():
    return dict(q=z(T, Hq, D, dtype=BF), k=z(T, Hkv, D, dtype=BF), q_weight=z(D), k_weight=z(D),
                q_out=z(T, Hq, D), k_out=z(T, Hkv, D), cos=z(9, D // 2), sin=z(9, D // 2), positions=z(T, dtype=I32))


def grad_kw():
    kw = {n: t for n, t in norm_kw().items() if n not in ("q_out", "k_out")}
    return dict(kw, d_q_out=z(T, Hq, D, dtype=BF), d_k_out=z(T, Hkv, D, dtype=BF), dq=z(T, Hq, D), dk=z(T, Hkv, D),
                dq_weight=z(D), dk_weight=z(D), workspace=z(16, dtype=torch.uint8))


def cache_kw():
    return dict(k_pages=z(P, Hkv, PAGE, D).to(E4), v_pages=z(P, Hkv, PAGE, D).to(E4), k_scales=z(P, Hkv, PAGE),
                v_scales=z(P, Hkv, PAGE))


def write_kw():
    return dict(cache_kw(), k=z(T, Hkv, D, dtype=BF), v=z(T, Hkv, D, dtype=BF), slots=z(T, dtype=I64))


def read_kw():
    return dict(cache_kw(), slots=z(T, dtype=I64), k_out=z(T, Hkv, D), v_out=z(T, Hkv, D))


def attend_kw():
    return dict(cache_kw(), q=z(B, W, Hq, D, dtype=BF), block_table=z(B, 4, dtype=I32), seq_lens=z(B, dtype=I32),
                out=z(B, W, Hq, D), lse=z(B, W, Hq), workspace=z(16, dtype=torch.uint8))


CALLS = {"kda_qk_norm_rope": norm_kw, "kda_qk_norm_rope_backward": grad_kw, "kda_kv_write": write_kw,
         "kda_kv_read": read_kw, "kda_paged_attention": attend_kw}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_matching_tensors_reach_the_device_check(name):
    with pytest.raises(ValueError, match=DEVICE_MSG):
        getattr(kda, name)(**CALLS[name]())


@pytest.mark.parametrize("name", sorted(CALLS))
def test_each_mismatched_tensor_is_refused(name):
    kw, n = CALLS[name](), 0
    for arg, t in kw.items():
        if arg == "workspace":
            continue
        grown = list(t.shape)
        grown[-1] += 1
        bad = [torch.zeros(*grown).to(t.dtype), t.unsqueeze(0), t.to(torch.float64)]
        if arg == "block_table":  # any number of pages
            bad = bad[1:]
        for b in bad:
            with pytest.raises((ValueError, TypeError)) as e:
                getattr(kda, name)(**dict(kw, **{arg: b}))
            assert DEVICE_MSG not in str(e.value), (name, arg)
            n += 1
    assert n > 10


def test_paired_and_ranged_arguments():
    kw = norm_kw()
    for missing in ("cos", "sin", "positions"):
        with pytest.raises(ValueError, match="cos, sin and positions"):
            kda.kda_qk_norm_rope(**dict(kw, **{missing: None}))
    with pytest.raises(ValueError, match="cos"):  # 10 channels are no multiple of 16
        kda.kda_qk_norm_rope(**dict(kw, cos=z(9, 5), sin=z(9, 5)))
    with pytest.raises(ValueError, match="cos"):  # more than the head has
        kda.kda_qk_norm_rope(**dict(kw, cos=z(9, 24), sin=z(9, 24)))
    for name, make in (("kda_kv_write", write_kw), ("kda_kv_read", read_kw), ("kda_paged_attention", attend_kw)):
        kw = make()
        with pytest.raises(ValueError, match="needs both"):
            getattr(kda, name)(**dict(kw, v_scales=None))
        with pytest.raises(ValueError, match="has none"):
            getattr(kda, name)(**dict(kw, k_pages=kw["k_pages"].to(BF), v_pages=kw["v_pages"].to(BF)))
        with pytest.raises(ValueError, match="multiple of 16"):
            cut = {n: kw[n][:, :, :8] for n in cache_kw()}
            getattr(kda, name)(**dict(kw, **cut))
    with pytest.raises(ValueError, match="multiple of the cache"):
        kda.kda_paged_attention(**dict(attend_kw(), q=z(B, W, 3, D), out=z(B, W, 3, D), lse=z(B, W, 3)))


def norm_args(**over):
    a = kda.QkNormRopeArgs(16, 16, 4 * 64, 2 * 64, 1, 16, 16, 16, 16, 16, 100, 64, 0, 1e-6, 5, 4, 2, 64, 16, 16, 4 * 64,
                           2 * 64, 1, None)
    for n, v in over.items():
        setattr(a, n, v)
    return a


@pytest.mark.parametrize("over,code", [
    (dict(d=48), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(in_dtype=7), INVALID), (dict(out_dtype=-1), INVALID),
    (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(rot=8), INVALID), (dict(rot=80), INVALID), (dict(rot=-16), INVALID),
    (dict(q=None), INVALID), (dict(k=8), INVALID), (dict(q_stride=4 * 64 - 8), INVALID), (dict(k_stride=2 * 64 + 4), INVALID),
    (dict(q_out_stride=0), INVALID), (dict(q_out=18), INVALID), (dict(k_out=None), INVALID), (dict(q_weight=4), INVALID),
    (dict(cos=None), INVALID), (dict(sin=4), INVALID), (dict(positions=2), INVALID), (dict(num_positions=-1), INVALID),
    (dict(T=2 ** 31), INVALID), (dict(T=2 ** 29), INVALID),
])
def test_norm_refusals(lib, over, code):
    assert lib.kda_qk_norm_rope(norm_args(**over), None) == code
    big = 1 << 24
    assert lib.kda_qk_norm_rope_backward(norm_args(**over), 16, 16, 1, 16, 16, 16, big, None) == code


def test_norm_backward_refusals(lib):
    need = lib.kda_qk_norm_rope_backward_workspace_size(5, 4, 2, 64)
    assert need == 608 * 2 * 64 * 4
    call = lambda dq=16, dk=16, dt=1, wq=16, wk=16, ws=16, n=need: lib.kda_qk_norm_rope_backward(  # noqa: E731
        norm_args(), dq, dk, dt, wq, wk, ws, n, None)
    assert call(dq=None) == call(dk=8) == call(dt=5) == call(wq=None) == call(wk=4) == call(ws=8) == INVALID
    assert call(ws=None) == call(n=need - 1) == WORKSPACE
    assert lib.kda_qk_norm_rope(None, None) == INVALID
    assert lib.kda_qk_norm_rope(norm_args(T=0, q=None, q_out=None), None) == 0
    for bad in ((-1, 4, 2, 64), (5, 0, 2, 64), (5, 4, 0, 64), (5, 4, 2, 65)):
        assert lib.kda_qk_norm_rope_backward_workspace_size(*bad) == 0


def cache(**over):
    c = kda.KvCache(16, 16, 16, 16, 1, 10, 16, 2, 64)
    for n, v in over.items():
        setattr(c, n, v)
    return c


BAD_CACHES = [(dict(type=2), INVALID), (dict(num_pages=-1), INVALID), (dict(page_size=0), INVALID),
              (dict(page_size=24), INVALID), (dict(page_size=-16), INVALID), (dict(Hkv=0), INVALID), (dict(d=80), UNSUPPORTED),
              (dict(k_pages=None), INVALID), (dict(v_pages=8), INVALID), (dict(k_scales=None), INVALID),
              (dict(v_scales=4), INVALID)]


@pytest.mark.parametrize("over,code", BAD_CACHES)
def test_cache_refusals(lib, over, code):
    c = cache(**over)
    assert lib.kda_kv_write(16, 16, 128, 128, 1, 3, 16, c, None, None) == code
    assert lib.kda_kv_read(c, 16, 3, 16, 16, 1, None, None) == code
    a = attn_args()
    a.cache = c
    assert lib.kda_paged_attention(a, None) == code


def test_write_and_read_refusals(lib):
    c = cache()
    w = lambda k=16, v=16, ks=128, vs=128, dt=1, t=3, s=16: lib.kda_kv_write(k, v, ks, vs, dt, t, s, c, None, None)  # noqa: E731
    assert w(k=None) == w(v=8) == w(ks=120) == w(vs=132) == w(dt=3) == w(t=-1) == w(s=None) == w(s=4) == INVALID
    assert w(t=2 ** 31) == w(t=2 ** 29) == INVALID
    assert w(k=None, v=None, s=None, t=0) == 0
    assert lib.kda_kv_write(16, 16, 128, 128, 1, 3, 16, None, None, None) == INVALID
    r = lambda s=16, t=3, k=16, v=16, dt=1: lib.kda_kv_read(c, s, t, k, v, dt, None, None)  # noqa: E731
    assert r(s=None) == r(s=12) == r(t=-1) == r(k=None) == r(v=2) == r(dt=9) == INVALID
    assert r(t=0, s=None, k=None, v=None) == 0


def attn_args(**over):
    a = kda.PagedAttentionArgs(16, 1, 2, 3, 4, cache(), 16, 5, 16, 0.1, 0.0, 0, 16, 1, None, 16, 1 << 40, None)
    for n, v in over.items():
        setattr(a, n, v)
    return a


@pytest.mark.parametrize("over,code", [
    (dict(q_dtype=4), INVALID), (dict(out_dtype=4), INVALID), (dict(B=-1), INVALID), (dict(W=0), INVALID),
    (dict(Hq=0), INVALID), (dict(Hq=3), INVALID), (dict(max_pages=-1), INVALID), (dict(window=-1), INVALID),
    (dict(softcap=-1.0), INVALID), (dict(softcap=float("nan")), INVALID), (dict(softcap=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(q=None), INVALID), (dict(out=8), INVALID),
    (dict(lse=2), INVALID), (dict(block_table=None), INVALID), (dict(block_table=2), INVALID),
    (dict(seq_lens=None), INVALID), (dict(seq_lens=6), INVALID), (dict(workspace=None), WORKSPACE),
    (dict(workspace=8), INVALID), (dict(workspace_bytes=1000), WORKSPACE), (dict(B=2 ** 30, W=8), INVALID),
])
def test_attention_refusals(lib, over, code):
    assert lib.kda_paged_attention(attn_args(**over), None) == code


def test_attention_sizes(lib):
    assert lib.kda_paged_attention(None, None) == INVALID
    assert lib.kda_paged_attention(attn_args(B=0, q=None, out=None, seq_lens=None, workspace=None), None) == 0
    size = kda.kda_paged_attention_workspace_size
    assert size(1, 1, 32, 8, 128) > 0 and size(1000, 1, 32, 8, 128) == size(1, 1, 32, 8, 128)
    for bad in ((-1, 1, 4, 2, 64), (1, 0, 4, 2, 64), (1, 1, 4, 3, 64), (1, 1, 4, 2, 65), (1, 1, 0, 2, 64), (1, 1, 4, 0, 64)):
        assert size(*bad) == 0
    for n, mirror in (("kda_qk_norm_rope_args", kda.QkNormRopeArgs), ("kda_kv_cache", kda.KvCache),
                      ("kda_paged_attention_args", kda.PagedAttentionArgs)):
        assert getattr(lib, n + "_bytes")() == ctypes.sizeof(mirror)
