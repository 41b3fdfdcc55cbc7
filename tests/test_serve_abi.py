"""The host checks of the paged-cache, tree-attention and log-probability entry points (no GPU): what is
refused before any CUDA call, and calls with nothing to do."""
import ctypes as C

import pytest
import torch

import shared_routed_expert_b200 as m
from shared_routed_expert_b200 import _lib, build

FAKE = 1 << 20          # aligned non-null addresses; the host checks never dereference them
OK, BAD, UNSUP, WS = _lib.MOE_OK, _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def cache(**kw):
    f = dict(k=FAKE, v=FAKE, page_stride=2 * 16 * 128, head_stride=16 * 128, slot_stride=128, num_pages=4, page_size=16,
             n_kv=2, head_dim=128, dtype=_lib.MOE_BF16, k_scale=1.0, v_scale=1.0)
    f.update(kw)
    return _lib.moe_kv_cache(**f)


def batch(**kw):
    f = dict(q_start=FAKE, ctx_len=FAKE, page_table=FAKE, B=2, max_pages=2, max_new=8)
    f.update(kw)
    return _lib.moe_kv_batch(**f)


BAD_CACHES = [
    (dict(k=None), BAD), (dict(v=FAKE + 8), BAD), (dict(num_pages=0), BAD), (dict(n_kv=0), BAD), (dict(head_dim=96), UNSUP),
    (dict(page_size=8), UNSUP), (dict(page_size=48), UNSUP), (dict(page_size=512), UNSUP), (dict(dtype=_lib.MOE_F32), UNSUP),
    (dict(slot_stride=64), BAD), (dict(slot_stride=132), BAD), (dict(head_stride=-2048), BAD),
    (dict(page_stride=(1 << 40)), BAD), (dict(k_scale=0.5), BAD), (dict(dtype=_lib.MOE_E4M3, v_scale=0.0), BAD),
    (dict(dtype=_lib.MOE_E4M3, k_scale=float("nan")), BAD), (dict(dtype=_lib.MOE_E4M3, k_scale=float("inf")), BAD),
    (dict(n_kv=2000), UNSUP),
]
BAD_BATCHES = [
    (dict(B=-1), BAD), (dict(B=4097), UNSUP), (dict(max_pages=0), BAD), (dict(q_start=None), BAD), (dict(ctx_len=FAKE + 2), BAD),
    (dict(page_table=None), BAD), (dict(max_new=-1), BAD), (dict(max_new=(1 << 20) + 1), UNSUP),
]


def append(L, c=None, b=None, **over):
    a = dict(T=4, n_q=4, rot=64, eps=1e-5, qkv=FAKE, qs=8 * 128, pos=FAKE, max_pos=10, qw=FAKE, kw=FAKE, cs=FAKE, qo=2 * FAKE,
             os=4 * 128, bad=None, st=None)
    a.update(over)
    return L.moe_qk_norm_rope_append(C.byref(c or cache()), C.byref(b or batch()), *a.values())


def attend(L, c=None, b=None, **over):
    a = dict(T=4, n_q=4, scale=0.1, q=FAKE, qs=512, mask=None, words=0, out=FAKE, os=512, lse=None, ws=FAKE, n=1 << 40, st=None)
    a.update(over)
    return L.moe_tree_attention(C.byref(c or cache()), C.byref(b or batch()), *a.values())


def compact(L, c=None, b=None, **over):
    a = dict(layers=1, ls=0, acc=FAKE, most=4, n=FAKE, bad=None, st=None)
    a.update(over)
    return L.moe_kv_compact(C.byref(c or cache()), C.byref(b or batch()), *a.values())


def logprobs(L, **over):
    a = dict(T=2, V=100, dt=_lib.MOE_F32, x=FAKE, stride=100, targets=FAKE, n=2, lp=FAKE, ent=None, ids=FAKE, top=FAKE, st=None)
    a.update(over)
    return L.moe_token_logprobs(*a.values())


@pytest.mark.parametrize("call", [append, attend, compact])
def test_bad_caches_and_batches_are_refused(L, call):
    for kw, want in BAD_CACHES:
        assert call(L, c=cache(**kw)) == want, kw
    for kw, want in BAD_BATCHES:
        assert call(L, b=batch(**kw)) == want, kw
    # strides over dimensions of size 1 are not looked at
    assert call(L, c=cache(num_pages=1, page_stride=3, n_kv=1, head_stride=-5), b=batch(B=0)) == OK


def test_null_structs(L):
    assert L.moe_qk_norm_rope_append(None, None, 1, 1, 0, 0.0, FAKE, 8, None, 0, None, None, None, FAKE, 8, None, None) == BAD
    assert L.moe_tree_attention(C.byref(cache()), None, 1, 2, 0.0, FAKE, 8, None, 0, FAKE, 8, None, FAKE, 1, None) == BAD
    assert L.moe_kv_compact(None, C.byref(batch()), 1, 0, FAKE, 1, FAKE, None, None) == BAD
    assert L.moe_tree_attention_workspace_size(None, 4, 4) == 0


def test_append_refusals(L):
    for kw, want in [(dict(T=-1), BAD), (dict(T=(1 << 20) + 1), UNSUP), (dict(n_q=3), BAD), (dict(n_q=0), BAD), (dict(eps=-1.0), BAD),
                     (dict(eps=float("nan")), BAD), (dict(qkv=None), BAD), (dict(qkv=FAKE + 8), BAD), (dict(qs=8 * 128 - 8), BAD),
                     (dict(qs=8 * 128 + 4), BAD), (dict(qo=None), BAD), (dict(os=504), BAD), (dict(pos=None), BAD),
                     (dict(max_pos=0), BAD), (dict(cs=None), BAD), (dict(cs=FAKE + 4), BAD), (dict(qw=FAKE + 2), BAD),
                     (dict(rot=130), UNSUP), (dict(rot=6), UNSUP), (dict(qo=FAKE), BAD)]:      # in place: one stride
        assert append(L, **kw) == want, kw
    assert append(L, T=0) == OK
    assert append(L, b=batch(B=0)) == OK


def test_attention_refusals(L):
    for kw, want in [(dict(T=-1), BAD), (dict(n_q=5), BAD), (dict(n_q=2048, qs=2048 * 128, os=2048 * 128), UNSUP),
                     (dict(scale=float("inf")), BAD), (dict(scale=float("nan")), BAD), (dict(q=None), BAD), (dict(q=FAKE + 2), BAD),
                     (dict(qs=511), BAD), (dict(qs=508), BAD), (dict(out=None), BAD), (dict(os=516), BAD), (dict(lse=FAKE + 2), BAD),
                     (dict(ws=None), BAD), (dict(ws=FAKE + 16), BAD), (dict(n=10), WS), (dict(words=1), BAD),
                     (dict(out=FAKE, os=520), BAD), (dict(mask=FAKE), BAD), (dict(mask=FAKE + 4, words=1), BAD), (dict(mask=FAKE, words=65), UNSUP)]:
        assert attend(L, **kw) == want, kw
    assert attend(L, mask=FAKE, words=1, b=batch(max_new=65)) == BAD
    for b in (batch(B=0), batch(max_new=0)):
        assert attend(L, b=b) == OK
    assert attend(L, T=0) == OK


def test_a_scale_that_overflows_with_the_keys_scale_is_refused(L):
    f8 = dict(dtype=_lib.MOE_E4M3, k_scale=1e30)
    assert attend(L, c=cache(**f8), b=batch(B=0), scale=1e8) == OK       # 1.4e38
    assert attend(L, c=cache(**f8), b=batch(B=0), scale=1e9) == BAD
    assert attend(L, b=batch(B=0), scale=3e38) == BAD                    # ... with log2 e


def test_compact_refusals(L):
    for kw, want in [(dict(layers=0), BAD), (dict(layers=5000), UNSUP), (dict(layers=2, ls=100), BAD), (dict(layers=2, ls=132), BAD),
                     (dict(acc=None), BAD), (dict(n=None), BAD), (dict(most=0), BAD), (dict(most=1025), UNSUP)]:
        assert compact(L, **kw) == want, kw
    assert compact(L, b=batch(B=0)) == OK


def test_logprobs_refusals(L):
    for kw, want in [(dict(T=-1), BAD), (dict(V=0), BAD), (dict(V=(1 << 24) + 1, stride=1 << 25), UNSUP), (dict(stride=99), BAD),
                     (dict(dt=_lib.MOE_E4M3), UNSUP), (dict(x=None), BAD), (dict(x=FAKE + 2), BAD), (dict(n=33), UNSUP),
                     (dict(V=1, n=2), BAD), (dict(targets=None), BAD), (dict(lp=None), BAD), (dict(ids=None), BAD),
                     (dict(top=None), BAD), (dict(n=0), BAD), (dict(n=-1), BAD), (dict(ent=FAKE + 1), BAD)]:
        assert logprobs(L, **kw) == want, kw
    assert logprobs(L, T=0) == OK


def test_counters_have_to_be_aligned(L):
    """The kernels add to them with 4-byte atomics, which an odd address would fault."""
    for off in (1, 2, 3):
        assert append(L, bad=FAKE + off) == BAD
        assert compact(L, bad=FAKE + off) == BAD
        assert append(L, bad=FAKE + off, b=batch(B=0)) == BAD and compact(L, bad=FAKE + off, b=batch(B=0)) == BAD
    assert append(L, bad=FAKE + 4, b=batch(B=0)) == OK and compact(L, bad=FAKE + 4, b=batch(B=0)) == OK


def test_arrays_without_elements_may_be_null(L):
    """An empty tensor's address is NULL: a step without rows or sequences is no error; what does not
    depend on them is still looked at."""
    none = dict(B=0, q_start=None, ctx_len=None, page_table=None, max_new=0)
    for b in (batch(), batch(**none)):
        assert append(L, b=b, T=0, qkv=None, qo=None, pos=None) == OK
        assert attend(L, b=b, T=0, q=None, out=None) == OK
        assert attend(L, b=b, T=0, q=None, out=None, mask=None, words=1) == OK
    assert compact(L, b=batch(**none), acc=None, n=None) == OK
    assert logprobs(L, T=0, x=None, targets=None, lp=None, ids=None, top=None) == OK
    assert logprobs(L, T=0, x=None, targets=None, lp=None, ids=None, top=None, n=0) == OK
    assert append(L, T=0, qkv=None, qo=None, pos=None, cs=None) == BAD
    assert append(L, T=0, qkv=None, qo=None, pos=None, rot=6) == UNSUP
    assert attend(L, T=0, q=None, out=None, ws=None) == BAD
    assert attend(L, T=0, q=None, out=None, n=10) == WS
    assert attend(L, T=4, mask=None, words=1) == BAD
    assert compact(L, b=batch(**none), acc=None, n=None, most=0) == BAD
    assert logprobs(L, T=0, x=None, targets=None, lp=None, ids=None, top=None, V=0) == BAD


def test_python_binding_refuses_tensors_that_do_not_fit():
    k = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    c = m.make_kv_cache(k, k.clone())
    assert (c.page_size, c.n_kv, c.head_dim, c.page_stride, c.head_stride, c.slot_stride) == (16, 2, 128, 4096, 2048, 128)
    n = m.make_kv_cache(k.view(4, 16, 2, 128).transpose(1, 2), k.clone().view(4, 16, 2, 128).transpose(1, 2))
    assert (n.page_size, n.n_kv, n.head_stride, n.slot_stride) == (16, 2, 128, 256)
    with pytest.raises(ValueError):
        m.make_kv_cache(k, k.transpose(1, 2))
    with pytest.raises(TypeError):
        m.make_kv_cache(k.float(), k.float())
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    b = m.make_kv_batch(i32(3), i32(2), i32(2, 4), 5)
    assert (b.B, b.max_pages, b.max_new) == (2, 4, 5)
    with pytest.raises(TypeError):
        m.make_kv_batch(i32(3).long(), i32(2), i32(2, 4), 5)
    with pytest.raises(ValueError):
        m.make_kv_batch(i32(2), i32(2), i32(2, 4), 5)
    q = torch.zeros(4, 4 * 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        m.moe_tree_attention(c, b, 4, q[:, :256], q, i32(4))
    with pytest.raises(TypeError):
        m.moe_tree_attention(c, b, 4, q.float(), q, i32(4))
    with pytest.raises(ValueError):
        m.moe_tree_attention(c, b, 4, q, q, i32(4), lse=torch.zeros(4, 3))
    with pytest.raises(TypeError):
        m.moe_token_logprobs(torch.zeros(2, 8, dtype=torch.float16), i32(2), torch.zeros(2))
    with pytest.raises(ValueError):
        m.moe_token_logprobs(torch.zeros(2, 8), i32(3), torch.zeros(2))
    with pytest.raises(ValueError):
        m.moe_qk_norm_rope_append(c, b, 4, 64, 1e-5, q, i32(4), None, None, torch.zeros(10, 64), q)


def test_alternatives_need_both_outputs():
    """Ids without log probabilities, or the other way round, are refused, not left unwritten."""
    ids, top = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    for kw in (dict(top_ids=ids), dict(top_logprobs=top), dict(top_ids=ids[:, :0], top_logprobs=top),
               dict(top_ids=ids, top_logprobs=top[:, :2])):
        with pytest.raises(ValueError, match="top"):
            m.moe_token_logprobs(torch.zeros(2, 8), None, None, **kw)


def test_layers_behind_the_allocation_are_refused():
    layers = torch.zeros(3, 4, 2, 16, 128, dtype=torch.bfloat16)
    more = torch.zeros(3, 4, 2, 16, 128, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    b = m.make_kv_batch(i32(3), i32(2), i32(2, 4), 5)
    one = layers[0].numel()
    for first, n, fits in ((0, 3, True), (0, 4, False), (1, 2, True), (1, 3, False)):
        c = m.make_kv_cache(layers[first], more[first])
        with pytest.raises(ValueError, match="CUDA device" if fits else "behind"):
            m.moe_kv_compact(c, b, i32(2, 4), i32(2), n_layers=n, layer_stride=one)
    c = m.make_kv_cache(layers[0], more[0].clone())          # V's layers are not there
    with pytest.raises(ValueError, match="behind"):
        m.moe_kv_compact(c, b, i32(2, 4), i32(2), n_layers=2, layer_stride=one)


def test_calls_run_on_the_device_of_their_tensors(monkeypatch):
    """Tensors of another device than the current one: it is made current for the launch; tensors of
    the CPU, or of several devices, are refused."""
    seen = []

    class on:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            seen.append(("enter", self.d))

        def __exit__(self, *exc):
            seen.append(("exit", self.d))

    class stream:
        cuda_stream = 77

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "device", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: stream)
    _lib._launch("f", lambda *a: seen.append(a) or 0, 1, None, 5)
    assert seen == [("enter", 1), (5, 77), ("exit", 1)]
    with pytest.raises(_lib.MoeError):
        _lib._launch("f", lambda *a: 2, 1, stream, 5)
    with pytest.raises(ValueError):
        _lib._launch("f", lambda *a: 0, -1, None)
    k = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    c = m.make_kv_cache(k, k.clone())
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    b = m.make_kv_batch(i32(3), i32(2), i32(2, 4), 5)
    q = torch.zeros(4, 4 * 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                          # everything on the CPU
        m.moe_tree_attention(c, b, 4, q, torch.empty_like(q), torch.zeros(1 << 10, dtype=torch.uint8))
    c.device = 0
    with pytest.raises(ValueError):                          # the cache elsewhere
        m.moe_tree_attention(c, b, 4, q, torch.empty_like(q), torch.zeros(1 << 10, dtype=torch.uint8))
    with pytest.raises(ValueError):
        m.moe_token_logprobs(torch.zeros(2, 8), i32(2), torch.zeros(2))
