"""ctypes binding of libsre_moe.so (include/moe.h). Argument marshalling only:
every step of the layer runs in the library's CUDA kernels. There is no CPU
path; if the library is missing, loading fails loudly."""
from __future__ import annotations

import ctypes as C
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsre_moe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE = 0, 1, 2, 3
MOE_ERR_CUDA, MOE_ERR_TIMEOUT, MOE_ERR_DEVICE = 4, 5, 6
MOE_F32, MOE_BF16, MOE_E4M3 = 0, 1, 2
(MOE_FFN_AUTO, MOE_FFN_SIMT, MOE_FFN_TCGEN05, MOE_FFN_TCGEN05_M128, MOE_FFN_TCGEN05_M256,
 MOE_FFN_TCGEN05_PAIR, MOE_FFN_TCGEN05_WIDE, MOE_FFN_TCGEN05_SWAP) = 0, 1, 2, 3, 4, 5, 6, 7
MOE_FFN_COMBINE_FOLD = 512         # flag: the fused layer's aggregation inside its down-projection
DTYPES = {"f32": MOE_F32, "bf16": MOE_BF16, "e4m3": MOE_E4M3}

EXPORTS = ("moe_workspace_size", "moe_route_topk", "moe_permute", "moe_grouped_ffn",
           "moe_combine", "moe_forward", "moe_quant_rows_e4m3", "moe_get_status",
           "moe_clear_status", "moe_status_string", "moe_launch_count", "moe_profile_enable",
           "moe_profile_reset", "moe_profile_read", "moe_inject_wait_timeout",
           "moe_permute_noalloc", "moe_qk_norm_rope", "moe_cast_f32_bf16", "moe_inject_fold_timeout",
           "moe_inject_route_timeout", "moe_qk_norm_rope_append", "moe_tree_attention",
           "moe_tree_attention_workspace_size", "moe_kv_compact", "moe_token_logprobs",
           "moe_inject_attention_timeout")


class MoeError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn}: {status_string(code)} (status {code})")


class moe_shape(C.Structure):
    _fields_ = [("T", C.c_int32), ("H", C.c_int32), ("I", C.c_int32), ("n_routed", C.c_int32),
                ("top_k", C.c_int32), ("shared_id", C.c_int32), ("shared_weight", C.c_float),
                ("renormalize", C.c_int32), ("act_dtype", C.c_int32), ("w_dtype", C.c_int32),
                ("routed_scale", C.c_float), ("bias_select_only", C.c_int32), ("out_f32", C.c_int32)]


class moe_kv_cache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("page_stride", C.c_int64), ("head_stride", C.c_int64),
                ("slot_stride", C.c_int64), ("num_pages", C.c_int32), ("page_size", C.c_int32), ("n_kv", C.c_int32),
                ("head_dim", C.c_int32), ("dtype", C.c_int32), ("k_scale", C.c_float), ("v_scale", C.c_float)]


class moe_kv_batch(C.Structure):
    _fields_ = [("q_start", C.c_void_p), ("ctx_len", C.c_void_p), ("page_table", C.c_void_p), ("B", C.c_int32),
                ("max_pages", C.c_int32), ("max_new", C.c_int32)]


_lib = None


def lib() -> C.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run python -m shared_routed_expert_b200.build")
        L = C.CDLL(LIB_PATH)
        p, i, u64, sz, f = C.c_void_p, C.c_int, C.c_uint64, C.c_size_t, C.c_float
        S = C.POINTER(moe_shape)
        L.moe_workspace_size.restype = sz
        L.moe_workspace_size.argtypes = [S, i]
        L.moe_route_topk.restype = i
        L.moe_route_topk.argtypes = [S, p, p, p, p, p, p, p, sz, p]
        L.moe_permute.restype = i
        L.moe_permute.argtypes = [S, p, p, p, p, p, p, sz, p]
        L.moe_grouped_ffn.restype = i
        L.moe_grouped_ffn.argtypes = [S, p, p, p, p, p, p, p, p, p, sz, i, p]
        L.moe_combine.restype = i
        L.moe_combine.argtypes = [S, p, p, p, p, p]
        L.moe_forward.restype = i
        L.moe_forward.argtypes = [S, p, p, p, p, p, p, p, i, p, p, sz, i, p]
        L.moe_quant_rows_e4m3.restype = i
        L.moe_quant_rows_e4m3.argtypes = [C.c_int32, C.c_int32, p, p, p, p]
        L.moe_get_status.restype = i
        L.moe_get_status.argtypes = [p, p]
        L.moe_clear_status.restype = i
        L.moe_clear_status.argtypes = [p, p]
        L.moe_status_string.restype = C.c_char_p
        L.moe_status_string.argtypes = [i]
        L.moe_launch_count.restype = u64
        L.moe_launch_count.argtypes = []
        L.moe_profile_enable.restype = None
        L.moe_profile_enable.argtypes = [i]
        L.moe_profile_reset.restype = None
        L.moe_profile_reset.argtypes = []
        L.moe_profile_read.restype = i
        L.moe_profile_read.argtypes = [C.c_char_p, C.POINTER(C.c_int64), C.POINTER(C.c_double)]
        L.moe_permute_noalloc.restype = i
        L.moe_permute_noalloc.argtypes = [S, p, p, p, p, p, p]
        L.moe_inject_wait_timeout.restype = None
        L.moe_inject_wait_timeout.argtypes = [i]
        L.moe_inject_fold_timeout.restype = None
        L.moe_inject_fold_timeout.argtypes = [i]
        L.moe_inject_route_timeout.restype = None
        L.moe_inject_route_timeout.argtypes = [i]
        L.moe_cast_f32_bf16.restype = i
        L.moe_cast_f32_bf16.argtypes = [sz, p, p, p]
        L.moe_qk_norm_rope.restype = i
        L.moe_qk_norm_rope.argtypes = [i, i, i, i, i, f, p, p, i, p, p, p, p, p]
        L.moe_inject_attention_timeout.restype = None
        L.moe_inject_attention_timeout.argtypes = [i]
        i64, KC, KB = C.c_int64, C.POINTER(moe_kv_cache), C.POINTER(moe_kv_batch)
        L.moe_qk_norm_rope_append.restype = i
        L.moe_qk_norm_rope_append.argtypes = [KC, KB, i, i, i, f, p, i64, p, i, p, p, p, p, i64, p, p]
        L.moe_tree_attention_workspace_size.restype = sz
        L.moe_tree_attention_workspace_size.argtypes = [KC, i, i]
        L.moe_tree_attention.restype = i
        L.moe_tree_attention.argtypes = [KC, KB, i, i, f, p, i64, p, i, p, i64, p, p, sz, p]
        L.moe_kv_compact.restype = i
        L.moe_kv_compact.argtypes = [KC, KB, i, i64, p, i, p, p, p]
        L.moe_token_logprobs.restype = i
        L.moe_token_logprobs.argtypes = [i, i, i, p, i64, p, i, p, p, p, p, p]
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().moe_status_string(code).decode()


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, rc: int):
    if rc != MOE_OK:
        raise MoeError(fn, rc)


def make_shape(cfg, T: int | None = None) -> moe_shape:
    """moe_shape of a LayerConfig-like object (T overrides cfg.T)."""
    return moe_shape(cfg.T if T is None else T, cfg.H, cfg.I, cfg.n_routed, cfg.top_k,
                     cfg.shared_id, cfg.shared_weight, int(cfg.renormalize),
                     DTYPES[cfg.act_dtype], DTYPES[cfg.w_dtype],
                     float(getattr(cfg, "routed_scale", 1.0)), int(getattr(cfg, "bias_select_only", False)),
                     int(getattr(cfg, "out_f32", False)))


def moe_workspace_size(shape: moe_shape, fuse_shared: bool = True) -> int:
    n = lib().moe_workspace_size(C.byref(shape), int(fuse_shared))
    if n == 0:
        raise MoeError("moe_workspace_size", MOE_ERR_INVALID_ARG)
    return n


def alloc_workspace(shape: moe_shape, fuse_shared: bool = True, device="cuda") -> torch.Tensor:
    n = moe_workspace_size(shape, fuse_shared)
    ws = torch.zeros(n + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + n]


def moe_route_topk(shape, x, router_w, router_bias, ids, weights, logits, ws, stream=None):
    _check("moe_route_topk", lib().moe_route_topk(
        C.byref(shape), _p(x), _p(router_w), _p(router_bias), _p(ids), _p(weights), _p(logits),
        _p(ws), ws.numel(), _stream(stream)))


def moe_permute(shape, ids, counts, offsets, perm, inv, ws, stream=None):
    _check("moe_permute", lib().moe_permute(
        C.byref(shape), _p(ids), _p(counts), _p(offsets), _p(perm), _p(inv), _p(ws), ws.numel(),
        _stream(stream)))


def moe_grouped_ffn(shape, x, perm, offsets, w13, s13, w2, s2, y, ws, impl=MOE_FFN_AUTO,
                    stream=None):
    _check("moe_grouped_ffn", lib().moe_grouped_ffn(
        C.byref(shape), _p(x), _p(perm), _p(offsets), _p(w13), _p(s13), _p(w2), _p(s2), _p(y),
        _p(ws), ws.numel(), impl, _stream(stream)))


def moe_combine(shape, y, inv, weights, out, stream=None):
    _check("moe_combine", lib().moe_combine(
        C.byref(shape), _p(y), _p(inv), _p(weights), _p(out), _stream(stream)))


def moe_forward(shape, x, router_w, router_bias, w13, s13, w2, s2, fuse_shared, out, ws,
                impl=MOE_FFN_AUTO, stream=None):
    _check("moe_forward", lib().moe_forward(
        C.byref(shape), _p(x), _p(router_w), _p(router_bias), _p(w13), _p(s13), _p(w2), _p(s2),
        int(fuse_shared), _p(out), _p(ws), ws.numel(), impl, _stream(stream)))


def moe_permute_noalloc(shape, ids, counts, offsets, perm, inv, stream=None):
    """moe_permute for callers that cannot allocate: the library's own fixed
    device scratch replaces the workspace (see include/moe.h)."""
    _check("moe_permute_noalloc", lib().moe_permute_noalloc(
        C.byref(shape), _p(ids), _p(counts), _p(offsets), _p(perm), _p(inv), _stream(stream)))


def moe_qk_norm_rope(cfg, qkv, positions, q_norm_w, k_norm_w, cos_sin, bad_positions=None, stream=None):
    """In place on the q and k heads of qkv [T, (n_q + 2 n_kv) d] bf16; cfg
    carries T, n_q, n_kv, d, rot, eps and max_pos = cos_sin rows."""
    _check("moe_qk_norm_rope", lib().moe_qk_norm_rope(
        qkv.shape[0], cfg.n_q, cfg.n_kv, cfg.d, cfg.rot, cfg.eps, _p(qkv), _p(positions), cos_sin.shape[0],
        _p(q_norm_w), _p(k_norm_w), _p(cos_sin if cfg.rot > 0 else None), _p(bad_positions), _stream(stream)))


def moe_cast_f32_bf16(inp, out, stream=None):
    """out (bf16) = inp (fp32) rounded to nearest even, same element count."""
    _check("moe_cast_f32_bf16", lib().moe_cast_f32_bf16(inp.numel(), _p(inp), _p(out), _stream(stream)))


def moe_quant_rows_e4m3(rows, cols, inp, codes, scales, stream=None):
    _check("moe_quant_rows_e4m3", lib().moe_quant_rows_e4m3(
        rows, cols, _p(inp), _p(codes), _p(scales), _stream(stream)))


# ---- paged cache, tree attention, log probabilities

# (the checks are written for speed: a decoding step calls these once per layer, and a
# launch is shorter than a few dozen attribute look-ups)

def _rows(name, t, dtype, device):
    """Row stride and row length of a tensor whose rows are dense: [T, n] or [T, heads, d]."""
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, not {dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}")
    stride, shape = t.stride(), t.shape
    if len(shape) == 2 and stride[1] == 1 and shape[0] > 1:
        return stride[0], shape[1]
    inner = 1
    for i in range(len(shape) - 1, 0, -1):
        if stride[i] != inner and shape[i] != 1:
            raise ValueError(f"{name}: the rows of a [T, ...] tensor have to be dense")
        inner *= shape[i]
    return (stride[0] if shape[0] > 1 else max(inner, stride[0])), inner


def _dense(name, t, dtype, shape, device):
    """Address of a contiguous tensor of that type and shape (None: any shape) on that device."""
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, not {dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} has to be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} is {tuple(t.shape)}, not {shape}")
    return t.data_ptr()


def _launch(name, fn, device, stream, *args):
    """Calls an entry point on `stream` (None: the device's current one) with the tensors'
    device current."""
    if device < 0:
        raise ValueError(f"{name}: the tensors have to be on a CUDA device")
    if device == torch._C._cuda_getDevice():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _stream(stream))
    if rc != MOE_OK:
        raise MoeError(name, rc)


def _device_of(t, cache, batch):
    """The device index that a call's tensor, cache and batch share."""
    device = t.get_device()
    if cache.device != device or batch.device != device:
        raise ValueError(f"the cache and the batch have to be on {t.device}, where the rows are")
    return device


def make_kv_cache(k, v, k_scale: float = 1.0, v_scale: float = 1.0) -> moe_kv_cache:
    """moe_kv_cache of K and V tensors [pages, kv heads, page size, head dim] (views of
    any layout with dense head rows, the same for both): bf16, or uint8 / float8_e4m3fn
    for E4M3 codes of value / scale. It keeps the tensors alive."""
    if k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride() or k.device != v.device or k.dim() != 4:
        raise ValueError("k and v: [pages, kv heads, page size, head dim], alike in type, strides and device")
    if k.stride(3) != 1:
        raise ValueError("the head dimension has to be dense")
    dt = {torch.bfloat16: MOE_BF16, torch.uint8: MOE_E4M3, torch.float8_e4m3fn: MOE_E4M3}.get(k.dtype)
    if dt is None:
        raise TypeError(f"a cache of {k.dtype}")
    c = moe_kv_cache(k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2), k.shape[0], k.shape[2],
                     k.shape[1], k.shape[3], dt, k_scale, v_scale)
    c.tensors, c.device = (k, v), k.get_device()
    # elements from a view's first to behind its last one, and to the end of its allocation
    c.extent = 1 + sum((n - 1) * s for n, s in zip(k.shape, k.stride())) if k.numel() else 0
    c.room = min(t.untyped_storage().nbytes() // t.element_size() - t.storage_offset() for t in (k, v))
    return c


def make_kv_batch(q_start, ctx_len, page_table, max_new: int) -> moe_kv_batch:
    """moe_kv_batch of int32 device tensors q_start [B + 1], ctx_len [B], page_table
    [B, max_pages]; it keeps them alive, and calls read what they hold at the time."""
    B = ctx_len.shape[0]
    i32, device = torch.int32, ctx_len.get_device()
    b = moe_kv_batch(_dense("q_start", q_start, i32, (B + 1,), device), _dense("ctx_len", ctx_len, i32, (B,), device),
                     _dense("page_table", page_table, i32, (B, page_table.shape[1]), device), B, page_table.shape[1], max_new)
    b.tensors, b.device = (q_start, ctx_len, page_table), device
    return b


def moe_qk_norm_rope_append(cache, batch, n_q: int, rot: int, eps: float, qkv, positions, q_norm_w, k_norm_w, cos_sin,
                            q_out, bad_tokens=None, stream=None):
    """qkv [T, (n_q + 2 n_kv) d] bf16 -> q_out [T, n_q d] bf16 and the cache (see
    include/moe.h); q_norm_w / k_norm_w None: no norm, rot 0: no rotation."""
    d, T, dev = cache.head_dim, qkv.shape[0], _device_of(qkv, cache, batch)
    bf16 = torch.bfloat16
    qs, qn = _rows("qkv", qkv, bf16, dev)
    os_, on = _rows("q_out", q_out, bf16, dev)
    width = (n_q + 2 * cache.n_kv) * d
    if qn != width or q_out.shape[0] != T or (on != n_q * d and on != width):
        raise ValueError("qkv [T, (n_q + 2 n_kv) d] and q_out [T, n_q d]")
    qw = None if q_norm_w is None else _dense("q_norm_w", q_norm_w, bf16, (d,), dev)
    kw = None if k_norm_w is None else _dense("k_norm_w", k_norm_w, bf16, (d,), dev)
    bad = None if bad_tokens is None else _dense("bad_tokens", bad_tokens, torch.int32, None, dev)
    max_pos, pos, cs = 0, None, None
    if rot > 0:
        max_pos = cos_sin.shape[0]
        pos = _dense("positions", positions, torch.int32, (T,), dev)
        cs = _dense("cos_sin", cos_sin, torch.float32, (max_pos, rot), dev)
    _launch("moe_qk_norm_rope_append", lib().moe_qk_norm_rope_append, dev, stream, cache, batch, T, n_q, rot, eps,
            qkv.data_ptr(), qs, pos, max_pos, qw, kw, cs, q_out.data_ptr(), os_, bad)


def moe_tree_attention_workspace_size(cache, n_q: int, T: int) -> int:
    n = lib().moe_tree_attention_workspace_size(C.byref(cache), n_q, T)
    if n == 0:
        raise MoeError("moe_tree_attention_workspace_size", MOE_ERR_INVALID_ARG)
    return n


def alloc_tree_attention_workspace(cache, n_q: int, T: int, device=None) -> torch.Tensor:
    """Zeroed workspace of moe_tree_attention for at most T rows over this cache."""
    n = moe_tree_attention_workspace_size(cache, n_q, T)
    ws = torch.zeros(n + 256, dtype=torch.uint8, device=cache.tensors[0].device if device is None else device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + n]


def moe_tree_attention(cache, batch, n_q: int, q, out, ws, tree_mask=None, lse=None, scale: float | None = None,
                       stream=None):
    """q [T, n_q d] bf16 over the cache -> out [T, n_q d] bf16, lse [T, n_q] fp32 or None;
    tree_mask [T, words] int64 (bit j: the row sees its sequence's new token j) or None
    for a chain; scale None: 1 / sqrt(head dim)."""
    T, d, dev = q.shape[0], cache.head_dim, _device_of(q, cache, batch)
    qs, qn = _rows("q", q, torch.bfloat16, dev)
    os_, on = _rows("out", out, torch.bfloat16, dev)
    if out.shape[0] != T or qn != n_q * d or on != qn:
        raise ValueError("q and out: [T, n_q d]")
    ls = None if lse is None else _dense("lse", lse, torch.float32, (T, n_q), dev)
    words, mask = 0, None
    if tree_mask is not None:
        words = tree_mask.shape[1]
        mask = _dense("tree_mask", tree_mask, torch.int64, (T, words), dev)
    wp = _dense("ws", ws, torch.uint8, None, dev)
    _launch("moe_tree_attention", lib().moe_tree_attention, dev, stream, cache, batch, T, n_q,
            d ** -0.5 if scale is None else scale, q.data_ptr(), qs, mask, words, out.data_ptr(), os_, ls, wp, ws.numel())


def moe_kv_compact(cache, batch, accepted, n_accepted, n_layers: int = 1, layer_stride: int = 0, bad_seqs=None,
                   stream=None):
    """Moves accepted [B, max_accept] int32 new tokens' keys and values to the front of
    their sequences' new tokens, in place, in n_layers caches layer_stride elements apart
    (the cache is the first one, all layers lie in its tensors' allocations)."""
    B, most, dev = batch.B, accepted.shape[1], _device_of(accepted, cache, batch)
    if n_layers > 1 and (n_layers - 1) * layer_stride + cache.extent > cache.room:
        raise ValueError("the layers reach behind the cache's allocation")
    acc = _dense("accepted", accepted, torch.int32, (B, most), dev)
    n = _dense("n_accepted", n_accepted, torch.int32, (B,), dev)
    bad = None if bad_seqs is None else _dense("bad_seqs", bad_seqs, torch.int32, None, dev)
    _launch("moe_kv_compact", lib().moe_kv_compact, dev, stream, cache, batch, n_layers, layer_stride, acc, most, n, bad)


def moe_token_logprobs(logits, targets, logprobs, entropy=None, top_ids=None, top_logprobs=None, stream=None):
    """logits [T, V] (bf16 or fp32, dense rows) and targets [T] int32 -> logprobs [T],
    entropy [T], top_ids / top_logprobs [T, n], each fp32 (ids int32) or None."""
    T, V = logits.shape
    dt, dev = logits.dtype, logits.get_device()
    code = MOE_BF16 if dt == torch.bfloat16 else MOE_F32 if dt == torch.float32 else None
    if code is None:
        raise TypeError(f"logits are {dt}, not bf16 or fp32")
    f32 = torch.float32
    tg = None if targets is None else _dense("targets", targets, torch.int32, (T,), dev)
    lp = None if logprobs is None else _dense("logprobs", logprobs, f32, (T,), dev)
    en = None if entropy is None else _dense("entropy", entropy, f32, (T,), dev)
    if (top_ids is None) != (top_logprobs is None) or (top_ids is not None and top_ids.shape != top_logprobs.shape):
        raise ValueError("top_ids and top_logprobs: both [T, n], or neither")
    n = 0 if top_ids is None else top_ids.shape[1]
    ids = top = None
    if n:
        ids = _dense("top_ids", top_ids, torch.int32, (T, n), dev)
        top = _dense("top_logprobs", top_logprobs, f32, (T, n), dev)
    _launch("moe_token_logprobs", lib().moe_token_logprobs, dev, stream, T, V, code, logits.data_ptr(),
            _rows("logits", logits, dt, dev)[0], tg, n, lp, en, ids, top)


def moe_get_status(ws, stream=None) -> int:
    return lib().moe_get_status(_p(ws), _stream(stream))


def moe_clear_status(ws, stream=None):
    _check("moe_clear_status", lib().moe_clear_status(_p(ws), _stream(stream)))


def moe_launch_count() -> int:
    return int(lib().moe_launch_count())


_prof_on = False


def moe_profile_enable(on: bool):
    global _prof_on
    lib().moe_profile_enable(int(on))
    _prof_on = bool(on)


def profile_enabled() -> bool:
    """Whether per-kernel event timing was last switched on through this module."""
    return _prof_on


def moe_profile_reset():
    lib().moe_profile_reset()


def moe_inject_wait_timeout(n_calls: int):
    lib().moe_inject_wait_timeout(int(n_calls))


def moe_inject_fold_timeout(n_calls: int):
    lib().moe_inject_fold_timeout(int(n_calls))


def moe_inject_route_timeout(n_calls: int):
    lib().moe_inject_route_timeout(int(n_calls))


def moe_inject_attention_timeout(n_calls: int):
    lib().moe_inject_attention_timeout(int(n_calls))


def moe_profile_read(name: str):
    n = C.c_int64()
    ms = C.c_double()
    _check("moe_profile_read", lib().moe_profile_read(name.encode(), C.byref(n), C.byref(ms)))
    return n.value, ms.value
