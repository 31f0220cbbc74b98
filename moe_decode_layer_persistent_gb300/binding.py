"""ctypes binding of libmk.so: the mk_* C ABI with the same names.

Argument marshalling only: every step of the decode layer runs in the CUDA
library.  Tensors are passed as device pointers (torch tensors are accepted
for convenience; only ``data_ptr()`` is read).  Loading fails loudly if the
library has not been built -- there is no CPU fallback.
"""

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmk.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libmk.so not built (run __graft_entry__.build()): %s" % LIB_PATH)
_lib = ctypes.CDLL(LIB_PATH)

MK_OK = 0
STATUS_NAMES = {0: "MK_OK", 1: "MK_ERR_INVALID_ARG", 2: "MK_ERR_UNSUPPORTED", 3: "MK_ERR_CUDA",
                4: "MK_ERR_OOM", 5: "MK_ERR_TIMEOUT", 6: "MK_ERR_DEVICE_FAULT"}
MK_FFN_MOE_NVFP4 = 0
MK_FFN_DENSE_SWIGLU_BF16 = 1
MK_FIRST_LAYER = 0x1
MK_FUSE_NEXT_QKV = 0x2
MK_TOPK_RENORM = 0x4
MK_PREFETCH_NEXT_KV = 0x8
MK_ERR_INVALID_ARG = 1
MK_BF16, MK_FP16 = 0, 1
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}

_vp = ctypes.c_void_p


class MkError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__("%s -> %s" % (fn, STATUS_NAMES.get(status, status)))


class mk_layer_config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("window", ctypes.c_int32), ("ffn_kind", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("pooled_dim", ctypes.c_int32), ("expert_inter", ctypes.c_int32),
                ("dense_inter", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
                ("max_ctx", ctypes.c_int32), ("rms_eps", ctypes.c_float),
                ("flags", ctypes.c_uint32), ("prefetch_experts", ctypes.c_int32),
                ("wait_timeout_ns", ctypes.c_uint64)]


class mk_prefetch_stats(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_uint64), ("predicted", ctypes.c_uint64),
                ("active", ctypes.c_uint64), ("hits", ctypes.c_uint64)]


_WEIGHT_FIELDS = ["attn_norm_w", "w_qkv", "w_o", "ffn_norm_w", "w_router", "w_pool", "w_unpool",
                  "exp_gate_q", "exp_gate_s", "exp_gate_ts", "exp_up_q", "exp_up_s", "exp_up_ts",
                  "exp_down_q", "exp_down_s", "exp_down_ts", "w_gate", "w_up", "w_down",
                  "next_attn_norm_w", "next_w_qkv"]


class mk_layer_weights(ctypes.Structure):
    _fields_ = [(n, _vp) for n in _WEIGHT_FIELDS]


class mk_step_io(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int32), ("ctx_len", ctypes.c_int32),
                ("x_in", _vp), ("x_out", _vp), ("q_in", _vp), ("k_cache", _vp),
                ("v_cache", _vp), ("next_k_cache", _vp), ("next_v_cache", _vp),
                ("q_out", _vp), ("topk_idx_out", _vp), ("topk_w_out", _vp),
                ("tree_mask", ctypes.POINTER(ctypes.c_uint16))]


class mk_stack_io(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int32), ("ctx_len", ctypes.c_int32),
                ("x_in", _vp), ("x_out", _vp), ("k_caches", ctypes.POINTER(_vp)),
                ("v_caches", ctypes.POINTER(_vp)), ("topk_idx_out", _vp), ("topk_w_out", _vp),
                ("tree_mask", ctypes.POINTER(ctypes.c_uint16))]


class mk_layer_info(ctypes.Structure):
    _fields_ = [("grid", ctypes.c_int32), ("threads", ctypes.c_int32),
                ("smem_bytes", ctypes.c_int32), ("tmem_cols", ctypes.c_int32),
                ("scratch_bytes", ctypes.c_int64)]


_i32, _i64 = ctypes.c_int32, ctypes.c_int64


class mk_slots_io(ctypes.Structure):
    _fields_ = [("n_requests", _i32), ("n_rows", _i32), ("page_size", _i32), ("max_pages", _i32),
                ("table_stride", _i64), ("n_pages", _i32), ("n_free", _i32), ("prefix_len", _i32),
                ("cached_lens", _vp), ("new_lens", _vp), ("free_pages", _vp), ("free_head", _vp),
                ("block_table", _vp), ("cu_rows", _vp), ("lens", _vp), ("positions", _vp),
                ("slots", _vp), ("row_request", _vp), ("summary", _vp)]


class mk_rope_config(ctypes.Structure):
    _fields_ = [("head_dim", _i32), ("rot_dim", _i32), ("layout", _i32), ("scaling", _i32),
                ("theta", ctypes.c_double), ("factor", ctypes.c_double), ("orig_ctx", _i32),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("attn_factor", ctypes.c_double)]


class mk_rope_io(ctypes.Structure):
    _fields_ = [("n_rows", _i32), ("n_q_heads", _i32), ("n_kv_heads", _i32),
                ("head_dim", _i32), ("dtype", _i32),
                ("q", _vp), ("q_stride", _i64), ("q_out", _vp), ("q_out_stride", _i64),
                ("k", _vp), ("k_stride", _i64), ("v", _vp), ("v_stride", _i64),
                ("positions", _vp), ("slots", _vp), ("k_cache", _vp), ("v_cache", _vp),
                ("n_slots", _i64)]


class mk_prefix_attn_io(ctypes.Structure):
    _fields_ = [("n_requests", _i32), ("n_rows", _i32), ("n_q_heads", _i32), ("n_kv_heads", _i32),
                ("head_dim", _i32), ("dtype", _i32), ("page_size", _i32), ("n_pages", _i32),
                ("prefix_len", _i32), ("max_pages", _i32), ("table_stride", _i64),
                ("window", _i32), ("scale", ctypes.c_float), ("q", _vp), ("q_stride", _i64),
                ("k_cache", _vp), ("v_cache", _vp), ("prefix_pages", _vp), ("block_table", _vp),
                ("lens", _vp), ("cu_rows", _vp), ("tree_mask", _vp), ("out", _vp),
                ("out_stride", _i64), ("lse", _vp)]


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_c = ctypes
_lib_mk_layer_create = _sig("mk_layer_create", _c.c_int,
                            [_c.POINTER(mk_layer_config), _c.POINTER(mk_layer_weights),
                             _c.POINTER(_vp)])
_lib_mk_decode_step = _sig("mk_decode_step", _c.c_int, [_vp, _c.POINTER(mk_step_io), _vp])
_lib_mk_layer_status = _sig("mk_layer_status", _c.c_int, [_vp])
_lib_mk_layer_clear_status = _sig("mk_layer_clear_status", _c.c_int, [_vp])
_lib_mk_layer_destroy = _sig("mk_layer_destroy", None, [_vp])
_lib_mk_stack_create = _sig("mk_stack_create", _c.c_int, [_c.POINTER(_vp), _c.c_int32, _c.POINTER(_vp)])
_lib_mk_stack_step = _sig("mk_stack_step", _c.c_int, [_vp, _c.POINTER(mk_stack_io), _vp])
_lib_mk_stack_status = _sig("mk_stack_status", _c.c_int, [_vp])
_lib_mk_layer_prefetch_stats = _sig("mk_layer_prefetch_stats", _c.c_int, [_vp, _vp])
_lib_mk_stack_prefetch_stats = _sig("mk_stack_prefetch_stats", _c.c_int, [_vp, _vp])
_lib_mk_stack_destroy = _sig("mk_stack_destroy", None, [_vp])
_lib_mk_status_string = _sig("mk_status_string", _c.c_char_p, [_c.c_int])
_lib_mk_layer_get_info = _sig("mk_layer_get_info", _c.c_int, [_vp, _c.POINTER(mk_layer_info)])
_lib_mk_selftest_quantize = _sig("mk_selftest_quantize", _c.c_int,
                                 [_vp, _c.c_int32, _c.c_int32, _vp, _vp, _vp, _vp])
_lib_mk_selftest_mma = _sig("mk_selftest_mma", _c.c_int,
                            [_c.c_int32, _vp, _vp, _vp, _vp, _c.c_int32, _vp, _vp])

_lib_mk_get_timestamps = _sig("mk_get_timestamps", _c.c_int, [_vp, _c.c_void_p, _c.c_size_t])

_lib_mk_selftest_sync = _sig("mk_selftest_sync", _c.c_int,
                             [_c.c_int32, _c.c_int32, _c.POINTER(_c.c_double)])

_lib_mk_decode_step_noalloc = _sig("mk_decode_step_noalloc", _c.c_int,
                                   [_c.POINTER(mk_layer_config), _c.POINTER(mk_layer_weights),
                                    _c.POINTER(mk_step_io), _vp])

_lib_mk_build_slots = _sig("mk_build_slots", _c.c_int, [_c.POINTER(mk_slots_io), _vp])
_lib_mk_rope_create = _sig("mk_rope_create", _c.c_int, [_c.POINTER(mk_rope_config), _c.POINTER(_vp)])
_lib_mk_rope_destroy = _sig("mk_rope_destroy", None, [_vp])
_lib_mk_rope_apply = _sig("mk_rope_apply", _c.c_int, [_vp, _c.POINTER(mk_rope_io), _vp])
_lib_mk_prefix_attn_workspace = _sig("mk_prefix_attn_workspace", _c.c_int,
                                     [_c.POINTER(mk_prefix_attn_io), _c.POINTER(_i64)])
_lib_mk_prefix_attn = _sig("mk_prefix_attn", _c.c_int,
                           [_c.POINTER(mk_prefix_attn_io), _vp, _i64, _vp])
_lib_mk_prefix_attn_status = _sig("mk_prefix_attn_status", _c.c_int, [_vp])

EXPORTED = ["mk_layer_create", "mk_decode_step", "mk_decode_step_noalloc", "mk_layer_status", "mk_layer_clear_status",
            "mk_layer_destroy", "mk_stack_create", "mk_stack_step", "mk_stack_status",
            "mk_stack_destroy", "mk_status_string", "mk_layer_get_info", "mk_get_timestamps",
            "mk_layer_prefetch_stats", "mk_stack_prefetch_stats",
            "mk_build_slots", "mk_rope_create", "mk_rope_destroy", "mk_rope_apply",
            "mk_prefix_attn_workspace", "mk_prefix_attn", "mk_prefix_attn_status",
            "mk_selftest_quantize", "mk_selftest_mma", "mk_selftest_sync"]


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, st):
    if st != MK_OK:
        raise MkError(fn, st)


def mk_status_string(status):
    return _lib_mk_status_string(int(status)).decode()


def make_config(wl, flags=0, max_ctx=None, timeout_ns=0, window=None, prefetch_experts=None):
    """mk_layer_config from a workload/layer shape dict.  prefetch_experts:
    experts of the previous step prefetched into L2 (MoE; None = 0, off)."""
    c = mk_layer_config()
    c.hidden = wl["hidden"]
    c.n_q_heads = wl["n_q_heads"]
    c.n_kv_heads = wl["n_kv_heads"]
    c.head_dim = wl["head_dim"]
    c.window = wl["window"] if window is None else window
    if wl["ffn"] == "moe":
        c.ffn_kind = MK_FFN_MOE_NVFP4
        c.n_experts, c.top_k = wl["n_experts"], wl["top_k"]
        c.pooled_dim, c.expert_inter = wl["pooled_dim"], wl["expert_inter"]
    else:
        c.ffn_kind = MK_FFN_DENSE_SWIGLU_BF16
        c.dense_inter = wl["dense_inter"]
    c.max_tokens = 16
    c.max_ctx = max_ctx if max_ctx is not None else wl["ctx"] + 16
    c.rms_eps = 1e-6
    c.flags = flags
    if prefetch_experts is None:
        prefetch_experts = 0
    c.prefetch_experts = prefetch_experts
    c.wait_timeout_ns = timeout_ns
    return c


def mk_layer_create(cfg, weights):
    """cfg: mk_layer_config; weights: dict name -> tensor (missing = NULL)."""
    w = mk_layer_weights()
    for n in _WEIGHT_FIELDS:
        setattr(w, n, _ptr(weights.get(n)))
    h = _vp()
    _check("mk_layer_create", _lib_mk_layer_create(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(h)))
    return h.value


def _tree(io, tree_mask):
    """Host array of the token-tree masks (kept alive with the io struct)."""
    if tree_mask is None:
        return
    arr = (ctypes.c_uint16 * len(tree_mask))(*[int(m) for m in tree_mask])
    io.tree_mask = ctypes.cast(arr, ctypes.POINTER(ctypes.c_uint16))
    io._tree = arr


def make_step_io(T, ctx, x_in, x_out, k_cache, v_cache, q_in=None, next_k_cache=None,
                 next_v_cache=None, q_out=None, topk_idx_out=None, topk_w_out=None, tree_mask=None):
    """tree_mask: optional list of T ancestor-or-self bitmasks (token tree)."""
    io = mk_step_io()
    io.n_tokens, io.ctx_len = T, ctx
    io.x_in, io.x_out, io.q_in = _ptr(x_in), _ptr(x_out), _ptr(q_in)
    io.k_cache, io.v_cache = _ptr(k_cache), _ptr(v_cache)
    io.next_k_cache, io.next_v_cache, io.q_out = _ptr(next_k_cache), _ptr(next_v_cache), _ptr(q_out)
    io.topk_idx_out, io.topk_w_out = _ptr(topk_idx_out), _ptr(topk_w_out)
    _tree(io, tree_mask)
    return io


def mk_decode_step(layer, io, stream=None):
    _check("mk_decode_step", _lib_mk_decode_step(layer, ctypes.byref(io), _stream(stream)))


def mk_decode_step_noalloc(cfg, weights, io, stream=None):
    """One decode step without any device allocation (scratch in the
    library's fixed static array; small layers only)."""
    w = mk_layer_weights()
    for n in _WEIGHT_FIELDS:
        setattr(w, n, _ptr(weights.get(n)))
    _check("mk_decode_step_noalloc", _lib_mk_decode_step_noalloc(
        ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(io), _stream(stream)))


def mk_layer_status(layer):
    return _lib_mk_layer_status(layer)


def mk_layer_clear_status(layer):
    _check("mk_layer_clear_status", _lib_mk_layer_clear_status(layer))


def mk_layer_destroy(layer):
    _lib_mk_layer_destroy(layer)


def mk_layer_get_info(layer):
    info = mk_layer_info()
    _check("mk_layer_get_info", _lib_mk_layer_get_info(layer, ctypes.byref(info)))
    return {f: getattr(info, f) for f, _ in mk_layer_info._fields_}


def mk_stack_create(layers):
    arr = (_vp * len(layers))(*layers)
    h = _vp()
    _check("mk_stack_create", _lib_mk_stack_create(arr, len(layers), ctypes.byref(h)))
    return h.value


def make_stack_io(T, ctx, x_in, x_out, k_caches, v_caches, topk_idx_out=None, topk_w_out=None,
                  tree_mask=None):
    io = mk_stack_io()
    io.n_tokens, io.ctx_len = T, ctx
    io.x_in, io.x_out = _ptr(x_in), _ptr(x_out)
    kc = (_vp * len(k_caches))(*[_ptr(t) for t in k_caches])
    vc = (_vp * len(v_caches))(*[_ptr(t) for t in v_caches])
    io.k_caches = ctypes.cast(kc, ctypes.POINTER(_vp))
    io.v_caches = ctypes.cast(vc, ctypes.POINTER(_vp))
    io._keep = (kc, vc)
    io.topk_idx_out, io.topk_w_out = _ptr(topk_idx_out), _ptr(topk_w_out)
    _tree(io, tree_mask)
    return io


def mk_stack_step(stack, io, stream=None):
    _check("mk_stack_step", _lib_mk_stack_step(stack, ctypes.byref(io), _stream(stream)))


def mk_stack_status(stack):
    return _lib_mk_stack_status(stack)


def _stats_dict(st):
    return {f: int(getattr(st, f)) for f, _ in mk_prefetch_stats._fields_}


def mk_layer_prefetch_stats(layer):
    st = mk_prefetch_stats()
    _check("mk_layer_prefetch_stats", _lib_mk_layer_prefetch_stats(layer, ctypes.byref(st)))
    return _stats_dict(st)


def mk_stack_prefetch_stats(stack):
    st = mk_prefetch_stats()
    _check("mk_stack_prefetch_stats", _lib_mk_stack_prefetch_stats(stack, ctypes.byref(st)))
    return _stats_dict(st)


def mk_stack_destroy(stack):
    _lib_mk_stack_destroy(stack)


def mk_selftest_quantize(x, codes, scales, s_row, stream=None):
    rows, K = x.shape
    _check("mk_selftest_quantize", _lib_mk_selftest_quantize(
        _ptr(x), rows, K, _ptr(codes), _ptr(scales), _ptr(s_row), _stream(stream)))


def mk_selftest_mma(fp4, a, a_scales, b, b_scales, K, out, stream=None):
    _check("mk_selftest_mma", _lib_mk_selftest_mma(
        int(fp4), _ptr(a), _ptr(a_scales), _ptr(b), _ptr(b_scales), K, _ptr(out), _stream(stream)))


def mk_get_timestamps(layer, grid):
    """Self-timing stamps of the layer's last step: uint64 array [grid, 10, 16]."""
    import numpy as np
    buf = np.zeros((grid, 10, 16), dtype=np.uint64)
    _check("mk_get_timestamps", _lib_mk_get_timestamps(layer, buf.ctypes.data, buf.size))
    return buf


SYNC_MODES = {"flag_hop": 0, "sentinel_hop": 1, "acquire_poll": 2, "fence": 3}


def mk_selftest_sync(mode, iters=10000):
    """ns per operation of an intra-GPU synchronisation primitive (see mk_selftest.h)."""
    m = SYNC_MODES[mode] if isinstance(mode, str) else mode
    out = _c.c_double()
    _check("mk_selftest_sync", _lib_mk_selftest_sync(m, iters, _c.byref(out)))
    return out.value


# ------------------------------------------- batched decoding over a paged cache
# The library sees addresses only, so that a tensor of another type, on another
# device or with other strides would be misread: these are refused here, as
# MK_ERR_INVALID_ARG.

def _refuse(fn):
    raise MkError(fn, MK_ERR_INVALID_ARG)


def _dtype_of(fn, t):
    import torch
    if t.dtype is torch.bfloat16:
        return MK_BF16
    if t.dtype is torch.float16:
        return MK_FP16
    _refuse(fn)


def _dense(fn, t, elem, n=None):
    """Address of a contiguous CUDA tensor of whole numbers or floats of `elem`
    bytes (None: NULL), with `n` values if given."""
    if t is None:
        return None
    if not t.is_cuda or t.element_size() != elem or not t.is_contiguous() or (
            n is not None and t.numel() != n):
        _refuse(fn)
    return t.data_ptr()


def _ints(fn, t, elem, n=None):
    if t is not None and (t.is_floating_point() or t.is_complex()):
        _refuse(fn)
    return _dense(fn, t, elem, n)


def _heads(fn, t, like=None):
    """(address, rows, heads, head_dim, elements between rows) of a tensor
    [rows, heads, d] whose heads lie side by side."""
    if not t.is_cuda or t.dim() != 3 or (like is not None and t.dtype != like.dtype):
        _refuse(fn)
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if (s2 != 1 and d > 1) or (s1 != d and h > 1):
        _refuse(fn)
    return t.data_ptr(), n, h, d, s0 if n > 1 else max(s0, h * d)


def _pool(fn, t, like):
    """(address, pages, page size) of a pool [pages, page_size, heads, d]."""
    if t.dim() != 4 or t.dtype != like.dtype:
        _refuse(fn)
    return _dense(fn, t, 2), t.shape[0], t.shape[1]


def _table(fn, t):
    """(address, rows, columns, elements between rows) of an int32 table."""
    if not t.is_cuda or t.dim() != 2 or t.element_size() != 4 or t.is_floating_point() or (
            t.shape[1] > 1 and t.stride(1) != 1):
        _refuse(fn)
    return t.data_ptr(), t.shape[0], t.shape[1], max(t.stride(0), t.shape[1])


def make_slots_io(cached_lens, new_lens, free_pages, free_head, block_table, cu_rows, lens,
                  positions, slots, row_request, summary, page_size, n_pages, prefix_len=0):
    """mk_slots_io of CUDA tensors (int32; slots int64).  free_head and
    row_request may be None."""
    fn = "make_slots_io"
    b, n = cached_lens.numel(), positions.numel()
    table, rows, cols, stride = _table(fn, block_table)
    if rows != b:
        _refuse(fn)
    return mk_slots_io(b, n, page_size, cols, stride, n_pages, free_pages.numel(), prefix_len,
                       _ints(fn, cached_lens, 4), _ints(fn, new_lens, 4, b),
                       _ints(fn, free_pages, 4), _ints(fn, free_head, 4, 1), table,
                       _ints(fn, cu_rows, 4, b + 1), _ints(fn, lens, 4, b), _ints(fn, positions, 4),
                       _ints(fn, slots, 8, n), _ints(fn, row_request, 4, n),
                       _ints(fn, summary, 4, 4))


def mk_build_slots(io, stream=None):
    _check("mk_build_slots", _lib_mk_build_slots(ctypes.byref(io), _stream(stream)))


def make_rope_config(head_dim, rot_dim=None, layout="half", theta=10000.0, scaling="none",
                     factor=1.0, orig_ctx=0, beta_fast=0.0, beta_slow=0.0, attn_factor=0.0):
    return mk_rope_config(head_dim, head_dim if rot_dim is None else rot_dim, ROPE_LAYOUTS[layout],
                          ROPE_SCALINGS[scaling], theta, factor, orig_ctx, beta_fast, beta_slow,
                          attn_factor)


def mk_rope_create(cfg):
    h = _vp()
    _check("mk_rope_create", _lib_mk_rope_create(ctypes.byref(cfg), ctypes.byref(h)))
    return h.value


def mk_rope_destroy(rope):
    _lib_mk_rope_destroy(rope)


def make_rope_io(q, q_out, k, v, positions, slots, k_cache, v_cache):
    """mk_rope_io of CUDA tensors: q, q_out [rows, q heads, d], k, v [rows, kv
    heads, d] (views with a row stride), positions int32, slots int64, caches
    [pages, page_size, kv heads, d].  q or k (with v) may be None."""
    fn = "make_rope_io"
    like = q if q is not None else k
    if like is None:
        _refuse(fn)
    n = like.shape[0]
    dt = _dtype_of(fn, like)
    qp = qop = kp = vp = kc = vc = None
    qs = qos = ks = vs = hq = hk = n_slots = 0
    if q is not None:
        qp, _, hq, d, qs = _heads(fn, q)
        qop, no, ho, do, qos = _heads(fn, q_out, q)
        if (no, ho, do) != (n, hq, d):
            _refuse(fn)
    if k is not None:
        kp, nk, hk, dk, ks = _heads(fn, k, like)
        kc, pages, page = _pool(fn, k_cache, like)
        n_slots = pages * page
        if nk != n or dk != like.shape[2] or k_cache.shape[2:] != k.shape[1:]:
            _refuse(fn)
        if v is not None:
            vp, _, _, _, vs = _heads(fn, v, like)
            vc = _pool(fn, v_cache, like)[0]
            if v.shape != k.shape or v_cache.shape != k_cache.shape:
                _refuse(fn)
    elif v is not None:
        _refuse(fn)
    return mk_rope_io(n, hq, hk, like.shape[2], dt, qp, qs, qop, qos, kp, ks, vp, vs,
                      _ints(fn, positions, 4, n), _ints(fn, slots, 8, n), kc, vc, n_slots)


def mk_rope_apply(rope, io, stream=None):
    _check("mk_rope_apply", _lib_mk_rope_apply(rope, ctypes.byref(io), _stream(stream)))


def make_prefix_attn_io(q, k_cache, v_cache, out, lens, cu_rows, block_table, prefix_pages=None,
                        prefix_len=0, window=0, scale=0.0, tree_mask=None, lse=None):
    """mk_prefix_attn_io of CUDA tensors: q, out [rows, q heads, d] (views with
    a row stride), caches [pages, page_size, kv heads, d], lens, cu_rows,
    block_table [requests, pages] and prefix_pages int32, tree_mask int64
    [rows], lse float32 [rows, q heads]."""
    fn = "make_prefix_attn_io"
    qp, n, hq, d, qs = _heads(fn, q)
    op, no, ho, do, os_ = _heads(fn, out, q)
    kp, pages, page = _pool(fn, k_cache, q)
    vp = _pool(fn, v_cache, q)[0]
    table, b, cols, stride = _table(fn, block_table)
    if (no, ho, do) != (n, hq, d) or v_cache.shape != k_cache.shape or k_cache.shape[3] != d:
        _refuse(fn)
    if prefix_len > 0 and (prefix_pages is None or prefix_pages.numel() * page < prefix_len):
        _refuse(fn)
    if lse is not None and not lse.is_floating_point():
        _refuse(fn)
    return mk_prefix_attn_io(b, n, hq, k_cache.shape[2], d, _dtype_of(fn, q), page, pages,
                             prefix_len, cols, stride, window, scale, qp, qs, kp, vp,
                             _ints(fn, prefix_pages, 4), table, _ints(fn, lens, 4, b),
                             _ints(fn, cu_rows, 4, b + 1), _ints(fn, tree_mask, 8, n), op, os_,
                             _dense(fn, lse, 4, n * hq))


def mk_prefix_attn_workspace(io):
    out = _i64()
    _check("mk_prefix_attn_workspace",
           _lib_mk_prefix_attn_workspace(ctypes.byref(io), ctypes.byref(out)))
    return out.value


def mk_prefix_attn(io, workspace, stream=None):
    _check("mk_prefix_attn", _lib_mk_prefix_attn(
        ctypes.byref(io), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def mk_prefix_attn_status(workspace):
    return _lib_mk_prefix_attn_status(_ptr(workspace))
