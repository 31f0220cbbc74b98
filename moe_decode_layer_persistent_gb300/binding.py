"""ctypes binding of libmk.so: the mk_* C ABI with the same names.

Argument marshalling only: every step of the decode layer runs in the CUDA
library.  Tensors are passed as device pointers (torch tensors are accepted
for convenience; only ``data_ptr()`` is read).  Loading fails loudly if the
library has not been built -- there is no CPU fallback.
"""

import ctypes
import os
import struct

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
ACTS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3}

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


class mk_kvq_cache(ctypes.Structure):
    _fields_ = [("n_pages", _i32), ("page_size", _i32), ("n_kv_heads", _i32), ("head_dim", _i32),
                ("k_codes", _vp), ("k_scales", _vp), ("v_codes", _vp), ("v_scales", _vp),
                ("k_exp", _vp), ("v_exp", _vp)]


class mk_qkv_append_io(ctypes.Structure):
    _fields_ = [("n_rows", _i32), ("n_q_heads", _i32), ("n_kv_heads", _i32), ("head_dim", _i32),
                ("dtype", _i32), ("bits", _i32), ("eps", ctypes.c_float),
                ("q", _vp), ("q_stride", _i64), ("q_out", _vp), ("q_out_stride", _i64),
                ("k", _vp), ("k_stride", _i64), ("v", _vp), ("v_stride", _i64),
                ("positions", _vp), ("slots", _vp), ("q_norm", _vp), ("k_norm", _vp),
                ("k_cache", _vp), ("v_cache", _vp), ("n_slots", _i64), ("kvq", mk_kvq_cache)]


class mk_kvq_read_io(ctypes.Structure):
    _fields_ = [("kvq", mk_kvq_cache), ("n_rows", _i32), ("dtype", _i32), ("slots", _vp),
                ("k_out", _vp), ("v_out", _vp)]


class mk_kvq_attn_io(ctypes.Structure):
    _fields_ = [("n_requests", _i32), ("n_rows", _i32), ("n_q_heads", _i32), ("dtype", _i32),
                ("max_pages", _i32), ("window", _i32), ("scale", ctypes.c_float),
                ("table_stride", _i64), ("kvq", mk_kvq_cache), ("q", _vp), ("q_stride", _i64),
                ("block_table", _vp), ("lens", _vp), ("cu_rows", _vp), ("tree_mask", _vp),
                ("out", _vp), ("out_stride", _i64), ("lse", _vp)]


class mk_linear_io(ctypes.Structure):
    _fields_ = [("n_rows", _i32), ("n_in", _i32), ("n_out", _i32), ("dtype", _i32), ("act", _i32),
                ("x", _vp), ("x_stride", _i64), ("w", _vp), ("w_stride", _i64), ("bias", _vp),
                ("residual", _vp), ("residual_stride", _i64), ("out", _vp), ("out_stride", _i64)]


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
_lib_mk_selftest_attn_waits = _sig("mk_selftest_attn_waits", _c.c_int,
                                   [_c.POINTER(mk_prefix_attn_io), _vp, _i64, _c.c_uint64, _i32,
                                    _i32, _vp])
_lib_mk_qkv_append = _sig("mk_qkv_append", _c.c_int, [_vp, _c.POINTER(mk_qkv_append_io), _vp])
_lib_mk_kvq_read = _sig("mk_kvq_read", _c.c_int, [_c.POINTER(mk_kvq_read_io), _vp])
_lib_mk_kvq_attn_workspace = _sig("mk_kvq_attn_workspace", _c.c_int,
                                  [_c.POINTER(mk_kvq_attn_io), _c.POINTER(_i64)])
_lib_mk_kvq_attn = _sig("mk_kvq_attn", _c.c_int, [_c.POINTER(mk_kvq_attn_io), _vp, _i64, _vp])
_lib_mk_kvq_attn_status = _sig("mk_kvq_attn_status", _c.c_int, [_vp])
_lib_mk_linear_workspace = _sig("mk_linear_workspace", _c.c_int,
                                [_c.POINTER(mk_linear_io), _c.POINTER(_i64)])
_lib_mk_linear = _sig("mk_linear", _c.c_int, [_c.POINTER(mk_linear_io), _vp, _i64, _vp])
_lib_mk_selftest_kvq_waits = _sig("mk_selftest_kvq_waits", _c.c_int,
                                  [_c.POINTER(mk_kvq_attn_io), _vp, _i64, _c.c_uint64, _i32, _i32, _vp])
_lib_mk_selftest_linear_waits = _sig("mk_selftest_linear_waits", _c.c_int,
                                     [_c.POINTER(mk_linear_io), _vp, _i64, _c.c_uint64, _i32, _i32,
                                      _i32, _vp])
_lib_mk_linear_status = _sig("mk_linear_status", _c.c_int, [_vp])

EXPORTED = ["mk_layer_create", "mk_decode_step", "mk_decode_step_noalloc", "mk_layer_status", "mk_layer_clear_status",
            "mk_layer_destroy", "mk_stack_create", "mk_stack_step", "mk_stack_status",
            "mk_stack_destroy", "mk_status_string", "mk_layer_get_info", "mk_get_timestamps",
            "mk_layer_prefetch_stats", "mk_stack_prefetch_stats",
            "mk_build_slots", "mk_rope_create", "mk_rope_destroy", "mk_rope_apply",
            "mk_prefix_attn_workspace", "mk_prefix_attn", "mk_prefix_attn_status",
            "mk_qkv_append", "mk_kvq_read", "mk_kvq_attn_workspace", "mk_kvq_attn", "mk_kvq_attn_status",
            "mk_linear_workspace", "mk_linear", "mk_linear_status",
            "mk_selftest_quantize", "mk_selftest_mma", "mk_selftest_sync", "mk_selftest_attn_waits",
            "mk_selftest_kvq_waits", "mk_selftest_linear_waits"]


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
# MK_ERR_INVALID_ARG.  A serving loop makes these structs in every step: each
# tensor is looked at once, and the fields are packed together.

_torch = None
_pack_slots = struct.Struct("@4iqiii11P").pack
_pack_rope = struct.Struct("@5iPqPqPqPqPPPPq").pack
_pack_attn = struct.Struct("@10iqifPqPPPPPPPPqP").pack
# (those of mk_kvq_cache, 4i6P, inside the others' without padding: 8-byte aligned)
_pack_kvq = struct.Struct("@4i6P").pack
_pack_append = struct.Struct("@6if" + "Pq" * 4 + "6Pq64s").pack
_pack_read = struct.Struct("@64s2i3P").pack
_pack_kvq_attn = struct.Struct("@6ifq64sPq5PqP").pack
_pack_linear = struct.Struct("@5iPqPqPPqPq").pack


def _load_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _refuse(fn):
    raise MkError(fn, MK_ERR_INVALID_ARG)


def _device_of(fn, t):
    d = t.get_device()
    if d < 0:
        _refuse(fn)
    return d


def _vec(fn, t, dtype, dev, n=None):
    """Address of a contiguous tensor of `dtype` on CUDA device `dev` (None: 0),
    with `n` values if given."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or (
            n is not None and t.numel() != n):
        _refuse(fn)
    return t.data_ptr()


def _kind(fn, T, t):
    if t.dtype is T.bfloat16:
        return MK_BF16
    if t.dtype is T.float16:
        return MK_FP16
    _refuse(fn)


def _rows(fn, t, shape, dtype, dev):
    """(address, elements between rows) of a tensor [rows, heads, d] whose heads
    lie side by side; of a single row, whose stride says nothing, one that every call
    takes."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _refuse(fn)
    n, h, d = shape
    s0, s1, s2 = t.stride()
    if (s2 != 1 and d > 1) or (s1 != d and h > 1):
        _refuse(fn)
    return t.data_ptr(), s0 if n > 1 or (s0 >= h * d and s0 % 8 == 0) else h * d


def _table(fn, t, dtype, dev):
    """(address, rows, columns, elements between rows) of a table."""
    if t.dtype is not dtype or t.dim() != 2 or t.get_device() != dev:
        _refuse(fn)
    rows, cols = t.shape
    s0, s1 = t.stride()
    if cols > 1 and s1 != 1:
        _refuse(fn)
    return t.data_ptr(), rows, cols, s0 if rows > 1 else max(s0, cols)


def make_slots_io(cached_lens, new_lens, free_pages, free_head, block_table, cu_rows, lens,
                  positions, slots, row_request, summary, page_size, n_pages, prefix_len=0):
    """mk_slots_io of CUDA tensors (int32; slots int64).  free_head and
    row_request may be None."""
    fn = "make_slots_io"
    T = _torch or _load_torch()
    i32, dev = T.int32, _device_of(fn, cu_rows)
    b, n = cached_lens.numel(), positions.numel()
    table, rows, cols, stride = _table(fn, block_table, i32, dev)
    if rows != b:
        _refuse(fn)
    return mk_slots_io.from_buffer_copy(_pack_slots(
        b, n, page_size, cols, stride, n_pages, free_pages.numel(), prefix_len,
        _vec(fn, cached_lens, i32, dev), _vec(fn, new_lens, i32, dev, b),
        _vec(fn, free_pages, i32, dev), _vec(fn, free_head, i32, dev, 1), table,
        _vec(fn, cu_rows, i32, dev, b + 1), _vec(fn, lens, i32, dev, b),
        _vec(fn, positions, i32, dev), _vec(fn, slots, T.int64, dev, n),
        _vec(fn, row_request, i32, dev, n), _vec(fn, summary, i32, dev, 4)))


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
    T = _torch or _load_torch()
    like = q if q is not None else k
    if like is None or like.dim() != 3 or (k is None and v is not None):
        _refuse(fn)
    dt, dev = like.dtype, _device_of(fn, like)
    n, hq, d = like.shape
    qp = qop = kp = vp = kc = vc = qs = qos = ks = vs = hk = n_slots = 0
    if q is not None:
        qp, qs = _rows(fn, q, q.shape, dt, dev)
        qop, qos = _rows(fn, q_out, q.shape, dt, dev)
    else:
        hq = 0
    if k is not None:
        hk = k.shape[1]
        kp, ks = _rows(fn, k, (n, hk, d), dt, dev)
        kc = _vec(fn, k_cache, dt, dev)
        pool = k_cache.shape
        if len(pool) != 4 or pool[2] != hk or pool[3] != d:
            _refuse(fn)
        n_slots = pool[0] * pool[1]
        if v is not None:
            vp, vs = _rows(fn, v, (n, hk, d), dt, dev)
            vc = _vec(fn, v_cache, dt, dev)
            if v_cache.shape != pool:
                _refuse(fn)
    return mk_rope_io.from_buffer_copy(_pack_rope(
        n, hq, hk, d, _kind(fn, T, like), qp, qs, qop, qos, kp, ks, vp, vs,
        _vec(fn, positions, T.int32, dev, n), _vec(fn, slots, T.int64, dev, n), kc, vc, n_slots))


def mk_rope_apply(rope, io, stream=None):
    _check("mk_rope_apply", _lib_mk_rope_apply(rope, ctypes.byref(io), _stream(stream)))


def make_prefix_attn_io(q, k_cache, v_cache, out, lens, cu_rows, block_table, prefix_pages=None,
                        prefix_len=0, window=0, scale=0.0, tree_mask=None, lse=None):
    """mk_prefix_attn_io of CUDA tensors: q, out [rows, q heads, d] (views with
    a row stride), caches [pages, page_size, kv heads, d], lens, cu_rows,
    block_table [requests, pages] and prefix_pages int32, tree_mask int64
    [rows], lse float32 [rows, q heads]."""
    fn = "make_prefix_attn_io"
    T = _torch or _load_torch()
    i32, dt, dev = T.int32, q.dtype, _device_of(fn, q)
    shape, pool = q.shape, k_cache.shape
    if len(shape) != 3 or len(pool) != 4:
        _refuse(fn)
    n, hq, d = shape
    pages, page, hk, dk = pool
    qp, qs = _rows(fn, q, shape, dt, dev)
    op, os_ = _rows(fn, out, shape, dt, dev)
    table, b, cols, stride = _table(fn, block_table, i32, dev)
    if v_cache.shape != pool or dk != d:
        _refuse(fn)
    if prefix_len > 0 and (prefix_pages is None or prefix_pages.numel() * page < prefix_len):
        _refuse(fn)
    io = mk_prefix_attn_io.from_buffer_copy(_pack_attn(
        b, n, hq, hk, d, _kind(fn, T, q), page, pages, prefix_len, cols, stride, window, scale,
        qp, qs, _vec(fn, k_cache, dt, dev), _vec(fn, v_cache, dt, dev),
        _vec(fn, prefix_pages, i32, dev), table, _vec(fn, lens, i32, dev, b),
        _vec(fn, cu_rows, i32, dev, b + 1), _vec(fn, tree_mask, T.int64, dev, n), op, os_,
        _vec(fn, lse, T.float32, dev, n * hq)))
    io.device = dev  # (an attribute beside the fields: the workspace has to be there too)
    return io


def mk_prefix_attn_workspace(io):
    out = _i64()
    _check("mk_prefix_attn_workspace",
           _lib_mk_prefix_attn_workspace(ctypes.byref(io), ctypes.byref(out)))
    return out.value


def mk_prefix_attn(io, workspace, stream=None):
    if not workspace.is_contiguous() or workspace.get_device() != getattr(io, "device", workspace.get_device()):
        _refuse("mk_prefix_attn")
    _check("mk_prefix_attn", _lib_mk_prefix_attn(
        ctypes.byref(io), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def mk_prefix_attn_status(workspace):
    return _lib_mk_prefix_attn_status(_ptr(workspace))


WITHHOLD = {"nothing": 0, "scores": 1, "weights": 2, "row_tile": 3, "buffers": 4}


def mk_selftest_attn_waits(io, workspace, wait_ns, withhold="nothing", which=0, stream=None):
    """mk_prefix_attn with short waits and a hand-off withheld; returns the status."""
    if not workspace.is_contiguous():
        _refuse("mk_selftest_attn_waits")
    return _lib_mk_selftest_attn_waits(
        ctypes.byref(io), workspace.data_ptr(), workspace.numel() * workspace.element_size(), wait_ns,
        WITHHOLD[withhold], which, _stream(stream))


# ------------------------- the attention half of a layer over a cache in 4 bits

def make_kvq_cache(k_codes, k_scales, v_codes, v_scales, k_exp=None, v_exp=None):
    """mk_kvq_cache of CUDA tensors: codes uint8 [pages, kv heads, page_size, d/2],
    scales uint8 [pages, kv heads, page_size, d/16], exps int32 [kv heads] or None."""
    fn = "make_kvq_cache"
    T = _torch or _load_torch()
    u8, dev = T.uint8, _device_of(fn, k_codes)
    shape = k_codes.shape
    if len(shape) != 4:
        _refuse(fn)
    pages, heads, page, half = shape
    groups = (pages, heads, page, half // 8)
    if half % 8 or v_codes.shape != shape or k_scales.shape != groups or v_scales.shape != groups:
        _refuse(fn)
    c = mk_kvq_cache.from_buffer_copy(_pack_kvq(
        pages, page, heads, 2 * half, _vec(fn, k_codes, u8, dev), _vec(fn, k_scales, u8, dev),
        _vec(fn, v_codes, u8, dev), _vec(fn, v_scales, u8, dev), _vec(fn, k_exp, T.int32, dev, heads),
        _vec(fn, v_exp, T.int32, dev, heads)))
    c.device = dev  # (an attribute beside the fields: other tensors have to be there too)
    return c


def _kvq_on(fn, kvq, dev):
    if getattr(kvq, "device", dev) != dev:
        _refuse(fn)
    return bytes(kvq)


def make_qkv_append_io(q, q_out, k, v, positions, slots, q_norm=None, k_norm=None, eps=1e-6,
                       k_cache=None, v_cache=None, kvq=None):
    """mk_qkv_append_io of CUDA tensors: q, q_out [rows, q heads, d], k, v [rows, kv
    heads, d] (views with a row stride), positions int32 (None without a rotation),
    slots int64, norms [d]; the cache as [pages, page_size, kv heads, d] tensors or
    as a mk_kvq_cache.  q or k (with v) may be None."""
    fn = "make_qkv_append_io"
    T = _torch or _load_torch()
    like = q if q is not None else k
    if like is None or like.dim() != 3 or (k is None and v is not None):
        _refuse(fn)
    dt, dev = like.dtype, _device_of(fn, like)
    n, hq, d = like.shape
    qp = qop = kp = vp = kc = vc = qs = qos = ks = vs = hk = n_slots = 0
    bits, four = 16, bytes(64)
    if q is not None:
        qp, qs = _rows(fn, q, q.shape, dt, dev)
        qop, qos = _rows(fn, q_out, q.shape, dt, dev)
    else:
        hq = 0
    if k is not None:
        hk = k.shape[1]
        kp, ks = _rows(fn, k, (n, hk, d), dt, dev)
        if v is not None:
            vp, vs = _rows(fn, v, (n, hk, d), dt, dev)
        if kvq is not None:
            bits, four = 4, _kvq_on(fn, kvq, dev)
            if kvq.n_kv_heads != hk or kvq.head_dim != d or k_cache is not None or v_cache is not None:
                _refuse(fn)
        else:
            kc = _vec(fn, k_cache, dt, dev)
            pool = k_cache.shape if k_cache is not None else ()
            if len(pool) != 4 or pool[2] != hk or pool[3] != d:
                _refuse(fn)
            n_slots = pool[0] * pool[1]
            if v is not None:
                vc = _vec(fn, v_cache, dt, dev)
                if v_cache is None or v_cache.shape != pool:
                    _refuse(fn)
    return mk_qkv_append_io.from_buffer_copy(_pack_append(
        n, hq, hk, d, _kind(fn, T, like), bits, eps, qp, qs, qop, qos, kp, ks, vp, vs,
        _vec(fn, positions, T.int32, dev, n), _vec(fn, slots, T.int64, dev, n),
        _vec(fn, q_norm, dt, dev, d), _vec(fn, k_norm, dt, dev, d), kc, vc, n_slots, four))


def mk_qkv_append(rope, io, stream=None):
    """rope: of mk_rope_create, or None (no rotation)."""
    _check("mk_qkv_append", _lib_mk_qkv_append(rope, ctypes.byref(io), _stream(stream)))


def make_kvq_read_io(kvq, slots, k_out, v_out):
    """mk_kvq_read_io: rows `slots` (int64; None: all, in order) of the cache as
    k_out, v_out [rows, kv heads, d], bf16 or fp16; either may be None."""
    fn = "make_kvq_read_io"
    T = _torch or _load_torch()
    like = k_out if k_out is not None else v_out
    if like is None:
        _refuse(fn)
    dt, dev = like.dtype, _device_of(fn, like)
    n = kvq.n_pages * kvq.page_size if slots is None else slots.numel()
    size = n * kvq.n_kv_heads * kvq.head_dim
    return mk_kvq_read_io.from_buffer_copy(_pack_read(
        _kvq_on(fn, kvq, dev), n, _kind(fn, T, like), _vec(fn, slots, T.int64, dev),
        _vec(fn, k_out, dt, dev, size), _vec(fn, v_out, dt, dev, size)))


def mk_kvq_read(io, stream=None):
    _check("mk_kvq_read", _lib_mk_kvq_read(ctypes.byref(io), _stream(stream)))


def make_kvq_attn_io(q, kvq, out, lens, cu_rows, block_table, window=0, scale=0.0, tree_mask=None,
                     lse=None):
    """mk_kvq_attn_io of CUDA tensors: q, out [rows, q heads, d] (views with a row
    stride), lens, cu_rows, block_table [requests, pages] int32, tree_mask int64
    [rows], lse float32 [rows, q heads]."""
    fn = "make_kvq_attn_io"
    T = _torch or _load_torch()
    i32, dt, dev = T.int32, q.dtype, _device_of(fn, q)
    shape = q.shape
    if len(shape) != 3 or kvq.head_dim != shape[2]:
        _refuse(fn)
    n, hq, _ = shape
    qp, qs = _rows(fn, q, shape, dt, dev)
    op, os_ = _rows(fn, out, shape, dt, dev)
    table, b, cols, stride = _table(fn, block_table, i32, dev)
    io = mk_kvq_attn_io.from_buffer_copy(_pack_kvq_attn(
        b, n, hq, _kind(fn, T, q), cols, window, scale, stride, _kvq_on(fn, kvq, dev), qp, qs, table,
        _vec(fn, lens, i32, dev, b), _vec(fn, cu_rows, i32, dev, b + 1),
        _vec(fn, tree_mask, T.int64, dev, n), op, os_, _vec(fn, lse, T.float32, dev, n * hq)))
    io.device = dev
    return io


def _with_workspace(fn, call, io, workspace, stream):
    if not workspace.is_contiguous() or workspace.get_device() != getattr(io, "device", workspace.get_device()):
        _refuse(fn)
    _check(fn, call(ctypes.byref(io), workspace.data_ptr(),
                    workspace.numel() * workspace.element_size(), _stream(stream)))


def mk_kvq_attn_workspace(io):
    out = _i64()
    _check("mk_kvq_attn_workspace",
           _lib_mk_kvq_attn_workspace(ctypes.byref(io), ctypes.byref(out)))
    return out.value


def mk_kvq_attn(io, workspace, stream=None):
    _with_workspace("mk_kvq_attn", _lib_mk_kvq_attn, io, workspace, stream)


def mk_kvq_attn_status(workspace):
    return _lib_mk_kvq_attn_status(_ptr(workspace))


def _matrix(fn, t, rows, cols, dtype, dev):
    """(address, elements between rows) of a [rows, cols] matrix with contiguous rows; of
    a single row, whose stride says nothing, one that every call takes."""
    if t.shape != (rows, cols) or t.dtype is not dtype or t.get_device() != dev:
        _refuse(fn)
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        _refuse(fn)
    return t.data_ptr(), s0 if rows > 1 or (s0 >= cols and s0 % 8 == 0) else -(-cols // 8) * 8


def make_linear_io(x, w, out, bias=None, act="none", residual=None):
    """mk_linear_io of CUDA tensors: x [rows, in], w [out, in], out and residual
    [rows, out] (views with a row stride), bias [out]."""
    fn = "make_linear_io"
    T = _torch or _load_torch()
    dt, dev = x.dtype, _device_of(fn, x)
    if x.dim() != 2 or w.dim() != 2:
        _refuse(fn)
    (m, k), n = x.shape, w.shape[0]
    xp, xs = _matrix(fn, x, m, k, dt, dev)
    wp, ws = _matrix(fn, w, n, k, dt, dev)
    op, os_ = _matrix(fn, out, m, n, dt, dev)
    rp, rs = _matrix(fn, residual, m, n, dt, dev) if residual is not None else (0, 0)
    io = mk_linear_io.from_buffer_copy(_pack_linear(
        m, k, n, _kind(fn, T, x), ACTS[act], xp, xs, wp, ws, _vec(fn, bias, dt, dev, n), rp, rs, op, os_))
    io.device = dev
    return io


def mk_linear_workspace(io):
    out = _i64()
    _check("mk_linear_workspace", _lib_mk_linear_workspace(ctypes.byref(io), ctypes.byref(out)))
    return out.value


def mk_linear(io, workspace, stream=None):
    _with_workspace("mk_linear", _lib_mk_linear, io, workspace, stream)


def mk_linear_status(workspace):
    return _lib_mk_linear_status(_ptr(workspace))


WITHHOLD_LINEAR = {"nothing": 0, "copies": 1, "stage": 2, "sums": 3, "columns": 4}


def mk_selftest_linear_waits(io, workspace, wait_ns, withhold="nothing", which=0, half=0, stream=None):
    """mk_linear with short waits and a hand-off withheld; returns the status."""
    if not workspace.is_contiguous():
        _refuse("mk_selftest_linear_waits")
    return _lib_mk_selftest_linear_waits(
        ctypes.byref(io), workspace.data_ptr(), workspace.numel() * workspace.element_size(), wait_ns,
        WITHHOLD_LINEAR[withhold], which, half, _stream(stream))


WITHHOLD_KVQ = {"nothing": 0, "scores": 1, "weights": 2, "keys": 3, "values": 4, "keys_used": 5, "values_used": 6,
                "row_tile": 7, "half": 8, "taken": 9}


def mk_selftest_kvq_waits(io, workspace, wait_ns, withhold="nothing", which=0, stream=None):
    """mk_kvq_attn with short waits and a hand-off withheld; returns the status."""
    if not workspace.is_contiguous():
        _refuse("mk_selftest_kvq_waits")
    return _lib_mk_selftest_kvq_waits(
        ctypes.byref(io), workspace.data_ptr(), workspace.numel() * workspace.element_size(), wait_ns,
        WITHHOLD_KVQ[withhold], which, _stream(stream))
