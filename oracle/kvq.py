"""The attention half of a batched layer over a paged cache in 4 bits, in
float64: the codes of a cache (mk_kvq_cache in include/mk.h), norms with the
rotation (mk_qkv_append), the projection (mk_linear).  Attention over decoded
pools is batch.prefix_attn without a prefix."""

import math

import numpy as np

from . import batch

# the finite E4M3 values that are not negative, by their codes
E4M3 = np.array([m / 512 if e == 0 else (8 + m) / 8 * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])


def e4m3(x):
    """Codes of the E4M3 values nearest to x >= 0, ties to the even code, at most 448."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(E4M3, x, side="left"), 1, 126)
    below, above = x - E4M3[hi - 1], E4M3[hi] - x
    return np.where((below < above) | ((below == above) & (hi % 2 == 1)), hi - 1, hi)


def encode(y, e=0):
    """y [..., d] as (codes uint8 [..., d/2], scales uint8 [..., d/16]); e: exponent,
    whatever broadcasts against y without its last axis."""
    z = np.asarray(y, dtype=np.float64) / 2.0 ** np.asarray(e, dtype=np.float64)[..., None]
    g = z.reshape(*z.shape[:-1], -1, 16)
    with np.errstate(invalid="ignore", divide="ignore"):
        nan = np.isnan(g).any(-1)
        top = np.where(nan, 0.0, np.abs(g).max(-1))
        # top / 7 is off by a rounding: a tie between two scales is one of 7 times them
        scale = e4m3(np.minimum(top, 1e6) / 7)
        other = np.clip(scale + np.where(7 * E4M3[scale] < top, 1, -1), 0, 126)
        tie = np.abs(top - 7 * E4M3[scale]) == np.abs(top - 7 * E4M3[other])
        scale = np.where(tie & (scale % 2 == 1), other, scale)
        s = E4M3[scale][..., None]
        n = np.where((s > 0) & ~nan[..., None], np.clip(np.rint(g / np.where(s > 0, s, 1.0)), -8, 7), 0.0)
    n = (np.nan_to_num(n) + 8).astype(np.uint8).reshape(*z.shape[:-1], -1, 2)
    return n[..., 0] | n[..., 1] << 4, np.where(nan, 0x7F, scale).astype(np.uint8)


def decode(codes, scales, e=0):
    """The values that codes and scales stand for; NaN scales give NaN."""
    table = np.full(256, np.nan)
    table[:127], table[128:255] = E4M3, -E4M3
    n = np.stack([codes & 15, codes >> 4], -1).astype(np.float64).reshape(*scales.shape, 16) - 8
    v = (n * table[scales][..., None]).reshape(*codes.shape[:-1], -1)
    return v * 2.0 ** np.asarray(e, dtype=np.float64)[..., None]


def decode_pool(codes, scales, exps):
    """[pages, heads, page, ...] pools as values [pages, page, heads, d]."""
    return decode(codes, scales, np.asarray(exps)[:, None]).transpose(0, 2, 1, 3)


def norm(x, w=None, eps=1e-6):
    if w is None:
        return np.asarray(x, dtype=np.float64)
    x = np.asarray(x, dtype=np.float64)
    return x * w / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def norm_rope(x, w, eps, positions, rot, layout, f, m):
    """(values, bound of the pair that each was made from: (|n_a| + |n_b|) m)."""
    n = norm(x, w, eps)
    if not rot:
        return n, np.abs(n)
    y = batch.rope(n, positions, rot, layout, f, m)
    mag = np.abs(n)
    one, two = ((slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half"
                else (slice(0, rot, 2), slice(1, rot, 2)))
    both = (mag[..., one] + mag[..., two]) * m
    mag[..., one] = mag[..., two] = both
    return y, mag


def linear(x, w, bias=None, act="none", residual=None):
    """(out, sum of |products|)."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    y = x @ w.T
    if bias is not None:
        y = y + bias
    if act == "silu":
        y = y / (1 + np.exp(-np.clip(y, -700, None)))
    elif act == "gelu":
        y = 0.5 * y * (1 + np.vectorize(math.erf)(y / math.sqrt(2)) if y.size else 1)
    elif act == "gelu_tanh":
        y = 0.5 * y * (1 + np.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    if residual is not None:
        y = y + residual
    return y, np.abs(x) @ np.abs(w).T
