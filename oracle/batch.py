"""The operators of a batched step over a paged KV cache, one request and one
row at a time, in float64 and Python integers: slot maps from request lengths,
rotary positions, attention with a prefix that all requests share.  The
definitions are those of include/mk.h (mk_build_slots, mk_rope_apply,
mk_prefix_attn); the token-tree visibility is layer.visible_keys'."""

import math

import numpy as np


def build_slots(cached, new, free_pages, head, table, n_rows, page, n_pages, prefix=0):
    """Returns a dict of table (a copy with the new pages), cu_rows, lens,
    positions, slots, row_request, summary."""
    B, width = table.shape
    table = table.copy()
    n_free = len(free_pages)
    head = min(max(int(head), 0), n_free)
    cu, lens = [0], []
    positions, slots, request = [0] * n_rows, [-1] * n_rows, [-1] * n_rows
    taken = refused = asked = row = 0
    for b in range(B):
        c, n = int(cached[b]), int(new[b])
        rows = max(n, 0)
        fits = c >= 0 and n >= 0 and c + n <= width * page and row + rows <= n_rows
        need = -(-(c + n) // page) - -(-c // page) if fits else 0
        granted = fits and (need == 0 or head + asked + need <= n_free)
        if granted:
            for i in range(need):
                table[b, -(-c // page) + i] = free_pages[head + asked + i]
            taken += need
        else:
            refused += 1
        asked += need
        lens.append(c + n if granted else min(max(c, 0), width * page))
        for i in range(rows):
            if row + i >= n_rows:
                break
            positions[row + i] = min(prefix + c + i, 2**31 - 1)
            request[row + i] = b
            if granted:
                p = int(table[b, (c + i) // page])
                if 0 <= p < n_pages:
                    slots[row + i] = p * page + (c + i) % page
        row += rows
        cu.append(min(row, n_rows))
    return dict(table=table, cu_rows=np.array(cu), lens=np.array(lens), positions=np.array(positions),
                slots=np.array(slots), row_request=np.array(request),
                summary=np.array([head + taken, min(row, n_rows), refused, min(asked, 2**31 - 1)]))


def rope_frequencies(rot, theta=10000.0, scaling="none", factor=1.0, orig_ctx=0, beta_fast=32.0,
                     beta_slow=1.0, attn_factor=0.0):
    """(radians per position of each pair, factor m on the rotated values)."""
    if scaling == "base":
        theta = theta * factor ** (rot / (rot - 2))
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    m = 1.0
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        g = np.clip((orig_ctx * f / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow), 0.0, 1.0)
        f = f * g + f / factor * (1 - g)
        m = 0.1 * math.log(factor) + 1.0
    return f, attn_factor or m


def rope(x, positions, rot, layout, f, m):
    """x [rows, heads, d] with the first rot values of every head rotated."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    a = np.asarray(positions, dtype=np.float64)[:, None] * f
    c, s = m * np.cos(a)[:, None], m * np.sin(a)[:, None]
    one, two = ((slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half"
                else (slice(0, rot, 2), slice(1, rot, 2)))
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y


def visible(i, n, length, prefix, window=0, mask=None):
    """(prefix keys, own keys) that row i of a request with n rows and `length`
    own keys sees; mask: the row's tree word."""
    base = max(0, length - n)
    depth = i if mask is None else bin(int(mask)).count("1") - 1
    p = prefix + base + depth
    low = p - window + 1 if window else 0
    pre = range(max(0, low), prefix)
    own = []
    for j in range(max(0, low - prefix), length):
        if mask is None:
            seen = j <= base + i
        else:
            seen = j < base or (j - base < 64 and (int(mask) >> (j - base)) & 1)
        if seen:
            own.append(j)
    return list(pre), own


def prefix_attn(q, k_pool, v_pool, prefix_pages, prefix, table, lens, cu, window=0, scale=None,
                tree=None):
    """q [rows, Hq, d]; pools [pages, page, Hkv, d].  Returns (out, lse, weight)
    with weight[r, h] = sum_j softmax_j |v_j| per value, the scale of the
    rounding errors of the weights; rows behind cu[-1] are NaN.  A page outside
    the pool reads as zeros."""
    N, Hq, d = q.shape
    pages, page, Hkv, _ = k_pool.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out, weight = np.full((N, Hq, d), np.nan), np.full((N, Hq, d), np.nan)
    lse = np.full((N, Hq), np.nan)
    zero = np.zeros((page, Hkv, d))

    def rows_of(pool, ids, keys):
        got = [pool[ids[j // page]][j % page] if 0 <= ids[j // page] < pages else zero[0]
               for j in keys]
        return np.array(got, dtype=np.float64).reshape(len(got), Hkv, d)

    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        length = min(max(int(lens[b]), 0), table.shape[1] * page)
        for i in range(n):
            r = int(cu[b]) + i
            pre, own = visible(i, n, length, prefix, window, None if tree is None else tree[r])
            k = np.concatenate([rows_of(k_pool, prefix_pages, pre), rows_of(k_pool, table[b], own)])
            v = np.concatenate([rows_of(v_pool, prefix_pages, pre), rows_of(v_pool, table[b], own)])
            for h in range(Hq):
                g = h // (Hq // Hkv)
                if not len(k):
                    out[r, h], weight[r, h], lse[r, h] = 0, 0, -np.inf
                    continue
                s = scale * (k[:, g] @ q[r, h].astype(np.float64))
                top = s.max()
                w = np.exp(s - top)
                lse[r, h] = top + math.log(w.sum())
                w /= w.sum()
                out[r, h], weight[r, h] = w @ v[:, g], w @ np.abs(v[:, g])
    return out, lse, weight
