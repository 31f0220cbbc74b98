"""GPU parity of the batched operators (mk_build_slots, mk_rope_apply,
mk_prefix_attn) with the float64 oracle, through the binding.

Tolerances, from the arithmetic, with u = eps / 2 of the tensors' type (half a
step, relative to the value), tiny = half the spacing of its subnormals and
v = 2^-24, half a step of float32:

rope: the angle is off by 2^-33 turns (truncated phase) and v half turns (32
  bits to float), below 2^-21.6 rad together; the frequency, held in 53 bits,
  adds 2^-51 pos f rad, below 2^-21 up to pos 2^30.  cos and sin add 2 ulp
  (2^-23) and the factor m another v, so that each is off by less than
  2^-20 m.  With the two products and the sum, 3 v:
    |err| <= (|x_a| + |x_b|) m 2^-19.5 + u |y| + tiny.
attention: a score is a sum of d exact products in float32, each partial sum
  off by 2 v (a tensor core may truncate), and sum |q_i k_i| <= |q| |k|: with
  e_s = scale 2 d v max|q| max|k| + 2^-20 (exp2 and its argument's rounding) a
  weight is relatively off by e_s; rounding it adds u, or tiny where it
  underflows (the largest weight is at least 1).  A quotient doubles e_s.  Sums
  of n keys in chunks of 16 and of the partial results add (n / 16 + 64) 2 v.
  With W = sum_j w_j |v_j| over the softmax weights (the oracle's third output):
    |out err| <= W (u + 2 e_s + (n / 16 + 64) 2 v) + n tiny max|v| + u |out| + tiny,
    |lse err| <= e_s + (n + 64) v + 4 v |lse|.
"""

import math

import numpy as np
import pytest
import torch

from oracle import batch as ob
from oracle import layer as ol
from moe_decode_layer_persistent_gb300 import synth
import layer_harness as H
import oracle_io as oio

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}               # torch.finfo(t).eps / 2
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}
V = 2.0 ** -24
CANARY = -1152.0                                          # exact in bf16 and fp16


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda()


def norm(x):
    """The largest 2-norm of a head's values."""
    return float(np.sqrt(np.max(np.sum(x * x, axis=-1), initial=0.0)))


def np64(t):
    return t.detach().cpu().double().numpy()


def rounded(rng, shape, dtype, scale=1.0):
    """N(0, scale^2) values of the type, as float64, and the CUDA tensor."""
    t = torch.from_numpy(rng.standard_normal(shape) * scale).to(TORCH[dtype])
    return t.double().numpy(), t.cuda()


# ------------------------------------------------------------------ slots

def run_slots(mk, cached, new, free, head, table, n_rows, page, n_pages, prefix=0, stream=None,
              no_head=False, no_request=False):
    B = len(cached)
    t = dev(table)
    guard = torch.full((B + 2, table.shape[1] + 3), -77, dtype=torch.int32, device="cuda")
    guard[1:B + 1, :table.shape[1]] = t
    view = guard[1:B + 1, :table.shape[1]]
    out = dict(cu_rows=dev([-5] * (B + 1)), lens=dev([-5] * B), positions=dev([-5] * n_rows),
               slots=dev([-5] * n_rows, torch.int64), row_request=dev([-5] * n_rows),
               summary=dev([-5] * 4))
    io = mk.make_slots_io(dev(cached), dev(new), dev(free), None if no_head else dev([head]), view,
                          out["cu_rows"], out["lens"], out["positions"], out["slots"],
                          None if no_request else out["row_request"], out["summary"], page,
                          n_pages, prefix)
    mk.mk_build_slots(io, stream)
    mk.mk_build_slots(io, stream)      # the same inputs again: the same outputs
    torch.cuda.synchronize()
    out["table"] = view
    assert bool((guard[0] == -77).all()) and bool((guard[-1] == -77).all())
    assert bool((guard[:, table.shape[1]:] == -77).all())
    return {k: v.cpu().numpy() for k, v in out.items()}


def check_slots(mk, cached, new, free, head, table, n_rows, page, n_pages, prefix=0, **kw):
    want = ob.build_slots(cached, new, free, head, table, n_rows, page, n_pages, prefix)
    got = run_slots(mk, cached, new, free, head, table, n_rows, page, n_pages, prefix, **kw)
    for k in want:
        if k == "row_request" and kw.get("no_request"):
            assert np.all(got[k] == -5)
            continue
        assert np.array_equal(got[k], want[k]), k
    return got


def batch_lengths(rng, B, width, page, n_pages, hi_new, fill=0.7):
    cached = rng.integers(0, int(width * page * fill) + 1, B)
    new = rng.integers(0, hi_new + 1, B)
    ids = rng.permutation(n_pages)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        held = -(-int(cached[b]) // page)
        table[b, :held] = ids[at:at + held]
        at += held
    return cached, new, table, ids[at:]


@pytest.mark.parametrize("B,width,page,hi_new,spare", [
    (1, 1, 16, 1, 0), (1, 8, 1, 5, 3), (31, 9, 16, 17, 2), (32, 5, 7, 40, 0), (33, 5, 64, 1, 9),
    (300, 6, 16, 30, 5), (1000, 40, 16, 3, 1), (5000, 3, 128, 2, 0)])
def test_slots(cuda_lib, B, width, page, hi_new, spare):
    rng = np.random.default_rng(B)
    n_pages = B * width + 50
    cached, new, table, free = batch_lengths(rng, B, width, page, n_pages, hi_new)
    check_slots(cuda_lib, cached, new, free, 3 % (len(free) + 1), table, int(new.sum()) + spare,
                page, n_pages, prefix=1000)


@pytest.mark.parametrize("what", ["short", "none", "head_low", "head_high", "rows_short", "no_rows",
                                  "bad_lengths", "bad_pages", "all_idle", "no_head", "no_request"])
def test_slots_edges(cuda_lib, what):
    rng = np.random.default_rng(7)
    B, width, page, n_pages = 700, 8, 16, 7000
    cached, new, table, free = batch_lengths(rng, B, width, page, n_pages, 40)
    head, n_rows, kw = 2, int(new.sum()), {}
    if what == "short":
        free = free[:350]
    elif what == "none":
        free = free[:0]
    elif what == "head_low":
        head = -9
    elif what == "head_high":
        head = len(free) + 9
    elif what == "rows_short":
        n_rows //= 2
    elif what == "no_rows":
        n_rows = 0
    elif what == "bad_lengths":
        cached[[0, 5, 400]], new[[5, 9, 650]] = -3, -2
        cached[[77, 78]] = [width * page + 1, 2 ** 31 - 1]
        new[[300]] = 2 ** 31 - 1                      # its rows end behind every buffer
        n_rows = 5000
    elif what == "bad_pages":
        table[::3, 0], free = -1, free.copy()
        table[1::3, 0] = n_pages
        free[::5] = n_pages + 3
    elif what == "all_idle":
        new[:] = 0
        n_rows = 7
    elif what == "no_head":
        head, kw = 0, dict(no_head=True)
    elif what == "no_request":
        kw = dict(no_request=True)
    check_slots(cuda_lib, cached, new, free, head, table, n_rows, page, n_pages, **kw)


@pytest.mark.parametrize("cached,new,spare", [
    ([5], [131072], 0), ([0, 63, 64, 1000], [70001, 0, 64, 30000], 9), ([100] * 32, [4096] * 32, 1),
    ([10, 20], [3, 5], 100000)])
def test_slots_few_requests_many_rows(cuda_lib, cached, new, spare):
    page = 64
    held = [-(-c // page) for c in cached]
    width = max(-(-(c + n) // page) for c, n in zip(cached, new)) + 1
    n_pages = sum(held) + sum(new) // page + 2 * len(new)
    ids = np.random.default_rng(sum(new)).permutation(n_pages)
    table = np.full((len(cached), width), -1)
    for b, h in enumerate(held):
        table[b, :h] = ids[sum(held[:b]):sum(held[:b + 1])]
    check_slots(cuda_lib, cached, new, ids[sum(held):], 0, table, sum(new) + spare, page, n_pages, prefix=7)


def test_slots_empty_batch(cuda_lib):
    got = check_slots(cuda_lib, np.zeros(0, int), np.zeros(0, int), np.arange(4), 1,
                      np.zeros((0, 3), int), 5, 16, 10)
    assert got["summary"].tolist() == [1, 0, 0, 0] and got["slots"].tolist() == [-1] * 5


# ------------------------------------------------------------------- rope

def check_rope(mk, rng, n, hq, hk, d, rot, layout, dtype, positions, scaling="none", factor=1.0,
               orig_ctx=0, in_place=False, no_v=False, no_q=False, stream=None, attn_factor=0.0):
    page = 16
    pages = n // page + 3
    x, qkv = rounded(rng, (n, hq + 2 * hk + 1, d), dtype)   # one head more: the rows have a gap
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:hq + 2 * hk]
    kc0, kc = rounded(rng, (pages, page, hk, d), dtype)
    vc0, vc = rounded(rng, (pages, page, hk, d), dtype)
    slots = rng.permutation(pages * page)[:n]
    if n > 3:
        slots[[1, n - 1]] = [-1, pages * page]              # rows without a place
    kept = kc.clone(), vc.clone()
    out = torch.full((n, hq + 1, d), CANARY, dtype=TORCH[dtype], device="cuda")
    q_out = q if in_place else out[:, :hq]
    cfg = mk.make_rope_config(d, rot, layout=layout, scaling=scaling, factor=factor,
                              orig_ctx=orig_ctx, attn_factor=attn_factor)
    rope = mk.mk_rope_create(cfg)
    io = mk.make_rope_io(None if no_q else q, None if no_q else q_out, k, None if no_v else v,
                         dev(positions), dev(slots, torch.int64), kc, None if no_v else vc)
    mk.mk_rope_apply(rope, io, stream)
    torch.cuda.synchronize()
    mk.mk_rope_destroy(rope)
    f, m = ob.rope_frequencies(rot, scaling=scaling, factor=factor, orig_ctx=orig_ctx,
                               attn_factor=attn_factor)

    def close(got, src):
        want = ob.rope(src, positions, rot, layout, f, m)
        mag = np.abs(src).copy()
        one, two = ((slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half"
                    else (slice(0, rot, 2), slice(1, rot, 2)))
        both = mag[..., one] + mag[..., two]
        tol = np.zeros_like(mag)
        for s in (one, two):
            tol[..., s] = both * m * 2.0 ** -19.5 + U[dtype] * np.abs(want[..., s]) + TINY[dtype]
        err = np.abs(got - want)
        assert np.all(err <= tol), (err / np.maximum(tol, 1e-300))[..., :rot].max()

    if not no_q:
        close(np64(q_out), x[:, :hq])
        if not in_place:
            assert bool((out[:, hq] == CANARY).all())
    live = (slots >= 0) & (slots < pages * page)
    flat = lambda t: t.view(pages * page, hk, d)  # noqa: E731
    got_k = np64(flat(kc))
    close(np.where(live[:, None, None], got_k[np.clip(slots, 0, pages * page - 1)],
                   ob.rope(x[:, hq:hq + hk], positions, rot, layout, f, m)), x[:, hq:hq + hk])
    others = np.setdiff1d(np.arange(pages * page), slots[live])
    assert torch.equal(flat(kc)[others], flat(kept[0])[others])
    assert torch.equal(flat(vc)[others], flat(kept[1])[others])
    want_v = flat(kept[1])[slots[live]] if no_v else v[torch.from_numpy(live).cuda()]
    assert torch.equal(flat(vc)[slots[live]], want_v)
    if not in_place:                                        # the inputs are as they were
        assert np.array_equal(np64(qkv), x)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,hq,hk,d,rot,dtype", [
    (1, 4, 1, 64, 64, "bf16"), (16, 32, 8, 128, 128, "bf16"), (5, 6, 2, 64, 16, "fp16"),
    (37, 8, 8, 128, 32, "bf16"), (3, 1, 1, 256, 256, "fp16"), (9, 5, 5, 80, 32, "bf16"),
    (700, 3, 1, 24, 16, "fp16")])
def test_rope(cuda_lib, layout, n, hq, hk, d, rot, dtype):
    rng = np.random.default_rng(n)
    check_rope(cuda_lib, rng, n, hq, hk, d, rot, layout, dtype, rng.integers(0, 40000, n))


@pytest.mark.parametrize("kw", [
    dict(scaling="linear", factor=8.0), dict(scaling="base", factor=4.0),
    dict(scaling="parts", factor=16.0, orig_ctx=4096),
    dict(scaling="parts", factor=16.0, orig_ctx=4096, attn_factor=0.75),
    dict(in_place=True), dict(no_v=True), dict(no_q=True), dict(in_place=True, layout="interleaved")])
def test_rope_variants(cuda_lib, kw):
    kw = dict(dict(layout="half"), **kw)
    rng = np.random.default_rng(11)
    check_rope(cuda_lib, rng, 50, 8, 2, 128, 64, dtype="bf16", positions=rng.integers(0, 1 << 20, 50), **kw)


def test_rope_far_and_odd_positions(cuda_lib):
    rng = np.random.default_rng(12)
    pos = np.array([0, 1, -1, 2 ** 20 + 1, 2 ** 24 + 1, 2 ** 30 - 1, 2 ** 30, -2 ** 30])
    check_rope(cuda_lib, rng, len(pos), 4, 1, 64, 64, "half", "fp16", pos)


def test_rope_moves_cache_rows_in_place(cuda_lib):
    """k and v are the very rows that the slots name: k turns there, v stays."""
    rng = np.random.default_rng(13)
    k0, kc = rounded(rng, (4, 16, 2, 64), "bf16")
    _, vc = rounded(rng, (4, 16, 2, 64), "bf16")
    kept = vc.clone()
    pos = np.arange(20, 30)
    rope = cuda_lib.mk_rope_create(cuda_lib.make_rope_config(64))
    flat_k, flat_v = kc.view(64, 2, 64), vc.view(64, 2, 64)
    io = cuda_lib.make_rope_io(None, None, flat_k[20:30], flat_v[20:30], dev(pos), dev(pos, torch.int64), kc, vc)
    cuda_lib.mk_rope_apply(rope, io)
    torch.cuda.synchronize()
    cuda_lib.mk_rope_destroy(rope)
    want = k0.reshape(64, 2, 64).copy()
    f, m = ob.rope_frequencies(64)
    want[20:30] = ob.rope(want[20:30], pos, 64, "half", f, m)
    err = np.abs(np64(flat_k) - want)
    assert err.max() <= 4 * 2 * 2.0 ** -19.5 + U["bf16"] * np.abs(want).max()
    assert np.all(err[:20] == 0) and np.all(err[30:] == 0) and torch.equal(vc, kept)


# -------------------------------------------------------------- attention

def make_attn(rng, lens, news, prefix, hq, hk, d, dtype, page, window=0, tree=False, q_scale=1.0,
              extra_rows=2, ramp=0.0):
    """Inputs of one call; every key that no row sees is NaN (page tails,
    unused pages, prefix keys below every window)."""
    B, G = len(lens), hq // hk
    n = int(sum(news))
    width = max(1, max(-(-max(a, 1) // page) for a in lens))
    first = -(-prefix // page)
    held = [-(-max(a, 0) // page) for a in lens]
    n_pages = first + sum(held) + 2
    ids = rng.permutation(n_pages)
    table = np.full((B, width), n_pages + 99)
    at = first
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    prefix_pages = ids[:first]
    cu = np.concatenate([[0], np.cumsum(news)]).astype(int)
    q0, q = rounded(rng, (n + extra_rows, hq + 1, d), dtype, q_scale)
    k0, k = rounded(rng, (n_pages, page, hk, d), dtype)
    v0, v = rounded(rng, (n_pages, page, hk, d), dtype)
    words = None
    if tree:
        words = []
        for m in news:
            mine = []
            for i in range(m):
                up = int(rng.integers(-1, i)) if i else -1
                mine.append((1 << i) | (mine[up] if up >= 0 else 0))
            words += mine
        words += [0] * extra_rows
    seen = np.zeros((n_pages, page), bool)
    for b in range(B):
        for i in range(news[b]):
            pre, own = ob.visible(i, news[b], min(max(lens[b], 0), width * page), prefix, window,
                                  None if words is None else words[cu[b] + i])
            for j in pre:
                seen[prefix_pages[j // page], j % page] = True
            for j in own:
                seen[table[b, j // page], j % page] = True
    if ramp:   # scores that grow along the keys: the running maximum moves all the time
        for b in range(B):
            for j in range(prefix):
                k0[prefix_pages[j // page], j % page] *= 1 + ramp * j / max(1, prefix)
        k.copy_(torch.from_numpy(k0).to(k.dtype))
        k0 = np64(k)
    hide = torch.from_numpy(~seen).cuda()
    k[hide], v[hide] = float("nan"), float("nan")
    return dict(n=n, q0=q0[:, :hq], q=q[:, :hq], k0=k0, v0=v0, k=k, v=v, table=table, prefix=prefix,
                prefix_pages=prefix_pages, lens=np.array(lens), cu=cu, window=window, words=words,
                dtype=dtype, d=d, hq=hq)


def call_attn(mk, a, stream=None, workspace=None, scale=0.0):
    rows = a["q"].shape[0]
    whole = torch.full((rows, a["hq"] + 1, a["d"]), CANARY, dtype=a["q"].dtype, device="cuda")
    a["whole"], a["out"] = whole, whole[:, :a["hq"]]
    a["lse"] = torch.full((rows, a["hq"]), CANARY, dtype=torch.float32, device="cuda")
    words = None if a["words"] is None else torch.tensor(
        [w - (1 << 64) if w >> 63 else w for w in a["words"]], dtype=torch.int64, device="cuda")
    a["keep"] = (dev(a["lens"]), dev(a["cu"]), dev(a["table"]), dev(a["prefix_pages"]), words)
    io = mk.make_prefix_attn_io(a["q"], a["k"], a["v"], a["out"], *a["keep"][:4], a["prefix"],
                                window=a["window"], tree_mask=words, lse=a["lse"], scale=scale)
    if workspace is None:
        workspace = torch.empty(mk.mk_prefix_attn_workspace(io), dtype=torch.uint8, device="cuda")
    a["workspace"], a["io"] = workspace, io
    mk.mk_prefix_attn(io, workspace, stream)


def check_attn(mk, a, scale=None):
    torch.cuda.synchronize()
    assert mk.mk_prefix_attn_status(a["workspace"]) == 0
    n, d, dt = a["n"], a["d"], a["dtype"]
    want, lse, weight = ob.prefix_attn(a["q0"][:n], a["k0"], a["v0"], a["prefix_pages"], a["prefix"],
                                       a["table"], a["lens"], a["cu"], a["window"], scale, a["words"])
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    keys = a["prefix"] + max(0, int(a["lens"].max(initial=0)))
    e_s = sc * 2 * d * V * norm(a["q0"]) * norm(a["k0"]) + 2.0 ** -20
    vmax = np.abs(a["v0"]).max()
    tol = weight * (U[dt] + 2 * e_s + (keys / 16 + 64) * 2 * V) + keys * TINY[dt] * vmax + U[dt] * np.abs(want) + TINY[dt]
    got, got_lse = np64(a["out"])[:n], np64(a["lse"])[:n]
    assert np.all(np.isfinite(got))
    err = np.abs(got - want)
    assert np.all(err <= tol), ("out", (err / np.maximum(tol, 1e-300)).max())
    empty = np.isinf(lse)
    assert np.array_equal(np.isinf(got_lse), empty) and np.all(got_lse[empty] < 0)
    e = np.abs(got_lse[~empty] - lse[~empty])
    assert np.all(e <= e_s + (keys + 64) * V + 4 * V * np.abs(lse[~empty])), ("lse", e.max())
    # rows behind the last request and the values beside out are left as they were
    assert bool((a["whole"][n:] == CANARY).all()) and bool((a["whole"][:, a["hq"]:] == CANARY).all())
    assert bool((a["lse"][n:] == CANARY).all())


ATTN = {
    # name: lens, news, prefix, hq, hk, d, dtype, page, more
    "one_key": ([1], [1], 0, 4, 1, 64, "bf16", 16, {}),
    "no_key": ([0, 3, 0], [1, 1, 2], 0, 2, 1, 64, "bf16", 16, {}),
    "prefix_only": ([0, 0], [1, 3], 77, 4, 2, 128, "bf16", 16, {}),
    "idle_requests": ([20, 0, 33, 5, 40], [0, 0, 2, 0, 1], 50, 4, 1, 128, "bf16", 16, {}),
    "all_idle": ([20, 7], [0, 0], 50, 4, 1, 128, "bf16", 16, {}),
    "tile_ends": ([127, 128, 129, 255, 256, 257], [1, 1, 1, 2, 2, 3], 128, 8, 2, 128, "bf16", 64, {}),
    "prefix_127": ([16, 17], [1, 1], 127, 4, 2, 64, "fp16", 16, {}),
    "prefix_129": ([15, 16], [2, 1], 129, 4, 2, 64, "bf16", 32, {}),
    "mha": ([30, 90, 200], [3, 1, 2], 300, 3, 3, 128, "fp16", 128, {}),
    "group_6": ([60, 61, 300], [5, 7, 16], 260, 12, 2, 64, "bf16", 16, {}),
    "group_7": ([60, 61, 140], [19, 7, 37], 130, 7, 1, 128, "bf16", 32, {}),
    "group_64": ([40, 9], [4, 3], 200, 64, 1, 64, "bf16", 16, {}),
    "rows_127": ([9] * 127, [1] * 127, 64, 2, 2, 64, "bf16", 16, {}),
    "rows_257": ([5] * 257, [1] * 257, 140, 1, 1, 64, "fp16", 16, {}),
    "chunk": ([350, 20], [300, 3], 150, 4, 2, 128, "bf16", 64, {}),
    "chunk_fp16": ([200, 130], [140, 130], 20, 2, 1, 64, "fp16", 256, {}),
    "few_keys_for_rows": ([3, 0, 8], [7, 2, 8], 30, 4, 1, 128, "bf16", 16, {}),
    "window_1": ([20, 5, 300], [4, 5, 2], 100, 4, 2, 64, "bf16", 16, dict(window=1)),
    "window_40": ([20, 50, 300, 41], [4, 5, 2, 1], 100, 4, 2, 128, "bf16", 16, dict(window=40)),
    "window_200": ([20, 250, 300], [4, 16, 2], 333, 4, 2, 64, "fp16", 32, dict(window=200)),
    "window_wide": ([20, 50], [4, 5], 100, 4, 2, 64, "bf16", 16, dict(window=100000)),
    "tree": ([40, 300, 16], [16, 9, 16], 100, 8, 2, 128, "bf16", 16, dict(tree=True)),
    "tree_64": ([64, 100], [64, 64], 40, 4, 1, 64, "fp16", 16, dict(tree=True)),
    "tree_window": ([140, 300, 20], [16, 9, 5], 200, 4, 1, 128, "bf16", 16, dict(tree=True, window=64)),
    "large_scores": ([100, 60], [4, 4], 400, 8, 2, 128, "bf16", 16, dict(q_scale=6.0, ramp=4.0)),
    "large_scores_fp16": ([100, 60], [4, 4], 400, 8, 2, 64, "fp16", 16, dict(q_scale=6.0, ramp=4.0)),
    "many_requests": ([(7 * i) % 90 + 1 for i in range(300)], [1] * 300, 90, 4, 1, 64, "bf16", 16, {}),
    "many_items": ([(3 * i) % 11 + 1 for i in range(300)], [1] * 300, 3, 32, 8, 64, "bf16", 16, {}),
    "many_items_128": ([(3 * i) % 7 + 1 for i in range(160)], [1] * 160, 2, 32, 4, 128, "fp16", 16, {}),
    "requests_900": ([(5 * i) % 200 + 1 for i in range(900)], [i % 3 for i in range(900)], 40, 2, 1, 64,
                     "bf16", 16, {}),
    "rows_65": ([70, 40], [33, 1], 300, 2, 1, 128, "bf16", 16, {}),
    "rows_64_65_128_129": ([40, 41, 70, 90], [32, 33, 64, 65], 0, 2, 1, 64, "bf16", 16, {}),
    "prefix_in_many_pieces": ([3, 2], [3, 2], 6000, 4, 2, 64, "bf16", 64, {}),
    "long": ([1500, 40, 700], [2, 2, 1], 2100, 4, 1, 128, "bf16", 1024, {}),
}


@pytest.mark.parametrize("name", list(ATTN))
def test_prefix_attn(cuda_lib, name):
    lens, news, prefix, hq, hk, d, dtype, page, more = ATTN[name]
    a = make_attn(np.random.default_rng(len(name)), lens, news, prefix, hq, hk, d, dtype, page, **more)
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)


def test_prefix_attn_scale(cuda_lib):
    a = make_attn(np.random.default_rng(1), [30, 9], [2, 1], 100, 4, 2, 64, "bf16", 16)
    call_attn(cuda_lib, a, scale=0.03125)
    check_attn(cuda_lib, a, scale=0.03125)


@pytest.mark.parametrize("name", ["one_key", "prefix_only", "no_key", "tile_ends", "chunk", "window_40", "tree_window",
                                  "prefix_in_many_pieces", "long"])
def test_prefix_attn_rows_of_nan(cuda_lib, name):
    """A row whose q holds a NaN: out and lse are NaN as the formula has it (a row
    without keys still gets 0 and -inf), and no other row's result is."""
    lens, news, prefix, hq, hk, d, dtype, page, more = ATTN[name]
    a = make_attn(np.random.default_rng(len(name)), lens, news, prefix, hq, hk, d, dtype, page, **more)
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)
    out, lse = a["out"].clone(), a["lse"].clone()
    bad = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    bad[:a["n"]:3, ::2] = True                    # some rows, some of their heads
    a["q"][:, :, 5][bad] = float("nan")
    call_attn(cuda_lib, a)
    torch.cuda.synchronize()
    keys = bad & ~torch.isinf(lse)
    assert bool(torch.isnan(a["out"][keys]).all()) and bool(torch.isnan(a["lse"][keys]).all())
    a["out"][keys], a["lse"][keys] = out[keys], lse[keys]
    check_attn(cuda_lib, a)                       # the others, and those without keys


@pytest.mark.parametrize("window,dtype,d", [(64, "bf16", 64), (100, "fp16", 128), (300, "bf16", 128)])
def test_prefix_attn_window_of_rows_that_see_one_another(cuda_lib, window, dtype, d):
    """Tree words in which every row sees rows behind it too, so that no row has
    depth 0 and the windows of all start later: keys below the lowest window
    hold NaN, in the prefix and among the requests' own."""
    a = make_attn(np.random.default_rng(window), [140, 300, 20, 90], [16, 9, 5, 64], 200, 4, 1, d, dtype, 16,
                  window=window, tree=True)
    news = [int(m) for m in np.diff(a["cu"])]
    a["words"] = [(1 << m) - 1 for m in news for _ in range(m)] + [0] * (len(a["words"]) - a["n"])
    pages, page = a["k"].shape[:2]
    seen = np.zeros((pages, page), bool)
    for b, m in enumerate(news):
        for i in range(m):
            pre, own = ob.visible(i, m, int(a["lens"][b]), a["prefix"], window, a["words"][int(a["cu"][b]) + i])
            for j in pre:
                seen[a["prefix_pages"][j // page], j % page] = True
            for j in own:
                seen[a["table"][b, j // page], j % page] = True
    hide = torch.from_numpy(~seen).cuda()
    a["k"][hide], a["v"][hide] = float("nan"), float("nan")
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("top", [0, 100, 299, 300, 431])
def test_prefix_attn_largest_scores(cuda_lib, dtype, top):
    """Scores up to 2^26, one far above the others: that key's value alone.  Its
    weight is 2^e, with e the rounding of the row's maximum, and goes into the
    product rounded, into the sum not; the output is rounded once more.  The score
    is exact, its product with scale log2(e), the way back and that factor itself
    round to 32 bits."""
    a = make_attn(np.random.default_rng(top), [132, 132], [1, 2], 300, 2, 1, 64, dtype, 16)
    c = np.random.default_rng(top).integers(0, 255, 432)
    c[top] = 255
    keys = torch.from_numpy(c * 2.0 ** 8).to(a["k"])           # score: 2^13 * 2^8 c / 8 = 2^18 c
    a["q"].zero_()
    a["q"][:, :, 3] = 2.0 ** 13
    for b in range(2):
        for j in range(432):
            page = a["prefix_pages"][j // 16] if j < 300 else a["table"][b, (j - 300) // 16]
            at = (int(page), j % 16 if j < 300 else (j - 300) % 16)
            a["k"][at] = 0
            a["k"][at][0, 3] = keys[j]
    call_attn(cuda_lib, a)
    torch.cuda.synchronize()
    assert cuda_lib.mk_prefix_attn_status(a["workspace"]) == 0
    for row, b in ((0, 0), (2, 1)) if top == 431 else ((0, 0), (1, 1), (2, 1)):
        page = a["prefix_pages"][top // 16] if top < 300 else a["table"][b, (top - 300) // 16]
        v = a["v0"][int(page), top % 16 if top < 300 else (top - 300) % 16, 0]
        err = np.abs(np64(a["out"])[row] - v)
        assert np.all(err <= 2.1 * U[dtype] * np.abs(v) + TINY[dtype]), err.max()
        lse = np64(a["lse"])[row]
        assert np.all(np.abs(lse - 255 * 2.0 ** 18) <= 8 * V * 255 * 2.0 ** 18), lse


def test_prefix_attn_table_with_gaps(cuda_lib):
    """A block table whose rows are wider than the pages in use (table_stride >
    max_pages), as a view: the entries beside it are not read."""
    a = make_attn(np.random.default_rng(12), [300, 45, 1, 700], [8, 3, 1, 2], 130, 8, 2, 128, "bf16", 16)
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)
    want, lse = a["out"].clone(), a["lse"].clone()
    rows, cols = a["table"].shape
    wide = torch.full((rows + 2, cols + 5), 2 ** 30, dtype=torch.int32, device="cuda")
    view = wide[1:rows + 1, 2:cols + 2]
    view.copy_(a["keep"][2])
    io = cuda_lib.make_prefix_attn_io(a["q"], a["k"], a["v"], a["out"], a["keep"][0], a["keep"][1], view, a["keep"][3],
                                      a["prefix"], lse=a["lse"])
    assert (io.max_pages, io.table_stride) == (cols, cols + 5)
    a["whole"].fill_(CANARY)
    cuda_lib.mk_prefix_attn(io, a["workspace"])
    check_attn(cuda_lib, a)
    assert torch.equal(a["out"], want) and torch.equal(a["lse"], lse)


def test_prefix_attn_bad_tables_and_lengths(cuda_lib):
    """Pages outside the pool read as zeros; lengths are cut to the table."""
    a = make_attn(np.random.default_rng(2), [40, 9, 60], [2, 1, 4], 100, 4, 2, 64, "bf16", 16)
    a["k"].copy_(torch.from_numpy(a["k0"]))
    a["v"].copy_(torch.from_numpy(a["v0"]))
    a["table"][0, 1], a["table"][2, 0] = -1, 2 ** 31 - 1
    a["prefix_pages"][3] = 10 ** 6
    a["table"][1] = a["table"][2]
    a["lens"] = np.array([40, 10 ** 9, 60])
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)


def test_prefix_attn_is_repeatable_and_needs_no_clean_workspace(cuda_lib):
    a = make_attn(np.random.default_rng(3), [300, 45, 700, 2], [8, 3, 1, 2], 900, 8, 2, 128, "bf16", 16)
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)
    first, lse = a["out"].clone(), a["lse"].clone()
    a["workspace"].fill_(0xFF)
    cuda_lib.mk_prefix_attn(a["io"], a["workspace"])
    torch.cuda.synchronize()
    assert torch.equal(a["out"], first) and torch.equal(a["lse"], lse)


def test_prefix_attn_workspace_too_small(cuda_lib):
    a = make_attn(np.random.default_rng(4), [30], [1], 40, 4, 1, 64, "bf16", 16)
    call_attn(cuda_lib, a)
    torch.cuda.synchronize()
    with pytest.raises(cuda_lib.MkError) as e:
        cuda_lib.mk_prefix_attn(a["io"], a["workspace"][:-1])
    assert e.value.status == 1


def test_prefix_attn_no_rows(cuda_lib):
    """Nothing to attend to: outputs stay, the status is that of a call."""
    a = make_attn(np.random.default_rng(5), [30], [0], 40, 4, 1, 64, "bf16", 16, extra_rows=0)
    a["q"] = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    a["hq"] = 4
    io = cuda_lib.make_prefix_attn_io(a["q"], a["k"], a["v"], torch.empty_like(a["q"]), dev([30]), dev([0, 0]),
                                      dev(a["table"]), dev(a["prefix_pages"]), 40)
    ws = torch.full((cuda_lib.mk_prefix_attn_workspace(io),), 0xFF, dtype=torch.uint8, device="cuda")
    cuda_lib.mk_prefix_attn(io, ws)
    torch.cuda.synchronize()
    assert cuda_lib.mk_prefix_attn_status(ws) == 0


def test_prefix_attn_rows_before_the_first_request(cuda_lib):
    a = make_attn(np.random.default_rng(8), [30, 9, 40], [2, 1, 3], 100, 4, 2, 64, "bf16", 16)
    a["cu"] = np.array([2, 2, 3, 6])
    call_attn(cuda_lib, a)
    b = dict(a, n=4, cu=a["cu"] - 2)
    for name in ("q0", "whole", "out", "lse"):
        b[name] = a[name][2:]
    check_attn(cuda_lib, b)
    assert bool((a["whole"][:2] == CANARY).all()) and bool((a["lse"][:2] == CANARY).all())


@pytest.mark.parametrize("cu", [[0, 3, 1, 6], [6, 0, 6, 0], [2 ** 31 - 1, 0, -2 ** 31, 6]])
def test_prefix_attn_falling_rows(cuda_lib, cu):
    """Rows that would belong to several requests: the status says so, nothing
    beside the outputs is touched, and the next call is well again."""
    a = make_attn(np.random.default_rng(9), [30, 9, 40], [2, 1, 3], 100, 4, 2, 64, "bf16", 16)
    right = a["cu"]
    call_attn(cuda_lib, a)
    size = a["workspace"].numel()
    room = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    b = dict(a, cu=np.array(cu))
    call_attn(cuda_lib, b, workspace=room[:size])
    torch.cuda.synchronize()
    assert cuda_lib.mk_prefix_attn_status(room) == 1
    assert bool((room[size:] == 0x5A).all()) and bool((b["whole"][:, b["hq"]:] == CANARY).all())
    assert bool((b["whole"][6:] == CANARY).all())
    a["cu"] = right
    call_attn(cuda_lib, a, workspace=room[:size])
    check_attn(cuda_lib, a)


def test_prefix_attn_far_pages(cuda_lib):
    """Slots whose byte offset passes 32 bits: a pool of 4.6 GB per cache, keys at
    its end."""
    rng = np.random.default_rng(6)
    a = make_attn(rng, [100, 17], [2, 1], 70, 4, 2, 128, "bf16", 64)
    pages = 140000
    big = {}
    for name in ("k", "v"):
        pool = torch.zeros(pages, 64, 2, 128, dtype=torch.bfloat16, device="cuda")
        pool[-a[name].shape[0]:] = a[name]
        big[name] = pool
    shift = pages - a["k"].shape[0]
    far = dict(a, k=big["k"], v=big["v"], table=np.where(a["table"] < a["k"].shape[0], a["table"] + shift, -1),
               prefix_pages=a["prefix_pages"] + shift)
    call_attn(cuda_lib, a)
    call_attn(cuda_lib, far)
    check_attn(cuda_lib, a)
    assert torch.equal(far["out"][:a["n"]], a["out"][:a["n"]]) and torch.equal(far["lse"], a["lse"])


def test_rope_far_slots(cuda_lib):
    """Cache rows whose byte offset passes 32 bits."""
    rope = cuda_lib.mk_rope_create(cuda_lib.make_rope_config(64))
    pages = 140000
    kc, vc = (torch.zeros(pages, 64, 2, 128, dtype=torch.bfloat16, device="cuda").view(pages, 64, 4, 64) for _ in range(2))
    _, k = rounded(np.random.default_rng(7), (3, 4, 64), "bf16")
    at = pages * 64 - 3
    io = cuda_lib.make_rope_io(None, None, k, k, dev([0, 0, 0]), dev([at, at + 1, at + 2], torch.int64), kc, vc)
    cuda_lib.mk_rope_apply(rope, io)
    torch.cuda.synchronize()
    cuda_lib.mk_rope_destroy(rope)
    assert torch.equal(kc.view(-1, 4, 64)[-3:], k) and torch.equal(vc.view(-1, 4, 64)[-3:], k)   # position 0


def test_largest_batch(cuda_lib):
    """65536 requests of one token each: every row sees its own key alone, so that
    its output is that key's value to the bit and its lse the key's score."""
    B, page, hq, d = 65536, 16, 2, 64
    gen = torch.Generator(device="cuda").manual_seed(1)
    zero, one = (torch.full((B,), x, dtype=torch.int32, device="cuda") for x in (0, 1))
    free = torch.randperm(B, generator=gen, device="cuda").int()
    table = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
    cu, lens, positions, request = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (B + 1, B, B, B))
    slots, summary = torch.empty(B, dtype=torch.int64, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
    cuda_lib.mk_build_slots(cuda_lib.make_slots_io(zero, one, free, None, table, cu, lens, positions, slots, request,
                                                   summary, page, B))
    q, k, v = (torch.randn(B, h, d, generator=gen, device="cuda").bfloat16() for h in (hq, 1, 1))
    kc, vc = (torch.full((B, page, 1, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rope = cuda_lib.mk_rope_create(cuda_lib.make_rope_config(d))
    qr, out = torch.empty_like(q), torch.empty_like(q)
    cuda_lib.mk_rope_apply(rope, cuda_lib.make_rope_io(q, qr, k, v, positions, slots, kc, vc))
    lse = torch.empty(B, hq, device="cuda")
    io = cuda_lib.make_prefix_attn_io(qr, kc, vc, out, lens, cu, table, lse=lse)
    ws = torch.empty(cuda_lib.mk_prefix_attn_workspace(io), dtype=torch.uint8, device="cuda")
    cuda_lib.mk_prefix_attn(io, ws)
    torch.cuda.synchronize()
    cuda_lib.mk_rope_destroy(rope)
    assert cuda_lib.mk_prefix_attn_status(ws) == 0
    assert summary.tolist() == [B, B, 0, B]
    assert torch.equal(slots, free.long() * page) and torch.equal(cu, torch.arange(B + 1, dtype=torch.int32, device="cuda"))
    assert torch.equal(qr, q)                                    # position 0
    assert torch.equal(out, v.expand(B, hq, d))
    # 64 partial sums, each off by 2 V of the absolute sum; scale, log2(e), their product
    # with it and ln(2) round the score six times; exp2 and log2 of a sum near 1
    score = (q.double() * k.double()).sum(-1) / 8
    size = (q.double() * k.double()).abs().sum(-1) / 8
    assert bool(((lse.double() - score).abs() <= 64 * 2 * V * size + 6 * V * score.abs() + 2.0 ** -21).all())


# ------------------------------------------- together, streams and graphs

def _step(mk, rng, B, page, prefix, hq, hk, d, dtype, n_rows):
    """Buffers of a batched step: lengths, table, pool with a rotated prefix."""
    width = 8
    first = -(-prefix // page)
    n_pages = first + B * width + 8
    s = dict(B=B, page=page, prefix=prefix, hq=hq, hk=hk, d=d, dtype=dtype, n_pages=n_pages)
    ids = rng.permutation(n_pages)
    s["ids"] = ids
    cached = rng.integers(0, width * page - 20, B)
    s["cached0"], s["new0"] = cached, rng.integers(1, 5, B)
    table = np.full((B, width), -1)
    at = first
    for b in range(B):
        held = -(-int(cached[b]) // page)
        table[b, :held] = ids[at:at + held]
        at += held
    s["table0"], s["free0"] = table, ids[at:]
    s["kc0"], s["k_cache"] = rounded(rng, (n_pages, page, hk, d), dtype)
    s["vc0"], s["v_cache"] = rounded(rng, (n_pages, page, hk, d), dtype)
    s["x0"], s["qkv"] = rounded(rng, (n_rows, hq + 2 * hk, d), dtype)
    s["cached"], s["new"], s["table"] = dev(cached), dev(s["new0"]), dev(table)
    s["free"], s["prefix_pages"] = dev(s["free0"]), dev(ids[:first])
    z = lambda n, t=torch.int32: torch.zeros(n, dtype=t, device="cuda")  # noqa: E731
    s["cu"], s["lens"], s["positions"], s["slots"] = z(B + 1), z(B), z(n_rows), z(n_rows, torch.int64)
    s["summary"] = z(4)
    s["q"], s["out"] = torch.empty_like(s["qkv"][:, :hq].contiguous()), torch.zeros(n_rows, hq, d, dtype=TORCH[dtype], device="cuda")
    s["rope"] = mk.mk_rope_create(mk.make_rope_config(d))
    s["io"] = (mk.make_slots_io(s["cached"], s["new"], s["free"], None, s["table"], s["cu"], s["lens"],
                                s["positions"], s["slots"], None, s["summary"], page, n_pages, prefix),
               mk.make_rope_io(s["qkv"][:, :hq], s["q"], s["qkv"][:, hq:hq + hk], s["qkv"][:, hq + hk:],
                               s["positions"], s["slots"], s["k_cache"], s["v_cache"]),
               mk.make_prefix_attn_io(s["q"], s["k_cache"], s["v_cache"], s["out"], s["lens"], s["cu"],
                                      s["table"], s["prefix_pages"], prefix))
    s["workspace"] = torch.empty(mk.mk_prefix_attn_workspace(s["io"][2]), dtype=torch.uint8, device="cuda")
    return s


def _run_step(mk, s, stream=None):
    mk.mk_build_slots(s["io"][0], stream)
    mk.mk_rope_apply(s["rope"], s["io"][1], stream)
    mk.mk_prefix_attn(s["io"][2], s["workspace"], stream)


def _check_step(mk, s):
    """The step against the oracle's three operators in a row, each of the
    later ones on the GPU's own (rounded) outputs of the one before."""
    assert mk.mk_prefix_attn_status(s["workspace"]) == 0
    n_rows = s["qkv"].shape[0]
    want = ob.build_slots(s["cached0"], s["new0"], s["free0"], 0, s["table0"], n_rows, s["page"],
                          s["n_pages"], s["prefix"])
    for k in ("cu_rows", "lens", "positions", "slots"):
        assert np.array_equal(s[{"cu_rows": "cu"}.get(k, k)].cpu().numpy(), want[k]), k
    used = int(want["cu_rows"][-1])
    f, m = ob.rope_frequencies(s["d"])
    x = np64(s["qkv"])
    hq, hk = s["hq"], s["hk"]
    q = ob.rope(x[:, :hq], want["positions"], s["d"], "half", f, m)
    k = ob.rope(x[:, hq:hq + hk], want["positions"], s["d"], "half", f, m)
    tol = lambda w: 2 * np.abs(x).max() * 2.0 ** -19.5 + U[s["dtype"]] * np.abs(w) + TINY[s["dtype"]]  # noqa: E731
    assert np.all(np.abs(np64(s["q"])[:used] - q[:used]) <= tol(q[:used]))
    flat = np64(s["k_cache"]).reshape(-1, hk, s["d"])
    at = want["slots"][:used]
    live = at >= 0
    assert np.all(np.abs(flat[at[live]] - k[:used][live]) <= tol(k[:used][live]))
    a = dict(n=used, q0=np64(s["q"]), k0=np64(s["k_cache"]), v0=np64(s["v_cache"]))
    out, _, weight = ob.prefix_attn(a["q0"][:used], a["k0"], a["v0"], s["ids"], s["prefix"],
                                    want["table"], want["lens"], want["cu_rows"])
    keys = s["prefix"] + int(want["lens"].max())
    d, dt = s["d"], s["dtype"]
    e_s = 2 * math.sqrt(d) * V * norm(a["q0"]) * norm(a["k0"]) + 2.0 ** -20
    bound = weight * (U[dt] + 2 * e_s + (keys / 16 + 64) * 2 * V) + keys * TINY[dt] * np.abs(a["v0"]).max() + U[dt] * np.abs(out) + TINY[dt]
    assert np.all(np.abs(np64(s["out"])[:used] - out) <= bound)
    assert bool((s["out"][used:] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_step_of_all_three(cuda_lib, dtype):
    s = _step(cuda_lib, np.random.default_rng(21), 9, 16, 100, 8, 2, 64, dtype, 48)
    _run_step(cuda_lib, s)
    torch.cuda.synchronize()
    _check_step(cuda_lib, s)
    cuda_lib.mk_rope_destroy(s["rope"])


def test_two_captured_steps_on_two_streams(cuda_lib):
    """Two graphs with workspaces of their own replay at the same time; lengths
    that change between replays are read anew."""
    steps = [_step(cuda_lib, np.random.default_rng(30 + i), 6 + i, 16, 64, 8, 2, 64, "bf16", 40) for i in range(2)]
    graphs, streams = [], [torch.cuda.Stream() for _ in steps]
    for s, st in zip(steps, streams):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            _run_step(cuda_lib, s, torch.cuda.current_stream())
        graphs.append(g)
    for again in range(3):
        rng = np.random.default_rng(40 + again)
        for s in steps:
            s["new0"] = rng.integers(0, 5, s["B"])
            s["new"].copy_(dev(s["new0"]))
            s["out"].zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        for s in steps:
            _check_step(cuda_lib, s)
    for s in steps:
        cuda_lib.mk_rope_destroy(s["rope"])


def test_layer_chain_with_positions(cuda_lib):
    """Two dense layers with rotary positions between them: the first layer's
    fused QKV writes the second one's q and cache rows, mk_rope_apply turns
    them where they are, the second layer starts from them; held to the layer
    contract against the oracle on the same inputs."""
    wl = dict(synth.WORKLOADS["tiny_layer"], ffn="dense", dense_inter=256, fuse_next=True)
    T, ctx = 8, 100
    work, _ = H.prepare(wl, "host", T=T, ctx=ctx)
    c, W = work["cfgs"][0], dict(work["Ws"][0])
    nxt = work["next"]
    kc, vc = (t.clone() for t in work["caches"][0])
    nkc, nvc = (t.clone() for t in (nxt["k_cache"], nxt["v_cache"]))
    max_ctx = min(kc.shape[0], nkc.shape[0])
    x0 = work["x_in"][:T].contiguous()
    x1, x2 = torch.zeros_like(x0), torch.zeros_like(x0)
    hq, hk, d = c["n_q_heads"], c["n_kv_heads"], c["head_dim"]
    q = torch.zeros(T, hq, d, dtype=torch.bfloat16, device="cuda")
    W["next_attn_norm_w"], W["next_w_qkv"] = nxt["attn_norm_w"], nxt["w_qkv"]
    first = cuda_lib.mk_layer_create(cuda_lib.make_config(
        c, flags=cuda_lib.MK_FIRST_LAYER | cuda_lib.MK_FUSE_NEXT_QKV, max_ctx=max_ctx), W)
    second = cuda_lib.mk_layer_create(cuda_lib.make_config(c, flags=0, max_ctx=max_ctx), work["Ws"][0])
    rope = cuda_lib.mk_rope_create(cuda_lib.make_rope_config(d, theta=500.0))
    pos = np.arange(ctx, ctx + T)
    rows_k, rows_v = nkc[ctx:ctx + T], nvc[ctx:ctx + T]
    pool = lambda t: t[:max_ctx].view(1, max_ctx, hk, d)  # noqa: E731
    turn = cuda_lib.make_rope_io(q, q, rows_k, rows_v, dev(pos), dev(pos, torch.int64), pool(nkc), pool(nvc))
    cuda_lib.mk_decode_step(first, cuda_lib.make_step_io(T, ctx, x0, x1, kc, vc, next_k_cache=nkc, next_v_cache=nvc, q_out=q))
    torch.cuda.synchronize()
    before = np64(q), np64(nkc), np64(nvc)
    cuda_lib.mk_rope_apply(rope, turn)
    cuda_lib.mk_decode_step(second, cuda_lib.make_step_io(T, ctx, x1, x2, nkc, nvc, q_in=q))
    torch.cuda.synchronize()
    status = cuda_lib.mk_layer_status(first), cuda_lib.mk_layer_status(second)
    for layer in (first, second):
        cuda_lib.mk_layer_destroy(layer)
    cuda_lib.mk_rope_destroy(rope)
    assert status == (0, 0)
    f, m = ob.rope_frequencies(d, theta=500.0)
    turned = before[1].copy()
    turned[ctx:ctx + T] = ob.rope(before[1][ctx:ctx + T], pos, d, "half", f, m)
    H.assert_close("q", np64(q), ob.rope(before[0], pos, d, "half", f, m))
    H.assert_close("k", np64(nkc), turned)
    assert np.array_equal(np64(nvc), before[2])
    r = ol.layer_forward(oio.oracle_cfg(c), oio.np_weights(work["Ws"][0]), np64(x1), np64(nkc), np64(nvc), ctx,
                         q_in=np64(q), first_layer=False)
    H.assert_close("x_out", np64(x2), r["x_out"])


# ------------------------------------------------------- waits that run out

@pytest.fixture(scope="module")
def waiting(cuda_lib):
    """A call whose CTAs hold pairs of row tiles, solos, or both, several pieces
    each: 64 requests of one token, 8 heads on 2, behind 40,000 keys (on 152 SMs
    the pairs' work ends in the middle of a CTA's)."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    B, prefix, page, hq, hk, d = 64, 40000, 64, 8, 2, 64
    first, held = prefix // page, 5
    pages = first + B * held
    q = torch.randn(B, hq, d, generator=gen, device="cuda").bfloat16()
    kc, vc = (torch.randn(pages, page, hk, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    ids = torch.randperm(pages, generator=gen, device="cuda").int()
    out = torch.full((B, hq, d), CANARY, dtype=torch.bfloat16, device="cuda")
    lens, cu = torch.full((B,), 300, dtype=torch.int32, device="cuda"), torch.arange(B + 1, dtype=torch.int32, device="cuda")
    io = cuda_lib.make_prefix_attn_io(q, kc, vc, out, lens, cu, ids[first:].view(B, held), ids[:first], prefix)
    size = cuda_lib.mk_prefix_attn_workspace(io)
    room = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    cuda_lib.mk_prefix_attn(io, room[:size])
    torch.cuda.synchronize()
    assert cuda_lib.mk_prefix_attn_status(room) == 0
    return dict(io=io, ws=room[:size], guard=room[size:], out=out, want=out.clone(),
                keep=(q, kc, vc, ids, lens, cu), kept=(kc.clone(), vc.clone()))


def test_attention_waits_that_do_not_run_out(cuda_lib, waiting):
    waiting["out"].fill_(CANARY)
    assert cuda_lib.mk_selftest_attn_waits(waiting["io"], waiting["ws"], 2 * 10 ** 9) == 0
    assert torch.equal(waiting["out"], waiting["want"])


@pytest.mark.parametrize("what,which", [("scores", 0), ("scores", 3), ("weights", 0), ("weights", 2),
                                        ("row_tile", 0), ("row_tile", 1), ("buffers", 0), ("buffers", 1)])
def test_attention_gives_up_and_recovers(cuda_lib, waiting, what, which):
    """A hand-off that never comes: within the limit (1 ms) every warp of the CTA
    gives up, its copies and products are waited for, the status says so, nothing
    beside outputs and workspace is touched; the next call on the same workspace
    is well, to the bit."""
    status = cuda_lib.mk_selftest_attn_waits(waiting["io"], waiting["ws"], 10 ** 6, what, which)
    assert cuda_lib.STATUS_NAMES[status] == "MK_ERR_TIMEOUT"
    assert cuda_lib.mk_prefix_attn_status(waiting["ws"]) == status
    assert bool((waiting["guard"] == 0x5A).all())
    assert all(torch.equal(a, b) for a, b in zip(waiting["keep"][1:3], waiting["kept"]))
    waiting["out"].fill_(CANARY)
    cuda_lib.mk_prefix_attn(waiting["io"], waiting["ws"])
    torch.cuda.synchronize()
    assert cuda_lib.mk_prefix_attn_status(waiting["ws"]) == 0
    assert torch.equal(waiting["out"], waiting["want"])


def test_rope_of_an_idle_step(cuda_lib):
    """A step without rows, through the binding: nothing happens."""
    pool = torch.full((2, 16, 2, 64), CANARY, dtype=torch.bfloat16, device="cuda")
    qkv = torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    rope = cuda_lib.mk_rope_create(cuda_lib.make_rope_config(64))
    for q in (qkv[:, :4], None):
        io = cuda_lib.make_rope_io(q, None if q is None else torch.empty_like(q), qkv[:, 4:6], qkv[:, 6:], none, none.long(), pool, pool.clone())
        cuda_lib.mk_rope_apply(rope, io)
    cuda_lib.mk_rope_apply(rope, cuda_lib.make_rope_io(qkv, torch.empty_like(qkv), None, None, none, None, None, None))
    torch.cuda.synchronize()
    cuda_lib.mk_rope_destroy(rope)
    assert bool((pool == CANARY).all())
