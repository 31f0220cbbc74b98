"""GPU parity of the attention half of a batched layer over a cache in 4 bits
(mk_linear, mk_qkv_append, mk_kvq_read, mk_kvq_attn) with the float64 oracle,
through the binding.

Tolerances, from the arithmetic, with u = eps / 2 of the tensors' type, tiny = half
the spacing of its subnormals and v = 2^-24, half a step of float32:

append: what a value is made from is off by less than 2^-20 of its pair's
  magnitude (the angle 2^-25 rad, sine and cosine 2 ulp, weight, factor and
  products 4 v, the root of the mean 6 v):
    |err| <= (|n_a| + |n_b|) m 2^-20 + u |y| + tiny.
  Codes and scales are the oracle's: what is near a border is worked out in 64 bits.
attention: a score is a sum of d exact products in float32, each partial sum off by
  2 v, and sum |q_i k_i| <= |q| |k|; q is off by 2^-25 of its row's largest value:
  with e_s = scale 3 d v max|q| max|k| + 2^-19 (exp2, its argument, the reference's
  rounding) a weight is relatively off by e_s; rounding it to fp16 adds 2^-11, or,
  where it underflows, 2^-25 against a largest weight of at least 2^-10.  A
  quotient doubles e_s.  Sums of n keys in chunks of 16 and of the partial results
  add (n / 16 + 64) 2 v.  With W = sum_j w_j |v_j| over the softmax weights:
    |out err| <= W (2^-11 + 2 e_s + (n / 16 + 64) 2 v) + n 2^-15 2^-10 max|v| + u |out| + tiny,
    |lse err| <= e_s + (n + 64) v + 4 v |lse|.
linear: products are exact in float32, sums of n_in in chunks of 16 and of up to 64
  parts off by (n_in / 16 + 64) 2 v of S = |x| |w|^T; an activation has a slope of
  at most 1.13 and adds 2^-20 (1 + |y|):
    |err| <= 1.13 S (n_in / 16 + 64) 2 v + 2^-20 (1 + |y|) + u |y| + tiny.
"""

import math

import numpy as np
import pytest
import torch

from oracle import batch as ob
from oracle import kvq as ok

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}               # torch.finfo(t).eps / 2
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}
V = 2.0 ** -24
CANARY = -1152.0                                          # exact in bf16 and fp16


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda()


def np64(t):
    return t.detach().cpu().double().numpy()


def rounded(rng, shape, dtype, scale=1.0):
    """N(0, scale^2) values of the type, as float64, and the CUDA tensor."""
    t = torch.from_numpy(rng.standard_normal(shape) * scale).to(TORCH[dtype])
    return t.double().numpy(), t.cuda()


# ----------------------------------------------------------------- append

def pool(rng, pages, heads, page, d):
    """Pools of any codes and scales that are numbers."""
    return [torch.from_numpy(x).cuda() for x in (
        rng.integers(0, 256, (pages, heads, page, d // 2), dtype=np.uint8),
        rng.integers(0, 126, (pages, heads, page, d // 16), dtype=np.uint8))]


def check_append(mk, rng, n, hq, hk, d, rot, layout, dtype, positions, bits, norm=True, page=16, scaling="none",
                 factor=1.0, orig_ctx=0, eps=1e-6, in_place=False, no_v=False, no_q=False, no_k=False, exps=True,
                 stream=None, by=1.0, change=None):
    pages = n // page + 3
    x, qkv = rounded(rng, (n, hq + 2 * hk + 1, d), dtype, by)   # one head more: the rows have a gap
    if change is not None:
        change(x)
        qkv.copy_(torch.from_numpy(x))
        x = np64(qkv)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:hq + 2 * hk]
    slots = rng.permutation(pages * page)[:n]
    if n > 3:
        slots[[1, n - 1]] = [-1, pages * page]              # rows without a place
    live = (slots >= 0) & (slots < pages * page)
    wq, wk = [rounded(rng, (d,), dtype) if norm else (None, None) for _ in range(2)]
    out = torch.full((n, hq + 1, d), CANARY, dtype=TORCH[dtype], device="cuda")
    q_out = q if in_place else out[:, :hq]
    rope = mk.mk_rope_create(mk.make_rope_config(d, rot, layout=layout, scaling=scaling, factor=factor,
                                                 orig_ctx=orig_ctx)) if rot else None
    e = [rng.integers(-3, 4, hk) if exps else np.zeros(hk, int) for _ in range(2)]
    kw = dict(q_norm=wq[1], k_norm=wk[1], eps=eps)
    if bits == 16:
        caches = [rounded(rng, (pages, page, hk, d), dtype)[1] for _ in range(2)]
        kw.update(k_cache=None if no_k else caches[0], v_cache=None if no_v or no_k else caches[1])
    else:
        caches = pool(rng, pages, hk, page, d) + pool(rng, pages, hk, page, d)
        ex = [dev(a) if exps else None for a in e]
        if not no_k:
            kw.update(kvq=mk.make_kvq_cache(*caches, *ex))
    kept = [c.clone() for c in caches]
    pos, at = dev(positions) if rot else None, None if no_k else dev(slots, torch.int64)
    io = mk.make_qkv_append_io(None if no_q else q, None if no_q else q_out, None if no_k else k,
                               None if no_v or no_k else v, pos, at, **kw)
    mk.mk_qkv_append(rope, io, stream)
    torch.cuda.synchronize()
    mk.mk_rope_destroy(rope)
    f, m = ob.rope_frequencies(rot or 16, scaling=scaling, factor=factor, orig_ctx=orig_ctx)

    def want(src, w):
        with np.errstate(invalid="ignore"):
            return ok.norm_rope(src, w, eps, positions, rot, layout, f, m)

    def close(got, wanted):
        y, mag = wanted
        tol = mag * 2.0 ** -20 + U[dtype] * np.abs(y) + TINY[dtype]
        assert np.all(np.abs(got - y) <= tol), (np.abs(got - y) / np.maximum(tol, 1e-300)).max()

    if not no_q:
        close(np64(q_out), want(x[:, :hq], wq[0]))
        if not in_place:
            assert bool((out[:, hq] == CANARY).all())
    if not in_place:                                        # the inputs are as they were
        assert np.array_equal(np64(qkv), x, equal_nan=True)
    if no_k:
        return
    at = slots[live]
    others = np.setdiff1d(np.arange(pages * page), at)
    yk = want(x[:, hq:hq + hk], wk[0])
    if bits == 16:
        flat = [c.view(pages * page, hk, d) for c in caches]
        close(np64(flat[0])[at], [a[live] for a in yk])
        old = [c.view(pages * page, hk, d) for c in kept]
        assert torch.equal(flat[1][at], old[1][at] if no_v else v[torch.from_numpy(live).cuda()])
    else:
        flat = [c.transpose(1, 2).reshape(pages * page, hk, -1) for c in caches]
        old = [c.transpose(1, 2).reshape(pages * page, hk, -1) for c in kept]
        for (y, a) in ((yk[0], 0), (x[:, hq + hk:hq + 2 * hk], 2)):
            codes, scales = ok.encode(y[live], e[a // 2][None])
            if a and no_v:
                codes, scales = old[2][at].cpu().numpy(), old[3][at].cpu().numpy()
            assert np.array_equal(flat[a + 1][at].cpu().numpy(), scales)
            assert np.array_equal(flat[a][at].cpu().numpy(), codes)
    for a, b in zip(flat, old):
        assert torch.equal(a[others], b[others])


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,hq,hk,d,rot,dtype", [
    (1, 4, 1, 64, 64, "bf16"), (16, 32, 8, 128, 128, "bf16"), (5, 6, 2, 64, 16, "fp16"),
    (37, 8, 8, 128, 32, "bf16"), (3, 1, 1, 256, 256, "fp16"), (9, 5, 5, 80, 48, "bf16"),
    (700, 3, 1, 32, 16, "fp16"), (2, 33, 17, 16, 16, "bf16"), (400, 32, 8, 128, 128, "fp16")])
def test_append(cuda_lib, bits, layout, n, hq, hk, d, rot, dtype):
    rng = np.random.default_rng(n)
    check_append(cuda_lib, rng, n, hq, hk, d, rot, layout, dtype, rng.integers(0, 40000, n), bits)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("kw", [
    dict(norm=False), dict(norm=False, rot=0), dict(rot=0), dict(scaling="linear", factor=8.0),
    dict(scaling="base", factor=4.0), dict(scaling="parts", factor=16.0, orig_ctx=4096), dict(eps=0.5),
    dict(in_place=True), dict(no_v=True), dict(no_q=True), dict(no_k=True), dict(exps=False), dict(page=256),
    dict(in_place=True, layout="interleaved"), dict(by=1e-3), dict(by=300.0), dict(by=1e-3, norm=False)])
def test_append_variants(cuda_lib, bits, kw):
    kw = dict(dict(layout="half", rot=64), **kw)
    rng = np.random.default_rng(11)
    check_append(cuda_lib, rng, 50, 8, 2, 128, dtype="bf16", positions=rng.integers(0, 1 << 20, 50), bits=bits, **kw)


@pytest.mark.parametrize("layout,d,rot,scaling", [
    ("half", 128, 32, "none"), ("half", 64, 64, "none"), ("interleaved", 128, 24, "linear"), ("interleaved", 80, 8, "none"),
    ("half", 128, 16, "parts")])
@pytest.mark.parametrize("n", [60, 1100, 4000])
def test_append_groups_as_given(cuda_lib, layout, d, rot, scaling, n):
    """Without norms: groups that the rotation leaves out, wholly or in part, and rows at
    position 0, whose values have few bits and are often on borders."""
    rng = np.random.default_rng(n + d)
    positions = rng.integers(0, 3, n) * rng.integers(0, 1 << 17, n)
    check_append(cuda_lib, rng, n, 2, 2, d, rot, layout, "bf16", positions, 4, norm=False, scaling=scaling,
                 factor=1.0 if scaling == "none" else 4.0, orig_ctx=4096 if scaling == "parts" else 0)


def test_append_head_of_eight(cuda_lib):
    rng = np.random.default_rng(2)
    check_append(cuda_lib, rng, 70, 5, 3, 8, 8, "interleaved", "bf16", rng.integers(0, 4000, 70), 16)


def test_append_many_codes(cuda_lib):
    """Codes of a million values, some hundred of which lie near a border in 32 bits."""
    rng = np.random.default_rng(3)
    for n, layout in ((1000, "half"), (4100, "interleaved")):   # rows on CTAs of 64 threads and of a warp
        check_append(cuda_lib, rng, n, 5, 3, 128, 128, layout, "bf16", rng.integers(0, 1 << 20, n), 4, scaling="parts",
                     factor=8.0, orig_ctx=8192)
    check_append(cuda_lib, rng, 4100, 33, 1, 64, 32, "half", "fp16", rng.integers(0, 1 << 20, 4100), 16)


def test_append_ties_infinities_and_nan(cuda_lib):
    """Values on borders between codes and scales (without a rotation they stay
    there), zeros, infinities; a NaN takes its group along."""
    def change(x):
        r = np.random.default_rng(4)
        x[:] = np.round(x * 8) / 4                                       # multiples of a quarter
        x[::3, :, ::16] = 7 * 2.0 ** r.integers(-3, 3, x[::3, :, ::16].shape)  # a power of two as scale
        x[1::7] = 0
        x[2::7, :, :16] = 7 * 17 / 16 * 2.0 ** -2                        # ties between scales
        x[3::7, :, 5], x[4::7, :, 40] = np.inf, -np.inf
        x[5::7, :, 20] = np.nan
    for dtype in ("bf16", "fp16"):
        rng = np.random.default_rng(5)
        check_append(cuda_lib, rng, 90, 1, 4, 64, 0, "half", dtype, None, 4, norm=False, no_q=True, change=change)


def test_read(cuda_lib):
    rng = np.random.default_rng(6)
    for dtype, d, page, heads, pages in (("bf16", 128, 64, 8, 5), ("fp16", 64, 16, 3, 7), ("bf16", 80, 32, 1, 1)):
        pools = pool(rng, pages, heads, page, d) + pool(rng, pages, heads, page, d)
        for s in pools[1::2]:
            s.copy_(torch.from_numpy(rng.integers(40, 80, s.shape, dtype=np.uint8)))
        exps = [rng.integers(-3, 4, heads) for _ in range(2)]
        on_gpu = [dev(e) for e in exps]
        kvq = cuda_lib.make_kvq_cache(*pools, *on_gpu)
        n = pages * page
        want = [ok.decode_pool(pools[i].cpu().numpy(), pools[i + 1].cpu().numpy(), exps[i // 2]).reshape(n, heads, d)
                for i in (0, 2)]
        slots = rng.integers(-2, n + 2, 45)
        for sl in (None, slots):
            rows = n if sl is None else len(sl)
            out = [torch.full((rows, heads, d), CANARY, dtype=TORCH[dtype], device="cuda") for _ in range(2)]
            at = None if sl is None else dev(sl, torch.int64)
            cuda_lib.mk_kvq_read(cuda_lib.make_kvq_read_io(kvq, at, *out))
            for got, w in zip(out, want):
                if sl is not None:
                    w = np.where(((sl >= 0) & (sl < n))[:, None, None], w[np.clip(sl, 0, n - 1)], 0)
                assert np.array_equal(np64(got), w)
        one = torch.zeros(n, heads, d, dtype=TORCH[dtype], device="cuda")
        cuda_lib.mk_kvq_read(cuda_lib.make_kvq_read_io(kvq, None, None, one))
        assert np.array_equal(np64(one), want[1])


# -------------------------------------------------------------- attention

def make_attn(rng, lens, news, hq, hk, d, dtype, page, window=0, tree=False, q_scale=1.0, extra_rows=2, exps=True,
              k_scale=1.0):
    """Inputs of one call; what no row sees has NaN scales."""
    B = len(lens)
    n = int(sum(news))
    width = max(1, max(-(-max(a, 1) // page) for a in lens))
    held = [-(-max(a, 0) // page) for a in lens]
    n_pages = sum(held) + 2
    ids = rng.permutation(n_pages)
    table = np.full((B, width), n_pages + 99)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    cu = np.concatenate([[0], np.cumsum(news)]).astype(int)
    q0, q = rounded(rng, (n + extra_rows, hq + 1, d), dtype, q_scale)
    e = [rng.integers(-2, 2, hk) if exps else np.zeros(hk, int) for _ in range(2)]
    pools = []
    for by in (k_scale, 1.0):
        pools += list(ok.encode(rng.standard_normal((n_pages, hk, page, d)) * by))
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
    a = dict(n=n, q0=q0[:, :hq], q=q[:, :hq], table=table, lens=np.array(lens), cu=cu, window=window, words=words,
             dtype=dtype, d=d, hq=hq, hk=hk, page=page, pools=pools, exps=e, news=list(news))
    hide_unseen(a)
    return a


def hide_unseen(a):
    pages, _, page, _ = a["pools"][0].shape
    seen = np.zeros((pages, page), bool)
    for b in range(len(a["lens"])):
        for i in range(a["news"][b]):
            _, own = ob.visible(i, a["news"][b], min(max(int(a["lens"][b]), 0), a["table"].shape[1] * page), 0, a["window"],
                                None if a["words"] is None else a["words"][a["cu"][b] + i])
            for j in own:
                seen[a["table"][b, j // page], j % page] = True
    p, r = np.nonzero(~seen)
    for scales in a["pools"][1::2]:
        scales[p, :, r] = np.where(np.arange(a["d"] // 16) % 2, 0xFF, 0x7F)


def call_attn(mk, a, stream=None, workspace=None, scale=0.0, lse=True):
    rows = a["q"].shape[0]
    whole = torch.full((rows, a["hq"] + 1, a["d"]), CANARY, dtype=a["q"].dtype, device="cuda")
    a["whole"], a["out"] = whole, whole[:, :a["hq"]]
    a["lse"] = torch.full((rows, a["hq"]), CANARY, dtype=torch.float32, device="cuda")
    words = None if a["words"] is None else torch.tensor(
        [w - (1 << 64) if w >> 63 else w for w in a["words"]], dtype=torch.int64, device="cuda")
    a["dev"] = [torch.from_numpy(x).cuda() for x in a["pools"]] + [dev(e) for e in a["exps"]]
    a["keep"] = (dev(a["lens"]), dev(a["cu"]), dev(a["table"]), words)
    kvq = mk.make_kvq_cache(*a["dev"])
    io = mk.make_kvq_attn_io(a["q"], kvq, a["out"], *a["keep"][:3], window=a["window"], tree_mask=words,
                             lse=a["lse"] if lse else None, scale=scale)
    if workspace is None:
        workspace = torch.empty(mk.mk_kvq_attn_workspace(io), dtype=torch.uint8, device="cuda")
    a["workspace"], a["io"], a["kvq"] = workspace, io, kvq
    mk.mk_kvq_attn(io, workspace, stream)


def check_attn(mk, a, scale=None, skip=None):
    torch.cuda.synchronize()
    assert mk.mk_kvq_attn_status(a["workspace"]) == 0
    n, d, dt = a["n"], a["d"], a["dtype"]
    k, v = (ok.decode_pool(a["pools"][i], a["pools"][i + 1], a["exps"][i // 2]) for i in (0, 2))
    want, lse, weight = ob.prefix_attn(a["q0"][:n], k, v, [], 0, a["table"], a["lens"], a["cu"], a["window"], scale,
                                       a["words"])
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    keys = max(0, int(np.minimum(a["lens"], a["table"].shape[1] * a["page"]).max(initial=0)))
    top = lambda x: float(np.sqrt(np.max(np.nansum(x * x, axis=-1), initial=0.0)))  # noqa: E731
    e_s = sc * 3 * d * V * top(a["q0"]) * top(k) + 2.0 ** -19
    vmax = np.nanmax(np.abs(v), initial=0.0)
    tol = (weight * (2.0 ** -11 + 2 * e_s + (keys / 16 + 64) * 2 * V) + keys * 2.0 ** -25 * vmax
           + U[dt] * np.abs(want) + TINY[dt])
    got, got_lse = np64(a["out"])[:n], np64(a["lse"])[:n]
    use = np.ones(n, bool) if skip is None else ~skip[:n]
    got, got_lse, want, lse, tol = got[use], got_lse[use], want[use], lse[use], tol[use]
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
    # name: lens, news, hq, hk, d, dtype, page, more
    "one_key": ([1], [1], 4, 1, 64, "bf16", 16, {}),
    "no_key": ([0, 3, 0], [1, 1, 2], 2, 1, 64, "bf16", 16, {}),
    "idle_requests": ([20, 0, 33, 5, 40], [0, 0, 2, 0, 1], 4, 1, 128, "bf16", 16, {}),
    "all_idle": ([20, 7], [0, 0], 4, 1, 128, "bf16", 16, {}),
    "tile_ends": ([15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129], [1] * 6 + [2] * 3 + [3] * 3, 8, 2, 128,
                  "bf16", 64, {}),
    "tile_ends_64": ([15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129], [1] * 12, 8, 1, 64, "fp16", 16, {}),
    "mha": ([30, 90, 200], [3, 1, 2], 3, 3, 128, "fp16", 128, {}),
    "group_6": ([60, 61, 300], [5, 7, 16], 12, 2, 64, "bf16", 16, {}),
    "group_7": ([60, 61, 140], [19, 7, 37], 7, 1, 128, "bf16", 32, {}),
    "group_9": ([60, 161], [1, 2], 9, 1, 128, "fp16", 32, {}),
    "group_64": ([40, 9], [4, 3], 64, 1, 64, "bf16", 16, {}),
    "group_64_128": ([70, 300], [1, 1], 128, 2, 128, "bf16", 16, {}),
    "rows_8_9": ([100, 101, 40], [2, 2, 3], 8, 2, 128, "bf16", 16, {}),
    "chunk": ([350, 20], [300, 3], 4, 2, 128, "bf16", 64, {}),
    "chunk_fp16": ([200, 130], [140, 130], 2, 1, 64, "fp16", 256, {}),
    "few_keys_for_rows": ([3, 0, 8], [7, 2, 8], 4, 1, 128, "bf16", 16, {}),
    "window_1": ([20, 5, 300], [4, 5, 2], 4, 2, 64, "bf16", 16, dict(window=1)),
    "window_40": ([20, 50, 300, 41], [4, 5, 2, 1], 4, 2, 128, "bf16", 16, dict(window=40)),
    "window_200": ([20, 250, 700], [4, 16, 2], 4, 2, 64, "fp16", 32, dict(window=200)),
    "window_wide": ([20, 50], [4, 5], 4, 2, 64, "bf16", 16, dict(window=100000)),
    "tree": ([40, 300, 16], [16, 9, 16], 8, 2, 128, "bf16", 16, dict(tree=True)),
    "tree_64": ([64, 100], [64, 64], 4, 1, 64, "fp16", 16, dict(tree=True)),
    "tree_window": ([140, 300, 20], [16, 9, 5], 4, 1, 128, "bf16", 16, dict(tree=True, window=64)),
    "large_scores": ([100, 460], [4, 4], 8, 2, 128, "bf16", 16, dict(q_scale=16.0)),
    "large_scores_fp16": ([100, 460], [4, 4], 8, 2, 64, "fp16", 16, dict(q_scale=16.0)),
    "small_q": ([100, 60], [4, 4], 8, 2, 128, "bf16", 16, dict(q_scale=1e-20)),
    "large_keys": ([100, 60], [2, 1], 8, 2, 128, "bf16", 16, dict(q_scale=2.0 ** -12, k_scale=500.0)),
    "many_requests": ([(7 * i) % 90 + 1 for i in range(300)], [1] * 300, 4, 1, 64, "bf16", 16, {}),
    "many_items": ([(3 * i) % 11 + 1 for i in range(300)], [1] * 300, 32, 8, 64, "bf16", 16, {}),
    "requests_900": ([(5 * i) % 200 + 1 for i in range(900)], [i % 3 for i in range(900)], 2, 1, 64, "bf16", 16, {}),
    "long": ([1500, 40, 3700], [2, 2, 1], 4, 1, 128, "bf16", 1024, {}),
    "long_64": ([9000], [1], 8, 1, 64, "fp16", 64, {}),
    "verify": ([600, 555, 91, 16], [16, 9, 13, 16], 8, 2, 128, "bf16", 16, {}),
    "rows_32_33": ([200, 300, 64], [8, 9, 16], 4, 1, 128, "fp16", 16, {}),
    "rows_64_65_128_129": ([240, 141, 270, 290], [32, 33, 64, 65], 2, 1, 64, "bf16", 16, {}),
}


@pytest.mark.parametrize("name", list(ATTN))
def test_attn(cuda_lib, name):
    lens, news, hq, hk, d, dtype, page, more = ATTN[name]
    a = make_attn(np.random.default_rng(len(name)), lens, news, hq, hk, d, dtype, page, **more)
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)


@pytest.mark.parametrize("name,lens,news,hq,hk,d,dtype,page,more", [
    # many key tiles per worker, items whole and in parts one after the other
    ("one_token", [2000 - 13 * i for i in range(64)], [1] * 64, 8, 8, 64, "bf16", 64, {}),
    ("one_token_128", [1900 - 41 * i for i in range(40)], [1] * 40, 32, 8, 128, "fp16", 128, {}),
    ("two_tokens", [1500 - 17 * i for i in range(50)], [2 + i % 2 for i in range(50)], 20, 4, 64, "fp16", 32, {}),
    ("folded_whole", [130 + (37 * i) % 300 for i in range(300)], [8] * 300, 4, 1, 64, "bf16", 16, {}),
    ("folded_128", [150 + (37 * i) % 700 for i in range(120)], [5 + i % 9 for i in range(120)], 4, 1, 128, "bf16", 32,
     dict(tree=True)),
    ("folded_long", [3000, 2500, 2900, 700, 5, 3100], [24] * 4 + [5, 24], 8, 8, 128, "fp16", 64, {}),
    ("folded_window", [1400 - 9 * i for i in range(40)], [17] * 40, 4, 2, 64, "bf16", 16, dict(window=600)),
    ("tiles_of_80_rows", [700 - 11 * i for i in range(18)], [80] * 18, 4, 4, 64, "bf16", 32, {}),
    ("tiles_of_128_rows", [900 - 7 * i for i in range(12)], [150] * 12, 2, 2, 128, "fp16", 64, {}),
    ("mixed", [40 + (53 * i) % 900 for i in range(90)], [(1, 30, 2, 70)[i % 4] for i in range(90)], 4, 2, 64, "bf16", 16, {}),
])
def test_attn_many_tiles_per_worker(cuda_lib, name, lens, news, hq, hk, d, dtype, page, more):
    a = make_attn(np.random.default_rng(len(name)), lens, news, hq, hk, d, dtype, page, **more)
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)
    first, lse = a["out"].clone(), a["lse"].clone()
    for _ in range(3):
        cuda_lib.mk_kvq_attn(a["io"], a["workspace"])
    torch.cuda.synchronize()
    assert torch.equal(a["out"], first) and torch.equal(a["lse"], lse)


def test_attn_scale_and_no_lse(cuda_lib):
    a = make_attn(np.random.default_rng(1), [30, 109], [2, 1], 4, 2, 64, "bf16", 16, exps=False)
    call_attn(cuda_lib, a, scale=0.03125)
    check_attn(cuda_lib, a, scale=0.03125)
    out, lse = a["out"].clone(), a["lse"].clone()
    call_attn(cuda_lib, a, scale=0.03125, lse=False)
    torch.cuda.synchronize()
    assert torch.equal(a["out"], out) and bool((a["lse"] == CANARY).all())


@pytest.mark.parametrize("name", ["one_key", "no_key", "tile_ends", "chunk", "window_40", "tree_window", "long", "verify"])
def test_attn_rows_of_nan(cuda_lib, name):
    """A row whose q holds a NaN: out and lse are NaN (a row without keys still gets
    0 and -inf), and no other row's result is."""
    lens, news, hq, hk, d, dtype, page, more = ATTN[name]
    a = make_attn(np.random.default_rng(len(name)), lens, news, hq, hk, d, dtype, page, **more)
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
def test_attn_window_of_rows_that_see_one_another(cuda_lib, window, dtype, d):
    """Tree words in which every row sees rows behind it too, so that no row has
    depth 0 and the windows of all start later: what lies below has NaN scales."""
    a = make_attn(np.random.default_rng(window), [140, 300, 20, 90], [16, 9, 5, 64], 4, 1, d, dtype, 16, window=window,
                  tree=True)
    a["words"] = [(1 << m) - 1 for m in a["news"] for _ in range(m)] + [0] * 2
    hide_unseen(a)
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)


@pytest.mark.parametrize("n", [160, 270, 400])
def test_attn_parts_below_every_window(cuda_lib, n):
    """The same with many requests: an item that a CTA has whole, its rows twice in the
    tile, and behind it the first part of one that no row sees any key of."""
    a = make_attn(np.random.default_rng(n), [128 * (2 + i % 3) + 203 for i in range(n)], [40] * n, 1, 1, 64, "bf16", 16,
                  window=64, tree=True)
    a["words"] = [(1 << 40) - 1] * (40 * n) + [0] * 2
    hide_unseen(a)
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)


def test_attn_rising_scores(cuda_lib):
    """Scores that rise along the keys by far more than fp16 holds: the reference
    that weights are taken against moves all the time."""
    for d, new in ((128, 1), (64, 3), (128, 16)):
        a = make_attn(np.random.default_rng(d), [700, 333], [new, 1], 4, 1, d, "bf16", 16, exps=False)
        codes, scales = a["pools"][:2]
        for b in range(2):
            for j in range(a["lens"][b]):
                page = a["table"][b, j // 16]
                scales[page, :, j % 16] = ok.e4m3(0.01 + j / 90.0)
        a["q"].abs_()
        a["q0"] = np64(a["q"])
        codes[:] = codes | 0x88
        call_attn(cuda_lib, a)
        check_attn(cuda_lib, a)


def test_attn_bad_tables_and_lengths(cuda_lib):
    """Pages outside the pool read as zeros; lengths are cut to the table."""
    a = make_attn(np.random.default_rng(2), [40, 9, 60], [2, 1, 4], 4, 2, 64, "bf16", 16)
    for s in a["pools"][1::2]:
        s[:] = 56
    a["table"][0, 1], a["table"][2, 0] = -1, 2 ** 31 - 1
    a["table"][1] = a["table"][2]
    a["lens"] = np.array([40, 10 ** 9, -7])
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)


def test_attn_table_with_gaps(cuda_lib):
    a = make_attn(np.random.default_rng(12), [300, 45, 1, 700], [8, 3, 1, 2], 8, 2, 128, "bf16", 16)
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)
    want, lse = a["out"].clone(), a["lse"].clone()
    rows, cols = a["table"].shape
    wide = torch.full((rows + 2, cols + 5), 2 ** 30, dtype=torch.int32, device="cuda")
    view = wide[1:rows + 1, 2:cols + 2]
    view.copy_(a["keep"][2])
    io = cuda_lib.make_kvq_attn_io(a["q"], a["kvq"], a["out"], a["keep"][0], a["keep"][1], view, lse=a["lse"])
    a["whole"].fill_(CANARY)
    cuda_lib.mk_kvq_attn(io, a["workspace"])
    check_attn(cuda_lib, a)
    assert torch.equal(a["out"], want) and torch.equal(a["lse"], lse)


def test_attn_is_repeatable_and_needs_no_clean_workspace(cuda_lib):
    a = make_attn(np.random.default_rng(3), [300, 45, 1700, 2], [8, 3, 1, 2], 8, 2, 128, "bf16", 16)
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)
    first, lse = a["out"].clone(), a["lse"].clone()
    a["workspace"].fill_(0xFF)
    cuda_lib.mk_kvq_attn(a["io"], a["workspace"])
    torch.cuda.synchronize()
    assert torch.equal(a["out"], first) and torch.equal(a["lse"], lse)


def test_attn_rows_before_the_first_request(cuda_lib):
    a = make_attn(np.random.default_rng(13), [30, 90], [3, 2], 4, 2, 64, "bf16", 16)
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)
    want = a["out"].clone()
    a["keep"][1][0] = 2                              # the first request has one row left, its last
    a["whole"].fill_(CANARY)
    cuda_lib.mk_kvq_attn(a["io"], a["workspace"])
    torch.cuda.synchronize()
    assert bool((a["whole"][:2] == CANARY).all()) and torch.equal(a["out"][2:5], want[2:5])


def test_attn_on_streams_and_in_graphs(cuda_lib):
    calls = [make_attn(np.random.default_rng(20 + i), [400 + i, 77], [1 + 2 * i, 1], 8, 2, 128, "bf16", 16) for i in range(3)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for a, s in zip(calls, streams):
        with torch.cuda.stream(s):
            call_attn(cuda_lib, a, stream=s)
    for a in calls:
        check_attn(cuda_lib, a)
    for a in calls:
        a["want"] = a["out"].clone(), a["lse"].clone()
        a["whole"].fill_(CANARY)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cuda_lib.mk_kvq_attn(a["io"], a["workspace"], torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert bool((a["whole"] == CANARY).all())
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a["out"], a["want"][0])
        a["keep"][0][0] -= 9                         # other lengths in the same graph
        a["lens"][0] -= 9
        g.replay()
        hide = [s.copy() for s in a["pools"][1::2]]
        check_attn(cuda_lib, a)
        del hide


def test_attn_without_pages(cuda_lib):
    """A table without columns, and a pool without pages, which reads as zeros."""
    a = make_attn(np.random.default_rng(14), [0, 0], [1, 9], 8, 2, 128, "bf16", 16)
    a["table"] = np.zeros((2, 0), int)
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)
    for new in (1, 9):
        a = make_attn(np.random.default_rng(15), [40, 200], [1, new], 8, 2, 128, "bf16", 16)
        a["pools"] = [p[:0] for p in a["pools"]]
        call_attn(cuda_lib, a)
        torch.cuda.synchronize()
        assert bool((a["out"][:a["n"]] == 0).all())
        want = np.log([40.0] + [200.0 - new + i + 1 for i in range(new)])
        assert np.abs(np64(a["lse"])[:a["n"]] - want[:, None]).max() < 1e-5


def test_attn_many_requests(cuda_lib):
    """More requests than a CTA has threads, several per thread; rows for either kernel."""
    rng = np.random.default_rng(16)
    for news in ([int(i % 7 == 0) for i in range(3000)], [20 * int(i % 150 == 3) for i in range(1200)]):
        lens = [int(n + rng.integers(0, 60)) if n else int(rng.integers(0, 60)) for n in news]
        a = make_attn(rng, lens, news, 4, 1, 64, "fp16", 16)
        call_attn(cuda_lib, a)
        check_attn(cuda_lib, a)


def far_pools(d, heads, page):
    """Pools whose codes pass 4 GB, their last pages' numbers."""
    pages = (1 << 32) // (heads * page * d // 2) + 40
    big = [torch.empty(pages, heads, page, w, dtype=torch.uint8, device="cuda") for w in (d // 2, d // 16) * 2]
    return big, pages


@pytest.mark.parametrize("new", [1, 12])
def test_attn_pages_beyond_four_gigabytes(cuda_lib, new):
    a = make_attn(np.random.default_rng(17), [700, 333], [new, 1], 32, 8, 128, "bf16", 128)
    big, pages = far_pools(128, 8, 128)
    small = a["pools"][0].shape[0]
    for b, p in zip(big, a["pools"]):
        b[pages - small:] = torch.from_numpy(p).cuda()
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)
    want, lse = a["out"].clone(), a["lse"].clone()
    table = a["keep"][2] + (pages - small)
    kvq = cuda_lib.make_kvq_cache(*big, *a["dev"][4:])
    io = cuda_lib.make_kvq_attn_io(a["q"], kvq, a["out"], a["keep"][0], a["keep"][1], table, lse=a["lse"])
    a["whole"].fill_(CANARY)
    cuda_lib.mk_kvq_attn(io, a["workspace"])
    torch.cuda.synchronize()
    assert torch.equal(a["out"], want) and torch.equal(a["lse"], lse)


def test_append_and_read_beyond_four_gigabytes(cuda_lib):
    rng = np.random.default_rng(18)
    big, pages = far_pools(128, 8, 64)
    kvq = cuda_lib.make_kvq_cache(*big)
    k0, k = rounded(rng, (5, 8, 128), "bf16")
    v0, v = rounded(rng, (5, 8, 128), "bf16")
    slots = dev([pages * 64 - 1, pages * 64 - 70, 3, pages * 64, pages * 32 + 17], torch.int64)
    cuda_lib.mk_qkv_append(None, cuda_lib.make_qkv_append_io(None, None, k, v, None, slots, kvq=kvq))
    out = [torch.empty(5, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cuda_lib.mk_kvq_read(cuda_lib.make_kvq_read_io(kvq, slots, *out))
    for x, got in ((k0, out[0]), (v0, out[1])):
        want = ok.decode(*ok.encode(x))
        want[3] = 0
        assert np.array_equal(np64(got), want)


def test_append_captured_and_replayed(cuda_lib):
    """A captured call reads its tensors when it is replayed."""
    rng = np.random.default_rng(19)
    n, hq, hk, d = 40, 8, 2, 64
    pools = pool(rng, 4, hk, 16, d) + pool(rng, 4, hk, 16, d)
    kvq = cuda_lib.make_kvq_cache(*pools)
    _, qkv = rounded(rng, (n, hq + 2 * hk, d), "bf16")
    positions, slots = dev(np.arange(n)), dev(rng.permutation(64)[:n], torch.int64)
    q_out = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
    rope = cuda_lib.mk_rope_create(cuda_lib.make_rope_config(d))
    io = cuda_lib.make_qkv_append_io(qkv[:, :hq], q_out, qkv[:, hq:hq + hk], qkv[:, hq + hk:], positions, slots, kvq=kvq)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        cuda_lib.mk_qkv_append(rope, io, torch.cuda.current_stream())
    x, again = rounded(rng, (n, hq + 2 * hk, d), "bf16")
    qkv.copy_(again)
    positions += 1000
    g.replay()
    torch.cuda.synchronize()
    f, m = ob.rope_frequencies(d)
    y, _ = ok.norm_rope(x[:, hq:hq + hk], None, 0, np.arange(n) + 1000, d, "half", f, m)
    codes, scales = ok.encode(y)
    got = [p.transpose(1, 2).reshape(64, hk, -1)[slots].cpu().numpy() for p in pools[:2]]
    cuda_lib.mk_rope_destroy(rope)
    assert np.array_equal(got[0], codes) and np.array_equal(got[1], scales)


# ----------------------------------------------------------------- linear

def check_linear(mk, rng, m, k, n, dtype, bias=False, act="none", residual=False, in_place=False, gap=8, stream=None,
                 by=1.0, pad=3):
    x0, x = rounded(rng, (m, k + gap), dtype, by)
    w0, w = rounded(rng, (n, k + gap), dtype, k ** -0.5)
    x[:, k:], w[:, k:] = float("nan"), float("nan")          # what lies between the rows is not read
    b0, b = rounded(rng, (n,), dtype) if bias else (None, None)
    whole = torch.full((m + 1, n + pad), CANARY, dtype=TORCH[dtype], device="cuda")
    out = whole[:m, :n]
    r0, r = rounded(rng, (m, n + pad + 2 * (pad & 1)), dtype) if residual else (None, None)
    if residual:
        r0, r = r0[:, :n], r[:, :n]
        if in_place:
            out.copy_(r)
            r = out
    io = mk.make_linear_io(x[:, :k], w[:, :k], out, bias=b, act=act, residual=r)
    ws = torch.full((mk.mk_linear_workspace(io),), 0xFF, dtype=torch.uint8, device="cuda")
    mk.mk_linear(io, ws, stream)
    torch.cuda.synchronize()
    assert mk.mk_linear_status(ws) == 0
    want, s = ok.linear(x0[:, :k], w0[:, :k], b0, act, r0)
    tol = 1.13 * s * (k / 16 + 64) * 2 * V + 2.0 ** -20 * (1 + np.abs(want)) + U[dtype] * np.abs(want) + TINY[dtype]
    err = np.abs(np64(out) - want)
    assert np.all(err <= tol), (err / tol).max()
    assert bool((whole[m:] == CANARY).all()) and bool((whole[:, n:] == CANARY).all())
    if not in_place:
        first = out.clone()
        ws.fill_(0x55)
        mk.mk_linear(io, ws, stream)
        torch.cuda.synchronize()
        assert torch.equal(out, first)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m,k,n", [
    (1, 8, 1), (1, 64, 128), (2, 256, 384), (3, 72, 130), (16, 4096, 256), (17, 1000, 129), (31, 136, 100),
    (64, 2048, 640), (65, 520, 255), (100, 4096, 257), (127, 64, 127), (128, 128, 256), (129, 192, 513),
    (250, 1024, 1031), (256, 320, 999), (257, 8, 7), (600, 264, 300), (1000, 512, 1500), (2100, 136, 2600),
    (90, 72, 23000)])
def test_linear(cuda_lib, dtype, m, k, n):
    check_linear(cuda_lib, np.random.default_rng(m + k + n), m, k, n, dtype, bias=bool(n & 1), residual=bool(m & 1))


@pytest.mark.parametrize("m,k,n", [(5, 200, 77), (300, 200, 264)])
@pytest.mark.parametrize("kw", [
    dict(act="silu"), dict(act="gelu"), dict(act="gelu_tanh"), dict(act="silu", bias=True, residual=True),
    dict(residual=True, in_place=True), dict(residual=True, in_place=True, act="gelu"), dict(gap=0),
    dict(act="silu", by=100.0), dict(act="gelu_tanh", by=100.0)])
def test_linear_variants(cuda_lib, m, k, n, kw):
    check_linear(cuda_lib, np.random.default_rng(9), m, k, n, "bf16", **kw)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m,k,n", [
    (1, 8, 4), (5, 200, 76), (64, 2048, 640), (127, 64, 132), (250, 1024, 1036), (257, 8, 12), (600, 264, 300),
    (1000, 512, 1500), (2101, 136, 2604), (90, 72, 23000)])
@pytest.mark.parametrize("kw", [
    dict(), dict(residual=True, bias=True, act="gelu"), dict(residual=True, in_place=True, act="silu")])
def test_linear_outputs_in_fours(cuda_lib, dtype, m, k, n, kw):
    check_linear(cuda_lib, np.random.default_rng(m + k + n), m, k, n, dtype, pad=4, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_linear_activations_over_their_range(cuda_lib, act, dtype):
    """Every value of the type from -40 to 40, one by one, by way of a row with a single 1.
    Each function has an exponential 2^E whose E is off by three roundings of itself, and is
    off by 2^-18.5 beside that; the oracle's 1 + erf and 1 + tanh are off by 2^-53, and what
    lies below 2^-126 may be zero."""
    import torch as T
    bits = T.arange(0, 1 << 16, dtype=T.int32, device="cuda").to(T.int16)
    y = bits.view(TORCH[dtype])
    y = y[T.isfinite(y) & (y.float().abs() <= 40)]
    y = y[: y.numel() // 8 * 8]
    n = y.numel()
    w = T.zeros(n, 8, dtype=y.dtype, device="cuda")
    w[:, 3] = y
    x = T.zeros(1, 8, dtype=y.dtype, device="cuda")
    x[0, 3] = 1.0
    out = T.empty(1, n, dtype=y.dtype, device="cuda")
    io = cuda_lib.make_linear_io(x, w, out, act=act)
    ws = T.empty(cuda_lib.mk_linear_workspace(io), dtype=T.uint8, device="cuda")
    cuda_lib.mk_linear(io, ws)
    T.cuda.synchronize()
    want, _ = ok.linear(np64(x), np64(w), None, act, None)
    got, a = np64(out)[0], np.abs(np64(y))
    e = math.log2(math.e) * {"silu": a, "gelu": a * a / 2, "gelu_tanh": 2 * 0.79789 * (a + 0.044716 * a ** 3)}[act]
    tol = (2.0 ** -18.5 + 3 * np.minimum(e, 130.0) * V + U[dtype]) * np.abs(want[0]) + TINY[dtype] + (a + 1) * 2.0 ** -53
    assert np.all(np.abs(got - want[0]) <= tol), (np.abs(got - want[0]) / tol).max()


def test_linear_takes_infinities_and_nan_as_they_come(cuda_lib):
    x = torch.zeros(40, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(200, 64, dtype=torch.bfloat16, device="cuda")
    x[3, 5], x[4, 6], x[7, 0] = float("inf"), float("nan"), 2.0
    out = torch.empty(40, 200, dtype=torch.bfloat16, device="cuda")
    for act in ("none", "silu", "gelu", "gelu_tanh"):
        io = cuda_lib.make_linear_io(x, w, out, act=act)
        ws = torch.empty(cuda_lib.mk_linear_workspace(io), dtype=torch.uint8, device="cuda")
        cuda_lib.mk_linear(io, ws)
        torch.cuda.synchronize()
        assert bool(torch.isinf(out[3]).all()) and bool(torch.isnan(out[4]).all()) and bool((out[0] == 0).all())
        assert bool((out[7] > 1.7).all()) and bool(torch.isfinite(out[5:]).all())


def test_linear_on_streams_and_in_graphs(cuda_lib):
    """Calls of every kind side by side, then captured and replayed on other inputs."""
    rng = np.random.default_rng(40)
    calls = []
    for m, k, n in ((3, 1024, 256), (300, 512, 700), (2100, 64, 2600), (40, 128, 24000)):
        x0, x = rounded(rng, (m, k), "bf16")
        w0, w = rounded(rng, (n, k), "bf16", k ** -0.5)
        out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        io = cuda_lib.make_linear_io(x, w, out, act="silu")
        ws = torch.empty(cuda_lib.mk_linear_workspace(io), dtype=torch.uint8, device="cuda")
        calls.append((x0, x, w0, w, out, io, ws))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        for c, s in zip(calls, streams):
            cuda_lib.mk_linear(c[5], c[6], s)
    torch.cuda.synchronize()

    def check():
        for x0, _, w0, _, out, _, ws in calls:
            assert cuda_lib.mk_linear_status(ws) == 0
            want, s = ok.linear(x0, w0, act="silu")
            k = x0.shape[1]
            tol = 1.13 * s * (k / 16 + 64) * 2 * V + 2.0 ** -20 * (1 + np.abs(want)) + U["bf16"] * np.abs(want) + TINY["bf16"]
            assert np.all(np.abs(np64(out) - want) <= tol)

    check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c in calls:
            cuda_lib.mk_linear(c[5], c[6], torch.cuda.current_stream())
    for i, c in enumerate(calls):
        x0, x = rounded(rng, c[0].shape, "bf16")
        c[1].copy_(x)
        calls[i] = (x0,) + c[1:]
    for c in calls:
        c[4].fill_(CANARY)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    check()


def test_linear_without_rows(cuda_lib):
    x, w = (torch.zeros(n, 64, dtype=torch.bfloat16, device="cuda") for n in (0, 5))
    io = cuda_lib.make_linear_io(x, w, torch.zeros(0, 5, dtype=torch.bfloat16, device="cuda"))
    ws = torch.full((cuda_lib.mk_linear_workspace(io),), 0xFF, dtype=torch.uint8, device="cuda")
    cuda_lib.mk_linear(io, ws)
    torch.cuda.synchronize()
    assert cuda_lib.mk_linear_status(ws) == 0


@pytest.mark.parametrize("m,k,n", [
    (1, 2048, 9771), (3, 72, 10068), (16, 512, 4900), (40, 4096, 1000), (70, 2500 * 4, 264), (128, 640, 2050), (200, 328, 1999),
    (400, 256, 3300), (33, 24, 19000), (64, 4096, 6144)])
@pytest.mark.parametrize("kw", [dict(pad=4, residual=True, act="silu"), dict(bias=True)])
def test_linear_few_rows_and_many_outputs(cuda_lib, m, k, n, kw):
    check_linear(cuda_lib, np.random.default_rng(m + k + n), m, k, n, "bf16", **kw)


def test_attn_without_rows(cuda_lib):
    a = make_attn(np.random.default_rng(23), [30, 9], [0, 0], 4, 1, 64, "bf16", 16)
    a["q"], a["n"] = a["q"][:0], 0
    call_attn(cuda_lib, a)
    torch.cuda.synchronize()
    assert cuda_lib.mk_kvq_attn_status(a["workspace"]) == 0


# ---------------------------------------------------------- all of them

def test_a_step_through_all_operators(cuda_lib):
    """Projection, slots, norms with rotation and cache write, attention, projection
    onto the residual stream, twice: the second step attends to the first one's keys.
    The oracle goes on from what each operator was given, so that each is held to its
    own tolerance."""
    mk = cuda_lib
    rng = np.random.default_rng(30)
    H, hq, hk, d, page, B, width = 512, 8, 2, 64, 16, 5, 8
    n_pages = B * width
    w_qkv0, w_qkv = rounded(rng, ((hq + 2 * hk) * d, H), "bf16", H ** -0.5)
    w_o0, w_o = rounded(rng, (H, hq * d), "bf16", (hq * d) ** -0.5)
    b0, bias = rounded(rng, ((hq + 2 * hk) * d,), "bf16", 0.1)
    (wq0, wq), (wk0, wk) = (rounded(rng, (d,), "bf16") for _ in range(2))
    pools = [torch.zeros(n_pages, hk, page, w, dtype=torch.uint8, device="cuda") for w in (d // 2, d // 16) * 2]
    exps = np.array([1, -1]), np.array([0, 2])
    on_gpu = [dev(e) for e in exps]
    kvq = mk.make_kvq_cache(*pools, *on_gpu)
    table, head = dev(np.full((B, width), -1)), dev([0])
    free = dev(rng.permutation(n_pages))
    lens = dev([0] * B)
    rope = mk.mk_rope_create(mk.make_rope_config(d))
    f, m = ob.rope_frequencies(d)
    for news in ([5, 33, 0, 1, 16], [1, 1, 4, 1, 2]):
        n = sum(news)
        cu, new_lens, summary = dev([0] * (B + 1)), dev([0] * B), dev([0] * 4)
        positions, slots = dev([0] * n), dev([0] * n, torch.int64)
        new = dev(news)
        mk.mk_build_slots(mk.make_slots_io(lens, new, free, head, table, cu, new_lens, positions, slots, None,
                                           summary, page, n_pages))
        x0, x = rounded(rng, (n, H), "bf16")
        qkv = torch.empty(n, hq + 2 * hk, d, dtype=torch.bfloat16, device="cuda")
        io = mk.make_linear_io(x, w_qkv, qkv.view(n, -1), bias=bias)
        ws = torch.empty(mk.mk_linear_workspace(io), dtype=torch.uint8, device="cuda")
        mk.mk_linear(io, ws)
        made = np64(qkv)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        mk.mk_qkv_append(rope, mk.make_qkv_append_io(q, q, k, v, positions, slots, q_norm=wq, k_norm=wk, kvq=kvq))
        out = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
        aio = mk.make_kvq_attn_io(q, kvq, out, new_lens, cu, table)
        aws = torch.empty(mk.mk_kvq_attn_workspace(aio), dtype=torch.uint8, device="cuda")
        mk.mk_kvq_attn(aio, aws)
        x_out = torch.empty_like(x)
        oio = mk.make_linear_io(out.view(n, -1), w_o, x_out, residual=x)
        ows = torch.empty(mk.mk_linear_workspace(oio), dtype=torch.uint8, device="cuda")
        mk.mk_linear(oio, ows)
        torch.cuda.synchronize()
        lens, head = new_lens, summary[:1].clone()
        assert mk.mk_linear_status(ws) == mk.mk_kvq_attn_status(aws) == mk.mk_linear_status(ows) == 0

        want, s = ok.linear(x0, w_qkv0, b0)
        assert np.all(np.abs(made.reshape(n, -1) - want) <= s * (H / 16 + 64) * 2 * V + U["bf16"] * np.abs(want) + 1e-6)
        pos, sl = positions.cpu().numpy(), slots.cpu().numpy()
        yq, mag = ok.norm_rope(made[:, :hq], wq0, 1e-6, pos, d, "half", f, m)
        assert np.all(np.abs(np64(q) - yq) <= mag * 2.0 ** -20 + U["bf16"] * np.abs(yq))
        yk, _ = ok.norm_rope(made[:, hq:hq + hk], wk0, 1e-6, pos, d, "half", f, m)
        for i, y in ((0, yk), (2, made[:, hq + hk:])):
            codes, scales = ok.encode(y, exps[i // 2][None])
            got = [p.transpose(1, 2).reshape(n_pages * page, hk, -1)[slots].cpu().numpy() for p in pools[i:i + 2]]
            assert np.array_equal(got[0], codes) and np.array_equal(got[1], scales)
        kd, vd = (ok.decode_pool(pools[i].cpu().numpy(), pools[i + 1].cpu().numpy(), exps[i // 2]) for i in (0, 2))
        ao, _, weight = ob.prefix_attn(np64(q), kd, vd, [], 0, table.cpu().numpy(), lens.cpu().numpy(), cu.cpu().numpy())
        e_s = 3 * d ** 0.5 * V * np.abs(np64(q)).max() * d * np.abs(kd).max() + 2.0 ** -19
        assert np.all(np.abs(np64(out) - ao) <= weight * (2.0 ** -11 + 2 * e_s + 2.0 ** -15) + U["bf16"] * np.abs(ao) + 2.0 ** -18)
        want, s = ok.linear(np64(out).reshape(n, -1), w_o0, residual=x0)
        assert np.all(np.abs(np64(x_out) - want) <= s * (hq * d / 16 + 64) * 2 * V + U["bf16"] * np.abs(want) + 1e-6)
        assert np.array_equal(sl, slots.cpu().numpy())
    mk.mk_rope_destroy(rope)


# ------------------------------------------------------- waits that run out

LINEAR_WAITS = {  # one CTA per tile, several tiles each; clusters; pairs, several tiles each; clusters of pairs
    "single": (40, 1024, 60000), "split": (3, 16384, 256), "pair": (2100, 1024, 9000), "split_pair": (250, 2048, 8192)}


@pytest.fixture(scope="module", params=list(LINEAR_WAITS))
def linear_waiting(cuda_lib, request):
    m, k, n = LINEAR_WAITS[request.param]
    gen = torch.Generator(device="cuda").manual_seed(m)
    x, w = ((torch.randn(r, k, generator=gen, device="cuda") * k ** -0.25).bfloat16() for r in (m, n))
    out = torch.full((m, n), CANARY, dtype=torch.bfloat16, device="cuda")
    io = cuda_lib.make_linear_io(x, w, out, act="silu")
    room = torch.full((cuda_lib.mk_linear_workspace(io) + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    size = room.numel() - 4096
    cuda_lib.mk_linear(io, room[:size])
    torch.cuda.synchronize()
    assert cuda_lib.mk_linear_status(room) == 0
    return dict(name=request.param, io=io, ws=room[:size], guard=room[size:], out=out, want=out.clone(), keep=(x, w),
                kept=(x.clone(), w.clone()))


def test_linear_waits_that_do_not_run_out(cuda_lib, linear_waiting):
    a = linear_waiting
    a["out"].fill_(CANARY)
    assert cuda_lib.mk_selftest_linear_waits(a["io"], a["ws"], 2 * 10 ** 9) == 0
    assert torch.equal(a["out"], a["want"])


@pytest.mark.parametrize("what,which,half", [
    ("copies", 0, 0), ("copies", 2, 0), ("copies", 15, 0), ("copies", 0, 1), ("copies", 2, 1), ("copies", 15, 1),
    ("stage", 0, 0), ("stage", 3, 0), ("stage", 15, 0), ("sums", 0, 0), ("sums", 1, 0), ("columns", 0, 0), ("columns", 0, 1)])
def test_linear_gives_up_and_recovers(cuda_lib, linear_waiting, what, which, half):
    """A hand-off that never comes: within the limit (2 ms) every warp of the CTA, and of
    its cluster, gives up, the copies and products on their way are waited for, whoever
    issued them, the status says so, nothing beside the output and the workspace is
    touched; the next call on the same workspace is well, to the bit."""
    a = linear_waiting
    several = a["name"] in ("single", "pair")     # tiles per CTA
    if half and "pair" not in a["name"] or not several and (what == "columns" or (what, which) == ("sums", 1)):
        pytest.skip("no such hand-off")
    status = cuda_lib.mk_selftest_linear_waits(a["io"], a["ws"], 2 * 10 ** 6, what, which, half)
    assert cuda_lib.STATUS_NAMES[status] == "MK_ERR_TIMEOUT"
    assert cuda_lib.mk_linear_status(a["ws"]) == status
    assert bool((a["guard"] == 0x5A).all())
    assert all(torch.equal(x, y) for x, y in zip(a["keep"], a["kept"]))
    a["out"].fill_(CANARY)
    cuda_lib.mk_linear(a["io"], a["ws"])
    torch.cuda.synchronize()
    assert cuda_lib.mk_linear_status(a["ws"]) == 0
    assert torch.equal(a["out"], a["want"])


@pytest.fixture(scope="module")
def kvq_waiting(cuda_lib):
    """Requests of 32 rows per kv head: several items per CTA, whole ones, held twice in
    their tiles, and such as lie in two CTAs."""
    n = 700
    a = make_attn(np.random.default_rng(n), [130 + (37 * i) % 300 for i in range(n)], [8] * n, 4, 1, 64, "bf16", 16)
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)
    size = a["workspace"].numel()
    room = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    a.update(ws=room[:size], guard=room[size:], want=(a["out"].clone(), a["lse"].clone()),
             kept=[t.clone() for t in a["dev"] + [a["q"]]])
    return a


def test_attn_waits_that_do_not_run_out(cuda_lib, kvq_waiting):
    a = kvq_waiting
    a["whole"].fill_(CANARY)
    assert cuda_lib.mk_selftest_kvq_waits(a["io"], a["ws"], 2 * 10 ** 9) == 0
    assert torch.equal(a["out"][:a["n"]], a["want"][0][:a["n"]]) and torch.equal(a["lse"], a["want"][1])


@pytest.mark.parametrize("what,which", [(w, i) for w in (
    "scores", "weights", "keys", "values", "keys_used", "values_used") for i in (0, 1, 4)] + [
    ("row_tile", 0), ("row_tile", 1), ("row_tile", 2), ("half", 0), ("half", 1), ("taken", 0)])
def test_attn_gives_up_and_recovers(cuda_lib, kvq_waiting, what, which):
    """A hand-off that never comes: as for the projection."""
    a = kvq_waiting
    status = cuda_lib.mk_selftest_kvq_waits(a["io"], a["ws"], 2 * 10 ** 6, what, which)
    assert cuda_lib.STATUS_NAMES[status] == "MK_ERR_TIMEOUT"
    assert cuda_lib.mk_kvq_attn_status(a["ws"]) == status
    assert bool((a["guard"] == 0x5A).all()) and bool((a["whole"][a["n"]:] == CANARY).all())
    assert all(torch.equal(x, y) for x, y in zip(a["dev"] + [a["q"]], a["kept"]))
    a["whole"].fill_(CANARY)
    cuda_lib.mk_kvq_attn(a["io"], a["ws"])
    torch.cuda.synchronize()
    assert cuda_lib.mk_kvq_attn_status(a["ws"]) == 0
    assert torch.equal(a["out"][:a["n"]], a["want"][0][:a["n"]]) and torch.equal(a["lse"], a["want"][1])


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("n", [1, 9, 700])
def test_append_takes_q_out_between_the_rows_of_k_and_v(cuda_lib, bits, n):
    """q from elsewhere, q_out in a tensor that holds k and v too."""
    mk, rng, hq, hk, d, page = cuda_lib, np.random.default_rng(n + bits), 4, 2, 64, 16
    pages = n // page + 1
    q0, q = rounded(rng, (n, hq, d), "bf16")
    x0, x = rounded(rng, (n, hk + hq + hk, d), "bf16")
    k, q_out, v = x[:, :hk], x[:, hk:hk + hq], x[:, hk + hq:]
    slots = rng.permutation(pages * page)[:n]
    if bits == 16:
        caches = [torch.zeros(pages, page, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        kw = dict(k_cache=caches[0], v_cache=caches[1])
    else:
        caches = pool(rng, pages, hk, page, d) + pool(rng, pages, hk, page, d)
        kw = dict(kvq=mk.make_kvq_cache(*caches))
    pos = rng.integers(0, 9000, n)
    rope = mk.mk_rope_create(mk.make_rope_config(d))
    at = dev(slots, torch.int64)
    positions = dev(pos)
    mk.mk_qkv_append(rope, mk.make_qkv_append_io(q, q_out, k, v, positions, at, **kw))
    torch.cuda.synchronize()
    mk.mk_rope_destroy(rope)
    f, m = ob.rope_frequencies(d)
    yq, mag = ok.norm_rope(q0, None, 0, pos, d, "half", f, m)
    assert np.all(np.abs(np64(q_out) - yq) <= mag * 2.0 ** -20 + U["bf16"] * np.abs(yq) + TINY["bf16"])
    assert np.array_equal(np64(k), x0[:, :hk]) and np.array_equal(np64(v), x0[:, hk + hq:])
    yk, mag = ok.norm_rope(x0[:, :hk], None, 0, pos, d, "half", f, m)
    if bits == 16:
        got = np64(caches[0].view(-1, hk, d)[at])
        assert np.all(np.abs(got - yk) <= mag * 2.0 ** -20 + U["bf16"] * np.abs(yk) + TINY["bf16"])
        assert torch.equal(caches[1].view(-1, hk, d)[at], v)
    else:
        for y, i in ((yk, 0), (x0[:, hk + hq:], 2)):
            codes, scales = ok.encode(y)
            got = [p.transpose(1, 2).reshape(pages * page, hk, -1)[at].cpu().numpy() for p in caches[i:i + 2]]
            assert np.array_equal(got[0], codes) and np.array_equal(got[1], scales)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n", [5, 400, 4000])
def test_append_in_the_rows_of_the_cache(cuda_lib, layout, n):
    """k and v in the cache already, in the rows that they go to: rotated in place."""
    mk, rng, hk, d, page = cuda_lib, np.random.default_rng(n), 2, 64, 16
    pages = n // page + 2
    held = [rounded(rng, (pages, page, hk, d), "fp16") for _ in range(2)]
    first = 3
    rows = [c.view(-1, hk, d)[first:first + n] for _, c in held]
    pos = rng.integers(0, 9000, n)
    rope = mk.mk_rope_create(mk.make_rope_config(d, layout=layout))
    at, positions = dev(np.arange(first, first + n), torch.int64), dev(pos)
    mk.mk_qkv_append(rope, mk.make_qkv_append_io(None, None, rows[0], rows[1], positions, at, k_cache=held[0][1], v_cache=held[1][1]))
    torch.cuda.synchronize()
    mk.mk_rope_destroy(rope)
    f, m = ob.rope_frequencies(d)
    k0 = held[0][0].reshape(-1, hk, d)
    y, mag = ok.norm_rope(k0[first:first + n], None, 0, pos, d, layout, f, m)
    got = np64(held[0][1].view(-1, hk, d))
    assert np.all(np.abs(got[first:first + n] - y) <= mag * 2.0 ** -20 + U["fp16"] * np.abs(y) + TINY["fp16"])
    assert np.array_equal(got[:first], k0[:first]) and np.array_equal(got[first + n:], k0[first + n:])
    assert np.array_equal(np64(held[1][1]), held[1][0])


def test_one_row_of_tensors_with_odd_rows(cuda_lib):
    """x, w and the residual, q, k and v as single rows of tensors whose stride no call
    would take, and a residual that is the output under another stride."""
    mk, rng = cuda_lib, np.random.default_rng(41)
    x0, x = (a[2:3, :256] for a in rounded(rng, (3, 260), "bf16"))     # 16-byte aligned, as 2 * 260 is a multiple of 8
    w0, w = (a[2:3, :256] for a in rounded(rng, (3, 260), "bf16", 1 / 16))
    r0, r = rounded(rng, (1, 1), "bf16")
    out = torch.empty(1, 7, dtype=torch.bfloat16, device="cuda")[:, :1]
    out.copy_(r)
    io = mk.make_linear_io(x, w, out, residual=out.as_strided((1, 1), (24, 1)))
    ws = torch.empty(mk.mk_linear_workspace(io), dtype=torch.uint8, device="cuda")
    mk.mk_linear(io, ws)
    want, s = ok.linear(x0, w0, None, "none", r0)
    assert abs(np64(out) - want) <= s * (16 + 64) * 2 * V + U["bf16"] * abs(want)

    t0, t = rounded(rng, (2, 260), "bf16")
    q, k, v = (t[:1, a:b].unflatten(1, (-1, 64)) for a, b in ((0, 128), (128, 192), (192, 256)))
    pools = pool(rng, 1, 1, 16, 64) + pool(rng, 1, 1, 16, 64)
    slots = dev([5], torch.int64)
    mk.mk_qkv_append(None, mk.make_qkv_append_io(q, q, k, v, None, slots, kvq=mk.make_kvq_cache(*pools)))
    for i, a in ((0, 128), (2, 192)):
        codes, scales = ok.encode(t0[0, a:a + 64])
        assert np.array_equal(pools[i][0, 0, 5].cpu().numpy(), codes) and np.array_equal(pools[i + 1][0, 0, 5].cpu().numpy(), scales)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_attn_scales_up_to_the_largest(cuda_lib, new, dtype):
    """The largest scale that is taken, with rows of zeros, whose scores are 0; and with
    rows so small that their scores are ordinary ones."""
    for scale, by in ((1.7e38, 0.0), (2.0 ** 126, 2.0 ** -126 if dtype == "bf16" else 0.0), (2.0 ** 100, 2.0 ** -100 if dtype == "bf16" else 0.0)):
        a = make_attn(np.random.default_rng(new), [50, 200], [new, new], 4, 1, 64, dtype, 16, q_scale=by)
        call_attn(cuda_lib, a, scale=scale)
        check_attn(cuda_lib, a, scale=scale)


@pytest.mark.parametrize("news", [[3, 5, 2], [24, 40, 30]])
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("fp16", 128)])
def test_attn_empty_tree_words_under_a_window(cuda_lib, news, dtype, d):
    """A row with an empty word (a padded one) is at base - 1: its window begins a key
    earlier than all others', which here is the last of a key tile."""
    # (made without window and words, which would hide the key that the empty word's row sees)
    a = make_attn(np.random.default_rng(d), [base + n for base, n in zip((95, 191, 319), news)], news, 4, 1, d, dtype, 16)
    a["window"] = 64
    a["words"] = [0 if i == n // 2 else (1 << n) - 1 for n in news for i in range(n)] + [0] * 2
    hide_unseen(a)
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)


@pytest.mark.parametrize("news", [[3, 1, 2], [24, 64, 30], [2, 16, 9]])
@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("fp16", 128)])
def test_attn_tree_keys_that_no_row_sees(cuda_lib, news, window, dtype, d):
    """Words that leave their own row out, some of them empty (padded rows): what no row
    sees between the tree's keys has NaN scales like any other such key."""
    rng = np.random.default_rng(sum(news) + d)
    a = make_attn(rng, [base + n for base, n in zip((95, 141, 0), news)], news, 4, 1, d, dtype, 16)
    a["window"] = window
    words = []
    for n in news:
        kept = int(rng.integers(0, 1 << 62)) & ((1 << n) - 1)
        words += [kept & int(rng.integers(0, 1 << 62)) if i % 3 else 0 for i in range(n)]
    a["words"] = words + [0] * 2
    hide_unseen(a)
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)


@pytest.mark.parametrize("new", [1, 20])
def test_attn_pages_of_65536_keys(cuda_lib, new):
    """The largest page: requests that end inside it, and one that goes on into another."""
    a = make_attn(np.random.default_rng(new), [66000, 300, 65536], [new, 2, 1], 4, 1, 64, "bf16", 65536)
    call_attn(cuda_lib, a)
    check_attn(cuda_lib, a)


@pytest.mark.parametrize("bits", [4, 16])
def test_append_to_pages_of_65536_keys(cuda_lib, bits):
    rng = np.random.default_rng(42)
    check_append(cuda_lib, rng, 60, 4, 2, 64, 64, "half", "bf16", rng.integers(0, 1 << 20, 60), bits, page=65536)


def test_attention_takes_the_largest_page(cuda_lib):
    """Four kv heads of 128 in one page of 65536 keys: 16 MB of codes."""
    rng = np.random.default_rng(43)
    pools = pool(rng, 1, 4, 65536, 128) + pool(rng, 1, 4, 65536, 128)
    kvq = cuda_lib.make_kvq_cache(*pools)
    q0, q = rounded(rng, (2, 8, 128), "bf16")
    out, lse = torch.empty_like(q), torch.empty(2, 8, device="cuda")
    lens, cu, table = dev([700, 65536]), dev([0, 1, 2]), dev([[0], [0]])
    for s in pools[1::2]:
        s.copy_(torch.from_numpy(rng.integers(16, 32, s.shape, dtype=np.uint8)))
    io = cuda_lib.make_kvq_attn_io(q, kvq, out, lens, cu, table, lse=lse)
    ws = torch.empty(cuda_lib.mk_kvq_attn_workspace(io), dtype=torch.uint8, device="cuda")
    cuda_lib.mk_kvq_attn(io, ws)
    k, v = (ok.decode_pool(pools[i].cpu().numpy(), pools[i + 1].cpu().numpy(), np.zeros(4, int)) for i in (0, 2))
    want, want_lse, weight = ob.prefix_attn(q0, k, v, [], 0, np.zeros((2, 1), int), np.array([700, 65536]), np.array([0, 1, 2]))
    size = lambda x: float(np.sqrt((x * x).sum(-1).max()))  # noqa: E731
    e_s = 3 * 128 ** 0.5 * V * size(q0) * size(k) + 2.0 ** -19
    tol = weight * (2.0 ** -11 + 2 * e_s + (65536 / 16 + 64) * 2 * V) + 65536 * 2.0 ** -25 * np.abs(v).max() + U["bf16"] * np.abs(want) + TINY["bf16"]
    assert np.all(np.abs(np64(out) - want) <= tol)
    assert np.all(np.abs(np64(lse) - want_lse) <= e_s + (65536 + 64) * V + 4 * V * np.abs(want_lse))
