"""The attention half of a batched decoder layer over a paged KV cache in 4 bits, as a serving program calls its
operators: the projections with bias, activation and residual; the norms of q and k per head with the rotation and
the cache write; attention over the cache.  Each in plain torch operations and, where `own` is set, through the
library.

The cache: per token and KV head, codes of 4 bits in groups of 16 values along the head, with an E4M3 scale s per
group and a power of two 2^e per head: code n stands for (n - 8) s 2^e."""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # a decode batch: one token per request, normed heads, into 4 bits
        dict(name="append-decode", op="append", rows=64, q_heads=32, kv_heads=8, dim=128, rot=128, layout="half", scaling="none", norm=True, bits=4, dtype="bf16", positions=16384, page=64),
        # the verify tokens of a few requests, normed heads, a cache in 16 bits
        dict(name="append-verify16", op="append", rows=125, q_heads=32, kv_heads=8, dim=128, rot=128, layout="half", scaling="none", norm=True, bits=16, dtype="bf16", positions=32768, page=16),
        # prompt chunks of an odd length, interleaved pairs in half of the head, no norms, far positions
        dict(name="append-chunk", op="append", rows=777, q_heads=12, kv_heads=2, dim=64, rot=32, layout="interleaved", scaling="linear", norm=False, bits=4, dtype="fp16", positions=1 << 20, page=32),
        # a long prompt, positions scaled by parts, into 4 bits
        dict(name="append-prompt", op="append", rows=8192, q_heads=32, kv_heads=8, dim=128, rot=128, layout="half", scaling="parts", norm=True, bits=4, dtype="bf16", positions=131072, page=64),
        # two short requests on the tiny layer's heads: latency
        dict(name="kvq-tiny", op="attn", requests=2, new=1, ragged=False, tree=False, own_lo=100, own_hi=500, window=0, q_heads=4, kv_heads=1, dim=64, dtype="bf16", page=16),
        # plain decoding, one token per request, lengths all over the range
        dict(name="kvq-decode", op="attn", requests=64, new=1, ragged=False, tree=False, own_lo=32, own_hi=8192, window=0, q_heads=32, kv_heads=8, dim=128, dtype="bf16", page=64),
        # ragged token trees of 16 requests over the stack's context
        dict(name="kvq-tree", op="attn", requests=16, new=16, ragged=True, tree=True, own_lo=16, own_hi=16384, window=0, q_heads=32, kv_heads=8, dim=128, dtype="fp16", page=32),
        # few requests with very long contexts
        dict(name="kvq-long", op="attn", requests=3, new=2, ragged=True, tree=False, own_lo=60000, own_hi=131072, window=0, q_heads=32, kv_heads=8, dim=128, dtype="bf16", page=128),
        # the tiny layer's projection of one verify step: latency
        dict(name="linear-tiny", op="linear", rows=2, n_in=256, n_out=384, bias=True, act="none", residual=False, dtype="bf16"),
        # the projection to q, k and v of a decode batch
        dict(name="linear-qkv", op="linear", rows=64, n_in=4096, n_out=6144, bias=True, act="none", residual=False, dtype="bf16"),
        # the output projection of a batch of verify steps, onto the residual stream
        dict(name="linear-out", op="linear", rows=250, n_in=4096, n_out=4096, bias=False, act="none", residual=True, dtype="fp16"),
        # the draft layers' widening projection of a prompt, with its activation
        dict(name="linear-prompt", op="linear", rows=4096, n_in=4096, n_out=12288, bias=True, act="silu", residual=False, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    limits = {}
    for c in listed():
        w = work(c)
        b, f = limits.get(c["op"], (0, 0))
        limits[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    op = rng.choice(["append", "attn", "attn", "linear"])
    while True:
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        d = rng.choice([64, 128, 128])
        kv = rng.choice([1, 2, 4, 8])
        if op == "append":
            c = dict(op=op, rows=_log(rng, 1, 8192), q_heads=rng.choice([1, 2, 4, 6, 8]) * kv, kv_heads=kv, dim=d, rot=rng.choice([d // 4, d // 2, d, d]),
                     layout=rng.choice(["half", "half", "interleaved"]), scaling=rng.choice(["none", "linear", "base", "parts"]), norm=rng.random() < 0.7,
                     bits=rng.choice([4, 4, 16]), dtype=dtype, positions=_log(rng, 128, 1 << 20), page=rng.choice([16, 32, 64, 128]))
        elif op == "attn":
            new = _log(rng, 1, 16)
            hi = max(new, _log(rng, 16, 131072))
            c = dict(op=op, requests=_log(rng, 1, 128), new=new, ragged=rng.random() < 0.5, tree=rng.random() < 0.25, own_lo=_log(rng, 1, hi),
                     own_hi=hi, window=rng.choice([0, 0, 0, 128, 2048]), q_heads=rng.choice([1, 2, 4, 4, 6, 8]) * kv, kv_heads=kv,
                     dim=d, dtype=dtype, page=rng.choice([16, 32, 64, 128]))
            if c["requests"] * c["own_hi"] * kv > 1 << 22:
                continue
        else:
            c = dict(op=op, rows=_log(rng, 1, 8192), n_in=8 * _log(rng, 8, 1536), n_out=_log(rng, 64, 12288), bias=rng.random() < 0.5,
                     act=rng.choice(["none", "none", "silu", "gelu"]), residual=rng.random() < 0.5, dtype=dtype)
        w = work(c)
        if w["bytes"] <= limits[op][0] and w["flops"] <= limits[op][1]:
            return c


def _spread(n, lo, hi, step):
    """n whole numbers that cover [lo, hi] evenly, in a fixed order."""
    return [lo + int((hi - lo + 1) * ((0.5 + i * step) % 1.0)) for i in range(n)]


def _attn_lengths(c):
    """Per request: its keys (the new tokens' among them) and its new tokens."""
    new = _spread(c["requests"], 1, c["new"], 0.7548776662466927) if c["ragged"] else [c["new"]] * c["requests"]
    return [max(a, n) for a, n in zip(_spread(c["requests"], c["own_lo"], c["own_hi"], 0.6180339887498949), new)], new


def _append_pages(c):
    return -(-c["rows"] // c["page"]) + 1


def work(case):
    c = case
    if c["op"] == "append":
        head, kv = c["dim"] * 2, c["kv_heads"] * c["dim"]
        slots = _append_pages(c) * c["page"]
        read = c["rows"] * ((c["q_heads"] + 2 * c["kv_heads"]) * head + 12)
        # what the cache holds is returned: of 4 bits, the values that they stand for
        written = c["rows"] * (c["q_heads"] * head + (kv * 4 if c["bits"] == 16 else kv * 9 // 8)) + (slots * kv * 4 if c["bits"] == 4 else 0)
        return {"bytes": read + written, "flops": c["rows"] * (c["q_heads"] + c["kv_heads"]) * c["dim"] * 8}
    if c["op"] == "attn":
        lens, new = _attn_lengths(c)
        keys, seen = 0, 0  # a token tree is counted as the chain: its masks, and so the few keys less, come with the inputs
        for length, n in zip(lens, new):
            for i in range(n):
                seen += min(length - n + i + 1, c["window"] or 1 << 40)
            keys += min(length, c["window"] + n if c["window"] else length)
        return {"bytes": keys * c["kv_heads"] * c["dim"] * 9 // 8 + sum(new) * c["q_heads"] * (c["dim"] * 4 + 4), "flops": 4 * seen * c["q_heads"] * c["dim"]}
    m, n, k = c["rows"], c["n_out"], c["n_in"]
    return {"bytes": 2 * (m * k + n * k + m * n * (2 if c["residual"] else 1) + (n if c["bias"] else 0)), "flops": 2 * m * n * k}


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype).to("cuda")


def _exponents(s, heads):
    """The heads' powers of two, and these as numbers."""
    for name, e in (("k", [i % 3 - 1 for i in range(heads)]), ("v", [-(i % 2) for i in range(heads)])):
        s[name + "_exp"], s[name + "_unit"] = _ints(e), _ints([2.0 ** i for i in e], torch.float64)


def _pool(z):
    """(codes, scales) of a pool of values [pages, heads, page, d], in 4 bits."""
    g = z.view(*z.shape[:-1], -1, 16)
    s = (g.abs().amax(-1, keepdim=True) / 7).clamp(max=448).to(torch.float8_e4m3fn)
    f = s.to(torch.float32)
    n = torch.where(f > 0, torch.round(g / f).clamp(-8, 7), 0).add_(8).to(torch.uint8).view(*z.shape[:-1], -1, 2)
    return (n[..., 0] | n[..., 1] << 4).contiguous(), s.view(torch.uint8)[..., 0].contiguous()


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed * 7919 + 13)
    h = torch.Generator().manual_seed(seed * 7919 + 17)
    c, s = case, {"case": dict(case)}
    t = DTYPES[c["dtype"]]

    def rand(*shape, by=1.0, dtype=t):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * by).to(dtype)

    if c["op"] == "append":
        n, hq, hk, d, p = c["rows"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
        qkv = rand(n, hq + 2 * hk, d)  # the projection's output: q, k and v are views of it
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["q_out"] = torch.empty(n, hq, d, device="cuda", dtype=t)
        s["q_norm"], s["k_norm"] = ((1 + 0.2 * rand(2, d, dtype=torch.float32)).to(t) if c["norm"] else (None, None))
        s["positions"] = torch.randint(0, c["positions"], (n,), generator=g, device="cuda", dtype=torch.int32)
        pages = _append_pages(c)
        s["slots"] = torch.randperm(pages * p, generator=g, device="cuda", dtype=torch.int64)[:n].contiguous()
        s["slots"][n - 1 - seed % 2:n - 1] = -1  # a row without a place
        if c["bits"] == 16:
            s["k_cache"], s["v_cache"] = rand(pages, p, hk, d), rand(pages, p, hk, d)
        else:
            _exponents(s, hk)
            s["kc"], s["ks"] = _pool(rand(pages, hk, p, d, dtype=torch.float32))
            s["vc"], s["vs"] = _pool(rand(pages, hk, p, d, dtype=torch.float32))
            s["k_values"], s["v_values"] = (torch.empty(pages * p, hk, d, device="cuda", dtype=t) for _ in range(2))
        s["rope"] = dict(theta=10000.0, scaling=c["scaling"], factor=1.0 if c["scaling"] == "none" else 8.0, orig_ctx=8192)
        if own:  # the frequencies that a program sets up once
            from moe_decode_layer_persistent_gb300 import binding as mk
            s["handle"] = mk.mk_rope_create(mk.make_rope_config(d, c["rot"], layout=c["layout"], **s["rope"]))
    elif c["op"] == "attn":
        b, hq, hk, d, p = c["requests"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
        lens, new = _attn_lengths(c)
        order = torch.randperm(b, generator=h).tolist()
        lens, new = [lens[i] for i in order], [new[i] for i in order]
        n = sum(new)
        held = [-(-a // p) for a in lens]
        pages = sum(held) + 2
        perm = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int64)
        count, col = _ints(held, torch.int64), torch.arange(max(held), device="cuda")
        at = (torch.cumsum(count, 0) - count)[:, None] + col
        s["table"] = torch.where(col < count[:, None], perm[at.clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
        _exponents(s, hk)
        s["kc"], s["ks"] = _pool(rand(pages, hk, p, d, dtype=torch.float32))
        s["vc"], s["vs"] = _pool(rand(pages, hk, p, d, dtype=torch.float32))
        s["q"] = rand(n, hq, d)
        s["lens"], s["cu"], s["new"] = _ints(lens), _ints([0] + torch.tensor(new).cumsum(0).tolist()), c["new"]
        s["mask"] = None
        if c["tree"]:  # each token hangs on one before it, or on the request's last cached token
            masks = []
            for m in new:
                up = torch.randint(-1, 1 << 20, (m,), generator=h).tolist()
                mine = []
                for i in range(m):
                    mine.append((1 << i) | (mine[up[i] % i] if i and up[i] >= 0 else 0))
                masks += mine
            s["mask"] = _ints(masks, torch.int64)
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(n, hq, device="cuda", dtype=torch.float32)
        if own:  # the workspace that a program keeps
            from moe_decode_layer_persistent_gb300 import binding as mk
            s["workspace"] = torch.empty(mk.mk_kvq_attn_workspace(_attn_io(mk, s)), device="cuda", dtype=torch.uint8)
    else:
        m, n, k = c["rows"], c["n_out"], c["n_in"]
        s["x"], s["w"] = rand(m, k), rand(n, k, by=k ** -0.5)
        s["bias"] = rand(n, by=0.3) if c["bias"] else None
        s["residual"] = rand(m, n) if c["residual"] else None
        s["out"] = torch.empty(m, n, device="cuda", dtype=t)
        if own:
            from moe_decode_layer_persistent_gb300 import binding as mk
            s["workspace"] = torch.empty(mk.mk_linear_workspace(_linear_io(mk, s)), device="cuda", dtype=torch.uint8)
    return s


def _kvq(mk, s):
    return mk.make_kvq_cache(s["kc"], s["ks"], s["vc"], s["vs"], s["k_exp"], s["v_exp"])


def _attn_io(mk, s):
    return mk.make_kvq_attn_io(s["q"], _kvq(mk, s), s["out"], s["lens"], s["cu"], s["table"], window=s["case"]["window"], tree_mask=s["mask"], lse=s["lse"])


def _linear_io(mk, s):
    return mk.make_linear_io(s["x"], s["w"], s["out"], bias=s["bias"], act=s["case"]["act"], residual=s["residual"])


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        from moe_decode_layer_persistent_gb300 import binding as mk
        stream = torch.cuda.current_stream()
        if op == "append":
            if s["case"]["bits"] == 16:
                io = mk.make_qkv_append_io(s["q"], s["q_out"], s["k"], s["v"], s["positions"], s["slots"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                                           k_cache=s["k_cache"], v_cache=s["v_cache"])
                mk.mk_qkv_append(s["handle"], io, stream)
                return {"q_out": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}
            kvq = _kvq(mk, s)
            io = mk.make_qkv_append_io(s["q"], s["q_out"], s["k"], s["v"], s["positions"], s["slots"], q_norm=s["q_norm"], k_norm=s["k_norm"], kvq=kvq)
            mk.mk_qkv_append(s["handle"], io, stream)
            mk.mk_kvq_read(mk.make_kvq_read_io(kvq, None, s["k_values"], s["v_values"]), stream)
            return {"q_out": s["q_out"], "k": s["k_values"], "v": s["v_values"]}
        if op == "attn":
            mk.mk_kvq_attn(_attn_io(mk, s), s["workspace"], stream)
            return {"out": s["out"], "lse": s["lse"]}
        mk.mk_linear(_linear_io(mk, s), s["workspace"], stream)
        return s["out"]
    return {"append": _plain_append, "attn": _plain_attn, "linear": _plain_linear}[op](s)


def _frequencies(rot, rope):
    """Radians per position of each pair, in 64 bits, and the factor on the rotated values."""
    f = torch.pow(torch.tensor(rope["theta"], dtype=torch.float64), -torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    k = rope["factor"]
    if rope["scaling"] == "linear":
        return f / k, 1.0
    if rope["scaling"] == "base":
        theta = rope["theta"] * k ** (rot / (rot - 2))
        return torch.pow(torch.tensor(theta, dtype=torch.float64), -torch.arange(0, rot, 2, dtype=torch.float64) / rot), 1.0
    if rope["scaling"] == "parts":
        keep = ((rope["orig_ctx"] * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return f * (keep + (1 - keep) / k), 0.1 * math.log(k) + 1.0
    return f, 1.0


def _e4m3(x):
    """x >= 0 rounded to the nearest E4M3 value, ties to even, at most 448."""
    y = x.clamp(min=2.0 ** -6)
    step = y / torch.frexp(y).mantissa * 0.0625  # (a power of two, exactly; exp2 need not be exact)
    return (torch.round(x / step) * step).clamp(max=448.0)


def _values(codes, scales, unit):
    """The values [..., heads, page, d] that a pool's codes stand for, in 32 bits."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).view(*scales.shape, 16).float() - 8
    return (n * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2) * unit.float()[:, None, None]


def _plain_append(s):
    c = s["case"]
    rot, hk, d, p = c["rot"], c["kv_heads"], c["dim"], c["page"]
    f, m = _frequencies(rot, s["rope"])
    angle = s["positions"].double()[:, None] * f.to(s["q"].device)
    cos, sin = (torch.cos(angle) * m)[:, None], (torch.sin(angle) * m)[:, None]

    def turned(x, w, t):
        y, co, si = x.to(t), cos.to(t), sin.to(t)
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.to(t)
        if c["layout"] == "half":
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            parts = torch.cat([a * co - b * si, b * co + a * si], -1)
        else:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            parts = torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2)
        return torch.cat([parts, y[..., rot:]], -1)

    q_out = turned(s["q"], s["q_norm"], torch.float32).to(s["q"].dtype)
    put = s["slots"] >= 0
    at = s["slots"][put]
    if c["bits"] == 16:
        s["k_cache"].view(-1, hk, d)[at] = turned(s["k"], s["k_norm"], torch.float32).to(s["k"].dtype)[put]
        s["v_cache"].view(-1, hk, d)[at] = s["v"][put]
        return {"q_out": q_out, "k": s["k_cache"], "v": s["v_cache"]}
    # the codes, in 64 bits: values lie next to their borders
    seven = torch.full((1,), 7.0, dtype=torch.float64, device=at.device)  # (a division by a number is a product with its reciprocal)
    for x, codes, scales, unit in ((turned(s["k"], s["k_norm"], torch.float64), s["kc"], s["ks"], s["k_unit"]), (s["v"].double(), s["vc"], s["vs"], s["v_unit"])):
        z = (x[put] / unit[:, None]).view(-1, hk, d // 16, 16)
        scale = _e4m3(z.abs().amax(-1, keepdim=True) / seven)
        n = torch.where(scale > 0, torch.round(z / scale).clamp(-8, 7), 0).add(8).to(torch.uint8).view(-1, hk, d // 2, 2)
        page, row = at // p, at % p
        codes[page, :, row] = n[..., 0] | n[..., 1] << 4
        scales[page, :, row] = scale[..., 0].to(torch.float8_e4m3fn).view(torch.uint8)
    k, v = (_values(*z).transpose(1, 2).reshape(-1, hk, d).to(s["q"].dtype) for z in ((s["kc"], s["ks"], s["k_unit"]), (s["vc"], s["vs"], s["v_unit"])))
    return {"q_out": q_out, "k": k, "v": v}


def _plain_attn(s):
    c = s["case"]
    hk, d, t, b = c["kv_heads"], c["dim"], s["new"], c["requests"]
    g, n = c["q_heads"] // hk, s["q"].shape[0]
    dev = s["q"].device
    lens, cu = s["lens"].long(), s["cu"].long()
    new = cu[1:] - cu[:-1]
    r = torch.arange(n, device=dev)
    req = torch.searchsorted(cu[1:], r, right=True)
    i = r - cu[req]
    base = lens[req] - new[req]
    bits = None if s["mask"] is None else s["mask"][:, None] >> torch.arange(t, device=dev) & 1
    pos = base + (i if bits is None else bits.sum(1) - 1)
    low = pos - c["window"] + 1 if c["window"] else torch.zeros_like(pos)
    pages = s["table"].long().clamp(min=0)
    k, v = (_values(x[pages], y[pages], e).transpose(1, 2).flatten(2, 3) for x, y, e in ((s["kc"], s["ks"], s["k_unit"]), (s["vc"], s["vs"], s["v_unit"])))
    width = k.shape[2]
    qb = torch.zeros(b, t, hk, g, d, device=dev)
    qb[req, i] = s["q"].float().view(n, hk, g, d) / math.sqrt(d)
    score = torch.matmul(qb.permute(0, 2, 1, 3, 4).reshape(b, hk, t * g, d), k.transpose(2, 3)).view(b, hk, t, g, width).permute(0, 2, 1, 3, 4)[req, i]
    key = torch.arange(width, device=dev)
    fresh = key - base[:, None]
    if bits is None:
        see = fresh <= i[:, None]
    else:
        see = (fresh < 0) | ((fresh < new[req][:, None]) & (bits.gather(1, fresh.clamp(0, t - 1)) > 0))
    see &= key >= low[:, None]
    score = score.masked_fill(~see[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - top)
    total = weight.sum(-1)
    wb = torch.zeros(b, t, hk, g, width, device=dev)
    wb[req, i] = weight
    out = torch.matmul(wb.permute(0, 2, 1, 3, 4).reshape(b, hk, t * g, width), v).view(b, hk, t, g, d).permute(0, 2, 1, 3, 4)[req, i]
    return {"out": (out / total[..., None]).reshape(n, hk * g, d).to(s["q"].dtype), "lse": (top[..., 0] + torch.log(total)).reshape(n, hk * g)}


def _activated(y, act):
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y / math.sqrt(2.0)))
    return y


def _plain_linear(s):
    y = torch.matmul(s["x"].float(), s["w"].float().t())
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _activated(y, s["case"]["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


def _e4m3_values():
    """The finite E4M3 values that are not negative, by their codes."""
    return torch.tensor([m / 512 if e == 0 else (8 + m) / 8 * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127], dtype=torch.float64, device="cuda")


def _decoded(codes, scales, exp):
    """Float64 values [..., d] of codes [..., d / 2] of one head."""
    table = _e4m3_values()
    c = codes.long()
    v = torch.empty(*c.shape[:-1], 2 * c.shape[-1], dtype=torch.float64, device="cuda")
    v[..., 0::2], v[..., 1::2] = c % 16 - 8, torch.div(c, 16, rounding_mode="floor") - 8
    return v * torch.repeat_interleave(table[scales.long()], 16, -1) * 2.0 ** exp


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "linear":
        y = s["x"].double() @ s["w"].double().transpose(0, 1)
        if c["bias"]:
            y += s["bias"].double()
        if c["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif c["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        return y + s["residual"].double() if c["residual"] else y
    hk, d, p = c["kv_heads"], c["dim"], c["page"]
    if c["op"] == "append":
        rot, rope = c["rot"], s["rope"]
        i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
        theta, k, m = rope["theta"], rope["factor"], 1.0
        if rope["scaling"] == "base":
            theta *= k ** (rot / (rot - 2.0))
        f = torch.exp(-2.0 * i / rot * math.log(theta))
        if rope["scaling"] == "linear":
            f = f / k
        elif rope["scaling"] == "parts":
            ramp = torch.clamp((rope["orig_ctx"] / (2 * math.pi / f) - 1.0) / 31.0, 0.0, 1.0)
            f, m = (1 - ramp) * f / k + ramp * f, 1.0 + 0.1 * math.log(k)
        z = torch.polar(torch.full_like(f, m).expand(c["rows"], -1).contiguous(), s["positions"].double()[:, None] * f)[:, None]

        def turn(x, w):
            y = x.double().clone()
            if w is not None:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + 1e-6) * w.double()
            one, two = (slice(0, rot // 2), slice(rot // 2, rot)) if c["layout"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
            u = torch.complex(y[..., one].contiguous(), y[..., two].contiguous()) * z
            y[..., one], y[..., two] = u.real, u.imag
            return y

        has = torch.nonzero(s["slots"] >= 0)[:, 0]
        at = s["slots"][has]
        found = {"q_out": turn(s["q"], s["q_norm"])}
        seven = torch.full((1, 1), 7.0, dtype=torch.float64, device="cuda")
        scales = _e4m3_values()
        for name, x in (("k", turn(s["k"], s["k_norm"])), ("v", s["v"].double())):
            if c["bits"] == 16:
                cache = s[name + "_cache"].double().flatten(0, 1)
                cache.index_copy_(0, at, x[has])
                found[name] = cache.view(s[name + "_cache"].shape)
                continue
            cache = torch.stack([_decoded(s[name + "c"][:, j], s[name + "s"][:, j], int(s[name + "_exp"][j])) for j in range(hk)], 2).flatten(0, 1)
            for j in range(hk):
                unit = 2.0 ** int(s[name + "_exp"][j])
                y = x[has, j].reshape(-1, 16) / unit
                big = y.abs().max(1, keepdim=True).values
                low = torch.searchsorted(scales, big / seven, right=True).clamp(1, len(scales) - 1) - 1  # the E4M3 scales around a seventh of it
                below, above = 7 * (big - 7 * scales[low]), 7 * (7 * scales[low + 1] - big)
                sc = torch.where((below < above) | ((below == above) & (low % 2 == 0)), scales[low], scales[low + 1])
                whole = torch.round(y / torch.where(sc > 0, sc, torch.ones_like(sc))).clamp(-8, 7) * sc
                cache[:, j].index_copy_(0, at, whole.view(-1, d) * unit)
            found[name] = cache
        return found
    g = c["q_heads"] // hk
    n = s["q"].shape[0]
    out = torch.empty(n, c["q_heads"], d, dtype=torch.float64, device="cuda")
    lse = torch.empty(n, c["q_heads"], dtype=torch.float64, device="cuda")
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    for b in range(c["requests"]):
        first, m, length = cu[b], cu[b + 1] - cu[b], lens[b]
        ids = s["table"][b, :-(-length // p)].long()
        see = torch.ones(m, length, dtype=torch.bool, device="cuda")
        for i in range(m):
            word = (2 << i) - 1 if s["mask"] is None else int(s["mask"][first + i])
            see[i, length - m:] = torch.tensor([word >> j & 1 for j in range(m)], dtype=torch.bool)
            if c["window"]:
                see[i, :max(0, min(length - m + bin(word).count("1") - c["window"], length - m))] = False
        for j in range(hk):
            keys, values = (_decoded(s[a + "c"][ids, j], s[a + "s"][ids, j], int(s[a + "_exp"][j])).flatten(0, 1)[:length] for a in "kv")
            q = s["q"][first:first + m, j * g:(j + 1) * g].double().reshape(m * g, d)
            score = (q @ keys.transpose(0, 1) / d ** 0.5).view(m, g, length)
            score = torch.where(see[:, None], score, torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
            part = torch.logsumexp(score, -1)
            out[first:first + m, j * g:(j + 1) * g] = (torch.exp(score - part[..., None]).view(m * g, length) @ values).view(m, g, d)
            lse[first:first + m, j * g:(j + 1) * g] = part
    return {"out": out, "lse": lse}
