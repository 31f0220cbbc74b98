"""The operators of a batched decoding step over a paged KV cache whose requests share a prefix, as a serving
program calls them: block tables and slot maps from the request lengths, rotary positions with the K/V write,
and attention with the shared prefix computed once for all.  Each in plain torch operations and, where `own` is
set, through the library."""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # a batch of verify steps: 16 requests, up to 16 new tokens each
        dict(name="slots-verify", op="slots", requests=16, new_lo=1, new_hi=16, cached_hi=1024, page=16, prefix=16384, free=1.0),
        # continuous decoding: one token per request, some requests idle, pages a little short
        dict(name="slots-decode", op="slots", requests=777, new_lo=0, new_hi=1, cached_hi=8192, page=16, prefix=0, free=0.9),
        # a large batch with prompts of odd lengths admitted in one step
        dict(name="slots-prompts", op="slots", requests=4096, new_lo=0, new_hi=96, cached_hi=4096, page=64, prefix=2048, free=1.0),
        # the 16 verify tokens of one request, on the heads of the decode layer
        dict(name="rope-verify", op="rope", rows=16, q_heads=32, kv_heads=8, dim=128, rot=128, layout="half", scaling="none", dtype="bf16", positions=16384, page=16),
        # a decode batch of odd size, interleaved pairs in a quarter of the head, positions far beyond the trained length
        dict(name="rope-decode", op="rope", rows=333, q_heads=12, kv_heads=2, dim=64, rot=16, layout="interleaved", scaling="linear", dtype="fp16", positions=1 << 20, page=32),
        # prompt chunks of a mid-sized batch, half of the head rotated
        dict(name="rope-chunk", op="rope", rows=2048, q_heads=32, kv_heads=8, dim=128, rot=64, layout="interleaved", scaling="base", dtype="bf16", positions=32768, page=64),
        # a long prompt, positions scaled by parts
        dict(name="rope-prompt", op="rope", rows=16384, q_heads=32, kv_heads=8, dim=128, rot=128, layout="half", scaling="parts", dtype="bf16", positions=131072, page=64),
        # two short requests on the tiny layer's heads: latency
        dict(name="attn-tiny", op="attn", requests=2, new=1, ragged=False, tree=False, prefix=500, own_lo=1, own_hi=40, window=0, q_heads=4, kv_heads=1, dim=64, dtype="bf16", page=16),
        # plain decoding, one token per request
        dict(name="attn-decode", op="attn", requests=64, new=1, ragged=False, tree=False, prefix=4096, own_lo=32, own_hi=1000, window=0, q_heads=32, kv_heads=8, dim=128, dtype="bf16", page=16),
        # ragged verify steps of 16 requests over the stack's context
        dict(name="attn-verify", op="attn", requests=16, new=16, ragged=True, tree=False, prefix=16384, own_lo=16, own_hi=1024, window=0, q_heads=32, kv_heads=8, dim=128, dtype="bf16", page=64),
        # token trees under the layer's sliding window
        dict(name="attn-tree-window", op="attn", requests=24, new=16, ragged=True, tree=True, prefix=8191, own_lo=16, own_hi=1500, window=2048, q_heads=32, kv_heads=8, dim=128, dtype="fp16", page=32),
        # the largest: 64 requests with 8 draft tokens over a prefix of 32k tokens
        dict(name="attn-long", op="attn", requests=64, new=8, ragged=False, tree=False, prefix=32768, own_lo=100, own_hi=2000, window=0, q_heads=32, kv_heads=8, dim=128, dtype="bf16", page=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    limits = {}
    for c in listed():
        w = work(c)
        b, f = limits.get(c["op"], (0, 0))
        limits[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    op = rng.choice(["slots", "rope", "attn", "attn"])
    while True:
        if op == "slots":
            lo = rng.choice([0, 0, 1])
            c = dict(op=op, requests=_log(rng, 1, 4096), new_lo=lo, new_hi=max(1, _log(rng, 1, 96)), cached_hi=_log(rng, 16, 8192),
                     page=rng.choice([16, 32, 64, 128]), prefix=_log(rng, 1, 32768), free=rng.choice([1.0, 1.0, 0.8]))
        elif op == "rope":
            d = rng.choice([64, 128])
            g, kv = rng.choice([1, 2, 4, 6, 8]), rng.choice([1, 2, 4, 8])
            c = dict(op=op, rows=_log(rng, 1, 16384), q_heads=g * kv, kv_heads=kv, dim=d, rot=rng.choice([d // 4, d // 2, d]),
                     layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "base", "parts"]),
                     dtype=rng.choice(["bf16", "fp16"]), positions=_log(rng, 128, 1 << 20), page=rng.choice([16, 32, 64, 128]))
        else:
            g, kv = rng.choice([1, 2, 4, 4, 6, 8]), rng.choice([1, 2, 4, 8])
            new = _log(rng, 1, 16)
            c = dict(op=op, requests=_log(rng, 1, 128), new=new, ragged=rng.random() < 0.5, tree=rng.random() < 0.25,
                     prefix=_log(rng, 1, 32768), own_lo=1, own_hi=max(new, _log(rng, 16, 2000)), window=rng.choice([0, 0, 0, 128, 2048]),
                     q_heads=g * kv, kv_heads=kv, dim=rng.choice([64, 128]), dtype=rng.choice(["bf16", "fp16"]), page=rng.choice([16, 32, 64, 128]))
        w = work(c)
        if w["bytes"] <= limits[op][0] and w["flops"] <= limits[op][1]:
            return c


def _spread(n, lo, hi, step):
    """n whole numbers that cover [lo, hi] evenly, in a fixed order."""
    return [lo + int((hi - lo + 1) * ((0.5 + i * step) % 1.0)) for i in range(n)]


def _slot_lengths(c):
    return _spread(c["requests"], 0, c["cached_hi"], 0.6180339887498949), _spread(c["requests"], c["new_lo"], c["new_hi"], 0.7548776662466927)


def _slot_pages(c):
    p = c["page"]
    return [-(-(a + n) // p) - -(-a // p) for a, n in zip(*_slot_lengths(c))]


def _attn_lengths(c):
    """Per request: its own keys (the new tokens' among them) and its new tokens."""
    new = _spread(c["requests"], 1, c["new"], 0.7548776662466927) if c["ragged"] else [c["new"]] * c["requests"]
    return [max(a, n) for a, n in zip(_spread(c["requests"], c["own_lo"], c["own_hi"], 0.6180339887498949), new)], new


def work(case):
    c = case
    if c["op"] == "slots":
        rows, pages = sum(_slot_lengths(c)[1]), sum(_slot_pages(c))
        return {"bytes": c["requests"] * (4 + 4 + 4 + 4 + 4) + pages * 8 + rows * (4 + 8 + 4), "flops": 0}
    if c["op"] == "rope":
        row = (c["q_heads"] + 2 * c["kv_heads"]) * c["dim"] * 2
        return {"bytes": c["rows"] * (2 * row + 12), "flops": c["rows"] * (c["q_heads"] + c["kv_heads"]) * c["rot"] * 3}
    lens, new = _attn_lengths(c)
    keys, seen = 0, 0  # a token tree is counted as the chain: its masks, and so the few keys less, come with the inputs
    for length, n in zip(lens, new):
        for i in range(n):
            seen += min(c["prefix"] + length - n + i + 1, c["window"] or 1 << 40)
        keys += min(length, c["window"] + n if c["window"] else length)
    prefix = min(c["prefix"], max(0, c["window"] - min(a - n for a, n in zip(lens, new)))) if c["window"] else c["prefix"]
    rows = sum(new)
    return {"bytes": (prefix + keys) * c["kv_heads"] * c["dim"] * 4 + rows * c["q_heads"] * (c["dim"] * 4 + 4),
            "flops": 4 * seen * c["q_heads"] * c["dim"]}


def _ints(v, device="cuda", dtype=torch.int32):
    return torch.tensor(v, dtype=dtype).to(device)


def _exclusive(t):
    return torch.cumsum(t, 0) - t


def _tables(counts, width, pages, g):
    """A block table of `width` columns with counts[b] pages for request b, drawn without repetition; the other entries -1."""
    n = torch.tensor(counts, dtype=torch.int64, device="cuda")
    perm = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    col = torch.arange(width, device="cuda")
    at = _exclusive(n)[:, None] + col
    return torch.where(col < n[:, None], perm[at.clamp(max=pages - 1)], -1).to(torch.int32).contiguous(), perm


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed * 7919 + 13)
    h = torch.Generator().manual_seed(seed * 7919 + 17)
    c, s = case, {"case": dict(case)}

    def shuffled(*lists):
        p = torch.randperm(len(lists[0]), generator=h).tolist()
        return [[v[i] for i in p] for v in lists]

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(DTYPES[c["dtype"]])

    if c["op"] == "slots":
        b, p = c["requests"], c["page"]
        cached, new = shuffled(*_slot_lengths(c))
        width = -(-(c["cached_hi"] + c["new_hi"]) // p)
        held = [-(-a // p) for a in cached]
        need = sum(_slot_pages(c))
        s["pages"] = sum(held) + need + 8
        s["table"], perm = _tables(held, width, s["pages"], g)
        s["free"] = perm[sum(held):sum(held) + int(need * c["free"]) + 4].contiguous()
        s["head"] = _ints([seed % 4])  # entries of the list that earlier steps took
        s["cached"], s["new"] = _ints(cached), _ints(new)
        n = sum(new) + 3  # the row buffers of a captured step are a little longer than the step
        s["cu"], s["lens"] = _ints([0] * (b + 1)), _ints([0] * b)
        s["positions"], s["slots"], s["request"] = _ints([0] * n), _ints([0] * n, dtype=torch.int64), _ints([0] * n)
        s["summary"] = _ints([0] * 4)
    elif c["op"] == "rope":
        n, hq, hk, d, p = c["rows"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
        qkv = rand(n, hq + 2 * hk, d)  # the projection's output: q, k and v are views of it
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["q_out"] = torch.empty(n, hq, d, device="cuda", dtype=qkv.dtype)
        s["positions"] = torch.randint(0, c["positions"], (n,), generator=g, device="cuda", dtype=torch.int32)
        pages = -(-n // p) + 3
        s["slots"] = torch.randperm(pages * p, generator=g, device="cuda", dtype=torch.int64)[:n].contiguous()
        s["slots"][n - 1 - seed % 2:n - 1] = -1  # a row without a place
        s["k_cache"], s["v_cache"] = rand(pages, p, hk, d), rand(pages, p, hk, d)
        s["rope"] = dict(theta=10000.0, scaling=c["scaling"], factor=1.0 if c["scaling"] == "none" else 8.0, orig_ctx=8192)
        if own:  # the frequencies that a program sets up once
            from moe_decode_layer_persistent_gb300 import binding as mk
            s["handle"] = mk.mk_rope_create(mk.make_rope_config(d, c["rot"], layout=c["layout"], **s["rope"]))
    else:
        b, hq, hk, d, p = c["requests"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
        lens, new = shuffled(*_attn_lengths(c))
        n = sum(new)
        first = -(-c["prefix"] // p)
        held = [-(-a // p) for a in lens]
        pages = first + sum(held) + 2
        table, _ = _tables([first] + held, max(first, -(-c["own_hi"] // p), -(-c["new"] // p)), pages, g)
        s["prefix_pages"] = table[0, :first].contiguous()
        s["table"] = table[1:, :max(held)].contiguous()
        s["k_cache"], s["v_cache"] = rand(pages, p, hk, d), rand(pages, p, hk, d)
        s["q"] = rand(n, hq, d)
        s["lens"] = _ints(lens)
        s["cu"] = _ints([0] + torch.tensor(new).cumsum(0).tolist())
        s["new"] = c["new"]
        s["mask"] = None
        if c["tree"]:  # each token hangs on one before it, or on the request's last cached token
            masks = []
            for m in new:
                up = torch.randint(-1, 1 << 20, (m,), generator=h).tolist()
                mine = []
                for i in range(m):
                    mine.append((1 << i) | (mine[up[i] % i] if i and up[i] >= 0 else 0))
                masks += mine
            s["mask"] = _ints(masks, dtype=torch.int64)
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(n, hq, device="cuda", dtype=torch.float32)
        if own:  # the workspace that a program keeps
            from moe_decode_layer_persistent_gb300 import binding as mk
            s["workspace"] = torch.empty(mk.mk_prefix_attn_workspace(_attn_io(mk, s)), device="cuda", dtype=torch.uint8)
    return s


def _attn_io(mk, s):
    c = s["case"]
    return mk.make_prefix_attn_io(s["q"], s["k_cache"], s["v_cache"], s["out"], s["lens"], s["cu"], s["table"], s["prefix_pages"], c["prefix"],
                                  window=c["window"], tree_mask=s["mask"], lse=s["lse"])


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        from moe_decode_layer_persistent_gb300 import binding as mk
        stream = torch.cuda.current_stream()
        if op == "slots":
            io = mk.make_slots_io(s["cached"], s["new"], s["free"], s["head"], s["table"], s["cu"], s["lens"], s["positions"], s["slots"],
                                  s["request"], s["summary"], s["case"]["page"], s["pages"], s["case"]["prefix"])
            mk.mk_build_slots(io, stream)
        elif op == "rope":
            io = mk.make_rope_io(s["q"], s["q_out"], s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"])
            mk.mk_rope_apply(s["handle"], io, stream)
        else:
            mk.mk_prefix_attn(_attn_io(mk, s), s["workspace"], stream)
        if op == "slots":
            return {k: s[k] for k in ("table", "cu", "lens", "positions", "slots", "request", "summary")}
        return {k: s[k] for k in (("q_out", "k_cache", "v_cache") if op == "rope" else ("out", "lse"))}
    return {"slots": _plain_slots, "rope": _plain_rope, "attn": _plain_attn}[op](s)


def _plain_slots(s):
    p, prefix = s["case"]["page"], s["case"]["prefix"]
    cached, new = s["cached"].long(), s["new"].long()
    rows, width, free = s["positions"].numel(), s["table"].shape[1], s["free"].numel()
    head = s["head"].long().clamp(0, free)
    n = new.clamp(min=0)
    cu = torch.cat([torch.zeros_like(head), torch.cumsum(n, 0)])
    fits = (cached >= 0) & (new >= 0) & (cached + new <= width * p) & (cu[1:] <= rows)
    before, after = (cached + p - 1) // p, (cached + n + p - 1) // p
    need = torch.where(fits, after - before, 0)
    upto = torch.cumsum(need, 0)
    granted = fits & ((need == 0) | (head + upto <= free))
    base = head + upto - need
    col = torch.arange(width, device=cached.device)
    entry = base[:, None] + col - before[:, None]
    fresh = granted[:, None] & (col >= before[:, None]) & (col < after[:, None])
    table = torch.where(fresh, s["free"][entry.clamp(0, free - 1)], s["table"])
    lens = torch.where(granted, cached + n, cached.clamp(0, width * p))
    r = torch.arange(rows, device=cached.device)
    used = cu[-1].clamp(max=rows)
    req = torch.searchsorted(cu[1:], r, right=True).clamp(max=cached.numel() - 1)
    at = cached[req] + r - cu[req]
    page = table[req, (at // p).clamp(0, width - 1)].long()
    ok = (r < used) & granted[req] & (page >= 0) & (page < s["pages"])
    slots = torch.where(ok, page * p + at % p, -1)
    summary = torch.stack([head[0] + torch.where(granted, need, 0).sum(), used, (~granted).sum(), need.sum()])
    i32 = torch.int32
    return {"table": table, "cu": cu.clamp(max=rows).to(i32), "lens": lens.to(i32), "positions": torch.where(r < used, prefix + at, 0).to(i32),
            "slots": slots, "request": torch.where(r < used, req, -1).to(i32), "summary": summary.to(i32)}


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


def _plain_rope(s):
    c = s["case"]
    rot = c["rot"]
    f, m = _frequencies(rot, s["rope"])
    angle = s["positions"].double()[:, None] * f.to(s["q"].device)
    cos, sin = (torch.cos(angle) * m).float()[:, None], (torch.sin(angle) * m).float()[:, None]

    def turned(x):
        y = x.float()
        if c["layout"] == "half":
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            parts = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            parts = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([parts, y[..., rot:]], -1).to(x.dtype)

    put = s["slots"] >= 0
    at = s["slots"][put]
    s["k_cache"].view(-1, c["kv_heads"], c["dim"])[at] = turned(s["k"])[put]
    s["v_cache"].view(-1, c["kv_heads"], c["dim"])[at] = s["v"][put]
    return {"q_out": turned(s["q"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attn(s):
    c = s["case"]
    hk, d, prefix, t = c["kv_heads"], c["dim"], c["prefix"], s["new"]
    g, n, b = c["q_heads"] // hk, s["q"].shape[0], c["requests"]
    dev = s["q"].device
    lens, cu = s["lens"].long(), s["cu"].long()
    new = cu[1:] - cu[:-1]
    scale = 1.0 / math.sqrt(d)
    r = torch.arange(n, device=dev)
    req = torch.searchsorted(cu[1:], r, right=True)
    i = r - cu[req]
    base = lens[req] - new[req]
    bits = None if s["mask"] is None else s["mask"][:, None] >> torch.arange(t, device=dev) & 1
    pos = prefix + base + (i if bits is None else bits.sum(1) - 1)
    low = pos - c["window"] + 1 if c["window"] else torch.zeros_like(pos)
    q = s["q"].float().view(n, hk, g, d) * scale
    # the prefix, for all rows at once
    kp = s["k_cache"][s["prefix_pages"].long()].view(-1, hk, d)[:prefix].float()
    vp = s["v_cache"][s["prefix_pages"].long()].view(-1, hk, d)[:prefix].float()
    sp = torch.matmul(q.permute(1, 0, 2, 3).reshape(hk, n * g, d), kp.permute(1, 2, 0)).view(hk, n, g, prefix)
    if c["window"]:
        sp = sp.masked_fill((torch.arange(prefix, device=dev) < low[:, None])[None, :, None], -math.inf)
    # each request's own keys, the requests padded to the longest
    pages = s["table"].long().clamp(min=0)
    ko = s["k_cache"][pages].view(b, -1, hk, d).permute(0, 2, 3, 1).float()
    vo = s["v_cache"][pages].view(b, -1, hk, d).permute(0, 2, 1, 3).float()
    width = ko.shape[-1]
    qb = torch.zeros(b, t, hk, g, d, device=dev)
    qb[req, i] = q
    so = torch.matmul(qb.permute(0, 2, 1, 3, 4).reshape(b, hk, t * g, d), ko).view(b, hk, t, g, width).permute(0, 2, 1, 3, 4)[req, i]
    key = torch.arange(width, device=dev)
    fresh = key - base[:, None]
    if bits is None:
        see = fresh <= i[:, None]
    else:
        see = (fresh < 0) | ((fresh < new[req][:, None]) & (bits.gather(1, fresh.clamp(0, t - 1)) > 0))
    see &= (prefix + key) >= low[:, None]
    so = so.masked_fill(~see[:, None, None], -math.inf).permute(1, 0, 2, 3)
    top = torch.maximum(sp.amax(-1) if prefix else so.amax(-1), so.amax(-1))[..., None]
    pp, po = torch.exp(sp - top), torch.exp(so - top)
    total = pp.sum(-1) + po.sum(-1)
    acc = torch.matmul(pp.view(hk, n * g, prefix), vp.permute(1, 0, 2)).view(hk, n, g, d)
    pb = torch.zeros(b, t, hk, g, width, device=dev)
    pb[req, i] = po.permute(1, 0, 2, 3)
    ob = torch.matmul(pb.permute(0, 2, 1, 3, 4).reshape(b, hk, t * g, width), vo).view(b, hk, t, g, d).permute(0, 2, 1, 3, 4)[req, i]
    acc = acc.permute(1, 0, 2, 3) + ob
    total = total.permute(1, 0, 2)
    return {"out": (acc / total[..., None]).reshape(n, hk * g, d).to(s["q"].dtype), "lse": (top[..., 0].permute(1, 0, 2) + torch.log(total)).reshape(n, hk * g)}


def exact(case, seed):
    if case["op"] == "slots":
        return None  # whole numbers
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
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

        def turn(x):
            y = x.double().clone()
            one, two = (slice(0, rot // 2), slice(rot // 2, rot)) if c["layout"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
            w = torch.complex(y[..., one].contiguous(), y[..., two].contiguous()) * z
            y[..., one], y[..., two] = w.real, w.imag
            return y

        kc, vc = s["k_cache"].double().flatten(0, 1), s["v_cache"].double().flatten(0, 1)
        has = torch.nonzero(s["slots"] >= 0)[:, 0]
        kc.index_copy_(0, s["slots"][has], turn(s["k"])[has])
        vc.index_copy_(0, s["slots"][has], s["v"].double()[has])
        return {"q_out": turn(s["q"]), "k_cache": kc.view(s["k_cache"].shape), "v_cache": vc.view(s["v_cache"].shape)}
    hk, d, g, prefix = c["kv_heads"], c["dim"], c["q_heads"] // c["kv_heads"], c["prefix"]
    n = s["q"].shape[0]
    out = torch.empty(n, c["q_heads"], d, dtype=torch.float64, device="cuda")
    lse = torch.empty(n, c["q_heads"], dtype=torch.float64, device="cuda")
    shared = [x[s["prefix_pages"].long()].flatten(0, 1)[:prefix].double() for x in (s["k_cache"], s["v_cache"])]
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    for b in range(c["requests"]):
        first, m, length = cu[b], cu[b + 1] - cu[b], lens[b]
        keys, values = (torch.cat([a, x[s["table"][b, :-(-length // c["page"])].long()].flatten(0, 1)[:length].double()]).transpose(0, 1)
                        for a, x in zip(shared, (s["k_cache"], s["v_cache"])))
        see = torch.ones(m, prefix + length, dtype=torch.bool, device="cuda")
        for i in range(m):
            word = (2 << i) - 1 if s["mask"] is None else int(s["mask"][first + i])
            for j in range(m):
                see[i, prefix + length - m + j] = bool(word >> j & 1)
            if c["window"]:
                p = prefix + length - m + bin(word).count("1") - 1
                see[i, :max(0, min(p - c["window"] + 1, prefix + length - m))] = False
        q = s["q"][first:first + m].double().view(m, hk, g, d).transpose(0, 1).reshape(hk, m * g, d)
        score = (q @ keys.transpose(1, 2) / d ** 0.5).view(hk, m, g, -1)
        score = torch.where(see[None, :, None], score, torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
        part = torch.logsumexp(score, -1)
        weight = torch.exp(score - part[..., None]).view(hk, m * g, -1)
        out[first:first + m] = (weight @ values).view(hk, m, g, d).transpose(0, 1).reshape(m, hk * g, d)
        lse[first:first + m] = part.transpose(0, 1).reshape(m, hk * g)
    return {"out": out, "lse": lse}
