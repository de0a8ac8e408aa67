"""Cases of the serving-step operators: building slot maps on the GPU, the fused
norm + rotation + cache write, and decode attention over shared prefixes.

``run`` computes each operator in plain torch operations (32-bit, rounded once at the end),
or, with ``own`` set, through this package's entry points.  ``exact`` gives the same
outputs from the definitions in 64 bits.
"""

import math

import torch

own = False

BLOCK = 16


def listed():
    return [
        # One decode step of a running batch: a token per sequence.
        {"name": "slots decode", "op": "slots", "seqs": 64, "ctx_lo": 128, "ctx_hi": 2048, "new_lo": 1, "new_hi": 1},
        # A verification step: a few drafts per sequence, their number differing by sequence.
        {"name": "slots verify", "op": "slots", "seqs": 256, "ctx_lo": 16, "ctx_hi": 16384, "new_lo": 2, "new_hi": 5},
        # Prompts admitted together: ragged lengths, empty tables.
        {"name": "slots prefill", "op": "slots", "seqs": 64, "ctx_lo": 0, "ctx_hi": 0, "new_lo": 1, "new_hi": 8191},
        # The smallest decode step, where latency is everything.
        {"name": "rope decode 8", "op": "rope", "tokens": 8, "hq": 32, "hkv": 8, "d": 128, "kv": "bf16",
         "rot": 128, "interleaved": False, "norm": True},
        # A continuous-batching decode step into an FP8 pool.
        {"name": "rope decode 256 fp8", "op": "rope", "tokens": 256, "hq": 32, "hkv": 8, "d": 128, "kv": "fp8",
         "rot": 128, "interleaved": False, "norm": True},
        # A large prefill chunk.
        {"name": "rope prefill bf16", "op": "rope", "tokens": 16384, "hq": 32, "hkv": 8, "d": 128, "kv": "bf16",
         "rot": 128, "interleaved": False, "norm": True},
        # An odd-sized prefill of an MHA layer into an INT8 pool, half of each head rotated in neighbouring pairs.
        {"name": "rope prefill int8", "op": "rope", "tokens": 4093, "hq": 32, "hkv": 32, "d": 64, "kv": "int8",
         "rot": 32, "interleaved": True, "norm": False},
        # A few samples of one short prompt.
        {"name": "prefix small", "op": "prefix", "groups": 1, "seqs": 4, "prefix_lo": 1024, "prefix_hi": 1024,
         "suffix_lo": 1, "suffix_hi": 120, "hq": 32, "hkv": 8, "d": 128, "kv": "bf16", "queries": 1},
        # Many requests about one long document.
        {"name": "prefix long", "op": "prefix", "groups": 1, "seqs": 64, "prefix_lo": 32768, "prefix_hi": 32768,
         "suffix_lo": 16, "suffix_hi": 300, "hq": 32, "hkv": 8, "d": 128, "kv": "bf16", "queries": 1},
        # Parallel sampling: groups of unequal size, each with a prompt of its own, MHA.
        {"name": "prefix groups", "op": "prefix", "groups": 16, "seqs": 117, "prefix_lo": 240, "prefix_hi": 2048,
         "suffix_lo": 1, "suffix_hi": 256, "hq": 32, "hkv": 32, "d": 128, "kv": "bf16", "queries": 1},
        # A large batch over one system prompt with an INT8 cache.
        {"name": "prefix large int8", "op": "prefix", "groups": 1, "seqs": 256, "prefix_lo": 16384, "prefix_hi": 16384,
         "suffix_lo": 16, "suffix_hi": 512, "hq": 32, "hkv": 8, "d": 128, "kv": "int8", "queries": 1},
        # Draft verification over two shared prompts, FP8 cache, head_dim 64.
        {"name": "prefix verify fp8", "op": "prefix", "groups": 2, "seqs": 48, "prefix_lo": 4000, "prefix_hi": 8192,
         "suffix_lo": 4, "suffix_hi": 400, "hq": 32, "hkv": 8, "d": 64, "kv": "fp8", "queries": 4},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["slots", "rope", "prefix", "rope", "prefix"])
    if op == "slots":
        kind = rng.choice(["decode", "verify", "prefill"])
        seqs = _log_int(rng, 1, 2048 if kind != "prefill" else 64)
        if kind == "prefill":
            return {"op": op, "seqs": seqs, "ctx_lo": 0, "ctx_hi": rng.choice([0, 100, 5000]), "new_lo": rng.choice([0, 1]),
                    "new_hi": _log_int(rng, 2, 8191)}
        return {"op": op, "seqs": seqs, "ctx_lo": rng.randint(0, 200), "ctx_hi": _log_int(rng, 256, 32768),
                "new_lo": rng.choice([0, 1, 2]) if kind == "verify" else 1,
                "new_hi": rng.randint(2, 8) if kind == "verify" else 1}
    hq, hkv = rng.choice([(32, 8), (32, 32), (16, 4), (8, 1), (28, 4), (4, 4), (24, 8)])
    d = rng.choice([64, 128])
    kv = rng.choice(["bf16", "int8", "fp8"])
    if op == "rope":
        return {"op": op, "tokens": _log_int(rng, 1, 8192 if hkv == 32 else 16384), "hq": hq, "hkv": hkv, "d": d,
                "kv": kv, "rot": rng.choice([d, d // 2]), "interleaved": rng.random() < 0.3, "norm": rng.random() < 0.8}
    queries = rng.choice([1, 1, 1, 2, 4])
    seqs = _log_int(rng, 2, 160)
    groups = min(seqs, _log_int(rng, 1, 24))
    # The largest listed case has 128 M pairs of a query head and a prefix token, and 32768 prefix tokens of 8 kv heads.
    room = min(64 * 1024 * 1024 // max(1, seqs * queries * hq), 300000 // (groups * hkv))
    hi = _log_int(rng, 16, max(16, min(32768, room)))
    return {"op": op, "groups": groups, "seqs": seqs, "prefix_lo": max(16, hi // rng.choice([1, 2, 8])), "prefix_hi": hi,
            "suffix_lo": queries, "suffix_hi": queries + _log_int(rng, 1, 400), "hq": hq, "hkv": hkv, "d": d, "kv": kv,
            "queries": queries}


# ---------------------------------------------------------------- the sizes of a case

def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], in no order, both ends among them where n allows it."""
    if n == 1 or lo == hi:
        return [hi] * n
    return [lo + ((i * 7919) % n) * (hi - lo) // (n - 1) for i in range(n)]


def _slots_sizes(c):
    n = c["seqs"]
    return _spread(n, c["ctx_lo"], c["ctx_hi"]), _spread(n, c["new_lo"], c["new_hi"])[::-1]


def _blocks(t):
    return -(-t // BLOCK)


def _prefix_sizes(c):
    """(first sequence of each group and the end, prefix tokens of each group, suffix tokens of each sequence)."""
    g, b = c["groups"], c["seqs"]
    weights = [1 + (i * 5) % 7 for i in range(g)]  # groups of unequal size, none empty
    starts, run = [0], 0
    for i in range(g):
        run += weights[i]
        starts.append(max(starts[-1] + 1, min(b - (g - 1 - i), run * b // sum(weights))))
    starts[-1] = b
    pre = [max(BLOCK, p // BLOCK * BLOCK) for p in _spread(g, c["prefix_lo"], c["prefix_hi"])]
    return starts, pre, _spread(b, c["suffix_lo"], c["suffix_hi"])


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _quantise(x, kv):
    """Codes and scales of rows [..., d]: s = max|x| / (127 or 448), the nearest code of x / s."""
    top = 127.0 if kv == "int8" else 448.0
    s = x.abs().amax(-1) / top
    y = torch.where(s[..., None] > 0, x / s[..., None], torch.zeros_like(x)).clamp(-top, top)
    if kv == "int8":
        return y.round().to(torch.int8), s
    return y.to(torch.float8_e4m3fn).view(torch.uint8), s


def _pool(nb, hkv, d, kv, gen):
    """A pool in use: K and V of unit size in every slot."""
    shape = (nb, hkv, BLOCK, d)
    s = {}
    for name in ("k", "v"):
        x = torch.randn(shape, generator=gen, device="cuda")
        if kv == "bf16":
            s[name] = x.to(torch.bfloat16)
        else:
            s[name], s[name + "_scale"] = _quantise(x, kv)
    return s


def prepare(case, seed):
    gen = _gen(seed)
    s = {"case": dict(case)}
    if case["op"] == "slots":
        ctx, new = _slots_sizes(case)
        have = [_blocks(t) for t in ctx]
        need = [_blocks(t + n) for t, n in zip(ctx, new)]
        width = max(max(need), 1) + 8
        nb = sum(need) + 64
        ids = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32)
        at = torch.cumsum(torch.tensor([0] + have, device="cuda"), 0)
        col = torch.arange(width, device="cuda")
        tables = torch.where(col < _ints(have)[:, None], ids[(at[:-1, None] + col).clamp(max=nb - 1)], -1)
        s.update(tables=tables.to(torch.int32).contiguous(), lens=_ints(ctx), new=_ints(new),
                 free=ids[sum(have):].clone(), used=_ints([seed % 16]), max_tokens=max(1, sum(new)), num_blocks=nb)
        if own:
            # The pool is what the ids belong to; one kv head of 64 dims stands for its layers.
            s["pool"] = _package().PagedKVPool(nb, 1, 64, "bf16")
            i32 = dict(dtype=torch.int32, device="cuda")
            s["out"] = dict(slot_mapping=torch.empty(s["max_tokens"], **i32), positions=torch.empty(s["max_tokens"], **i32),
                            query_starts=torch.empty(len(ctx) + 1, **i32), new_context_lens=torch.empty(len(ctx), **i32),
                            new_free_used=torch.empty(1, **i32))
    elif case["op"] == "rope":
        n, hq, hkv, d, rot = (case[k] for k in ("tokens", "hq", "hkv", "d", "rot"))
        # q, k and v lie side by side in a projection's output, heads of different size.
        x = torch.randn(n, hq + 2 * hkv, d, generator=gen, device="cuda")
        x = x * torch.exp(0.7 * torch.randn(1, hq + 2 * hkv, 1, generator=gen, device="cuda"))
        s["qkv"] = x.to(torch.bfloat16)
        s["qw"], s["kw"] = ((1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16) for _ in range(2))
        top = 32768
        angle = torch.arange(top, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        nb = _blocks(n) + 8
        if n <= 512:  # a decode step: every token somewhere else
            s["positions"] = torch.randint(0, top, (n,), generator=gen, device="cuda", dtype=torch.int32)
            s["slots"] = torch.randperm(nb * BLOCK, generator=gen, device="cuda")[:n].to(torch.int32)
        else:  # a prefill: runs of positions in scattered blocks
            t = torch.arange(n, device="cuda")
            s["positions"] = (t % 5000).to(torch.int32)
            block = torch.randperm(nb, generator=gen, device="cuda")
            s["slots"] = (block[t // BLOCK] * BLOCK + t % BLOCK).to(torch.int32)
        s.update(_pool(nb, hkv, d, case["kv"], gen))
        s["q_out"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
        if case["kv"] == "int8":
            s["k_values"], s["v_values"] = (torch.empty(s["k"].shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    else:
        starts, pre, suf = _prefix_sizes(case)
        hq, hkv, d, k = (case[x] for x in ("hq", "hkv", "d", "queries"))
        g, b = case["groups"], case["seqs"]
        gid = [i for i in range(g) for _ in range(starts[i + 1] - starts[i])]
        need = [sum(p // BLOCK for p in pre), sum(_blocks(t) for t in suf)]
        nb = sum(need) + 16
        ids = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32).tolist()
        rows, at, pre_ids = [], need[0], []
        for i in range(g):
            before = sum(p // BLOCK for p in pre[:i])
            pre_ids.append(ids[before:before + pre[i] // BLOCK])
        width = max(pre[gid[i]] // BLOCK + _blocks(suf[i]) for i in range(b)) + 4
        for i in range(b):
            n = _blocks(suf[i])
            row = pre_ids[gid[i]] + ids[at:at + n]
            rows.append(row + [-1] * (width - len(row)))
            at += n
        q = 1.5 * torch.randn((b, hq, d) if k == 1 else (b, k, hq, d), generator=gen, device="cuda")
        s.update(q=q.to(torch.bfloat16), tables=_ints(rows), lens=_ints([pre[gid[i]] + suf[i] for i in range(b)]),
                 starts=_ints(starts), prefix=_ints(pre), max_prefix=max(pre), max_suffix=max(suf), scale=d ** -0.5,
                 most=max(starts[i + 1] - starts[i] for i in range(g)), **_pool(nb, hkv, d, case["kv"], gen))
        s["out"] = torch.empty_like(s["q"])
    if own and case["op"] != "slots":
        pkv = _package()
        s["pool"] = pkv.PagedKVPool.from_tensors(s["k"], s["v"], s.get("k_scale"), s.get("v_scale"))
        if case["op"] == "prefix":
            bytes_ = pkv.shared_prefix_workspace_bytes(s["pool"], case["seqs"], case["hq"], case["groups"], s["max_prefix"],
                                                       s["max_suffix"], num_queries=case["queries"])
            s["workspace"] = torch.empty(bytes_, dtype=torch.uint8, device="cuda")
    return s


def _package():
    import paged_kv_cache_264_gb300
    return paged_kv_cache_264_gb300


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    if c["op"] == "slots":
        if own:
            out = _package().reserve_slots(s["pool"], s["tables"], s["lens"], s["new"], s["free"], s["max_tokens"],
                                           free_used=s["used"], **s["out"])
        else:
            out = _plain_slots(s)
        return {"tables": s["tables"], "slots": out[0], "positions": out[1], "starts": out[2], "lens": out[3], "used": out[4]}
    if c["op"] == "rope":
        hq, hkv = c["hq"], c["hkv"]
        q, k, v = s["qkv"][:, :hq], s["qkv"][:, hq:hq + hkv], s["qkv"][:, hq + hkv:]
        qw, kw = (s["qw"], s["kw"]) if c["norm"] else (None, None)
        if own:
            q_out = _package().norm_rope_and_cache(s["pool"], q, k, v, s["positions"], s["slots"], s["cos_sin"], qw, kw,
                                                   eps=1e-6, interleaved=c["interleaved"], out=s["q_out"])
        else:
            q_out = _plain_rope(s, q, k, v, qw, kw)
        out = {"q": q_out}
        for name in ("k", "v"):
            if c["kv"] == "bf16":
                out[name] = s[name]
            elif c["kv"] == "fp8":
                out[name], out[name + "_scale"] = s[name].view(torch.float8_e4m3fn), s[name + "_scale"]
            else:  # the values that the codes stand for
                out[name] = torch.mul(s[name], s[name + "_scale"][..., None], out=s[name + "_values"])
        return out
    if own:
        return _package().shared_prefix_decode(s["pool"], s["q"], s["tables"], s["lens"], s["starts"], s["prefix"], s["scale"],
                                               s["max_prefix"], s["max_suffix"], out=s["out"], workspace=s["workspace"])
    return _plain_prefix(s)


def _plain_slots(s):
    lens, new, free, tables = s["lens"], s["new"], s["free"], s["tables"]
    width = tables.shape[1]
    have, need = (lens + BLOCK - 1) // BLOCK, (lens + new + BLOCK - 1) // BLOCK
    ends = torch.cumsum(need - have, 0)
    starts = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0, dtype=torch.int32)])
    ok = (s["used"] + ends[-1] <= free.shape[0]) & (need <= width).all() & (starts[-1] <= s["max_tokens"])
    col = torch.arange(width, device=tables.device, dtype=torch.int32)
    at = s["used"] + (ends - (need - have))[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < need[:, None]) & ok
    tables.copy_(torch.where(fresh, free[at.clamp(0, free.shape[0] - 1)], tables))
    i = torch.arange(s["max_tokens"], device=tables.device, dtype=torch.int32)
    b = (torch.searchsorted(starts, i, right=True) - 1).clamp(max=lens.shape[0] - 1)
    live = (i < starts[-1]) & ok
    p = torch.where(live, lens[b] + i - starts[b], 0).to(torch.int32)
    slots = torch.where(live, tables[b, (p // BLOCK).long()] * BLOCK + p % BLOCK, -1).to(torch.int32)
    return (slots, p, torch.where(ok, starts, 0).to(torch.int32), torch.where(ok, lens + new, lens).to(torch.int32),
            torch.where(ok, s["used"] + ends[-1], s["used"]).to(torch.int32))


def _plain_rope(s, q, k, v, qw, kw):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    table = s["cos_sin"][s["positions"].long()]
    cos, sin = table[:, None, :half], table[:, None, half:]

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        if c["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., rot:]], -1)

    block, at = s["slots"].long() // BLOCK, s["slots"].long() % BLOCK
    for name, x in (("k", turned(k, kw)), ("v", v.float())):
        if c["kv"] == "bf16":
            s[name][block, :, at] = x.to(torch.bfloat16)
        else:
            s[name][block, :, at], s[name + "_scale"][block, :, at] = _quantise(x, c["kv"])
    s["q_out"].copy_(turned(q, qw))
    return s["q_out"]


def _rows(s, name, blocks):
    """fp32 rows of blocks [n, m]: [n, Hkv, m * 16, d]."""
    x = s[name][blocks]
    x = (x.view(torch.float8_e4m3fn) if s["case"]["kv"] == "fp8" else x).float()
    if s["case"]["kv"] != "bf16":
        x = x * s[name + "_scale"][blocks][..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_prefix(s):
    c = s["case"]
    g, b, hq, hkv, d, k = (c[x] for x in ("groups", "seqs", "hq", "hkv", "d", "queries"))
    grp, dev = hq // hkv, s["q"].device
    q = s["q"].float().view(b, k, hkv, grp, d).transpose(1, 2).reshape(b, hkv, k * grp, d) * s["scale"]
    starts = s["starts"].long()
    # the prefix of each group against all of the group's rows
    member = starts[:-1, None] + torch.arange(s["most"], device=dev)
    rows = q[member.clamp(max=b - 1)].transpose(1, 2).flatten(2, 3)
    nb = s["max_prefix"] // BLOCK
    inside = torch.arange(nb, device=dev) < (s["prefix"] // BLOCK)[:, None]
    blocks = torch.where(inside, s["tables"][starts[:-1], :nb], 0).long()
    x = rows @ _rows(s, "k", blocks).transpose(2, 3)
    x = x.masked_fill(~inside.repeat_interleave(BLOCK, 1)[:, None, None], float("-inf"))
    m1 = x.amax(-1, keepdim=True)
    x = torch.exp(x - m1)
    l1 = x.sum(-1, keepdim=True)
    o1 = x @ _rows(s, "v", blocks)
    gid = torch.searchsorted(s["starts"], torch.arange(b, device=dev, dtype=torch.int32), right=True) - 1
    place = torch.arange(b, device=dev) - starts[gid]
    m1, l1, o1 = (t.view(g, hkv, s["most"], k * grp, -1)[gid, :, place] for t in (m1, l1, o1))
    # each sequence's own tokens
    first = s["prefix"][gid]
    nb = _blocks(s["max_suffix"])
    col = (first // BLOCK)[:, None] + torch.arange(nb, device=dev)
    t = torch.arange(nb * BLOCK, device=dev)
    seen = (s["lens"] - first)[:, None] - (k - 1 - torch.arange(k, device=dev))
    seen = (t < seen[..., None]).repeat_interleave(grp, 1)
    blocks = torch.gather(s["tables"], 1, col.clamp(max=s["tables"].shape[1] - 1)).clamp(min=0).long()
    x = (q @ _rows(s, "k", blocks).transpose(2, 3)).masked_fill(~seen[:, None], float("-inf"))
    m = torch.maximum(m1, x.amax(-1, keepdim=True))
    x = torch.exp(x - m)
    o = x @ _rows(s, "v", blocks) + o1 * torch.exp(m1 - m)
    o = o / (x.sum(-1, keepdim=True) + l1 * torch.exp(m1 - m))
    return o.view(b, hkv, k, grp, d).transpose(1, 2).reshape(s["q"].shape).to(torch.bfloat16)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "slots":
        ctx, new = _slots_sizes(case)
        fresh = sum(_blocks(t + n) - _blocks(t) for t, n in zip(ctx, new))
        partly = sum(1 for t, n in zip(ctx, new) if t % BLOCK and n)
        return {"bytes": 8 * len(ctx) + 4 * fresh + 4 * partly + 8 * sum(new) + 4 * fresh + 8 * len(ctx) + 12, "flops": 0}
    if case["op"] == "rope":
        n, hq, hkv, d, rot = (case[k] for k in ("tokens", "hq", "hkv", "d", "rot"))
        kept = 2 * d if case["kv"] == "bf16" else d + 4
        return {"bytes": n * (2 * d * (hq + 2 * hkv) + 4 * rot + 8 + 2 * d * hq + 2 * hkv * kept) + 4 * d,
                "flops": n * (hq + hkv) * (4 * d + 3 * rot)}
    starts, pre, suf = _prefix_sizes(case)
    hq, hkv, d, k = (case[x] for x in ("hq", "hkv", "d", "queries"))
    row = 2 * hkv * (2 * d if case["kv"] == "bf16" else d + 4)
    size = [starts[i + 1] - starts[i] for i in range(case["groups"])]
    pairs = sum(n * p for n, p in zip(size, pre)) + sum(suf)
    return {"bytes": row * (sum(pre) + sum(suf)) + 4 * case["seqs"] * k * hq * d + 4 * (sum(pre) + sum(suf)) // BLOCK,
            "flops": 4 * pairs * k * hq * d}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"slots": _exact_slots, "rope": _exact_rope, "prefix": _exact_prefix}[case["op"]](s)


def _exact_slots(s):
    lens, new, free, used = (s[x].tolist() for x in ("lens", "new", "free", "used"))
    tables = s["tables"].tolist()
    slots, positions, starts, at = [], [], [0], used[0]
    for b, (t, n) in enumerate(zip(lens, new)):
        for p in range(t, t + n):
            if p % BLOCK == 0:
                tables[b][p // BLOCK] = free[at]
                at += 1
            slots.append(tables[b][p // BLOCK] * BLOCK + p % BLOCK)
            positions.append(p)
        starts.append(len(slots))
    rest = s["max_tokens"] - len(slots)
    return {"tables": _ints(tables), "slots": _ints(slots + [-1] * rest), "positions": _ints(positions + [0] * rest),
            "starts": _ints(starts), "lens": _ints([t + n for t, n in zip(lens, new)]), "used": _ints([at])}


def _value64(x, scale, kv):
    x = (x.view(torch.float8_e4m3fn).float() if kv == "fp8" else x).double()
    return x if kv == "bf16" else x * scale.double()[..., None]


def _exact_rope(s):
    c = s["case"]
    hq, hkv, rot, kv = c["hq"], c["hkv"], c["rot"], c["kv"]
    x = s["qkv"].double()
    if c["norm"]:
        w = torch.cat([s["qw"].double().expand(hq, -1), s["kw"].double().expand(hkv, -1)])
        size = x[:, :hq + hkv].pow(2).sum(-1, keepdim=True) / c["d"]
        x[:, :hq + hkv] *= w / (size + 1e-6).sqrt()
    # each rotated pair as a complex number times e^(i angle), of the angles' given cosines and sines
    turn = s["cos_sin"].double()[s["positions"].long()]
    turn = torch.complex(turn[:, :rot // 2], turn[:, rot // 2:])[:, None]
    one = torch.arange(rot // 2, device="cuda") * (2 if c["interleaved"] else 1)
    two = one + (1 if c["interleaved"] else rot // 2)
    z = torch.complex(x[:, :hq + hkv][..., one], x[:, :hq + hkv][..., two]) * turn
    y = x.clone()
    y[:, :hq + hkv, one], y[:, :hq + hkv, two] = z.real, z.imag
    out = {"q": y[:, :hq]}
    slots = s["slots"].long()
    for name, rows in (("k", y[:, hq:hq + hkv]), ("v", y[:, hq + hkv:])):
        if kv == "bf16":
            whole = s[name].double()
            whole[slots // BLOCK, :, slots % BLOCK] = rows
            out[name] = whole
            continue
        top = 127.0 if kv == "int8" else 448.0
        step = rows.abs().amax(-1) / top
        code = torch.where(step[..., None] > 0, rows / step[..., None], 0.0).clamp(-top, top)
        if kv == "int8":
            whole = _value64(s[name], s[name + "_scale"], kv)
            whole[slots // BLOCK, :, slots % BLOCK] = code.round() * step[..., None]
            out[name] = whole
        else:
            grid = torch.exp2(torch.clamp(torch.floor(torch.log2(code.abs().clamp(min=1e-9))), min=-6.0) - 3)
            whole, scale = s[name].view(torch.float8_e4m3fn).float().double(), s[name + "_scale"].double()
            whole[slots // BLOCK, :, slots % BLOCK] = (code / grid).round() * grid
            scale[slots // BLOCK, :, slots % BLOCK] = step
            out[name], out[name + "_scale"] = whole, scale
    return out


def _exact_prefix(s):
    c = s["case"]
    k, hkv, kv = c["queries"], c["hkv"], c["kv"]
    grp = c["hq"] // hkv
    q = s["q"].double().view(c["seqs"], k, hkv, grp, c["d"])
    out = torch.empty_like(q)
    starts, prefix, lens = (s[x].tolist() for x in ("starts", "prefix", "lens"))

    def rows(name, blocks, h):
        scale = None if kv == "bf16" else s[name + "_scale"][blocks, h]
        return _value64(s[name][blocks, h], scale, kv).flatten(0, 1)

    for g in range(c["groups"]):
        lo, hi = starts[g], starts[g + 1]
        shared = s["tables"][lo, :prefix[g] // BLOCK].long()
        for h in range(hkv):
            ks, vs = rows("k", shared, h), rows("v", shared, h)
            x1 = torch.einsum("bigd,td->bigt", q[lo:hi, :, h], ks) * s["scale"]
            for b in range(lo, hi):
                mine = s["tables"][b, prefix[g] // BLOCK:_blocks(lens[b])].long()
                x2 = torch.einsum("igd,td->igt", q[b, :, h], rows("k", mine, h)) * s["scale"]
                t = torch.arange(prefix[g], prefix[g] + x2.shape[-1], device="cuda")
                last = lens[b] - k + torch.arange(k, device="cuda")
                x2 = torch.where(t <= last[:, None, None], x2, float("-inf"))
                p = torch.softmax(torch.cat([x1[b - lo], x2], -1), -1)
                n = prefix[g]
                out[b, :, h] = torch.einsum("igt,td->igd", p[..., :n], vs) + torch.einsum(
                    "igt,td->igd", p[..., n:], rows("v", mine, h))
    return out.view(s["q"].shape)
