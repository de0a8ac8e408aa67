"""Cases of the prompt operators: attention of packed prompts over keys and values as they come
out of the projection, attention of prompt chunks over the paged cache, and reading a cache back.

``run`` computes each operator in plain torch operations (32-bit, rounded once at the end),
or, with ``own`` set, through this package's entry points.  ``exact`` gives the same
outputs from the definitions in 64 bits.
"""

import math

import torch

own = False

BLOCK = 16
PAD = 5  # rows behind the last sequence, as a step of fixed size has them: left as they were


def listed():
    return [
        # A few short questions admitted together: latency is everything.
        {"name": "prompt short", "op": "prompt", "seqs": 3, "ones": 0, "new_lo": 5, "new_hi": 60, "before_lo": 0, "before_hi": 0,
         "hq": 32, "hkv": 8, "d": 128, "kv": "bf16", "window": 0, "causal": True},
        # Prompts of a batch packed without padding, one kv head per query head.
        {"name": "prompt packed mha", "op": "prompt", "seqs": 64, "ones": 0, "new_lo": 128, "new_hi": 2048, "before_lo": 0,
         "before_hi": 0, "hq": 32, "hkv": 32, "d": 128, "kv": "bf16", "window": 0, "causal": True},
        # One long document.
        {"name": "prompt long", "op": "prompt", "seqs": 1, "ones": 0, "new_lo": 16384, "new_hi": 16384, "before_lo": 0,
         "before_hi": 0, "hq": 32, "hkv": 8, "d": 128, "kv": "bf16", "window": 0, "causal": True},
        # Ragged prompts of a sliding-window layer with small heads and seven query heads per kv head.
        {"name": "prompt window d64", "op": "prompt", "seqs": 7, "ones": 0, "new_lo": 1, "new_hi": 6007, "before_lo": 0,
         "before_hi": 0, "hq": 28, "hkv": 4, "d": 64, "kv": "bf16", "window": 1024, "causal": True},
        # A follow-up of a few words to two short conversations.
        {"name": "prefill small", "op": "prefill", "seqs": 2, "ones": 0, "new_lo": 9, "new_hi": 30, "before_lo": 17,
         "before_hi": 200, "hq": 32, "hkv": 8, "d": 128, "kv": "bf16", "window": 0, "causal": True},
        # The last chunk of a long prompt that is taken in pieces.
        {"name": "prefill chunk", "op": "prefill", "seqs": 1, "ones": 0, "new_lo": 2048, "new_hi": 2048, "before_lo": 14336,
         "before_hi": 14336, "hq": 32, "hkv": 8, "d": 128, "kv": "bf16", "window": 0, "causal": True},
        # A continuous-batching step: 60 sequences decode a token each beside four chunks, INT8 cache.
        {"name": "prefill mixed int8", "op": "prefill", "seqs": 64, "ones": 60, "new_lo": 300, "new_hi": 1023, "before_lo": 16,
         "before_hi": 8192, "hq": 32, "hkv": 8, "d": 128, "kv": "int8", "window": 0, "causal": True},
        # Short questions about documents that are in an FP8 cache already.
        {"name": "prefill extend fp8", "op": "prefill", "seqs": 24, "ones": 0, "new_lo": 17, "new_hi": 64, "before_lo": 2000,
         "before_hi": 8192, "hq": 32, "hkv": 8, "d": 128, "kv": "fp8", "window": 0, "causal": True},
        # One question about one long document, one kv head per query head: few rows, a long cache.
        {"name": "prefill long few", "op": "prefill", "seqs": 1, "ones": 0, "new_lo": 24, "new_hi": 24, "before_lo": 32744,
         "before_hi": 32744, "hq": 32, "hkv": 32, "d": 128, "kv": "bf16", "window": 0, "causal": True},
        # One short sequence read back.
        {"name": "gather small fp8", "op": "gather", "seqs": 1, "len_lo": 100, "len_hi": 100, "first_hi": 0, "hkv": 8, "d": 128,
         "kv": "fp8"},
        # A batch's INT8 caches read back to be moved elsewhere, from different positions on.
        {"name": "gather batch int8", "op": "gather", "seqs": 256, "len_lo": 16, "len_hi": 4096, "first_hi": 100, "hkv": 8,
         "d": 128, "kv": "int8"},
        # Long contexts read back whole.
        {"name": "gather long bf16", "op": "gather", "seqs": 8, "len_lo": 32768, "len_hi": 32768, "first_hi": 0, "hkv": 8,
         "d": 128, "kv": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


_HEADS = [(32, 8, 128), (32, 32, 128), (16, 4, 64), (28, 4, 128), (28, 4, 64), (8, 1, 64), (4, 4, 128), (32, 32, 64),
          (16, 2, 128), (71, 1, 64), (6, 2, 64)]


def draw(rng):
    op = rng.choice(["prompt", "prefill", "prompt", "prefill", "gather"])
    hq, hkv, d = rng.choice(_HEADS)
    kv = "bf16" if op == "prompt" else rng.choice(["bf16", "int8", "fp8"])
    if op == "gather":
        seqs = _log_int(rng, 1, 300)
        hi = _log_int(rng, 1, max(1, min(32768, 250000 * 8 * 128 // (seqs * hkv * d))))
        return {"op": op, "seqs": seqs, "len_lo": rng.choice([0, 1, hi // 2, hi]), "len_hi": hi,
                "first_hi": rng.choice([0, 0, 33, 1000]), "hkv": hkv, "d": d, "kv": kv}
    seqs = _log_int(rng, 1, 96)
    # Pairs of a query head and a token that it sees, of the largest listed case: 4.3 G; drawn ones have less.
    room = 4 * 10**9 * 128 // (hq * d)
    if op == "prompt":
        hi = _log_int(rng, 1, max(2, min(16384, int(math.sqrt(room / seqs)), 400000 * 4096 // (seqs * hq * d))))
        before = rng.choice([0, 0, 0, 40, 700])
    else:
        hi = _log_int(rng, 1, max(2, min(4096, 100000 // seqs)))
        before = _log_int(rng, 1, max(2, min(32768, room // (2 * seqs * hi), 2000000 // (seqs * hkv))))
    hi = max(1, min(hi, int(math.sqrt(before * before + 4 * room / seqs) - before) // 2))
    ones = rng.choice([0, 0, seqs // 2, seqs - 1]) if op == "prefill" else 0
    return {"op": op, "seqs": seqs, "ones": ones, "new_lo": rng.choice([0, 1, hi // 3, hi]), "new_hi": hi,
            "before_lo": rng.choice([0, before // 2]), "before_hi": before, "hq": hq, "hkv": hkv, "d": d, "kv": kv,
            "window": rng.choice([0, 0, 0, 100, 512, 2000]), "causal": op == "prefill" or before == 0 or rng.random() < 0.8} | (
        {"window": 0, "causal": False} if op == "prompt" and rng.random() < 0.15 else {})


# ---------------------------------------------------------------- the sizes of a case

def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], in no order, both ends among them where n allows it."""
    if n == 1 or lo == hi:
        return [hi] * n
    return [lo + ((i * 7919) % n) * (hi - lo) // (n - 1) for i in range(n)]


def _blocks(t):
    return -(-t // BLOCK)


def _sizes(c):
    """New tokens of each sequence and the tokens before them."""
    n, ones = c["seqs"], c["ones"]
    new = [1] * ones + _spread(n - ones, c["new_lo"], c["new_hi"])
    new = [new[(i * 5 + 3) % n] if n % 5 else new[(i * 7 + 3) % n] if n % 7 else new[i] for i in range(n)]
    return new, _spread(n, c["before_lo"], c["before_hi"])[::-1]


def _gather_sizes(c):
    n = c["seqs"]
    return _spread(n, c["len_lo"], c["len_hi"]), _spread(n, 0, c["first_hi"])[::-1]


def _starts(sizes):
    out = [0]
    for x in sizes:
        out.append(out[-1] + x)
    return out


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


def _channels(gen, d):
    """Sizes of a head's channels: a few keys' channels are some times as large as the others."""
    return torch.where(torch.rand(d, generator=gen, device="cuda") < 0.03, 4.0, 1.0)


def _pool(nb, hkv, d, kv, gen):
    """A pool in use: K and V in every slot."""
    shape = (nb, hkv, BLOCK, d)
    s = {}
    for name in ("k", "v"):
        x = torch.randn(shape, generator=gen, device="cuda")
        if name == "k":
            x = x * _channels(gen, d)
        if kv == "bf16":
            s[name] = x.to(torch.bfloat16)
        else:
            s[name], s[name + "_scale"] = _quantise(x, kv)
    return s


def _tables(lens, gen):
    """Block tables of sequences of these lengths, blocks in no order, and the pool's blocks."""
    nb = sum(_blocks(t) for t in lens) + 8
    ids = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32).tolist()
    width, rows, at = max(_blocks(t) for t in lens) + 3, [], 0
    for t in lens:
        rows.append(ids[at:at + _blocks(t)] + [-1] * (width - _blocks(t)))
        at += _blocks(t)
    return _ints(rows), nb


def _package():
    import paged_kv_cache_264_gb300
    return paged_kv_cache_264_gb300


def prepare(case, seed):
    gen = _gen(seed)
    c = dict(case)
    s = {"case": c}
    bf = dict(dtype=torch.bfloat16, device="cuda")
    if c["op"] == "gather":
        n, first = _gather_sizes(c)
        s["tables"], nb = _tables([a + b for a, b in zip(n, first)], gen)
        s.update(starts=_ints(_starts(n)), first=_ints(first), tokens=sum(n) + PAD, **_pool(nb, c["hkv"], c["d"], c["kv"], gen))
        shape = (sum(n) + PAD, c["hkv"], c["d"])
        s["k_out"], s["v_out"] = torch.zeros(shape, **bf), torch.zeros(shape, **bf)
        if own:
            s["pool"] = _package().PagedKVPool.from_tensors(s["k"], s["v"], s.get("k_scale"), s.get("v_scale"))
        return s
    new, before = _sizes(c)
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    n, lens = sum(new), [a + b for a, b in zip(new, before)]
    s.update(query_starts=_ints(_starts(new)), scale=d ** -0.5, max_context=max(lens))
    s["out"] = torch.zeros(n + PAD, hq, d, **bf)
    if c["op"] == "prompt":
        if c["before_hi"] == 0:  # q, k and v lie side by side in a projection's output
            x = torch.randn(n + PAD, hq + 2 * hkv, d, generator=gen, device="cuda")
            x[:, :hq] *= 1.5
            x[:, hq:hq + hkv] *= _channels(gen, d)
            x = x.to(torch.bfloat16)
            s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
            s["key_starts"] = None
        else:  # keys of earlier tokens were read back and lie in front of the new ones'
            s["q"] = (1.5 * torch.randn(n + PAD, hq, d, generator=gen, device="cuda")).to(torch.bfloat16)
            keys = torch.randn(sum(lens), hkv, d, generator=gen, device="cuda") * _channels(gen, d)
            s["k"] = keys.to(torch.bfloat16)
            s["v"] = torch.randn(sum(lens), hkv, d, generator=gen, device="cuda").to(torch.bfloat16)
            s["key_starts"] = _ints(_starts(lens))
        if own:
            # The layer's pool; the operator needs its heads and its device, not its blocks.
            s["pool"] = _package().PagedKVPool(8, hkv, d, "bf16")
            s["workspace"] = _workspace(s, c, s["k"].shape[0])
        return s
    s["q"] = (1.5 * torch.randn(n + PAD, hq, d, generator=gen, device="cuda")).to(torch.bfloat16)
    s["tables"], nb = _tables(lens, gen)
    s.update(lens=_ints(lens), **_pool(nb, hkv, d, c["kv"], gen))
    if own:
        s["pool"] = _package().PagedKVPool.from_tensors(s["k"], s["v"], s.get("k_scale"), s.get("v_scale"))
        s["workspace"] = _workspace(s, c, s["max_context"])
    return s


def _workspace(s, c, max_context):
    size = _package().prefill_workspace_bytes(s["pool"], c["seqs"], c["hq"], s["q"].shape[0], max_context)
    return torch.empty(size, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    if c["op"] == "gather":
        if own:
            _package().gather_cache(s["pool"], s["tables"], s["starts"], s["tokens"], first_positions=s["first"], k=s["k_out"],
                                    v=s["v_out"])
        else:
            _plain_gather(s)
        return {"k": s["k_out"], "v": s["v_out"]}
    if own:
        if c["op"] == "prompt":
            return _package().prompt_attention(s["pool"], s["q"], s["k"], s["v"], s["query_starts"], s["scale"],
                                               key_starts=s["key_starts"], causal=c["causal"], window=c["window"],
                                               out=s["out"], workspace=s["workspace"])
        return _package().paged_attention_prefill(s["pool"], s["q"], s["tables"], s["lens"], s["query_starts"], s["scale"],
                                                  s["max_context"], window=c["window"], out=s["out"],
                                                  workspace=s["workspace"])
    new, before = _sizes(c)
    at = key = 0
    for b, (n, earlier) in enumerate(zip(new, before)):
        t = n + earlier
        if n:
            if c["op"] == "prompt":
                k, v = s["k"][key:key + t].float().transpose(0, 1), s["v"][key:key + t].float().transpose(0, 1)
            else:
                k, v = (_rows(s, name, b, t) for name in ("k", "v"))
            _plain_attention(c, s["q"][at:at + n], k, v, s["scale"], s["out"][at:at + n])
        at += n
        key += t
    return s["out"]


def _rows(s, name, b, t):
    """fp32 rows of sequence b's first t tokens: [Hkv, t, d]."""
    blocks = s["tables"][b, :_blocks(t)].long()
    x = s[name][blocks]
    x = (x.view(torch.float8_e4m3fn) if s["case"]["kv"] == "fp8" else x).float()
    if s["case"]["kv"] != "bf16":
        x = x * s[name + "_scale"][blocks][..., None]
    return x.transpose(0, 1).flatten(1, 2)[:, :t]


def _plain_attention(c, q, k, v, scale, out):
    """q [n, Hq, d], k and v [Hkv, t, d]."""
    n, hq, d = q.shape
    hkv, t = k.shape[:2]
    rows = q.float().view(n, hkv, hq // hkv, d).permute(1, 2, 0, 3) * scale  # [Hkv, G, n, d]
    p = torch.arange(t - n, t, device=q.device)[:, None]
    col = torch.arange(t, device=q.device)
    seen = (col <= p) if c["causal"] else torch.ones(n, t, dtype=torch.bool, device=q.device)
    if c["window"]:
        seen = seen & (col > p - c["window"])
    heads = max(1, min(hkv, 2**30 // max(1, hq // hkv * n * t)))  # kv heads at a time, to bound the memory
    for h in range(0, hkv, heads):
        x = rows[h:h + heads].flatten(1, 2) @ k[h:h + heads].transpose(1, 2)
        x = x.view(-1, hq // hkv, n, t).masked_fill_(~seen, float("-inf"))
        x = x.sub_(x.amax(-1, keepdim=True).clamp_(min=-3e38)).exp_()
        total = x.sum(-1, keepdim=True)
        o = (x.flatten(1, 2) @ v[h:h + heads]).view(-1, hq // hkv, n, d)
        o = torch.where(total > 0, o / total, 0.0)
        g = hq // hkv
        out[:, h * g:(h + o.shape[0]) * g] = o.permute(2, 0, 1, 3).reshape(n, -1, d).to(torch.bfloat16)


def _plain_gather(s):
    c = s["case"]
    lens, first = _gather_sizes(c)
    n = sum(lens)
    starts = s["starts"]
    row = torch.arange(n, device=starts.device, dtype=torch.int32)
    b = torch.searchsorted(starts, row, right=True) - 1
    p = row - starts[b] + s["first"][b]
    block, at = s["tables"][b, (p // BLOCK).long()].long(), (p % BLOCK).long()
    for name in ("k", "v"):
        x = s[name][block, :, at]
        x = (x.view(torch.float8_e4m3fn) if c["kv"] == "fp8" else x).float()
        if c["kv"] != "bf16":
            x = x * s[name + "_scale"][block, :, at][..., None]
        s[name + "_out"][:n] = x.to(torch.bfloat16)


# ---------------------------------------------------------------- what a pass cannot do without

def _seen(c, n, t):
    """(pairs of a query and a token that it sees, tokens that some query sees) of one sequence."""
    w = c["window"] or 10**9
    if n == 0:
        return 0, 0
    if not c["causal"]:
        return n * t, t
    # query i sees min(w, t - n + i + 1) tokens
    full = max(0, min(n, t - w))  # the last queries, whose window is full
    part = n - full
    return part * (t - n + 1) + part * (part - 1) // 2 + full * w, min(t, w + n - 1)


def work(case):
    c = case
    if c["op"] == "gather":
        n = sum(_gather_sizes(c)[0])
        held = c["d"] * 2 if c["kv"] == "bf16" else c["d"] + 4
        return {"bytes": 2 * n * c["hkv"] * (held + 2 * c["d"]) + 4 * n // BLOCK, "flops": 0 if c["kv"] == "bf16" else 2 * n * c["hkv"] * c["d"]}
    new, before = _sizes(c)
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    both = [_seen(c, n, n + b) for n, b in zip(new, before)]
    row = 2 * hkv * (2 * d if c["kv"] == "bf16" else d + 4)
    tokens = sum(x[1] for x in both)
    return {"bytes": 4 * sum(new) * hq * d + row * tokens + (4 * tokens // BLOCK if c["op"] == "prefill" else 0),
            "flops": 4 * d * hq * sum(x[0] for x in both)}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "gather":
        return _exact_gather(s)
    new, before = _sizes(c)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    grp, at, key = c["hq"] // c["hkv"], 0, 0
    for b, (n, earlier) in enumerate(zip(new, before)):
        t = n + earlier
        for h in range(c["hkv"] if n else 0):
            if c["op"] == "prompt":
                k, v = s["k"][key:key + t, h].double(), s["v"][key:key + t, h].double()
            else:
                k, v = (_tokens64(s, name, b, 0, t, h) for name in ("k", "v"))
            for lo in range(0, n, 2048):
                hi = min(n, lo + 2048)
                end = t if not c["causal"] else earlier + hi  # tokens that one of these queries may see
                begin = 0 if not c["window"] else max(0, earlier + lo - c["window"] + 1)
                q = s["q"][at + lo:at + hi, h * grp:(h + 1) * grp].double()
                x = torch.einsum("igd,td->git", q, k[begin:end]) * s["scale"]
                away = (earlier + torch.arange(lo, hi, device="cuda"))[:, None] - torch.arange(begin, end, device="cuda")
                if c["causal"]:
                    x = torch.where(away >= 0, x, float("-inf"))
                if c["window"]:
                    x = torch.where(away < c["window"], x, float("-inf"))
                out[at + lo:at + hi, h * grp:(h + 1) * grp] = torch.einsum("git,td->igd", torch.softmax(x, -1), v[begin:end])
        at += n
        key += t
    return out


def _tokens64(s, name, b, first, last, h):
    """Tokens first .. last - 1 of sequence b, kv head h: [last - first, d]."""
    t = torch.arange(first, last, device="cuda")
    block = s["tables"][b].long()[t // BLOCK]
    x = s[name][block, h, t % BLOCK]
    if s["case"]["kv"] == "bf16":
        return x.double()
    x = (x.view(torch.float8_e4m3fn).float() if s["case"]["kv"] == "fp8" else x).double()
    return x * s[name + "_scale"][block, h, t % BLOCK].double()[:, None]


def _exact_gather(s):
    c = s["case"]
    out = {x: torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda") for x in ("k", "v")}
    at = 0
    for b, (n, first) in enumerate(zip(*_gather_sizes(c))):
        for name in ("k", "v") if n else ():
            for h in range(c["hkv"]):
                out[name][at:at + n, h] = _tokens64(s, name, b, first, first + n, h)
        at += n
    return out
