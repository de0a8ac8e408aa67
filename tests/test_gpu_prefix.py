"""shared_prefix_decode on the GPU against attention in 64 bits over the pool's own values.

Tolerance, before any run.  With w the softmax weights of a row, the output's rounding to bf16
moves it by at most 2^-8 |out|.  The weights enter the product over V in bf16: each moves by at
most 2^-8 of itself, numerator and denominator with it, so the output moves by at most
2^-8 (sum w |v| + |out|); INT8 and FP8 pools fold V's scale into the rounded weight, which the
same bound covers.  Logits are fp32 sums of up to 128 products (2^-24 times their absolute sum,
times log2 e and the scale), at most 2^-12 here, and move the output by as much of 2 sum w |v|."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build
from gpu_helpers import fill_pool_garbage

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


class Batch:
    """A batch of groups [(prefix tokens, [own tokens of each sequence])]; a prefix of None: the
    sequences are outside every group (between two groups: a group that shares nothing)."""

    def __init__(self, groups, hq, hkv, d, kv, k=1, seed=0, spare=3, q_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        inside = [i for i, (p, _) in enumerate(groups) if p is not None]
        groups = [(0 if p is None and inside and inside[0] < i < inside[-1] else p, own) for i, (p, own) in enumerate(groups)]
        self.hq, self.hkv, self.d, self.kv, self.k = hq, hkv, d, kv, k
        self.prefix = [p or 0 for p, own in groups for _ in own]
        self.own = [t for _, own in groups for t in own]
        self.b = len(self.own)
        nb = sum((p or 0) // 16 for p, _ in groups) + sum((t + 15) // 16 for t in self.own) + spare
        ids = torch.randperm(nb, generator=g).tolist()
        width = max((p + t + 15) // 16 for p, t in zip(self.prefix, self.own)) + 2
        rows, starts, lens, at, b = [], [], [], 0, 0
        for p, own in groups:
            shared = ids[at:at + (p or 0) // 16]
            at += len(shared)
            if p is not None:
                starts.append(b)
                lens.append(p)
            for t in own:
                n = (t + 15) // 16
                row = shared + ids[at:at + n]
                at += n
                rows.append(row + [10 ** 6] * (width - len(row)))  # entries past the end hold anything
                b += 1
            if p is not None:
                end = b
        self.starts = torch.tensor(starts + [end] if starts else [0], dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.tables = torch.tensor(rows, dtype=torch.int32, device="cuda")
        self.context = torch.tensor([p + t for p, t in zip(self.prefix, self.own)], dtype=torch.int32, device="cuda")
        self.max_prefix, self.max_own = max(lens + [0]), max(self.own + [1])
        self.pool = pkv.PagedKVPool(nb, hkv, d, kv)
        fill_pool_garbage(self.pool)
        gen = torch.Generator(device="cuda").manual_seed(seed + 1)
        slots = sorted({rows[b][t // 16] * 16 + t % 16 for b in range(self.b) for t in range(self.prefix[b] + self.own[b])})
        slots = torch.tensor(slots, dtype=torch.int32, device="cuda")
        if slots.numel():
            kv_new = torch.randn(2, slots.numel(), hkv, d, generator=gen, device="cuda").to(torch.bfloat16)
            kv_new[1] += 0.25
            self.pool.reshape_and_cache(kv_new[0].contiguous(), kv_new[1].contiguous(), slots)
        shape = (self.b, hq, d) if k == 1 else (self.b, k, hq, d)
        self.q = (q_scale * torch.randn(shape, generator=gen, device="cuda")).to(torch.bfloat16)
        self.scale = d ** -0.5

    def run(self, **kw):
        args = dict(q=self.q, block_tables=self.tables, context_lens=self.context, group_starts=self.starts,
                    prefix_lens=self.lens, scale=self.scale, max_prefix_len=self.max_prefix, max_suffix_len=self.max_own)
        return pkv.shared_prefix_decode(self.pool, **(args | kw))

    def values(self, name, b, t):
        """K or V of tokens 0 .. t - 1 of sequence b, [Hkv, t, d] in 64 bits."""
        blocks = self.tables[b, :(t + 15) // 16].long()
        x = (self.pool.k_cache if name == "k" else self.pool.v_cache)[blocks]
        x = (x.view(torch.float8_e4m3fn).float() if self.kv == "fp8" else x).double()
        if self.kv != "bf16":
            x = x * (self.pool.k_scale if name == "k" else self.pool.v_scale)[blocks].double()[..., None]
        return x.transpose(0, 1).flatten(1, 2)[:, :t]

    def reference(self, b, drop=()):
        """(output, sum w |v|) of sequence b in 64 bits, [k, Hq, d]; tokens in `drop` are not seen."""
        t = self.prefix[b] + self.own[b]
        k, v = self.values("k", b, t), self.values("v", b, t)
        q = self.q[b].double().view(self.k, self.hkv, self.hq // self.hkv, self.d)
        x = torch.einsum("ihgd,htd->ihgt", q, k) * self.scale
        seen = torch.arange(t, device="cuda") < (t - (self.k - 1 - torch.arange(self.k, device="cuda")))[:, None]
        if len(drop):
            seen[:, torch.tensor(drop, device="cuda")] = False
        w = torch.softmax(x.masked_fill(~seen[:, None, None], float("-inf")), -1)
        w, v = w.masked_fill(~seen[:, None, None], 0), torch.where(seen.any(0)[:, None], v, 0)
        out = torch.einsum("ihgt,htd->ihgd", w, v), torch.einsum("ihgt,htd->ihgd", w, v.abs())
        return tuple(o.reshape(self.k, self.hq, self.d) for o in out)

    def check(self, out, seqs=None, drop=()):
        for b in range(self.b) if seqs is None else seqs:
            ref, wv = self.reference(b, drop)
            got = out[b].double().view(ref.shape)
            tol = 2.0 ** -8 * (2 * ref.abs() + wv) + 2.0 ** -11 * wv
            err = (got - ref).abs()
            assert (err <= tol).all(), (b, err.max().item(), (err / tol).max().item(), got.isnan().sum().item())


GROUPS = {
    "one tile": [(128, [5, 1, 16, 40])],
    "one block": [(16, [1, 3])],
    "one sequence": [(272, [33])],
    "tail of a tile": [(144, [7, 9, 200]), (112, [20, 1])],
    "no own tokens": [(256, [0, 17, 0])],
    "mixed": [(None, [30, 700]), (2048, [1, 64, 65]), (0, [40, 50]), (528, [9]), (None, [1, 300])],
    "many rows": [(400, [1 + 3 * i for i in range(37)])],        # GQA of 8: 296 rows, two units
    "many small groups": [(16 * (1 + i % 9), [1 + i % 5] * (1 + i % 3)) for i in range(40)],
    "long": [(9008, [10, 20, 31])],
    "no group": [(None, [17, 80, 333])],
}


@pytest.mark.parametrize("name", sorted(GROUPS))
@pytest.mark.parametrize("hq,hkv,d,kv,k", [
    (8, 2, 128, "bf16", 1), (16, 2, 64, "bf16", 1), (6, 6, 128, "bf16", 1), (16, 2, 128, "int8", 1), (9, 3, 64, "int8", 1),
    (8, 1, 128, "fp8", 1), (16, 4, 64, "fp8", 1),
])
def test_groups(name, hq, hkv, d, kv, k):
    x = Batch(GROUPS[name], hq, hkv, d, kv, k, seed=len(name))
    out = x.run()
    assert x.pool.device_error() == 0
    x.check(out)
    x.pool.close()


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("int8", 128), ("fp8", 64)])
@pytest.mark.parametrize("hq,hkv,k", [(8, 2, 4), (4, 4, 2), (12, 4, 5), (32, 1, 16)])
def test_several_queries(kv, d, hq, hkv, k):
    """k draft tokens per sequence; the shortest own part leaves the first query the prefix only."""
    x = Batch([(192, [k - 1, k, 16, 17 + k]), (None, [k, 60]), (0, [k, 33])][:: 1 if hkv < 4 else 2], hq, hkv, d, kv, k, seed=k)
    out = x.run()
    assert x.pool.device_error() == 0
    x.check(out)
    x.pool.close()


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("n,hq,hkv", [(3, 128, 4), (4, 128, 4), (5, 128, 4), (8, 128, 4), (9, 128, 4), (33, 32, 2)])
def test_row_counts_around_the_tiles(kv, n, hq, hkv):
    """96, 128, 160, 256, 288 and 528 query rows per kv head."""
    x = Batch([(1600, [1 + i for i in range(n)])], hq, hkv, 128, kv, seed=n)
    out = x.run()
    assert x.pool.device_error() == 0
    x.check(out)
    x.pool.close()


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
def test_sharp_softmax_and_rising_logits(kv):
    """Large queries: the running maximum moves late and far, and most weights vanish."""
    x = Batch([(1040, [20, 300, 3])], 16, 2, 128, kv, seed=5, q_scale=30.0)
    x.check(x.run())
    # the last prefix tokens hold the largest logits of every row
    y = Batch([(1040, [20, 300, 3])], 16, 2, 128, kv, seed=6)
    blocks = y.tables[0, 60:65].long()
    n = 5 * 16
    key = 6.0 * y.q.float().mean((0, 1)).sign().expand(n, 2, 128).to(torch.bfloat16).contiguous()
    slots = (blocks[:, None] * 16 + torch.arange(16, device="cuda")).flatten().to(torch.int32)
    value = torch.randn(n, 2, 128, device="cuda").to(torch.bfloat16)
    y.pool.reshape_and_cache(key, value, slots)
    y.check(y.run())
    assert x.pool.device_error() == 0 and y.pool.device_error() == 0
    x.pool.close()
    y.pool.close()


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_same_as_decode_and_any_workspace(kv):
    x = Batch([(1024, [50, 3, 200, 9, 17]), (320, [5, 90])], 32, 8, 128, kv, seed=9)
    need = pkv.shared_prefix_workspace_bytes(x.pool, x.b, 32, 2, x.max_prefix, x.max_own)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten
    out = x.run(workspace=ws)
    x.check(out)
    ws.fill_(255)
    assert torch.equal(x.run(workspace=ws), out)                     # and the same to the bit every time
    into = torch.empty_like(out)
    assert x.run(out=into, workspace=ws) is into and torch.equal(into, out)
    whole = x.pool.decode(x.q, x.tables, x.context, x.scale, int(x.context.max()))
    for b in range(x.b):
        ref, wv = x.reference(b)
        # both sides are within the tolerance of the module's head
        assert ((whole[b].double() - out[b].double()).abs() <= 2 * (2.0 ** -8 * (2 * ref[0].abs() + wv[0]) + 2.0 ** -11 * wv[0])).all()
    # generous bounds and an explicit partition change the plan, not the result
    x.check(x.run(max_prefix_len=1024 + 160, max_suffix_len=900, partition_blocks=2))
    assert x.pool.device_error() == 0
    x.pool.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_bad_blocks_are_skipped(kv):
    x = Batch([(320, [40, 1])], 8, 2, 128, kv, seed=3)
    good = x.tables.clone()
    x.tables[0, 7] = -1
    x.tables[0, 11] = x.pool.num_blocks
    x.tables[1, 3] = -5  # another sequence's entry for the prefix is not read
    out = x.run()
    assert x.pool.device_error() == pkv.DEVERR_BLOCK_ID
    x.tables = good
    x.check(out, drop=list(range(112, 128)) + list(range(176, 192)))
    # a whole tile, and a whole prefix
    x.tables = good.clone()
    x.tables[0, 8:16] = 2 ** 31 - 1
    out = x.run()
    assert x.pool.device_error() == pkv.DEVERR_BLOCK_ID
    x.tables = good
    x.check(out, drop=list(range(128, 256)))
    x.tables = good.clone()
    x.tables[0, :20] = -1
    out = x.run()
    assert x.pool.device_error() == pkv.DEVERR_BLOCK_ID
    x.tables = good
    x.check(out, drop=list(range(320)))
    x.pool.close()


def test_bad_lengths_and_groups():
    x = Batch([(160, [40, 1, 30]), (48, [9, 9])], 8, 2, 128, "bf16", seed=4)
    ref = x.run()
    ctx = x.context.clone()
    for b, t in ((1, 159), (3, 0), (0, 160 + 41), (4, -3)):  # shorter than the prefix, empty, past max_suffix_len
        x.context = ctx.clone()
        x.context[b] = t
        out = x.run()
        assert x.pool.device_error() == pkv.DEVERR_CONTEXT_LEN
        assert (out[b] == 0).all()
        rest = [i for i in range(5) if i != b]
        assert torch.equal(out[rest], ref[rest])
    x.context = ctx
    starts, lens = x.starts.clone(), x.lens.clone()
    for s, n in (([0, 3, 6], [160, 48]), ([0, 4, 3], [160, 48]), ([-1, 3, 5], [160, 48]), ([0, 3, 5], [161, 48]),
                 ([0, 3, 5], [176, 48]), ([0, 3, 5], [160, -16])):
        out = x.run(group_starts=torch.tensor(s, dtype=torch.int32, device="cuda"),
                    prefix_lens=torch.tensor(n, dtype=torch.int32, device="cuda"))
        assert x.pool.device_error() == pkv.DEVERR_PREFIX | pkv.DEVERR_CONTEXT_LEN
        assert (out == 0).all()
    assert torch.equal(x.run(group_starts=starts, prefix_lens=lens), ref) and x.pool.device_error() == 0
    # empty groups, and one that covers nothing
    out = x.run(group_starts=torch.tensor([0, 0, 3, 3, 5, 5], dtype=torch.int32, device="cuda"),
                prefix_lens=torch.tensor([16, 160, 0, 48, 32], dtype=torch.int32, device="cuda"))
    x.check(out)
    assert x.pool.device_error() == 0
    x.pool.close()


def test_nan_reaches_only_the_rows_that_see_it():
    x = Batch([(160, [40, 1]), (48, [9, 9])], 8, 2, 128, "bf16", seed=4)
    ref = x.run().clone()
    x.pool.v_cache[x.tables[0, 3].long(), 1, 5, 7] = float("nan")  # prefix of the first group, kv head 1
    out = x.run()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[:2, 4:, 7] = True
    # a NaN in V poisons its own value of every head that sees it
    assert out[hit].isnan().all() or (out[hit] == 0).all()
    assert torch.equal(out[~hit], ref[~hit])
    x.pool.close()


def test_captured_and_replayed_with_other_groups():
    """Groups, lengths and tables live on the device: one capture serves them all."""
    one = Batch([(512, [30, 2, 64, 7, 90, 1])], 16, 4, 128, "bf16", seed=1)
    tables, context = one.tables.clone(), one.context.clone()
    starts, lens = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    starts[1:] = 6
    lens[0] = 512
    out = torch.empty_like(one.q)
    ws = torch.empty(pkv.shared_prefix_workspace_bytes(one.pool, 6, 16, 3, 512, 602), dtype=torch.uint8, device="cuda")

    def call():
        pkv.shared_prefix_decode(one.pool, one.q, tables, context, starts, lens, one.scale, 512, 602, out=out, workspace=ws)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call()
    for s, n in (([0, 6, 6, 6], [512, 0, 0]), ([0, 2, 5, 6], [512, 256, 0]), ([0, 0, 3, 6], [0, 16, 496]), ([2, 2, 2, 2], [0, 0, 0])):
        starts.copy_(torch.tensor(s, dtype=torch.int32))
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert one.pool.device_error() == 0
        one.check(out)  # however it is divided, the attention is the same
    one.pool.close()


def test_refusals():
    x = Batch([(160, [40, 1])], 8, 2, 128, "bf16", seed=4)
    before = pkv.launch_count()
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    for bad in (dict(group_starts=x.starts[:1]), dict(prefix_lens=x.lens.cpu()), dict(context_lens=x.context[:1]),
                dict(q=x.q[..., :64].contiguous()), dict(out=x.q[:1])):
        with pytest.raises(ValueError):
            x.run(**bad)
    with pytest.raises(TypeError):
        x.run(prefix_lens=x.lens.long())
    many = torch.zeros(4098, dtype=torch.int32, device="cuda")
    for bad in (dict(workspace=small), dict(max_prefix_len=-1), dict(max_suffix_len=0), dict(max_prefix_len=10 ** 5),
                dict(max_suffix_len=10 ** 5), dict(scale=float("nan")), dict(group_starts=many, prefix_lens=many[1:]),
                dict(q=x.q[:, :7].contiguous())):
        with pytest.raises(pkv.PagedKVError):
            x.run(**bad)
    assert pkv.launch_count() == before
    assert x.run(q=x.q[:0], block_tables=x.tables[:0], context_lens=x.context[:0]).shape == (0, 8, 128)
    x.pool.close()
