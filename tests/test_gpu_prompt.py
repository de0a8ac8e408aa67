"""paged_attention_prefill and prompt_attention on the GPU against 64-bit torch (prompt_reference.py
derives the tolerance)."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from gpu_helpers import fill_pool_garbage
from paged_kv_cache_264_gb300 import build
from prompt_reference import attend, cached, check, ints, starts_of, tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def make_cache(gen, lens, hkv, d, kv, extra_blocks=3):
    """A pool whose slots hold garbage but for the sequences' tokens, and their block tables."""
    need = [(t + 15) // 16 for t in lens]
    nb = sum(need) + extra_blocks
    ids = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32)
    tables = torch.full((len(lens), max(need + [1]) + 2), -1, dtype=torch.int32, device="cuda")
    slots, at = [], 0
    for b, t in enumerate(lens):
        mine = ids[at:at + need[b]]
        tables[b, :need[b]] = mine
        pos = torch.arange(t, device="cuda")
        slots.append(mine[pos // 16] * 16 + pos.int() % 16 if t else mine[:0])
        at += need[b]
    pool = pkv.PagedKVPool(nb, hkv, d, kv)
    fill_pool_garbage(pool)
    n = sum(lens)
    if n:
        k, v = (_randn(gen, n, hkv, d).to(torch.bfloat16) for _ in range(2))
        pool.reshape_and_cache(k, v, torch.cat(slots).to(torch.int32))
    return pool, tables


def check_prefill(pool, tables, q, out, new, lens, scale, window, what):
    at = 0
    for b, (n, t) in enumerate(zip(new, lens)):
        if n:
            k, v, missing = cached(pool, tables[b], t)
            ref = attend(q[at:at + n].double(), k, v, scale, window, missing=missing)
            check(out[at:at + n], *ref, t, (what, b, n, t), pool.dtype != "bf16")
        at += n


def run_prefill(seed, new, before, hq, hkv, d, kv, window=0, scale=None, pad=3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens = [a + b for a, b in zip(new, before)]
    pool, tables = make_cache(gen, lens, hkv, d, kv)
    n = sum(new)
    q = (1.5 * _randn(gen, n + pad, hq, d)).to(torch.bfloat16)
    q[n:] = float("nan")
    out = torch.full_like(q, 7.0)
    scale = d ** -0.5 if scale is None else scale
    got = pool.prefill(q, tables, ints(lens), starts_of(new), scale, max(lens), window=window, out=out)
    torch.cuda.synchronize()
    assert got is out and pool.device_error() == 0
    check_prefill(pool, tables, q, out, new, lens, scale, window, (new, before, hq, hkv, d, kv, window))
    assert (out[n:] == 7.0).all()  # rows behind the last sequence
    pool.close()


HEADS = [(4, 4, 128), (8, 2, 64), (7, 1, 128), (12, 4, 64), (28, 4, 128), (71, 1, 64), (160, 1, 64)]


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_prefill_heads(hq, hkv, d, kv):
    run_prefill(hq + d, [1, 5, 0, 40, 130, 17], [0, 30, 9, 111, 3, 200], hq, hkv, d, kv)


SIZES = [
    ([1], [0]), ([2], [126]), ([1], [127]), ([1], [128]), ([129], [0]), ([257], [1]), ([300, 1, 1, 64], [0, 500, 16, 63]),
    ([15, 16, 17, 31, 32, 33], [1, 0, 15, 16, 17, 112]), ([600], [700]), ([24], [4000]), ([1] * 40, list(range(0, 1200, 30))),
]


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("new,before", SIZES)
def test_prefill_sizes(new, before, kv):
    run_prefill(len(new) + new[0], new, before, 8, 2, 128, kv)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 128, 129, 500, 5000])
def test_prefill_windows(window, kv):
    run_prefill(window, [1, 70, 300, 5], [900, 0, 200, 1000], 8, 4, 64, kv, window=window)


@pytest.mark.parametrize("scale", [0.0, -0.125, 1e-3, 2.0])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_scales(scale, d):
    run_prefill(3, [50, 7], [100, 33], 4, 2, d, "bf16", scale=scale)
    run_prefill(4, [50, 7], [100, 33], 4, 2, d, "int8", scale=scale)


def test_prefill_released_blocks_behind_a_window():
    """Blocks before every query's window may be -1, and what lies before the window in its first block NaN."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    new, lens, w = [20, 1, 300], [700, 555, 900], 130
    pool, tables = make_cache(gen, lens, 2, 128, "bf16")
    q = _randn(gen, sum(new), 8, 128).to(torch.bfloat16)
    clean = [cached(pool, tables[b], t) for b, t in enumerate(lens)]
    for b, (n, t) in enumerate(zip(new, lens)):
        first = t - n - w + 1  # the first token that any query sees
        for pos in range(first // 16 * 16, first):
            pool.k_cache[tables[b, pos // 16], :, pos % 16] = float("nan")
            pool.v_cache[tables[b, pos // 16], :, pos % 16] = float("inf")
        tables[b, :first // 16] = -1
    out = pool.prefill(q, tables, ints(lens), starts_of(new), 0.1, max(lens), window=w)
    torch.cuda.synchronize()
    assert pool.device_error() == 0
    at = 0
    for (n, t), (k, v, _) in zip(zip(new, lens), clean):
        check(out[at:at + n], *attend(q[at:at + n].double(), k, v, 0.1, w), t, (n, t))
        at += n
    pool.close()


@pytest.mark.parametrize("hq,hkv,d,kv", [(4, 4, 128, "bf16"), (16, 1, 64, "bf16"), (8, 2, 128, "int8"), (4, 1, 64, "fp8")])
def test_prefill_long_contexts_are_cut_and_joined(hq, hkv, d, kv):
    """Few rows behind long contexts: the pieces' states, several for a row."""
    run_prefill(11, [3, 30, 1], [20000, 9000, 40], hq, hkv, d, kv)


def test_prefill_growing_logits():
    """Logits that pass the running maximum again and again, tile after tile, and rows of them apart."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    t, n, d = 1500, 200, 64
    pool, tables = make_cache(gen, [t], 1, d, "bf16")
    k = torch.zeros(t, 1, d, device="cuda")
    k[:, 0, 0] = torch.arange(t, device="cuda") / 16
    k[:, 0, 1] = -torch.arange(t, device="cuda") / 16
    v = _randn(gen, t, 1, d)
    pos = torch.arange(t, device="cuda")
    pool.reshape_and_cache(k.to(torch.bfloat16), v.to(torch.bfloat16), (tables[0, pos // 16] * 16 + pos % 16).to(torch.int32))
    q = torch.zeros(n, 4, d, device="cuda")
    q[::2, :, 0] = 1.0
    q[1::2, :, 1] = 1.0
    q[:, 3] = 0.0
    q = q.to(torch.bfloat16)
    out = pool.prefill(q, tables, ints([t]), starts_of([n]), 1.0, t)
    check_prefill(pool, tables, q, out, [n], [t], 1.0, 0, "growing")
    pool.close()


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("jump", [3.0, 40.0, 300.0, 20000.0])
def test_prefill_jumping_logits(jump, kv):
    """Logits that jump by any amount at any column: within a tile, between its halves, after thousands."""
    gen = torch.Generator(device="cuda").manual_seed(int(jump))
    t, n, d = 1100, 70, 64
    pool, tables = make_cache(gen, [t], 1, d, kv)
    k = 0.05 * _randn(gen, t, 1, d)
    k[:, 0, 0] = 0
    at = [3, 70, 130, 200, 270, 700, 701, 1000]  # tokens whose logit is a jump above all before
    for i, pos in enumerate(at):
        k[pos, 0, 0] = (i + 1) * jump
    v = _randn(gen, t, 1, d)
    pos = torch.arange(t, device="cuda")
    pool.reshape_and_cache(k.to(torch.bfloat16), v.to(torch.bfloat16), (tables[0, pos // 16] * 16 + pos % 16).to(torch.int32))
    q = _randn(gen, n, 4, d)
    q[:, :, 0] = torch.tensor([1.0, -1.0, 0.0, 0.125], device="cuda")
    q = q.to(torch.bfloat16)
    out = pool.prefill(q, tables, ints([t]), starts_of([n]), 1.0, t)
    check_prefill(pool, tables, q, out, [n], [t], 1.0, 0, ("jump", jump, kv))
    out = pool.prefill(q, tables, ints([300]), starts_of([n]), -1.0, t)
    check_prefill(pool, tables, q, out, [n], [300], -1.0, 0, ("jump", jump, kv))
    pool.close()


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
def test_prefill_values_of_any_size(kv):
    """Values whose sizes differ from token to token by any factor, zeros among them: a row's large values must not
    cost the small ones their weights where these are what a query sees."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    t, n, hkv, d = 700, 90, 2, 64
    pool, tables = make_cache(gen, [t], hkv, d, kv)
    k = _randn(gen, t, hkv, d)
    size = torch.exp2(torch.randint(-60, 60, (t, hkv, 1), generator=gen, device="cuda").float())
    v = _randn(gen, t, hkv, d) * size
    v[::7] = 0
    v[300:400] = 0
    pos = torch.arange(t, device="cuda")
    pool.reshape_and_cache(k.to(torch.bfloat16), v.to(torch.bfloat16), (tables[0, pos // 16] * 16 + pos % 16).to(torch.int32))
    q = (3 * _randn(gen, n, 4, d)).to(torch.bfloat16)
    for window in (0, 1, 20, 100):
        out = pool.prefill(q, tables, ints([t]), starts_of([n]), 0.125, t, window=window)
        check_prefill(pool, tables, q, out, [n], [t], 0.125, window, (kv, window))
    for seen in (95, 400):  # the last of it: values of zero alone, behind large logits too
        out = pool.prefill(q, tables, ints([seen]), starts_of([n]), 8.0, t, window=30)
        check_prefill(pool, tables, q, out, [n], [seen], 8.0, 30, (kv, seen))
    pool.close()


@pytest.mark.parametrize("t,tiny", [(700, 400), (700, 700), (6000, 3000)])
@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
def test_prefill_smallest_values_ahead_of_others(kv, t, tiny):
    """The smallest values that there are, a tile of them and more, must not cost the ones behind them their weights.
    Over codes V's scales count as at least 2^-98: a value of such a row moves by at most 448 * 2^-98 < 2^-89."""
    gen = torch.Generator(device="cuda").manual_seed(12)
    n, hkv, d = 40, 2, 128
    pool, tables = make_cache(gen, [t], hkv, d, kv)
    k, v = _randn(gen, t, hkv, d), _randn(gen, t, hkv, d)
    v[:tiny] *= torch.exp2(torch.randint(-124, -90, (tiny, hkv, 1), generator=gen, device="cuda").float())
    pos = torch.arange(t, device="cuda")
    pool.reshape_and_cache(k.to(torch.bfloat16), v.to(torch.bfloat16), (tables[0, pos // 16] * 16 + pos % 16).to(torch.int32))
    q = _randn(gen, n, 8, d).to(torch.bfloat16)
    out = pool.prefill(q, tables, ints([t]), starts_of([n]), 0.125, t)
    kc, vc, _ = cached(pool, tables[0], t)
    ref = attend(q.double(), kc, vc, 0.125)
    tol = tolerance(*ref, t, d, kv != "bf16") + 2.0 ** -89
    assert ((out.double() - ref[0]).abs() <= tol).all()
    pool.close()


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
def test_blocks_behind_two_to_the_31_elements(kv):
    gen = torch.Generator(device="cuda").manual_seed(13)
    t, n, hkv, d, blocks = 200, 9, 16, 128, 70000
    assert (blocks - 20) * 16 * hkv * d > 2 ** 31
    pool = pkv.PagedKVPool(blocks, hkv, d, kv)
    tables = (blocks - 1 - torch.randperm(13, generator=gen, device="cuda")).to(torch.int32)[None]
    k, v = (_randn(gen, t, hkv, d).to(torch.bfloat16) for _ in range(2))
    pos = torch.arange(t, device="cuda")
    pool.reshape_and_cache(k, v, (tables[0, pos // 16] * 16 + pos % 16).to(torch.int32))
    q = _randn(gen, n, 32, d).to(torch.bfloat16)
    wide = torch.cat([tables, torch.full((1, 400), -1, dtype=torch.int32, device="cuda")], 1)
    for most in (t, 5000):
        out = pool.prefill(q, wide, ints([t]), starts_of([n]), d ** -0.5, most)
        check_prefill(pool, tables, q, out, [n], [t], d ** -0.5, 0, (kv, most))
    for got, ref in zip(pool.gather_cache(tables, starts_of([t]), t), cached(pool, tables[0], t)):
        # over codes a product rounded to fp32 and to bf16
        assert ((got.double() - ref).abs() <= (0 if kv == "bf16" else 2.0 ** -8 + 2.0 ** -23) * ref.abs()).all()
    assert pool.device_error() == 0
    pool.close()


def test_prefill_matches_decode_for_single_tokens():
    gen = torch.Generator(device="cuda").manual_seed(6)
    lens = [1, 17, 200, 1025, 3000]
    pool, tables = make_cache(gen, lens, 8, 128, "int8")
    q = _randn(gen, 5, 32, 128).to(torch.bfloat16)
    out = pool.prefill(q, tables, ints(lens), starts_of([1] * 5), 128 ** -0.5, 3000)
    check_prefill(pool, tables, q, out, [1] * 5, lens, 128 ** -0.5, 0, "single")
    # the decode rounds its weights to 16 bits too, and its output: both are within the tolerance of the formula
    other = pool.decode(q, tables, ints(lens), 128 ** -0.5, 3000)
    for b, t in enumerate(lens):
        k, v, _ = cached(pool, tables[b], t)
        tol = 2 * tolerance(*attend(q[b:b + 1].double(), k, v, 128 ** -0.5), t, 128, True)
        assert not ((out[b].double() - other[b].double()).abs() > tol).any(), t
    pool.close()


@pytest.mark.parametrize("most", [300, 5000])  # short calls run without a plan
@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_prefill_bad_lengths_and_blocks(kv, most):
    gen = torch.Generator(device="cuda").manual_seed(7)
    new, lens = [10, 4, 6, 0, 30], [100, 40, 50, 33, 300]
    pool, tables = make_cache(gen, lens, 2, 64, kv)
    tables = torch.cat([tables, torch.full((5, 400), -1, dtype=torch.int32, device="cuda")], 1)
    q = _randn(gen, sum(new), 4, 64).to(torch.bfloat16)
    qs = starts_of(new)
    # lengths: fewer tokens than queries, more than max_context_len, negative for a sequence without queries
    given = [100, 3, most + 1, -5, 300]
    out = torch.full_like(q, 7.0)
    pool.prefill(q, tables, ints(given), qs, 0.125, most, out=out)
    assert pool.device_error() == pkv.DEVERR_CONTEXT_LEN
    assert (out[10:20] == 0).all()
    check_prefill(pool, tables, q[:10], out[:10], [10], [100], 0.125, 0, "good one")
    check_prefill(pool, tables[4:], q[20:], out[20:], [30], [300], 0.125, 0, "last one")
    # blocks that are not there
    tables[0, 2] = -1
    tables[4, 18] = pool.num_blocks  # the last, partly filled one
    tables[4, 0] = 2 ** 31 - 1
    out.fill_(7.0)
    pool.prefill(q, tables, ints(lens), qs, 0.125, most, out=out)
    assert pool.device_error() == pkv.DEVERR_BLOCK_ID
    check_prefill(pool, tables, q, out, new, lens, 0.125, 0, "missing blocks")
    # all of a sequence's blocks missing: nothing to see
    tables[1] = -1
    pool.prefill(q, tables, ints(lens), qs, 0.125, most, out=out)
    assert pool.device_error() == pkv.DEVERR_BLOCK_ID
    assert (out[10:14] == 0).all()
    pool.close()


@pytest.mark.parametrize("most", [20, 5000])
@pytest.mark.parametrize("starts", [[0, 4, 3, 12], [-1, 4, 8, 12], [0, 4, 8, 13], [0, 2 ** 31 - 1, 8, 12]])
def test_invalid_starts_write_nothing(starts, most):
    gen = torch.Generator(device="cuda").manual_seed(8)
    pool, tables = make_cache(gen, [20, 20, 20], 2, 64, "bf16")
    wide = torch.cat([tables, torch.full((3, 400), -1, dtype=torch.int32, device="cuda")], 1)
    x = _randn(gen, max(12, most), 4, 64).to(torch.bfloat16)
    out = torch.full_like(x, 7.0)
    bad = ints([s if s != 13 else max(13, most + 1) for s in starts])
    pool.prefill(x, wide, ints([20] * 3), bad, 0.125, most, out=out)
    assert pool.device_error() == pkv.DEVERR_QUERY
    pool.prompt_attention(x, x[:, :2], x[:, 2:], bad, 0.125, out=out)
    assert pool.device_error() == pkv.DEVERR_QUERY
    pool.prompt_attention(x, x[:, :2], x[:, 2:], starts_of([4, 4, 4]), 0.125, key_starts=bad, out=out)
    assert pool.device_error() == pkv.DEVERR_QUERY
    assert (out == 7.0).all()
    k, v = torch.full_like(x[:, :2].contiguous(), 7.0), torch.full_like(x[:, :2].contiguous(), 7.0)
    pool.gather_cache(tables, bad, x.shape[0], k=k, v=v)
    assert pool.device_error() == pkv.DEVERR_QUERY
    assert (k == 7.0).all() and (v == 7.0).all()
    pool.close()


# ---------------------------------------------------------------- packed keys and values

def run_prompt(seed, new, keys, hq, hkv, d, causal=True, window=0, scale=None, pad=3, fused=True):
    """keys None: the queries' own."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pool = pkv.PagedKVPool(2, hkv, d, "int8")  # its type does not matter
    n = sum(new)
    own = keys is None
    m = n if own else sum(keys)
    if own and fused:
        x = _randn(gen, n + pad, hq + 2 * hkv, d).to(torch.bfloat16)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        q, k, v = (_randn(gen, r + pad, h, d).to(torch.bfloat16) for r, h in ((n, hq), (m, hkv), (m, hkv)))
    q[n:] = float("nan")
    k[m:] = float("nan")
    v[m:] = float("inf")
    scale = d ** -0.5 if scale is None else scale
    out = torch.full((n + pad, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    keys = new if own else keys
    pool.prompt_attention(q, k, v, starts_of(new), scale, key_starts=None if own else starts_of(keys), causal=causal,
                          window=window, out=out)
    torch.cuda.synchronize()
    assert pool.device_error() == 0
    at = key = 0
    for nb, t in zip(new, keys):
        ref = attend(q[at:at + nb].double(), k[key:key + t].double(), v[key:key + t].double(), scale, window, causal)
        check(out[at:at + nb], *ref, t, (new, keys, hq, hkv, d, causal, window, nb, t))
        at, key = at + nb, key + t
    assert (out[n:] == 7.0).all()
    pool.close()


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_heads(hq, hkv, d, causal):
    run_prompt(hq + d, [1, 5, 0, 40, 130, 17, 300], None, hq, hkv, d, causal=causal)


@pytest.mark.parametrize("new", [[1], [16], [127], [128], [129], [256], [1000], [2049, 3, 70], [7] * 50, [0, 0, 5, 0]])
def test_prompt_sizes(new):
    run_prompt(len(new) + new[0], new, None, 8, 2, 128)
    run_prompt(len(new) + new[0], new, None, 4, 4, 64, causal=False, fused=False)


@pytest.mark.parametrize("window", [1, 17, 64, 128, 300, 2000])
def test_prompt_windows(window):
    run_prompt(window, [1, 200, 700], None, 8, 2, 128, window=window)
    run_prompt(window, [1, 200, 700], [50, 900, 701], 14, 2, 64, window=window)


@pytest.mark.parametrize("causal", [True, False])
def test_prompt_keys_of_their_own(causal):
    """More keys than queries, fewer (the first queries see nothing), none, and the other way round."""
    run_prompt(9, [5, 200, 40, 0, 7, 300], [100, 20, 0, 50, 7, 1111], 8, 2, 128, causal=causal)
    run_prompt(10, [1, 1, 1], [5000, 1, 129], 4, 4, 64, causal=causal)
    run_prompt(10, [3], [0], 4, 4, 64, causal=causal)


def test_prompt_long_keys_are_cut_and_joined():
    run_prompt(12, [20, 1], [9000, 17000], 4, 2, 128)
    run_prompt(13, [20, 1], [9000, 17000], 4, 2, 64, causal=False)
    run_prompt(14, [20, 1], [9000, 17000], 4, 2, 64, window=8000)


def test_prompt_neighbours_do_not_reach_one_another():
    """NaN and infinite keys and values of one sequence stay in it."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    pool = pkv.PagedKVPool(2, 2, 64, "bf16")
    new = [37, 20, 150]
    x = _randn(gen, sum(new), 8, 64).to(torch.bfloat16)
    x[37:57, 4:6] = float("nan")
    x[37:57, 6:] = float("inf")
    out = pool.prompt_attention(x[:, :4], x[:, 4:6], x[:, 6:], starts_of(new), 0.125)
    for lo, hi in ((0, 37), (57, 207)):
        ref = attend(x[lo:hi, :4].double(), x[lo:hi, 4:6].double(), x[lo:hi, 6:].double(), 0.125)
        check(out[lo:hi], *ref, 150, lo)
    assert out[37:57].isnan().all()
    # and a row's own NaN query stays in its row
    x = _randn(gen, sum(new), 8, 64).to(torch.bfloat16)
    x[60, 1] = float("nan")
    out = pool.prompt_attention(x[:, :4], x[:, 4:6], x[:, 6:], starts_of(new), 0.125)
    assert out[60, 1].isnan().all()
    assert out.isnan().sum() == 64
    pool.close()


# ---------------------------------------------------------------- how the calls are made

def test_streams_graphs_and_workspaces():
    gen = torch.Generator(device="cuda").manual_seed(3)
    new, lens = [50, 1, 7], [50, 2000, 900]
    pool, tables = make_cache(gen, lens, 2, 128, "fp8")
    q = _randn(gen, 58, 8, 128).to(torch.bfloat16)
    cl, qs = ints(lens), starts_of(new)
    expect = pool.prefill(q, tables, cl, qs, 0.1, 2000)
    # another stream, its memory taken here
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pool.prefill(q, tables, cl, qs, 0.1, 2000, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, expect)
    # two graphs that share a workspace, replayed with lengths that change between replays
    ws = torch.empty(pkv.prefill_workspace_bytes(pool, 3, 8, 58, 2000), dtype=torch.uint8, device="cuda")
    k, v = (_randn(gen, 58, 2, 128).to(torch.bfloat16) for _ in range(2))
    a, b = torch.empty_like(q), torch.empty_like(q)
    packed = pool.prompt_attention(q, k, v, qs, 0.1)
    pool.prefill(q, tables, cl, qs, 0.1, 2000, out=a, workspace=ws)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        pool.prefill(q, tables, cl, qs, 0.1, 2000, out=a, workspace=ws)
    with torch.cuda.graph(graphs[1]):
        pool.prompt_attention(q, k, v, qs, 0.1, out=b, workspace=ws)
    for _ in range(3):
        a.zero_()
        b.zero_()
        for g in graphs:
            g.replay()
        assert torch.equal(a, expect) and torch.equal(b, packed)
    qs.copy_(starts_of([20, 0, 30]))  # a step with fewer tokens
    cl.copy_(ints([50, 2000, 800]))
    a.fill_(7.0)
    graphs[0].replay()
    assert (a[50:] == 7.0).all()
    check_prefill(pool, tables, q[:50], a[:50], [20, 0, 30], [50, 2000, 800], 0.1, 0, "replay")
    assert pool.device_error() == 0
    pool.close()


def test_strided_rows_and_empty_calls():
    gen = torch.Generator(device="cuda").manual_seed(4)
    pool, tables = make_cache(gen, [90, 40], 2, 64, "bf16")
    wide = _randn(gen, 60, 11, 64).to(torch.bfloat16)
    q = wide[:, 3:7]
    out = torch.full((60, 9, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    new, lens = [50, 10], [90, 40]
    pool.prefill(q, tables, ints(lens), starts_of(new), 0.125, 90, out=out[:, 2:6])
    check_prefill(pool, tables, q, out[:, 2:6], new, lens, 0.125, 0, "strided")
    assert (out[:, :2] == 7.0).all() and (out[:, 6:] == 7.0).all()
    # rows before the first sequence, sequences without queries, no sequences, no rows
    o = torch.full((60, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    pool.prefill(q, tables, ints(lens), ints([20, 20, 30]), 0.125, 90, out=o)
    check_prefill(pool, tables[1:], q[20:30], o[20:30], [10], [40], 0.125, 0, "middle")
    assert (o[:20] == 7.0).all() and (o[30:] == 7.0).all()
    before = pkv.launch_count()
    assert pool.prefill(q[:0], tables, ints(lens), ints([0, 0, 0]), 0.125, 90).shape == (0, 4, 64)
    assert pool.prompt_attention(q[:0], q[:0, :2], q[:0, :2], ints([0]), 0.125).shape == (0, 4, 64)
    assert pkv.launch_count() == before
    assert (pool.prompt_attention(q[:5], q[:0, :2], q[:0, :2], ints([0, 5]), 0.125, key_starts=ints([0, 0])) == 0).all()
    assert pool.device_error() == 0
    pool.close()


def test_refusals():
    pool = pkv.PagedKVPool(8, 2, 64, "bf16", fill=0)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    q, k = torch.zeros(6, 4, 64, **bf), torch.zeros(6, 2, 64, **bf)
    tables, lens, qs = ints([[0, 1], [2, 3]]), ints([20, 20]), ints([0, 3, 6])
    before = pkv.launch_count()

    def refused(error, fn, *args, **kwargs):
        with pytest.raises(error):
            fn(*args, **kwargs)

    refused(TypeError, pool.prefill, q.float(), tables, lens, qs, 0.1, 20)
    refused(ValueError, pool.prefill, q[..., :32], tables, lens, qs, 0.1, 20)
    refused(ValueError, pool.prefill, q.transpose(0, 1), tables, lens, qs, 0.1, 20)
    refused(ValueError, pool.prefill, q, tables[:1], lens, qs, 0.1, 20)
    refused(ValueError, pool.prefill, q, tables, lens, qs[:2], 0.1, 20)
    refused(TypeError, pool.prefill, q, tables, lens.long(), qs, 0.1, 20)
    refused(ValueError, pool.prefill, q, tables, lens, qs, 0.1, 20, out=torch.zeros(5, 4, 64, **bf))
    refused(pkv.PagedKVError, pool.prefill, q, tables, lens, qs, 0.1, 33)   # more than the tables hold
    refused(pkv.PagedKVError, pool.prefill, q, tables, lens, qs, 0.1, 0)
    refused(pkv.PagedKVError, pool.prefill, q, tables, lens, qs, float("nan"), 20)
    refused(pkv.PagedKVError, pool.prefill, q, tables, lens, qs, 0.1, 20, window=-1)
    refused(pkv.PagedKVError, pool.prefill, torch.zeros(6, 3, 64, **bf), tables, lens, qs, 0.1, 20)  # 3 heads over 2
    refused(pkv.PagedKVError, pool.prefill, q, tables, lens, qs, 0.1, 20, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    refused(pkv.PagedKVError, pool.prefill, q.expand(6, 4, 64)[:1].expand(6, 4, 64), tables, lens, qs, 0.1, 20)  # rows on one another
    refused(ValueError, pool.prompt_attention, q, k, k[:5], qs, 0.1)
    refused(ValueError, pool.prompt_attention, q, q, q, qs, 0.1)
    refused(ValueError, pool.prompt_attention, q, k, k, qs, 0.1, key_starts=qs[:2])
    refused(pkv.PagedKVError, pool.prompt_attention, q, k, k, qs, 0.1, causal=False, window=5)
    refused(ValueError, pool.gather_cache, tables, qs[:2], 6)
    refused(ValueError, pool.gather_cache, tables, qs, -1)
    refused(ValueError, pool.gather_cache, tables, qs, 6, first_positions=qs)
    refused(ValueError, pool.gather_cache, tables, qs, 6, k=q)
    refused(pkv.PagedKVError, pkv.prefill_workspace_bytes, pool, 2, 4, 2 ** 30, 20)
    refused(pkv.PagedKVError, pkv.prefill_workspace_bytes, pool, -1, 4, 5, 20)
    torch.cuda.synchronize()
    assert pkv.launch_count() == before and pool.device_error() == 0
    pool.close()
