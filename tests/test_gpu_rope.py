"""norm_rope_and_cache and rope_table on the GPU against 64-bit torch.

Tolerances, before any run.  Queries and bf16 keys are rounded once to bf16, at most 2^-8 of the
value.  The fp32 arithmetic before that is off by less than 2^-18 of the pair's size |a| + |b|: the
mean of up to 128 squares and its root by less than 64 half steps of 2^-24 (a sum of 8, then 4
pairwise adds, the product, the root and the division), the products and the sum of the rotation
by 4, and the table's cosines by one half step each.  A quantised value is off by half a step
of its code on top: s / 2 for INT8; for E4M3 2^-4 of the value, or 2^-10 s where it is subnormal."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _reference(x, w, eps, table, pos, rot, interleaved):
    """(values, pair sizes |a| + |b|) in 64 bits."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    size = x.abs()
    if table is not None:
        cs = table.double()[pos.long()][:, None]
        c, s = cs[..., :rot // 2], cs[..., rot // 2:]
        i = torch.arange(rot // 2, device=x.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        xa, xb = x[..., a], x[..., b]
        y = x.clone()
        y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
        both = xa.abs() + xb.abs()
        size[..., a] = both
        size[..., b] = both
        x = y
    return x, size


def _check(got, ref, size, what):
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -18 * size + 1e-30
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), ((got.double() - ref).abs() / tol).max().item())


def _check_cache(pool, name, slots, ref, size, what):
    cache, scale = (pool.k_cache, pool.k_scale) if name == "k" else (pool.v_cache, pool.v_scale)
    live = slots >= 0
    blk, off = slots[live].long() // 16, slots[live].long() % 16
    got, ref, size = cache[blk, :, off], ref[live], size[live]
    if pool.dtype == "bf16":
        return _check(got, ref, size, what)
    top = 127.0 if pool.dtype == "int8" else 448.0
    s = scale[blk, :, off].double()
    amax = ref.abs().amax(-1)
    assert ((s - amax / top).abs() <= (2.0 ** -18 * size.amax(-1) + 2.0 ** -24 * amax) / top + 1e-45).all(), what
    val = (got.view(torch.float8_e4m3fn).float() if pool.dtype == "fp8" else got).double() * s[..., None]
    step = 0.5 * s[..., None].expand_as(ref) if pool.dtype == "int8" else \
        torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * s[..., None])
    # the code's half step, widened by the arithmetic's error in the value and in the scale
    tol = step * (1 + 2.0 ** -16) + 2.0 ** -17 * (size + amax[..., None]) + 1e-30
    assert ((val - ref).abs() <= tol).all(), (what, ((val - ref).abs() / tol).max().item())


def _inputs(n, hq, hkv, d, seed, fused=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, hq + 2 * hkv, d, generator=g, device="cuda") * \
        torch.exp(torch.randn(1, hq + 2 * hkv, 1, generator=g, device="cuda"))
    x = x.to(torch.bfloat16)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    w = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]
    return q, k, v, w


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,hq,hkv,rot,interleaved,norm,fused", [
    (1, 1, 1, 1.0, False, "both", True),
    (7, 32, 8, 1.0, False, "both", True),
    (5, 28, 4, 0.5, True, "k", False),
    (33, 24, 24, 0.75, False, "q", True),       # half of 48 or 96: partner lanes at no power of two
    (19, 9, 3, 0.25, False, "none", True),
    (40, 17, 1, 1.0, True, "both", False),
    (3, 8, 2, 0.0, False, "both", True),
])
def test_against_64_bits(kv, d, n, hq, hkv, rot, interleaved, norm, fused):
    q, k, v, (qw, kw) = _inputs(n, hq, hkv, d, seed=n, fused=fused)
    qw, kw = (qw if norm in ("both", "q") else None), (kw if norm in ("both", "k") else None)
    rot = int(rot * d)
    nb = n // 16 + 3
    pool = pkv.PagedKVPool(nb, hkv, d, kv, fill=0)
    g = torch.Generator(device="cuda").manual_seed(n + 1)
    slots = torch.randperm(nb * 16, generator=g, device="cuda")[:n].to(torch.int32)
    if n > 2:
        slots[1] = -1
    before = [t.clone() for t in (pool.k_cache, pool.v_cache)]
    table = pkv.rope_table(9000, rot) if rot else None
    pos = torch.randint(0, 9000, (n,), generator=g, device="cuda", dtype=torch.int32)
    out = pkv.norm_rope_and_cache(pool, q, k, v, pos if rot else None, slots, table, qw, kw, eps=1e-5,
                                  interleaved=interleaved)
    assert pool.device_error() == 0 and out.is_contiguous() and out.dtype == torch.bfloat16
    _check(out, *_reference(q, qw, 1e-5, table, pos, rot, interleaved), "q")
    kr, ks = _reference(k, kw, 1e-5, table, pos, rot, interleaved)
    _check_cache(pool, "k", slots, kr, ks, "k")
    # values go in exactly as reshape_and_cache writes them
    other = pkv.PagedKVPool(nb, hkv, d, kv, fill=0)
    other.reshape_and_cache(k.contiguous(), v.contiguous(), slots)
    assert torch.equal(pool.v_cache.view(torch.uint8), other.v_cache.view(torch.uint8))
    if kv != "bf16":
        assert torch.equal(pool.v_scale, other.v_scale)
    if rot == 0 and kw is None:
        assert torch.equal(pool.k_cache.view(torch.uint8), other.k_cache.view(torch.uint8))
    # no other slot is touched
    mask = torch.ones(nb * 16, dtype=torch.bool, device="cuda")
    mask[slots[slots >= 0].long()] = False
    for t, b in zip((pool.k_cache, pool.v_cache), before):
        t, b = (x.view(torch.uint8).transpose(1, 2).reshape(nb * 16, -1) for x in (t, b))
        assert torch.equal(t[mask], b[mask])
    # in place gives the same queries
    q2 = q.clone() if not fused else q
    ref = out.clone()
    pkv.norm_rope_and_cache(pool, q2, k, v, pos if rot else None, slots, table, qw, kw, eps=1e-5,
                            interleaved=interleaved, out=q2)
    assert torch.equal(q2, ref)
    pool.close()
    other.close()


def test_plain_copy_without_norm_and_rotation():
    for kv in ("bf16", "int8", "fp8"):
        q, k, v, _ = _inputs(50, 8, 4, 128, 5)
        a, b = (pkv.PagedKVPool(8, 4, 128, kv, fill=0) for _ in range(2))
        slots = torch.arange(50, dtype=torch.int32, device="cuda") + 13
        out = pkv.norm_rope_and_cache(a, q, k, v, None, slots)
        b.reshape_and_cache(k.contiguous(), v.contiguous(), slots)
        assert torch.equal(out, q)
        assert torch.equal(a.k_cache.view(torch.uint8), b.k_cache.view(torch.uint8))
        assert torch.equal(a.v_cache.view(torch.uint8), b.v_cache.view(torch.uint8))
        if kv != "bf16":
            assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)
        a.close()
        b.close()


def test_zero_rows_and_padding():
    """Rows of zeros normalise to zeros; padded tokens (slot -1) leave the pool as it was."""
    pool = pkv.PagedKVPool(2, 2, 64, "int8", fill=0)
    pool.k_cache.fill_(55)
    z = torch.zeros(4, 8, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([3, -1, -5, 20], dtype=torch.int32, device="cuda")
    out = pkv.norm_rope_and_cache(pool, z[:, :4], z[:, 4:6], z[:, 6:], torch.zeros(4, dtype=torch.int32, device="cuda"),
                                  slots, pkv.rope_table(4, 64), w, w)
    assert out.abs().max().item() == 0 and pool.device_error() == 0
    rows = pool.k_cache.transpose(1, 2).reshape(32, -1)
    assert (rows[[3, 20]] == 0).all() and (rows[[i for i in range(32) if i not in (3, 20)]] == 55).all()
    assert pool.k_scale[0, :, 3].tolist() == [0, 0]
    pool.close()


def test_bad_positions_and_slots():
    q, k, v, (qw, kw) = _inputs(5, 4, 2, 64, 9)
    pool = pkv.PagedKVPool(2, 2, 64, "bf16", fill=0)
    table = pkv.rope_table(100, 64)
    pos = torch.tensor([0, 100, 5, -1, 99], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 1, 32, 3, 4], dtype=torch.int32, device="cuda")
    out = pkv.norm_rope_and_cache(pool, q, k, v, pos, slots, table, qw, kw)
    assert pool.device_error() == pkv.DEVERR_POSITION | pkv.DEVERR_SLOT
    assert (out[[1, 3]] == 0).all() and (out[[0, 2, 4]].abs().amax((1, 2)) > 0).all()
    written = pool.v_cache.transpose(1, 2).reshape(32, -1).abs().amax(1) > 0
    assert written.nonzero().flatten().tolist() == [0, 4]
    pool.close()


def test_infinities_and_nan_stay_in_their_rows():
    q, k, v, (qw, kw) = _inputs(6, 4, 2, 128, 11)
    clean = pkv.PagedKVPool(1, 2, 128, "bf16", fill=0)
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    pos, table = slots + 40, pkv.rope_table(64, 128)
    ref = pkv.norm_rope_and_cache(clean, q, k, v, pos, slots, table, qw, kw).clone()
    q, k = q.clone(), k.clone()
    q[2, 1, 5], k[3, 0, 7] = float("nan"), float("inf")
    pool = pkv.PagedKVPool(1, 2, 128, "bf16", fill=0)
    out = pkv.norm_rope_and_cache(pool, q, k, v, pos, slots, table, qw, kw)
    assert out[2, 1].isnan().all() and not pool.k_cache[0, 0, 3].isfinite().all()
    keep = torch.ones(6, 4, dtype=torch.bool, device="cuda")
    keep[2, 1] = False
    assert torch.equal(out[keep], ref[keep])
    keep = torch.ones(2, 16, dtype=torch.bool, device="cuda")
    keep[0, 3] = False
    assert torch.equal(pool.k_cache[0][keep], clean.k_cache[0][keep])
    pool.close()
    clean.close()


def test_long_call_and_64_bit_offsets():
    """A prefill past 2^31 bytes of projection output, checked at both ends; far positions."""
    n, hq, hkv, d = 300000, 24, 4, 128  # 32 heads of 128: 4096 values a token, 2.5 GB
    x = torch.empty(n, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda")
    x[:64].normal_()
    x[64:-64] = x[0]
    x[-64:].normal_()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    nb = (n + 15) // 16
    pool = pkv.PagedKVPool(nb, hkv, d, "fp8")
    slots = torch.arange(n, dtype=torch.int32, device="cuda").flip(0).contiguous()
    table = pkv.rope_table(1 << 20, d)
    pos = torch.arange(n, dtype=torch.int32, device="cuda") + (1 << 20) - n
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    out = pkv.norm_rope_and_cache(pool, q, k, v, pos, slots, table, w, w)
    assert pool.device_error() == 0
    for at in (slice(0, 64), slice(n - 64, n)):
        _check(out[at], *_reference(q[at], w, 1e-6, table, pos[at], d, False), "q")
        kr, ks = _reference(k[at], w, 1e-6, table, pos[at], d, False)
        _check_cache(pool, "k", slots[at], kr, ks, "k")
    pool.close()


def test_rope_table_is_exact_to_a_half_step():
    for rot, base in ((64, 10000.0), (48, 5e5)):
        t = pkv.rope_table(70000, rot, base)
        p = torch.arange(70000, dtype=torch.float64, device="cuda")[:, None]
        a = p * base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        ref = torch.cat([a.cos(), a.sin()], 1)
        # half a step of fp32, and 70000 times the 2^-50 or so that the two powers may differ by
        assert ((t.double() - ref).abs() <= 2.0 ** -24 * ref.abs() + 70000 * 2.0 ** -50).all()


def test_refusals():
    pool = pkv.PagedKVPool(2, 2, 64, "bf16", fill=0)
    q, k, v, (qw, kw) = _inputs(4, 4, 2, 64, 1)
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    table = pkv.rope_table(16, 64)
    ok = dict(q=q, k=k, v=v, positions=slots, slot_mapping=slots, cos_sin=table, q_weight=qw, k_weight=kw)
    before = pkv.launch_count()
    wide = torch.zeros(4, 4, 65, dtype=torch.bfloat16, device="cuda")[..., :64]
    for bad in (dict(k=q), dict(v=v[:3]), dict(q=q.transpose(0, 1)), dict(q=wide), dict(slot_mapping=slots[:3]),
                dict(positions=slots[:2]), dict(q_weight=qw[:32]), dict(out=q[:, :2]), dict(k=k.cpu()),
                dict(positions=slots.cpu()), dict(cos_sin=table[:0])):
        with pytest.raises(ValueError):
            pkv.norm_rope_and_cache(pool, **(ok | bad))
    for bad in (dict(q=q.float()), dict(q_weight=qw.float()), dict(cos_sin=table.double()), dict(positions=None)):
        with pytest.raises(TypeError):
            pkv.norm_rope_and_cache(pool, **(ok | bad))
    for bad in (dict(cos_sin=torch.zeros(16, 24, device="cuda")), dict(cos_sin=torch.zeros(16, 80, device="cuda")),
                dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(pkv.PagedKVError):
            pkv.norm_rope_and_cache(pool, **(ok | bad))
    assert pkv.launch_count() == before
    assert pkv.norm_rope_and_cache(pool, q[:0], k[:0], v[:0], slots[:0], slots[:0], table).shape == (0, 4, 64)
    assert pkv.launch_count() == before
    pool.close()
