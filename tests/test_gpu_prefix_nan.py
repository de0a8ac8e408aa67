"""shared_prefix_decode with NaN and infinities among the keys, values and scales that a query sees: what
is NaN by the formula in 64 bits is NaN, and everything else keeps the tolerance of test_gpu_prefix,
whether the items over the sequences' own tokens join the prefix's states (two launches) or a merge
pass does (three).

To that tolerance comes what 32-bit weights cannot hold: 2^x below 2^-126 may be 0, so each of fewer than
2^11 tokens of |v| < 2^4 loses at most 2^-126 |v|, together less than 2^-111; 64 bits keep such weights
(one value of the test with far larger logits is 3e-153, where its row's largest weight meets a v of 0)."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build
from test_gpu_prefix import Batch

pytestmark = pytest.mark.gpu

JOINED, MERGED = {}, {"partition_blocks": 1}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _check(x, plan):
    launches = pkv.launch_count()
    out = x.run(**plan)
    assert pkv.launch_count() - launches == (3 if plan else 2)
    assert x.pool.device_error() == 0
    seen = 0
    for b in range(x.b):
        ref, wv = x.reference(b)
        got = out[b].double().view(ref.shape)
        nan = ref.isnan()
        seen += int(nan.sum())
        assert torch.equal(got.isnan(), nan), (b, int(nan.sum()), int(got.isnan().sum()))
        tol = 2.0 ** -8 * (2 * ref.abs() + wv) + 2.0 ** -11 * wv + 2.0 ** -111
        assert ((got - ref).abs() <= tol)[~nan].all(), b
    return seen


def _batch(kv, d=128, hq=8, hkv=2, own=(40, 1, 70), prefix=1024, **kw):
    return Batch([(prefix, list(own)), (48, [9, 33])], hq, hkv, d, kv, seed=31, **kw)


def _place(x, token, b=0):
    return x.tables[b, token // 16].long(), token % 16


@pytest.mark.parametrize("plan", [JOINED, MERGED], ids=["joined", "merged"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d,hq", [(128, 8), (64, 8), (128, 32)])
def test_key_of_the_prefix_bf16(plan, value, d, hq):
    """One value of one key: a NaN makes every logit of its heads' rows NaN, an infinity those that its
    sign in the query makes +inf; where it makes -inf the token weighs nothing."""
    x = _batch("bf16", d, hq)
    blk, at = _place(x, 700)
    x.pool.k_cache[blk, 1, at, 5] = value
    assert _check(x, plan) > 0
    x.pool.close()


@pytest.mark.parametrize("plan", [JOINED, MERGED], ids=["joined", "merged"])
@pytest.mark.parametrize("kv,d", [("int8", 128), ("int8", 64), ("fp8", 128), ("fp8", 64)])
@pytest.mark.parametrize("what", ["k", "v"])
def test_scale_of_the_prefix(plan, kv, d, what):
    x = _batch(kv, d)
    blk, at = _place(x, 1023)
    (x.pool.k_scale if what == "k" else x.pool.v_scale)[blk, 0, at] = float("nan")
    assert _check(x, plan) == 3 * 4 * d  # the first group's rows of kv head 0
    x.pool.close()


@pytest.mark.parametrize("plan", [JOINED, MERGED], ids=["joined", "merged"])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("d", [128, 64])
def test_fp8_codes_of_the_prefix(plan, what, d):
    x = _batch("fp8", d)
    blk, at = _place(x, 3)
    (x.pool.k_cache if what == "k" else x.pool.v_cache)[blk, 1, at, 9] = 0x7F
    assert _check(x, plan) == 3 * 4 * (d if what == "k" else 1)
    x.pool.close()


@pytest.mark.parametrize("plan", [JOINED, MERGED], ids=["joined", "merged"])
def test_value_of_the_prefix_bf16(plan):
    x = _batch("bf16")
    blk, at = _place(x, 130)
    x.pool.v_cache[blk, 0, at, 77] = float("nan")
    assert _check(x, plan) == 3 * 4  # its own value of every row of the group's kv head 0
    x.pool.close()


@pytest.mark.parametrize("plan", [JOINED, MERGED], ids=["joined", "merged"])
@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
def test_all_keys_of_a_prefix(plan, kv):
    """A state whose every logit is NaN has no maximum."""
    x = _batch(kv, prefix=144)
    blocks = x.tables[0, :9].long()
    if kv == "bf16":
        x.pool.k_cache[blocks, 0] = float("nan")
    else:
        x.pool.k_scale[blocks, 0] = float("nan")
    assert _check(x, plan) == 3 * 4 * 128
    x.pool.close()


@pytest.mark.parametrize("plan", [JOINED, MERGED], ids=["joined", "merged"])
def test_prefix_alone(plan):
    """The first of two query tokens of a sequence with one token of its own sees the prefix only."""
    x = _batch("bf16", own=(1, 1, 3), k=2, hq=4)
    blk, at = _place(x, 40)
    x.pool.k_cache[blk, 0, at, 0] = float("inf")
    x.pool.k_cache[blk, 1, at, 0] = float("nan")
    assert _check(x, plan) > 0
    x.pool.close()


@pytest.mark.parametrize("plan", [JOINED, MERGED], ids=["joined", "merged"])
@pytest.mark.parametrize("what", ["k", "v"])
def test_next_to_far_larger_logits(plan, what):
    """Own tokens whose logits lie so far above the prefix's that its weights are 0 in fp32: 0 times NaN
    is NaN all the same."""
    x = _batch("bf16", hq=2, own=(5, 6, 70))
    for b in range(3):
        blk, at = x.tables[b, 64].long(), 2
        x.pool.k_cache[blk, :, at] = 40 * x.q[b].sign()  # about 40 * 128 * 0.8 * scale = 360
    blk, at = _place(x, 900)
    (x.pool.k_cache if what == "k" else x.pool.v_cache)[blk, 0, at, 11] = float("nan")
    assert _check(x, plan) == 3 * (128 if what == "k" else 1)
    x.pool.close()


@pytest.mark.parametrize("plan", [JOINED, MERGED], ids=["joined", "merged"])
@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
def test_own_tokens(plan, kv):
    x = _batch(kv)
    for b, head in ((0, 0), (2, 1)):
        blk, at = x.tables[b, 64].long(), 0
        if kv == "bf16":
            x.pool.k_cache[blk, head, at, 3] = float("nan")
        else:
            x.pool.k_scale[blk, head, at] = float("nan")
    assert _check(x, plan) == 2 * 4 * 128
    x.pool.close()
