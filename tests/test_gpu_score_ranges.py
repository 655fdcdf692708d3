"""Scored attention on the GPU at the ends of what its options accept: caps and
scales whose products leave fp32, caps too wide for a fixed maximum, slopes of
any size."""

import numpy as np
import pytest

import oracle
from score_cases import batch, slopes_of

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_hkv_gb300 import binding  # noqa: E402
from paged_kv_cache_hkv_gb300.synth import RequestSpec, make_step  # noqa: E402
from test_gpu_scores import assert_within, expected, run  # noqa: E402


@pytest.fixture(autouse=True)
def _clear_errors():
    binding.pkv_get_device_errors(clear=True)
    yield


def times_power(bits, k):
    """bf16 bit patterns times 2^k (zeros stay)."""
    e = (bits >> 7) & 0xFF
    assert ((e == 0) | ((e.astype(int) + k > 0) & (e.astype(int) + k < 255))).all()
    return np.where(e == 0, bits, bits.astype(np.int32) + k * 128).astype(np.uint16)


# softcap, scale, power of two on q. The products of softcap and the powers of
# scale / softcap overflow fp32 in the first three and are subnormal in the
# fourth; the others are the corners of the accepted range.
EXTREMES = [(2e4, 2e8, -27), (1e5, 1e9, -30), (1e26, 1e28, -93), (0.5, 5.1e-5, 9),
            (1e30, 1e30, -100), (5e29, 1.0, 0), (1.0, 1e-30, 0), (1e-29, 1.0, 0), (1.0, 1e30, -100)]


@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("softcap,scale,power", EXTREMES)
def test_caps_and_scales_whose_products_leave_fp32(softcap, scale, power, d, alibi):
    """With q times 2^power the scores are of ordinary size (or the cap makes
    them small), so the oracle's bound is as tight as ever; rows of zeros in q
    and k give scores of exactly 0."""
    step = make_step(batch(2), num_q_heads=8, num_kv_heads=2, head_dim=d, seed=d, scale=scale)
    step.q[...] = times_power(step.q, power)
    step.q[3::7] = 0
    step.k[5::9] = 0
    scores = dict(softcap=softcap)
    if alibi:
        scores["alibi_slopes"] = slopes_of(8)
    assert_within(run(step, **scores).out_host(), *expected(step, **scores))


@pytest.mark.parametrize("power", [0, 5])
@pytest.mark.parametrize("softcap", [52.0, 60.0, 500.0, 880.0])
@pytest.mark.parametrize("d", [64, 128])
def test_caps_that_keep_the_running_maximum(d, softcap, power):
    """Caps above 51 without slopes: every score within the polynomial's range
    (power 0), or some tiles beyond it and some not (q of every other request
    times 32: a score's deviation is 48)."""
    step = make_step(batch(4), num_q_heads=8, num_kv_heads=4, head_dim=d, seed=d + 1,
                     scale=1.5 / d ** 0.5)
    for r in range(0, step.num_reqs, 2):
        rows = slice(step.query_start_loc[r], step.query_start_loc[r + 1])
        step.q[rows] = times_power(step.q[rows], power)
    scores = dict(softcap=softcap)
    assert_within(run(step, **scores).out_host(), *expected(step, **scores))


def nearest_values(step, begin, end, farthest=False):
    """bf16 bits [T, Hkv, D] of V at the key of each row's range that is nearest
    to the row's position (or farthest from it), zeros for an empty range."""
    slots = oracle.slot_mapping(step.block_table, step.query_start_loc, step.num_computed,
                                step.block_size)
    pool = oracle.kv_write(step.kv_cache, step.k, step.v, slots)
    want = np.zeros((step.num_tokens, step.num_kv_heads, step.head_dim), np.uint16)
    for r, s in enumerate(step.specs):
        for i in range(s.query_len):
            t, p = step.query_start_loc[r] + i, s.num_computed + i
            lo, hi = max(0, begin[t]), min(end[t], s.seq_len)
            if lo < hi:
                j = lo if farthest else max(min(p, hi - 1), lo)
                want[t] = pool[step.block_table[r][j // step.block_size], 1, j % step.block_size]
    return want


STEEP = [3.4e38, 2.3e38, 1e36, 5e29, 1e28, 1e20, 1e7, 1e4]


@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("ranges", ["causal", "far", "ahead"])
@pytest.mark.parametrize("d,sign,shared", [(64, 1, None), (128, 1, None), (64, -1, None),
                                           (128, -1, None), (64, 1, (64, 0, 4))])
def test_slopes_of_any_size(d, sign, shared, ranges, softcap):
    """A slope so steep that one key takes all the weight gives that key's
    value, bit for bit: the nearest one, or with a negative slope the farthest
    (the causal rows' first key; ties are not made)."""
    specs = [RequestSpec(64 + s, 1, shares_prefix=True) for s in (5, 300, 64, 0)]
    specs += [RequestSpec(131, 140), RequestSpec(0, 70), RequestSpec(600, 1)]
    step = make_step(specs, num_q_heads=8, num_kv_heads=2, head_dim=d, prefix_tokens=64, seed=d)
    pos = np.concatenate([np.arange(s.num_computed, s.seq_len) for s in specs]).astype(np.int32)
    begin, end = np.zeros_like(pos), pos + 1
    if ranges == "far":  # the nearest visible key is far away, or there is none
        begin, end = np.full_like(pos, 3), np.minimum(pos + 1, 40 + pos % 29)
        begin[::5] = 90  # behind the end: these rows see nothing
    elif ranges == "ahead" and sign > 0:  # keys on both sides: the row's own is the nearest
        end = pos + 60
    scores = dict(softcap=softcap, key_begin=begin.astype(np.int32), key_end=end.astype(np.int32),
                  alibi_slopes=(sign * np.array(STEEP)).astype(np.float32))
    out = run(step, shared_prefix=shared, **scores).out_host()
    want = nearest_values(step, begin, end, farthest=sign < 0)
    assert np.array_equal(out, np.repeat(want, 4, axis=1))
