"""Rows and expected results for the tests of the 8-bit pool."""

import numpy as np

import oracle
from paged_kv_cache_hkv_gb300.synth import f32_to_bf16_bits

INF, NAN = np.uint16(0x7F80), np.uint16(0x7FC1)


def odd_rows(num_tokens, hkv, d, seed):
    """bf16 rows [T, Hkv, D] of every kind a scale meets: ordinary ones, sizes
    over fp32's whole range, subnormals, zeros of both signs, largest values at and next
    to the border of two scales, ties between codes, infinities and NaNs."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((num_tokens, hkv, d)).astype(np.float32)
    kind = rng.integers(0, 10, size=(num_tokens, hkv))
    size = np.exp2(rng.integers(-140, 126, size=(num_tokens, hkv)).astype(np.float64))
    x = np.where((kind == 1)[..., None], x * size[..., None], x).astype(np.float32)
    x[kind == 2] *= 1e-3 ** rng.integers(0, 4, size=x[kind == 2].shape)  # a wide row
    x[kind == 3] = 0.0
    bits = f32_to_bf16_bits(x)
    bits[kind == 3] |= np.uint16(0x8000) * rng.integers(0, 2, size=bits[kind == 3].shape).astype(np.uint16)
    # ties and borders: few mantissa bits, largest element 1.75 * 2^k or one bf16 step off
    n = int((kind == 4).sum())
    if n:
        tie = (rng.integers(0, 2, (n, d)) << 15 | rng.integers(110, 127, (n, d)) << 7 |
               rng.integers(0, 32, (n, d)) << 2).astype(np.uint16)
        tie[:, 0] = (127 << 7) + 0x60 + rng.integers(-1, 2, n)
        bits[kind == 4] = tie
    bits[kind == 5] &= np.uint16(0x807F)  # subnormals
    bits[kind == 6] = np.where(rng.random(bits[kind == 6].shape) < 0.01, INF, bits[kind == 6])
    bits[kind == 7] = np.where(rng.random(bits[kind == 7].shape) < 0.01, NAN, bits[kind == 7])
    return bits


def random_slots(num_tokens, num_slots, seed, padding=0.1):
    rng = np.random.default_rng(seed)
    slots = rng.permutation(num_slots)[:num_tokens].astype(np.int64)
    return np.where(rng.random(num_tokens) < padding, -1 - rng.integers(0, 9, num_tokens), slots)


def quantised_step(step):
    """(codes, scales) of the step's pool and of it after the step's write, and the
    latter's values as a bf16 pool."""
    codes, scales = oracle.quantise_rows(step.kv_cache)
    slots = oracle.slot_mapping(step.block_table, step.query_start_loc, step.num_computed,
                                step.block_size)
    codes, scales = oracle.quant_write(codes, scales, step.k, step.v, slots)
    return codes, scales, oracle.quant_pool_bits(codes, scales)


def expected(step, pool, softcap=0.0, alibi_slopes=None, key_begin=None, key_end=None):
    """(out, bound) over the 8-bit pool's values: the scored oracle's bound (weights
    and output rounded to bf16, fp32 scores and sums), and what the decode kernel's
    f16 operands add below their normal numbers:
      - a q row is held as f16 under a power of two that brings its largest to 224 ..
        448. f16's 11 bits hold bf16's 8; elements below 2^-14 are off by 2^-25, so by
        less than 2^-32 of top = max|q|: a score by e = scale 2^-32 top sum|k_d| (the
        bound's D 2^-24 of |q||k| do not cover that where they are small), an output by
        2 e A <= 2 e max|v|;
      - a weight times V's scale is off by 2^-25 of the largest such product or less,
        and a code is 448 at most: of n keys by n 2^-25 448 max_j(w_j 2^v_j), and
        448 * 2^v < 2 max_d|v_jd|: n 2^-24 sum_j w_j max_d|v_jd|, the attention over
        rows that are their largest magnitude throughout."""
    args = (step.block_table, step.seq_lens, step.query_start_loc, step.num_computed, step.scale)
    kw = dict(softcap=softcap, slopes=alibi_slopes, key_begin=key_begin, key_end=key_end)
    out, bound = oracle.scored_attention(step.q, pool, *args, **kw)
    flat = pool.copy()
    flat[:, 1] = (pool[:, 1] & 0x7FFF).max(axis=-1, keepdims=True)
    reach, _ = oracle.scored_attention(step.q, flat, *args, **kw)
    B, group = step.block_size, step.num_q_heads // step.num_kv_heads
    for r, s in enumerate(step.specs):
        j = np.arange(s.seq_len)
        blk = step.block_table[r][j // B].astype(np.int64)
        k, v = (np.nan_to_num(np.abs(oracle.bf16_bits_to_f64(pool[blk, i, j % B]))) for i in (0, 1))
        rows = slice(int(step.query_start_loc[r]), int(step.query_start_loc[r]) + s.query_len)
        top = np.abs(oracle.bf16_bits_to_f64(step.q[rows])).max(axis=2)
        e = step.scale * 2.0 ** -32 * top * np.repeat(k.sum(axis=2).max(axis=0), group)
        more = 2 * (e * np.repeat(v.max(axis=(0, 2)), group))[..., None] + \
            s.seq_len * 2.0 ** -24 * reach[rows]
        bound[rows] += 1.1 * more * (bound[rows] > 0)
    return out, bound
