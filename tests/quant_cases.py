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
    """(out, bound) over the 8-bit pool's values: the scored oracle's bound (bf16
    weights and output, fp32 scores and sums), and what the decode's q adds: a q
    row is held as two e4m3 numbers under one power of two, exactly but for
    elements below 2^-6 / 224 of the row's largest, which are off by at most
    2^-14 / 224 < 2^-21 of it. A score is then off by at most
    e = scale 2^-21 max|q| sum|k_d|, an output by 2 e A <= 2 e max|v| over the seen keys."""
    out, bound = oracle.scored_attention(step.q, pool, step.block_table, step.seq_lens,
                                         step.query_start_loc, step.num_computed, step.scale,
                                         softcap=softcap, slopes=alibi_slopes,
                                         key_begin=key_begin, key_end=key_end)
    B, group = step.block_size, step.num_q_heads // step.num_kv_heads
    for r, s in enumerate(step.specs):
        L = s.seq_len
        j = np.arange(L)
        blk = step.block_table[r][j // B].astype(np.int64)
        k, v = (np.nan_to_num(np.abs(oracle.bf16_bits_to_f64(pool[blk, i, j % B]))) for i in (0, 1))
        reach = k.sum(axis=2).max(axis=0)  # [Hkv]
        top = v.max(axis=(0, 2))
        t0 = int(step.query_start_loc[r])
        q = np.abs(oracle.bf16_bits_to_f64(step.q[t0:t0 + s.query_len])).max(axis=2)
        e = step.scale * 2.0 ** -21 * q * np.repeat(reach, group)
        bound[t0:t0 + s.query_len] += (2.2 * e * np.repeat(top, group))[..., None] * \
            (bound[t0:t0 + s.query_len] > 0)
    return out, bound
