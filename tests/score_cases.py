"""Batches, key ranges and slopes for the tests of capped, biased and
range-masked attention."""

import numpy as np

from paged_kv_cache_hkv_gb300.synth import RequestSpec

NAN_BITS = np.uint16(0x7FC0)

# q heads, kv heads, head_dim, block size: every group size and block size
SHAPES = [(4, 2, 64, 16), (8, 1, 64, 32), (8, 1, 128, 8), (6, 6, 128, 16), (16, 4, 128, 32),
          (12, 6, 64, 8), (32, 8, 128, 16)]


def batch(seed=0):
    """Decodes of one to several hundred keys, chunks with and without a cache,
    a single-token prompt, in a mixed order."""
    rng = np.random.default_rng(seed)
    return [RequestSpec(0, 1), RequestSpec(int(rng.integers(100, 400)), 1), RequestSpec(0, 129),
            RequestSpec(15, 1), RequestSpec(16, 1), RequestSpec(int(rng.integers(1, 200)), 67),
            RequestSpec(int(rng.integers(400, 700)), 1), RequestSpec(131, 2), RequestSpec(7, 3)]


def slopes_of(num_q_heads):
    return (2.0 ** (-8.0 * np.arange(1, num_q_heads + 1) / num_q_heads)).astype(np.float32)


def key_ranges(step, mask, seed=0):
    """(key_begin, key_end) int32 [T] of a step's rows."""
    rng = np.random.default_rng(seed)
    T = step.num_tokens
    begin, end = np.zeros(T, np.int32), np.zeros(T, np.int32)
    for r, s in enumerate(step.specs):
        t0, c, n, L = int(step.query_start_loc[r]), s.num_computed, s.query_len, s.seq_len
        pos = np.arange(c, c + n)
        b, e = np.zeros(n, np.int64), pos + 1
        if mask == "documents":  # some of them padding that sees nothing
            cuts = np.unique(np.concatenate([[0], rng.integers(0, L + 1, size=max(1, L // 40)), [L]]))
            for a, z in zip(cuts[:-1], cuts[1:]):
                inside = (pos >= a) & (pos < z)
                b[inside] = a
                if rng.random() < 0.15 and z < L:
                    e[inside] = a
        elif mask == "prefix":
            e = np.maximum(pos + 1, rng.integers(1, L + 20))
        elif mask == "window":
            b = pos - int(rng.integers(1, 90)) + 1
        elif mask == "empty":  # most rows see nothing, and that in several ways
            way = rng.integers(0, 5, size=n)
            b = np.where(way == 0, 5, np.where(way == 1, L + 3, np.where(way == 2, 1 << 30, 0)))
            e = np.where(way == 0, 5, np.where(way == 3, -7, pos + 1))
            e = np.where(way == 1, 1 << 30, e)
        elif mask == "random":
            b = rng.integers(-3, L + 2, size=n)
            e = b + rng.integers(-2, L + 5, size=n)
        begin[t0:t0 + n], end[t0:t0 + n] = b, e
    return begin, end
