"""Pools in the middle of serving, for the tests of pkv_build_step_tables and
pkv_release_blocks."""

import numpy as np


def pool_state(computed, total, block_size, *, width=None, spare=20, prefix_blocks=0, sharers=(),
               seed=0, head=None):
    """Tables that hold the blocks of `computed` tokens per request, a ring of
    the other blocks and the reference counts. `total` tokens per request
    bound the pool. Requests in `sharers` start with the same prefix_blocks
    blocks."""
    rng = np.random.default_rng(seed)
    B = block_size
    have = [-(-int(c) // B) for c in computed]
    need = [-(-int(t) // B) for t in total]
    blocks = sum(max(h, n) for h, n in zip(have, need)) + prefix_blocks + spare
    order = rng.permutation(blocks).astype(np.int32)
    table = np.full((len(have), width or max(need + have + [1])), -1, np.int32)
    ref = np.zeros(blocks, np.int32)
    shared = order[:prefix_blocks]
    at = prefix_blocks
    for r, h in enumerate(have):
        first = 0
        if r in sharers:
            assert h >= prefix_blocks
            table[r, :prefix_blocks] = shared
            ref[shared] += 1
            first = prefix_blocks
        own = order[at:at + h - first]
        table[r, first:h] = own
        ref[own] = 1
        at += h - first
    free = order[at:]
    if prefix_blocks and not sharers:
        free = np.concatenate([shared, free])
    head = int(rng.integers(0, blocks)) if head is None else head % blocks  # a place of the ring
    queue = np.full(blocks, -9, np.int32)  # places that hold nothing
    queue[(head + np.arange(len(free))) % blocks] = free
    return table, ref, queue, np.array([head, len(free)], np.int32)
