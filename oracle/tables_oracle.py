"""Plain statement of the block bookkeeping around a step (test infrastructure
only): blocks popped from the head of a free queue for the requests' new
tokens ([P4] §3.3: popleft; [P2] §3.3: ceil(tokens / B) blocks), and given back
at its tail when their reference count reaches zero ([P1] §4.3.1, [P4] §3.3).
Readings the pages leave open: a request that the queue cannot serve, and
every later one that needs a block, gets none (first come, first served); a
sequence is released from its last block to its first.
"""

from __future__ import annotations

from collections import deque

import numpy as np

from .paged_oracle import blocks_for_tokens


def ring(queue, state):
    """The free queue as a deque."""
    head, count = (int(x) for x in state)
    return deque(int(queue[(head + i) % len(queue)]) for i in range(count))


def build_step_tables(block_table, num_computed, query_lens, queue, state, ref_cnt, block_size,
                      num_tokens=None):
    """Returns a dict of the new block_table, query_start_loc, seq_lens,
    slot_mapping, free_state and ref_cnt, and "denied" (bool [R])."""
    B = block_size
    table, ref = np.array(block_table), np.array(ref_cnt)
    free = ring(queue, state)
    R = len(num_computed)
    qsl, lens, slots = np.zeros(R + 1, np.int64), np.zeros(R, np.int32), []
    denied, full = np.zeros(R, bool), False
    for r in range(R):
        c, n = int(num_computed[r]), int(query_lens[r])
        qsl[r + 1] = qsl[r] + n
        have, total = int(blocks_for_tokens(c, B)), int(blocks_for_tokens(c + n, B))
        if total > have and (full or len(free) < total - have):
            full = denied[r] = True
            table[r, have:total] = -1
            slots += [-1] * n
            continue
        for e in range(have, total):
            table[r, e] = free.popleft()
            ref[table[r, e]] = 1
        lens[r] = c + n
        slots += [int(table[r, p // B]) * B + p % B for p in range(c, c + n)]
    T = len(slots) if num_tokens is None else num_tokens
    out = np.full(T, -1, np.int64)
    out[:min(T, len(slots))] = slots[:T]
    taken = int(state[1]) - len(free)
    return {"block_table": table, "query_start_loc": qsl.astype(np.int32), "seq_lens": lens,
            "slot_mapping": out, "ref_cnt": ref, "denied": denied,
            "free_state": np.array([(int(state[0]) + taken) % len(queue), len(free)], np.int32)}


def release_blocks(block_table, rows, tokens, queue, state, ref_cnt, block_size):
    """Returns a dict of the new free_queue, free_state and ref_cnt. A block
    released more often than held is freed once."""
    queue, ref = np.array(queue), np.array(ref_cnt)
    order, head = [], int(state[0])
    for r in rows:
        for e in range(int(blocks_for_tokens(tokens[r], block_size)) - 1, -1, -1):
            order.append(int(block_table[r][e]))
    drops = {}
    for b in order:
        drops[b] = drops.get(b, 0) + 1
    last = {b: x for x, b in enumerate(order)}
    count = int(state[1])
    for x, b in enumerate(order):
        if last[b] != x:
            continue
        held = int(ref[b])
        ref[b] = max(0, held - drops[b])
        if held > 0 and ref[b] == 0:
            queue[(head + count) % len(queue)] = b
            count += 1
    return {"free_queue": queue, "free_state": np.array([head, count], np.int32), "ref_cnt": ref}
