"""Model check of the scored prefill kernel's barrier protocol, on the CPU.

The roles are those of test_prefill_protocol.py with the K ring of two slots
and the V ring of three, and these differences: the
K-copy warp claims and publishes the next item before it waits for the Q
buffer, and a softmax agent looks at the next item at the current one's last
tile (it takes it when that tile is through) and leaves the current one's epilogue until it has the next item's first tile
in hand: it reads O just before it publishes that tile's P (the accumulator is
overwritten only after that) and stores the row afterwards. Agents also fill a
list of bad V rows per item and read it as they store; there are five, and
agent 0 empties, as it reads O of item i, the list of item i + 3. The model
checks that a store finds its item's list complete and with nothing else in it.
The K-copy warp writes a mask per tile into a ring of eight before it copies K;
the S thread, which waits for that copy, arrives on the tile's S barrier
itself, next to its commit, so that an agent that has waited for S may read the
mask. The model checks that each agent finds its own tile's.
"""

import random

import pytest

import test_prefill_protocol as plain
from test_prefill_protocol import ITEM_Q, N_SOFTMAX, S_BUFS, run, take

K_STAGES, V_STAGES = 2, 3


@pytest.fixture(autouse=True)
def _rings(monkeypatch):
    monkeypatch.setattr(plain, "K_STAGES", K_STAGES)
    monkeypatch.setattr(plain, "V_STAGES", V_STAGES)


def k_warp_ahead(cta, ring=8):
    T, it = 0, 0
    cta.masks = [None] * ring
    for i in range(S_BUFS):
        cta.b[f"s_full{i}"].count = 2

    def claim(j):
        slot = j % ITEM_Q
        if j >= ITEM_Q:
            yield ("wait", f"iq_free{slot}", (j - ITEM_Q) // ITEM_Q)
        cta.item_q[slot] = cta.claim()
        yield ("arrive", f"iq_full{slot}", 1)

    yield from claim(0)
    item = cta.item_q[0]
    while item is not None:
        if it > 0:
            yield ("wait", "q_free", it - 1)
        yield ("tma", "q_full")
        for _ in range(cta.items[item]):
            if T >= K_STAGES:
                Tp = T - K_STAGES
                yield ("wait", f"s_full{Tp % S_BUFS}", Tp // S_BUFS)
            cta.masks[T % len(cta.masks)] = T
            yield ("tma", f"k_full{T % K_STAGES}")
            T += 1
        it += 1
        yield from claim(it)
        item = cta.item_q[it % ITEM_Q]


def s_thread(cta):
    """The plain S thread with its own arrival next to each S commit."""
    for op in plain.s_thread(cta):
        yield op
        if op[0] == "commit" and op[2].startswith("s_full"):
            yield ("arrive", op[2], 1)


def agent(cta, a, lists=5, reset=3, publish_first=False):
    rng = random.Random(cta.rng.random())
    if not hasattr(cta, "lists"):
        cta.lists, cta.fills, cta.closed = [0] * lists, {}, set()
    T, it = 0, 0
    pend = None

    def load(i, last):
        yield ("wait", "o_full", i)
        yield ("wait", f"p_ready{last % S_BUFS}", last // S_BUFS)
        cta.closed.add(i)
        assert cta.lists[i % lists] == cta.fills.get(i, 0), f"list of item {i}"
        if a == 0:
            cta.lists[(i + reset) % lists] = 0
        cta.o_read[i] = cta.o_read.get(i, 0) + 1

    def store(i):
        for _ in range(2):  # others may run between the reads of the list
            yield ("step", None, None)
            assert cta.lists[i % lists] == cta.fills.get(i, 0), f"list of item {i}"

    item = yield from take(cta, 0, 1)
    while item is not None:
        nkv = cta.items[item]
        for kt in range(nkv):
            Tg = T + kt
            if kt == nkv - 1:
                yield ("wait", f"iq_full{(it + 1) % ITEM_Q}", (it + 1) // ITEM_Q)
                seen = cta.item_q[(it + 1) % ITEM_Q]
            yield ("wait", f"s_full{Tg % S_BUFS}", Tg // S_BUFS)
            assert cta.masks[Tg % len(cta.masks)] == Tg
            cta.s_read[Tg] = cta.s_read.get(Tg, 0) + 1
            if kt > 0 and rng.random() < 0.3:  # the max grew: rescale O
                Tp = Tg - 1
                yield ("wait", f"pv_done{Tp % S_BUFS}", Tp // S_BUFS)
                assert Tp in cta.pv_done and Tg not in cta.pv_issued
            if rng.random() < 0.5:  # a partly seen tile: look at its V rows
                yield ("wait", f"v_full{Tg % V_STAGES}", Tg // V_STAGES)
                if rng.random() < 0.7:
                    assert it not in cta.closed
                    cta.fills[it] = cta.fills.get(it, 0) + 1
                    cta.lists[it % lists] += 1
            if publish_first:
                yield ("arrive", f"p_ready{Tg % S_BUFS}", 1)
            if pend is not None:
                yield from load(*pend)
            if not publish_first:
                yield ("arrive", f"p_ready{Tg % S_BUFS}", 1)
            if pend is not None:
                yield from store(pend[0])
                pend = None
        pend = (it, T + nkv - 1)
        T += nkv
        it += 1
        item = yield from take(cta, it, 1)
        assert item == seen
    if pend is not None:
        yield from load(*pend)
        yield from store(pend[0])


ROLES = {"k": k_warp_ahead, "s": s_thread, "agent": agent}


@pytest.mark.parametrize("case", range(60))
def test_random_items_and_interleavings(case):
    rng = random.Random(1000 + case)
    items = [rng.choice([1, 1, 1, 2, 3, 4, rng.randint(1, 9)]) for _ in range(rng.randint(1, 14))]
    for s in range(30):
        run(items, seed=case * 1000 + s, roles_override=ROLES)


def test_all_one_tile_and_all_long():
    for items in ([1] * 20, [7] * 6, [2, 1, 1, 1, 2, 1, 3, 1, 1], [1, 2] * 8, [3, 4, 5, 1]):
        for s in range(60):
            run(items, seed=s, roles_override=ROLES)


PLANTED = {
    # P published before the previous item's O was read
    "epilogue_after_p": {"k": k_warp_ahead, "s": s_thread, "agent": lambda c, a: agent(c, a, publish_first=True)},
    # fewer lists: the one emptied is still read
    "three_lists": {"k": k_warp_ahead, "s": s_thread, "agent": lambda c, a: agent(c, a, lists=3, reset=2)},
    "four_lists": {"k": k_warp_ahead, "s": s_thread, "agent": lambda c, a: agent(c, a, lists=4, reset=3)},
    # a ring of masks as short as the K ring
    "three_masks": {"k": lambda c: k_warp_ahead(c, ring=3), "s": s_thread, "agent": agent},
    # the list emptied is one that others fill
    "reset_next": {"k": k_warp_ahead, "s": s_thread, "agent": lambda c, a: agent(c, a, reset=1)},
}


@pytest.mark.parametrize("mistake", sorted(PLANTED))
def test_model_catches_planted_mistakes(mistake):
    with pytest.raises(AssertionError):
        for s in range(300):
            run([1, 5, 2, 1, 1, 1, 6, 3, 1, 4, 1, 1], seed=s, roles_override=PLANTED[mistake])
    assert N_SOFTMAX > 1
