"""Model check of the scored prefill kernel's barrier protocol, on the CPU.

The roles are those of test_prefill_protocol.py with two differences: the
K-copy warp claims and publishes the next item before it waits for the Q
buffer, and a softmax agent leaves an item's epilogue until it has the next
item's first tile in hand, just before it publishes that tile's P (the
accumulator is overwritten only after that). Agents also fill a list of bad V
rows per item; there are four, and agent 0 empties, in the epilogue of item i,
the list of item i + 3. The model checks that an epilogue finds its item's
list complete and with nothing else in it.
"""

import random

import pytest

from test_prefill_protocol import ITEM_Q, K_STAGES, N_SOFTMAX, S_BUFS, V_STAGES, run, take


def k_warp_ahead(cta):
    T, it = 0, 0

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
            yield ("tma", f"k_full{T % K_STAGES}")
            T += 1
        it += 1
        yield from claim(it)
        item = cta.item_q[it % ITEM_Q]


def agent(cta, a, lists=4, reset=3, publish_first=False):
    rng = random.Random(cta.rng.random())
    if not hasattr(cta, "lists"):
        cta.lists, cta.fills, cta.closed = [0] * lists, {}, set()
    T, it = 0, 0
    pend = None

    def epilogue(i, last):
        yield ("wait", "o_full", i)
        yield ("wait", f"p_ready{last % S_BUFS}", last // S_BUFS)
        assert cta.lists[i % lists] == cta.fills.get(i, 0), f"list of item {i}"
        cta.closed.add(i)
        if a == 0:
            yield ("step", None, None)  # others may run between the read and the reset
            cta.lists[(i + reset) % lists] = 0
        cta.o_read[i] = cta.o_read.get(i, 0) + 1

    item = yield from take(cta, 0, 1)
    while item is not None:
        nkv = cta.items[item]
        for kt in range(nkv):
            Tg = T + kt
            yield ("wait", f"s_full{Tg % S_BUFS}", Tg // S_BUFS)
            cta.s_read[Tg] = cta.s_read.get(Tg, 0) + 1
            if kt > 0 and rng.random() < 0.3:  # the max grew: rescale O
                Tp = Tg - 1
                yield ("wait", f"pv_done{Tp % S_BUFS}", Tp // S_BUFS)
                assert Tp in cta.pv_done and Tg not in cta.pv_issued
            if rng.random() < 0.5:  # a partly seen tile: look at its V rows
                if Tg >= V_STAGES:
                    Tp = Tg - V_STAGES
                    yield ("wait", f"pv_done{Tp % S_BUFS}", Tp // S_BUFS)
                yield ("wait", f"v_full{Tg % V_STAGES}", Tg // V_STAGES)
                if rng.random() < 0.7:
                    assert it not in cta.closed
                    cta.fills[it] = cta.fills.get(it, 0) + 1
                    cta.lists[it % lists] += 1
            if publish_first:
                yield ("arrive", f"p_ready{Tg % S_BUFS}", 1)
            if pend is not None:
                yield from epilogue(*pend)
                pend = None
            if not publish_first:
                yield ("arrive", f"p_ready{Tg % S_BUFS}", 1)
        pend = (it, T + nkv - 1)
        T += nkv
        it += 1
        item = yield from take(cta, it, 1)
    if pend is not None:
        yield from epilogue(*pend)


ROLES = {"k": k_warp_ahead, "agent": agent}


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
    "epilogue_after_p": {"k": k_warp_ahead, "agent": lambda c, a: agent(c, a, publish_first=True)},
    # two lists
    "two_lists": {"k": k_warp_ahead, "agent": lambda c, a: agent(c, a, lists=2, reset=1)},
    # the list emptied is one that others fill
    "reset_next": {"k": k_warp_ahead, "agent": lambda c, a: agent(c, a, reset=1)},
}


@pytest.mark.parametrize("mistake", sorted(PLANTED))
def test_model_catches_planted_mistakes(mistake):
    with pytest.raises(AssertionError):
        for s in range(300):
            run([1, 5, 2, 1, 1, 1, 6, 3, 1, 4, 1, 1], seed=s, roles_override=PLANTED[mistake])
    assert N_SOFTMAX > 1
