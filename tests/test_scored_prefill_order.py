"""Who has seen whose shared-memory writes in the scored prefill with sixteen
softmax warps, on the CPU.

The barrier model of test_scored_prefill_protocol.py runs one operation at a
time, so it cannot tell a wait that orders memory from one that merely comes
later. Here every role carries the set of writes and reads that it is ordered
after: an arrival hands its role's set to the barrier's phase, a wait takes the
phase's set over. A commit of the tensor core and a copy's completion hand over
nothing (they stand for the asynchronous work alone).

With sixteen warps at head_dim 64 only half of the agents hold columns of O:
agents a < 2 do, agent a + 2 has the other keys of the same rows. Every agent
writes its part of an item's row sums at the item's last tile, into one of four
places; the O holders read both parts as they store the row. Agents also add to
the item's list of bad keys, one of five, which agent 0 empties three items
ahead. The model checks that each write and read is ordered after those it must
not overtake.
"""

import random

import pytest

import test_prefill_protocol as plain
from test_prefill_protocol import N_SOFTMAX, S_BUFS, run, take
from test_scored_prefill_protocol import K_STAGES, V_STAGES, k_warp_ahead, s_thread

HOLDERS, PLACES, LISTS = 2, 4, 5
assert N_SOFTMAX == 2 * HOLDERS


def knowing(cta, name, role):
    """The role's operations, with what it is ordered after kept in cta.known[name]."""
    if not hasattr(cta, "known"):
        cta.known, cta.handed = {}, {}
    known = cta.known.setdefault(name, set())
    op = next(role)
    while True:
        if op[0] == "arrive":  # (the phase cannot complete without this arrival)
            cta.handed.setdefault((op[1], cta.b[op[1]].phases), set()).update(known)
        yield op
        if op[0] == "wait":
            known |= cta.handed.get((op[1], op[2]), set())
        try:
            op = role.send(None)
        except StopIteration:
            return


@pytest.fixture(autouse=True)
def _rings(monkeypatch):
    monkeypatch.setattr(plain, "K_STAGES", K_STAGES)
    monkeypatch.setattr(plain, "V_STAGES", V_STAGES)
    for name in ("v_warp", "pv_thread"):
        role = getattr(plain, name)
        monkeypatch.setattr(plain, name, lambda cta, role=role, name=name: knowing(cta, name, role(cta)))


def agent(cta, a, both_waits=True, places=PLACES, reset=3):
    rng = random.Random(cta.rng.random())
    holds = a < HOLDERS

    def known(event):
        return event in cta.known[f"sm{a}"]

    def note(event):
        cta.known[f"sm{a}"].add(event)

    def load(i, last):
        yield ("wait", "o_full", i)
        if holds or both_waits:
            yield ("wait", f"p_ready{last % S_BUFS}", last // S_BUFS)
        if a == 0:
            for other in range(N_SOFTMAX):  # nobody adds to the list as it is emptied
                if i + reset >= LISTS:
                    assert known(("filled", i + reset - LISTS, other)), f"list of item {i + reset}"
            note(("emptied", i + reset))
        cta.o_read[i] = cta.o_read.get(i, 0) + 1

    def store(i):
        yield ("step", None, None)
        if holds:
            for part in (a, a + HOLDERS):
                assert known(("sums", i, part)), f"row sums of item {i} from agent {part}"
            note(("read", i, a))

    T, it, pend = 0, 0, None
    item = yield from take(cta, 0, 1)
    while item is not None:
        nkv = cta.items[item]
        for kt in range(nkv):
            Tg = T + kt
            yield ("wait", f"s_full{Tg % S_BUFS}", Tg // S_BUFS)
            cta.s_read[Tg] = cta.s_read.get(Tg, 0) + 1
            if rng.random() < 0.5:  # a partly seen tile: a bad key goes into the list
                yield ("wait", f"v_full{Tg % V_STAGES}", Tg // V_STAGES)
                assert it < 3 or known(("emptied", it)), f"list of item {it} not emptied yet"
            if kt == nkv - 1:
                note(("filled", it, a))
                assert it < places or known(("read", it - places, a % HOLDERS)), f"sums of {it - places}"
                note(("sums", it, a))
            if pend is not None:
                yield from load(*pend)
            yield ("arrive", f"p_ready{Tg % S_BUFS}", 1)
            if pend is not None:
                yield from store(pend[0])
                pend = None
        pend = (it, T + nkv - 1)
        T += nkv
        it += 1
        item = yield from take(cta, it, 1)
    if pend is not None:
        yield from load(*pend)
        yield from store(pend[0])


def roles(**kw):
    return {"k": lambda c: knowing(c, "k", k_warp_ahead(c)), "s": lambda c: knowing(c, "s", s_thread(c)),
            "agent": lambda c, a: knowing(c, f"sm{a}", agent(c, a, **kw))}


@pytest.mark.parametrize("case", range(40))
def test_every_write_is_seen_by_its_readers(case):
    rng = random.Random(case)
    items = [rng.choice([1, 1, 1, 2, 3, rng.randint(1, 6)]) for _ in range(rng.randint(1, 16))]
    for s in range(20):
        run(items, seed=case * 100 + s, roles_override=roles())


PLANTED = {
    # an agent without O that waits for the last PV only
    "o_full_only": dict(both_waits=False),
    # fewer places for the row sums: one is filled while it may be read
    "two_places": dict(places=2),
    # the list emptied is one that others fill
    "reset_next": dict(reset=1),
}


@pytest.mark.parametrize("mistake", sorted(PLANTED))
def test_model_catches_planted_mistakes(mistake):
    with pytest.raises(AssertionError):
        for s in range(200):
            run([1, 2, 1, 1, 3, 1, 1, 1, 2, 1, 1, 4, 1], seed=s, roles_override=roles(**PLANTED[mistake]))
