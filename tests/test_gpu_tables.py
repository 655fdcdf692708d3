"""pkv_build_step_tables and pkv_release_blocks against the oracle on the GPU
(every output equal), alone and as a serving loop uses them: release, build,
write, attend."""

import numpy as np
import pytest

import oracle
from parity import assert_close, bits_to_f64
from table_cases import pool_state

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_hkv_gb300 import binding, synth  # noqa: E402
from paged_kv_cache_hkv_gb300.runner import bf16_to_numpy  # noqa: E402


@pytest.fixture(autouse=True)
def _clear_errors():
    binding.pkv_get_device_errors(clear=True)
    yield


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def release_workspace(n, width):
    nbytes = binding.pkv_release_workspace_size(n, width)
    if not nbytes:
        return None
    return torch.full((nbytes,), 0xa5, dtype=torch.uint8, device="cuda")


class Device:
    """The buffers of a serving loop."""

    def __init__(self, table, ref, queue, state, B, in_place=True):
        self.B = B
        self.table, self.ref, self.queue, self.state = dev(table), dev(ref), dev(queue), dev(state)
        self.state_out = self.state if in_place else torch.full_like(self.state, -77)

    def build(self, c, n, T=None, slots=True, ref=True, stream=None):
        R = len(c)
        T = int(np.sum(n)) if T is None else T
        self.c, self.n = dev(c), dev(n)
        self.qsl = torch.full((R + 1,), -5, dtype=torch.int32, device="cuda")
        self.lens = torch.full((R,), -5, dtype=torch.int32, device="cuda")
        self.slots = torch.full((T,), -5, dtype=torch.int64, device="cuda") if slots else None
        binding.pkv_build_step_tables(
            self.table, self.qsl, self.lens, self.slots, self.c, self.n, self.queue, self.state,
            block_size=self.B, ref_cnt=self.ref if ref else None, free_state_out=self.state_out,
            num_tokens=T, stream=stream)
        torch.cuda.synchronize()

    def release(self, rows, tokens):
        binding.pkv_release_blocks(self.table, dev(rows), dev(tokens), self.queue, self.state,
                                   self.ref, block_size=self.B, free_state_out=self.state_out,
                                   workspace=release_workspace(len(rows), self.table.shape[1]))
        torch.cuda.synchronize()

    def check_build(self, want):
        for name, t in (("block_table", self.table), ("query_start_loc", self.qsl),
                        ("seq_lens", self.lens), ("slot_mapping", self.slots),
                        ("free_state", self.state_out), ("ref_cnt", self.ref)):
            assert np.array_equal(t.cpu().numpy(), want[name]), name

    def check_release(self, want):
        for name, t in (("free_queue", self.queue), ("free_state", self.state_out),
                        ("ref_cnt", self.ref)):
            assert np.array_equal(t.cpu().numpy(), want[name]), name


def lengths(kind, rng):
    if kind == "one":
        return np.array([0]), np.array([1])
    if kind == "decode":
        R = 65
        return rng.integers(0, 700, R), np.ones(R, np.int64)
    if kind == "mixed":
        c = rng.integers(0, 300, 90)
        n = np.where(rng.random(90) < 0.3, rng.integers(0, 400, 90), 1)
        c[::7] = 0
        return c, n
    if kind == "many":  # several requests per thread of the scan
        R = 5003
        return rng.integers(0, 100, R), np.where(rng.random(R) < 0.02, rng.integers(0, 300, R), 1)
    if kind == "long":  # one prompt that outweighs everything
        return np.array([3, 0, 40, 17]), np.array([1, 131071, 0, 5])
    if kind == "idle":
        return rng.integers(0, 90, 40), np.zeros(40, np.int64)
    raise ValueError(kind)


KINDS = ["one", "decode", "mixed", "many", "long", "idle"]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("kind", KINDS)
def test_build_matches_the_oracle(kind, B, in_place):
    rng = np.random.default_rng(B)
    c, n = lengths(kind, rng)
    table, ref, queue, state = pool_state(c, c + n, B, seed=B)
    want = oracle.build_step_tables(table, c, n, queue, state, ref, B)
    d = Device(table, ref, queue, state, B, in_place)
    d.build(c, n)
    d.check_build(want)
    if not in_place:
        assert np.array_equal(d.state.cpu().numpy(), state)
    assert np.array_equal(d.queue.cpu().numpy(), queue)
    assert binding.pkv_get_device_errors(clear=True) == 0


@pytest.mark.parametrize("kind", ["decode", "mixed", "many", "long"])
@pytest.mark.parametrize("part", [0.0, 0.3, 0.9])
def test_out_of_blocks_first_come_first_served(kind, part):
    rng = np.random.default_rng(7)
    c, n = lengths(kind, rng)
    B = 16
    table, ref, queue, state = pool_state(c, c + n, B, spare=0, seed=1)
    state[1] = int(state[1] * part)
    want = oracle.build_step_tables(table, c, n, queue, state, ref, B)
    assert want["denied"].any()
    d = Device(table, ref, queue, state, B)
    d.build(c, n)
    d.check_build(want)
    assert binding.pkv_get_device_errors(clear=True) == binding.DEVERR_NO_BLOCKS


def test_exactly_enough_blocks_and_the_ring_wraps():
    c, n = np.array([5, 0, 16]), np.array([30, 100, 1])
    for head in (0, 3, 11, 12):
        table, ref, queue, state = pool_state(c, c + n, 16, spare=0, head=head)
        want = oracle.build_step_tables(table, c, n, queue, state, ref, 16)
        assert not want["denied"].any() and want["free_state"][1] == 0
        d = Device(table, ref, queue, state, 16)
        d.build(c, n)
        d.check_build(want)
        assert binding.pkv_get_device_errors(clear=True) == 0


def test_padding_rows_no_requests_and_left_out_outputs():
    c, n = np.array([20, 3]), np.array([1, 9])
    table, ref, queue, state = pool_state(c, c + n, 16, width=7)
    want = oracle.build_step_tables(table, c, n, queue, state, ref, 16, num_tokens=50)
    d = Device(table, ref, queue, state, 16)
    d.build(c, n, T=50)
    d.check_build(want)
    d = Device(table, ref, queue, state, 16)
    d.build(c, n, slots=False, ref=False)
    assert np.array_equal(d.table.cpu().numpy(), want["block_table"])
    assert np.array_equal(d.ref.cpu().numpy(), ref)
    # no request, and no token
    d = Device(np.zeros((0, 4)), ref, queue, state, 16)
    d.build(np.zeros(0), np.zeros(0), T=5)
    assert d.qsl.tolist() == [0] and (d.slots == -1).all()
    assert np.array_equal(d.state.cpu().numpy(), state)
    d.build(np.zeros(0), np.zeros(0), T=0)
    assert binding.pkv_get_device_errors(clear=True) == 0


def test_bad_contents_are_flagged_and_hand_out_nothing():
    B = 16
    c = np.array([10, -1, 5, 2 ** 31 - 2, 20, 100, 7])
    n = np.array([10, 3, -4, 5, 1, 200, 2])  # 100 + 200 is more than the table's 8 entries
    ok = [0, 4, 6]
    good = np.where(np.isin(np.arange(7), ok), c, 0)
    table, ref, queue, state = pool_state(good, good + np.where(good > 0, 40, 0), B, width=8)
    d = Device(table, ref, queue, state, B)
    rows = np.maximum(n, 0)
    d.build(c, n, T=int(rows.sum()))
    assert binding.pkv_get_device_errors(clear=True) == binding.DEVERR_LENGTHS
    # the others are served as if the bad ones asked for nothing
    want = oracle.build_step_tables(table, good, np.where(np.isin(np.arange(7), ok), n, 0), queue,
                                    state, ref, B)
    assert np.array_equal(d.table.cpu().numpy(), want["block_table"])
    assert d.qsl.tolist() == np.concatenate([[0], np.cumsum(rows)]).tolist()
    assert np.array_equal(d.lens.cpu().numpy()[ok], want["seq_lens"][ok])
    assert (d.lens.cpu().numpy()[[1, 2, 3, 5]] == 0).all()
    slots = d.slots.cpu().numpy()
    for r in range(7):
        part = slots[int(rows[:r].sum()):int(rows[:r + 1].sum())]
        if r in ok:
            w = want["slot_mapping"][want["query_start_loc"][r]:want["query_start_loc"][r + 1]]
            assert np.array_equal(part, w)
        else:
            assert (part == -1).all()
    # more rows than num_tokens
    d = Device(table, ref, queue, state, B)
    d.build(np.array([10, 0, 0, 0, 20, 0, 7]), np.array([10, 0, 0, 0, 1, 0, 2]), T=11)
    assert binding.pkv_get_device_errors(clear=True) == binding.DEVERR_LENGTHS
    assert np.array_equal(d.slots.cpu().numpy(), want["slot_mapping"][:11])
    for bad_state in ([-1, 3], [len(queue), 3], [0, -2], [0, len(queue) + 1]):
        d = Device(table, ref, queue, np.array(bad_state), B)
        d.build(np.array([10, 0, 0, 0, 20, 0, 7]), np.array([30, 0, 0, 0, 1, 0, 2]))
        assert binding.pkv_get_device_errors(clear=True) == (binding.DEVERR_LENGTHS |
                                                             binding.DEVERR_NO_BLOCKS)
        assert d.state.tolist() == bad_state and d.lens.tolist() == [0, 0, 0, 0, 21, 0, 9]
        d.release(np.array([0]), np.array([10, 0, 0, 0, 20, 0, 7]))
        assert binding.pkv_get_device_errors(clear=True) == binding.DEVERR_LENGTHS
        assert d.state.tolist() == bad_state and np.array_equal(d.ref.cpu().numpy(), ref)
    # ids out of the pool in the queue, and a hole in the table
    q2 = queue.copy()
    q2[state[0]] = len(queue) + 3
    t2 = table.copy()
    t2[4, 1] = -1
    d = Device(t2, ref, q2, state, B)
    d.build(np.array([10, 0, 0, 0, 20, 0, 7]), np.array([30, 0, 0, 0, 1, 0, 2]))
    assert binding.pkv_get_device_errors(clear=True) == binding.DEVERR_BLOCK_RANGE
    assert d.table[0, 1] == -1 and d.slots[30] == -1


@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("kind", ["all", "some", "twice", "long", "many"])
def test_release_matches_the_oracle(kind, B):
    rng = np.random.default_rng(B)
    R, P = (3001, 6) if kind == "many" else (40, 6)
    tokens = rng.integers(P * B, 900, R)
    tokens[5] = 0
    if kind == "long":
        tokens[7] = 200000
    sharers = tuple(r for r in range(0, R, 3) if r != 5)
    table, ref, queue, state = pool_state(tokens, tokens, B, prefix_blocks=P, sharers=sharers,
                                          seed=B)
    rows = {"all": rng.permutation(R), "some": rng.permutation(R)[:9], "long": np.array([7]),
            "twice": np.array([3, 5, 3, 0, 8, 8, 1]), "many": rng.permutation(R)[:2900]}[kind]
    want = oracle.release_blocks(table, rows, tokens, queue, state, ref, B)
    d = Device(table, ref, queue, state, B, in_place=False)
    d.release(rows, tokens)
    d.check_release(want)
    assert np.array_equal(d.table.cpu().numpy(), table)
    flags = binding.pkv_get_device_errors(clear=True)
    assert flags == (binding.DEVERR_REF_COUNT if kind == "twice" else 0)
    if kind == "all":  # everything is back, and every count at zero
        assert want["free_state"][1] == len(queue) and (want["ref_cnt"] == 0).all()


def test_release_skips_what_is_out_of_range():
    tokens = np.array([40, 50, 16, 64])
    table, ref, queue, state = pool_state(tokens, tokens, 16)
    d = Device(table, ref, queue, state, 16)
    d.release(np.array([1, -1, 4, 2 ** 31 - 1]), tokens)
    want = oracle.release_blocks(table, [1], tokens, queue, state, ref, 16)
    d.check_release(want)
    assert binding.pkv_get_device_errors(clear=True) == binding.DEVERR_LENGTHS
    d = Device(table, ref, queue, state, 16)
    d.release(np.array([0, 1, 2]), np.array([-3, 50, 5000, 1]))
    d.check_release(want)
    assert binding.pkv_get_device_errors(clear=True) == binding.DEVERR_LENGTHS
    t2 = table.copy()
    t2[1, 0], t2[1, 2] = -1, len(queue)
    d = Device(t2, ref, queue, state, 16)
    d.release(np.array([1]), tokens)
    assert binding.pkv_get_device_errors(clear=True) == binding.DEVERR_BLOCK_RANGE
    assert d.state[1] == state[1] + 2
    # already free
    d = Device(table, np.zeros_like(ref), queue, state, 16)
    d.release(np.array([0, 0, 1]), tokens)
    assert binding.pkv_get_device_errors(clear=True) == binding.DEVERR_REF_COUNT
    assert np.array_equal(d.state.cpu().numpy(), state) and (d.ref == 0).all()
    d.release(np.zeros(0), tokens)
    assert np.array_equal(d.state.cpu().numpy(), state)


def test_many_steps_of_a_serving_loop():
    """Requests come, grow, share a prompt, end and come again, the pool
    running short now and then; all bookkeeping in place on the device."""
    rng = np.random.default_rng(3)
    B, R, W, blocks = 16, 24, 40, 100
    table = np.full((R, W), -1, np.int32)
    ref = np.zeros(blocks, np.int32)
    queue = rng.permutation(blocks).astype(np.int32)
    state = np.array([0, blocks], np.int32)
    d = Device(table, ref, queue, state, B)
    held = np.zeros(R, np.int64)
    seen_denied = 0
    for step in range(60):
        n = np.where(held > 0, 1, np.where(rng.random(R) < 0.4, rng.integers(1, 200, R), 0))
        n = np.where(rng.random(R) < 0.1, 0, n)
        want = oracle.build_step_tables(table, held, n, queue, state, ref, B)
        d.build(held, n)
        d.check_build(want)
        table, ref, state = want["block_table"], want["ref_cnt"], want["free_state"]
        seen_denied += want["denied"].any()
        held = np.where(want["denied"], held, held + n)
        # a request forks off another's whole blocks (a prefix in common)
        src, dst = rng.integers(0, R, 2)
        whole = held[src] // B
        if held[dst] == 0 and whole:
            table[dst, :whole] = table[src, :whole]
            ref[table[src, :whole]] += 1
            held[dst] = whole * B
            d.table.copy_(torch.from_numpy(table))
            d.ref.copy_(torch.from_numpy(ref))
        out = np.flatnonzero((held > 0) & (rng.random(R) < 0.12))
        want = oracle.release_blocks(table, out, held, queue, state, ref, B)
        d.release(out, held)
        d.check_release(want)
        queue, state, ref = want["free_queue"], want["free_state"], want["ref_cnt"]
        held[out] = 0
    assert seen_denied > 3
    assert binding.pkv_get_device_errors(clear=True) in (0, binding.DEVERR_NO_BLOCKS)


def test_the_step_they_build_is_attended():
    """release -> build -> write and attend in one stream, no table from the
    host; a denied request's rows are left as they were."""
    rng = np.random.default_rng(5)
    B, Hq, Hkv, D = 16, 8, 2, 64
    c = np.array([33, 0, 100, 16, 5, 200])
    n = np.array([1, 70, 1, 20, 1, 1])
    held = np.concatenate([c, [90]])  # one more row, to be released
    table, ref, queue, state = pool_state(held, np.concatenate([c + n, [90]]), B, width=16, spare=0,
                                          seed=2)
    state[1] = 1  # one free block: the release has to provide the others
    want_r = oracle.release_blocks(table, [6], held, queue, state, ref, B)
    want = oracle.build_step_tables(table[:6], c, n, want_r["free_queue"], want_r["free_state"],
                                    want_r["ref_cnt"], B)
    T = int(n.sum())
    blocks = len(queue)
    bits = lambda *s: synth.f32_to_bf16_bits(rng.standard_normal(s, dtype=np.float32))  # noqa: E731
    pool, q, k, v = bits(blocks, 2, B, Hkv, D), bits(T, Hq, D), bits(T, Hkv, D), bits(T, Hkv, D)
    up = lambda a: torch.from_numpy(a.view(np.int16)).cuda().view(torch.bfloat16)  # noqa: E731
    full = Device(table, ref, queue, state, B)
    binding.pkv_release_blocks(full.table, dev([6]), dev(held), full.queue, full.state, full.ref,
                               block_size=B)
    rows = full.table[:6]
    qsl, lens = dev(np.zeros(7)), dev(np.zeros(6))
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")
    cd, nd = dev(c), dev(n)
    binding.pkv_build_step_tables(rows, qsl, lens, slots, cd, nd, full.queue, full.state,
                                  block_size=B, ref_cnt=full.ref)
    kv, qd = up(pool), up(q)
    out = torch.full((T, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(binding.pkv_attention_workspace_size(6, Hq, kv), dtype=torch.uint8,
                     device="cuda")
    check = torch.empty_like(slots)
    binding.pkv_paged_attention_with_write(
        out, qd, kv, up(k), up(v), rows, lens, qsl, cd, max_query_len=70, max_seq_len=256,
        scale=0.125, workspace=ws, slot_mapping=check)
    torch.cuda.synchronize()
    assert np.array_equal(slots.cpu().numpy(), want["slot_mapping"])
    denied = want["denied"]
    assert denied.tolist() == [False, False, False, False, False, False] or denied.any()
    flags = binding.pkv_get_device_errors(clear=True)
    live = [r for r in range(6) if not denied[r]]
    pool2 = oracle.kv_write(pool, k, v, want["slot_mapping"])
    got = bf16_to_numpy(out)
    for r in range(6):
        t0, t1 = want["query_start_loc"][r], want["query_start_loc"][r + 1]
        if r in live:
            kvr = oracle.gather_request_kv(pool2, want["block_table"][r], int(c[r] + n[r]))
            ref_out = oracle.attend_rows(q[t0:t1], kvr, c[r] + np.arange(n[r]), 0.125)
            assert_close(got[t0:t1], ref_out)
        else:
            assert (bits_to_f64(got[t0:t1]) == 5.0).all()
    assert bool(flags & binding.DEVERR_NO_BLOCKS) == bool(denied.any())


def test_graph_replay_advances_the_queue_in_place():
    """One captured step of decodes replayed: every replay takes the next
    blocks; on a stream of its own."""
    B, R = 8, 50
    c = np.arange(R) * 3
    table, ref, queue, state = pool_state(c, c + 40, B)
    d = Device(table, ref, queue, state, B)
    cd, nd = dev(c), dev(np.ones(R))
    qsl, lens = dev(np.zeros(R + 1)), dev(np.zeros(R))
    slots = torch.zeros(R, dtype=torch.int64, device="cuda")
    calls = binding.TableCalls(block_table=d.table, query_start_loc=qsl, seq_lens=lens,
                               slot_mapping=slots, num_computed_tokens=cd, query_lens=nd,
                               free_queue=d.queue, free_state=d.state, ref_cnt=d.ref, block_size=B,
                               release_rows=dev([1, 2]), release_tokens=lens)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        calls.build()
        cd.copy_(lens)
    for _ in range(20):
        want = oracle.build_step_tables(table, c, np.ones(R, int), queue, state, ref, B)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(d.table.cpu().numpy(), want["block_table"])
        assert np.array_equal(slots.cpu().numpy(), want["slot_mapping"])
        assert np.array_equal(d.state.cpu().numpy(), want["free_state"])
        table, ref, state, c = want["block_table"], want["ref_cnt"], want["free_state"], c + 1
    calls.release(side)
    torch.cuda.synchronize()
    want = oracle.release_blocks(table, [1, 2], c, queue, state, ref, B)
    d.check_release(want)
    assert binding.pkv_get_device_errors(clear=True) == 0


@pytest.mark.parametrize("rows", [7, 1200])
def test_a_captured_release_and_build(rows):
    """Release and build captured together, small and large, replayed over a
    restored pool; the queue's state in place."""
    B, R, P = 16, 1300, 4
    rng = np.random.default_rng(rows)
    tokens = rng.integers(P * B, 400, R)
    table, ref, queue, state = pool_state(tokens, tokens, B, prefix_blocks=P, sharers=range(0, R, 2),
                                          width=40, seed=3)
    gone = rng.permutation(R)[:rows]
    d = Device(table, ref, queue, state, B)
    c, n = np.array([0, 0, 5]), np.array([100, 1, 300])
    fresh = np.full((3, 40), -1, np.int32)
    fresh[2, 0] = table[gone[0], 5]  # (any block: request 2 goes on in it)
    ft, qsl, lens = dev(fresh), dev(np.zeros(4)), dev(np.zeros(3))
    slots = torch.zeros(401, dtype=torch.int64, device="cuda")
    rel = binding.TableCalls(block_table=d.table, free_queue=d.queue, free_state=d.state,
                             ref_cnt=d.ref, block_size=B, release_rows=dev(gone),
                             release_tokens=dev(tokens))
    bld = binding.TableCalls(block_table=ft, query_start_loc=qsl, seq_lens=lens, slot_mapping=slots,
                             num_computed_tokens=dev(c), query_lens=dev(n), free_queue=d.queue,
                             free_state=d.state, ref_cnt=d.ref, block_size=B)
    want_r = oracle.release_blocks(table, gone, tokens, queue, state, ref, B)
    want = oracle.build_step_tables(fresh, c, n, want_r["free_queue"], want_r["free_state"],
                                    want_r["ref_cnt"], B)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        rel.release()
        bld.build()
    for _ in range(3):
        d.ref.copy_(torch.from_numpy(ref))
        d.queue.copy_(torch.from_numpy(queue))
        d.state.copy_(torch.from_numpy(state))
        ft.copy_(torch.from_numpy(fresh))
        slots.fill_(-9)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(ft.cpu().numpy(), want["block_table"])
        assert np.array_equal(slots.cpu().numpy(), want["slot_mapping"])
        assert np.array_equal(d.queue.cpu().numpy(), want_r["free_queue"])
        assert np.array_equal(d.state.cpu().numpy(), want["free_state"])
        assert np.array_equal(d.ref.cpu().numpy(), want["ref_cnt"])
    assert binding.pkv_get_device_errors(clear=True) == 0


def test_many_requests():
    """More than 64 requests per thread of the scan, and a release of as many."""
    rng = np.random.default_rng(0)
    R, B = 70001, 16
    c = rng.integers(0, 40, R)
    n = np.where(rng.random(R) < 0.01, rng.integers(0, 60, R), rng.integers(0, 2, R))
    table, ref, queue, state = pool_state(c, c + n, B, seed=0)
    want = oracle.build_step_tables(table, c, n, queue, state, ref, B)
    d = Device(table, ref, queue, state, B)
    d.build(c, n)
    d.check_build(want)
    rows = rng.permutation(R)[:65000]
    want = oracle.release_blocks(want["block_table"], rows, c + n, queue, want["free_state"],
                                 want["ref_cnt"], B)
    d.release(rows, c + n)
    d.check_release(want)
    assert binding.pkv_get_device_errors(clear=True) == 0


def test_two_pools_on_two_streams_at_once():
    rng = np.random.default_rng(1)
    runs = []
    for seed in (1, 2):
        c, n = lengths("many", rng)
        table, ref, queue, state = pool_state(c, c + n, 16, seed=seed)
        want = oracle.build_step_tables(table, c, n, queue, state, ref, 16)
        rows = rng.permutation(len(c))[:2000]
        after = oracle.release_blocks(want["block_table"], rows, c + n, queue, want["free_state"],
                                      want["ref_cnt"], 16)
        d = Device(table, ref, queue, state, 16)
        R, T = len(c), int(n.sum())
        args = (dev(np.zeros(R + 1)), dev(np.zeros(R)), torch.zeros(T, dtype=torch.int64, device="cuda"),
                dev(c), dev(n), dev(rows), release_workspace(2000, table.shape[1]))
        runs.append((d, args, torch.cuda.Stream(), after))
    torch.cuda.synchronize()
    for d, (qsl, lens, slots, c, n, rows, ws), s, _ in runs:
        binding.pkv_build_step_tables(d.table, qsl, lens, slots, c, n, d.queue, d.state,
                                      block_size=16, ref_cnt=d.ref, stream=s)
        binding.pkv_release_blocks(d.table, rows, lens, d.queue, d.state, d.ref, block_size=16,
                                   workspace=ws, stream=s)
    torch.cuda.synchronize()
    for d, _, _, after in runs:
        d.check_release(after)
    assert binding.pkv_get_device_errors(clear=True) == 0
