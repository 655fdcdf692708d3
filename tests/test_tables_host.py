"""Step tables and block release without a GPU: the oracle against the pages'
worked examples and invariants, a numpy restatement of the release kernel's
counting against the oracle, and the calls' refusals."""

import ctypes

import numpy as np
import pytest

import oracle
from paged_kv_cache_hkv_gb300 import binding, build
from table_cases import pool_state
from test_abi_host import FAKE, MISALIGNED
from test_abi_host import header_define as E


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return binding.load()


def _build(lib, **kw):
    a = dict(bt=FAKE, mb=8, qsl=FAKE, sl=FAKE, slots=FAKE, nc=FAKE, ql=FAKE, R=2, T=4, q=FAKE,
             st=FAKE, so=FAKE, ref=FAKE, nb=64, B=16)
    a.update(kw)
    return lib.pkv_build_step_tables(a["bt"], a["mb"], a["qsl"], a["sl"], a["slots"], a["nc"],
                                     a["ql"], a["R"], a["T"], a["q"], a["st"], a["so"], a["ref"],
                                     a["nb"], a["B"], None)


def _release(lib, **kw):
    a = dict(bt=FAKE, mb=8, R=2, rows=FAKE, tok=FAKE, n=2, q=FAKE, st=FAKE, so=FAKE, ref=FAKE, nb=64,
             B=16, ws=None, wsb=0)
    a.update(kw)
    return lib.pkv_release_blocks(a["bt"], a["mb"], a["R"], a["rows"], a["tok"], a["n"], a["q"],
                                  a["st"], a["so"], a["ref"], a["nb"], a["B"], a["ws"], a["wsb"],
                                  None)


ODD8 = ctypes.c_void_p(0x10004)


def test_build_refusals(lib):
    for k in ("R", "T", "mb"):
        assert _build(lib, **{k: -1}) == E("PKV_ERR_BAD_SHAPE")
    assert _build(lib, nb=0) == E("PKV_ERR_BAD_SHAPE")
    assert _build(lib, B=0) == E("PKV_ERR_BAD_SHAPE")
    assert _build(lib, B=12) == E("PKV_ERR_UNSUPPORTED")
    for k in ("bt", "qsl", "sl", "nc", "ql", "q", "st", "so"):
        assert _build(lib, **{k: None}) == E("PKV_ERR_NULL_POINTER"), k
        assert _build(lib, **{k: ctypes.c_void_p(0x10002)}) == E("PKV_ERR_MISALIGNED"), k
    assert _build(lib, ref=ctypes.c_void_p(0x10001)) == E("PKV_ERR_MISALIGNED")
    assert _build(lib, slots=ODD8) == E("PKV_ERR_MISALIGNED")
    assert MISALIGNED


def test_release_refusals(lib):
    for k in ("R", "n", "mb"):
        assert _release(lib, **{k: -1}) == E("PKV_ERR_BAD_SHAPE")
    assert _release(lib, nb=0) == E("PKV_ERR_BAD_SHAPE")
    assert _release(lib, B=64) == E("PKV_ERR_UNSUPPORTED")
    assert _release(lib, n=1 << 16, mb=1 << 13) == E("PKV_ERR_BAD_SHAPE")  # 2^29 entries
    for k in ("bt", "rows", "tok", "q", "st", "so", "ref"):
        assert _release(lib, **{k: None}) == E("PKV_ERR_NULL_POINTER"), k
        assert _release(lib, **{k: ctypes.c_void_p(0x10002)}) == E("PKV_ERR_MISALIGNED"), k


def _apart(names, step=1 << 24):
    return {n: ctypes.c_void_p((i + 1) * step) for i, n in enumerate(names)}


BUILD_ARRAYS = ("bt", "qsl", "sl", "slots", "nc", "ql", "q", "st", "so", "ref")
RELEASE_ARRAYS = ("bt", "rows", "tok", "q", "st", "so", "ref")


def test_overlapping_arrays_are_refused(lib):
    if pytest.importorskip("torch").cuda.is_available():
        pytest.skip("the accepted calls of this test must end at the device check: no GPU")
    ok = lambda s: s not in (E("PKV_ERR_BAD_SHAPE"), E("PKV_OK"))  # noqa: E731
    a = _apart(BUILD_ARRAYS)
    assert ok(_build(lib, **a)) and ok(_build(lib, **{**a, "so": a["st"]}))
    assert ok(_build(lib, **{**a, "ref": None})) and ok(_build(lib, **{**a, "slots": None}))
    # lengths updated in place, a table inside the queue, the last word of one in another
    for out, src in (("sl", "nc"), ("sl", "ql"), ("qsl", "ql"), ("bt", "q"), ("ref", "q"),
                     ("so", "q"), ("sl", "st"), ("ref", "st"), ("bt", "ref"), ("slots", "bt")):
        assert _build(lib, **{**a, out: a[src]}) == E("PKV_ERR_BAD_SHAPE"), (out, src)
    inside = ctypes.c_void_p(a["bt"].value + 4 * (2 * 8 - 1))
    behind = ctypes.c_void_p(a["bt"].value + 4 * 2 * 8)
    assert _build(lib, **{**a, "nc": inside}) == E("PKV_ERR_BAD_SHAPE")
    assert ok(_build(lib, **{**a, "nc": behind}))
    r = _apart(RELEASE_ARRAYS)
    assert ok(_release(lib, **r)) and ok(_release(lib, **{**r, "so": r["st"]}))
    for out, src in (("q", "bt"), ("ref", "rows"), ("so", "tok"), ("q", "ref"), ("q", "st")):
        assert _release(lib, **{**r, out: r[src]}) == E("PKV_ERR_BAD_SHAPE"), (out, src)


def test_release_workspace(lib):
    size = lib.pkv_release_workspace_size
    assert size(0, 100) == 0 and size(8, 300) == 0
    assert size(-1, 4) < 0 and size(4, -1) < 0 and size(1 << 16, 1 << 13) < 0
    big = size(1000, 400)
    assert big > 0
    kw = dict(n=1000, mb=400, R=1000)
    assert _release(lib, **kw) == E("PKV_ERR_WORKSPACE")
    assert _release(lib, ws=FAKE, wsb=big - 1, **kw) == E("PKV_ERR_WORKSPACE")
    assert _release(lib, ws=ctypes.c_void_p(0x10010), wsb=big, **kw) == E("PKV_ERR_WORKSPACE")


def test_binding_checks():
    torch = pytest.importorskip("torch")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        binding.pkv_release_blocks(i32(2, 4), i32(1), i32(2), i32(8), i32(2), i32(8), block_size=16)
    with pytest.raises(ValueError, match="ref_cnt"):
        binding._release_args(i32(2, 4), i32(1), i32(2), i32(8), i32(2), None, None, 16, None)
    with pytest.raises(ValueError, match="query_lens"):
        binding.TableCalls(block_table=i32(2, 4), free_queue=i32(8), free_state=i32(2), block_size=16)


def test_worked_examples_of_the_pages():
    """17 new tokens take 2 blocks; position 17 of a table [5, 12] is slot 193
    and position 32 of [7, 21, 9] is slot 144 when the queue hands out those
    blocks."""
    table = np.array([[5, -1, -1], [7, 21, -1]], np.int32)
    queue = np.array([12, 9, 3, 4], np.int32)
    ref = np.zeros(32, np.int32)
    out = oracle.build_step_tables(table, [16, 32], [2, 1], queue, [0, 4], ref, 16)
    assert out["block_table"].tolist() == [[5, 12, -1], [7, 21, 9]]
    assert out["slot_mapping"].tolist() == [192, 193, 144]
    assert out["query_start_loc"].tolist() == [0, 2, 3] and out["seq_lens"].tolist() == [18, 33]
    assert out["free_state"].tolist() == [2, 2]
    fresh = oracle.build_step_tables(np.full((1, 4), -1), [0], [17], queue, [1, 3], ref, 16)
    assert fresh["block_table"].tolist() == [[9, 3, -1, -1]]


@pytest.mark.parametrize("seed", range(6))
def test_oracle_agrees_with_the_slot_oracle_and_keeps_the_pool_whole(seed):
    """Slots are those of the finished table, no block is handed out twice,
    and build followed by release gives every block back."""
    rng = np.random.default_rng(seed)
    R, B = int(rng.integers(1, 30)), int(rng.choice([8, 16, 32]))
    c = rng.integers(0, 200, R)
    n = rng.integers(0, 60, R)
    table, ref, queue, state = pool_state(c, c + n, B, seed=seed)
    out = oracle.build_step_tables(table, c, n, queue, state, ref, B)
    want = oracle.slot_mapping(out["block_table"], out["query_start_loc"], c, B)
    assert np.array_equal(out["slot_mapping"], want)
    used = [b for r in range(R) for b in out["block_table"][r][:-(-int(c[r] + n[r]) // B)]]
    assert len(set(used)) == len(used)
    assert sorted(used + list(oracle.ring(queue, out["free_state"]))) == list(range(len(queue)))
    back = oracle.release_blocks(out["block_table"], range(R), c + n, queue, out["free_state"],
                                 out["ref_cnt"], B)
    assert sorted(oracle.ring(back["free_queue"], back["free_state"])) == list(range(len(queue)))
    assert (back["ref_cnt"] == 0).all()


def kernel_release(table, rows, tokens, queue, state, ref_cnt, B, order):
    """The release kernel's counting, its entries taken in a given order."""
    FREED, TOP = -(1 << 30), -(1 << 29)
    ref, queue = np.array(ref_cnt), np.array(queue)
    blocks = []
    for r in rows:
        for e in range(-(-int(tokens[r]) // B) - 1, -1, -1):
            blocks.append(int(table[r][e]))
    for x in order:
        b = blocks[x]
        old, ref[b] = int(ref[b]), ref[b] - 1
        if old == 1:
            ref[b] += FREED
        elif old <= 0:
            ref[b] += 1
    for x in order:
        b = blocks[x]
        if ref[b] < TOP:
            ref[b] = max(int(ref[b]), FREED + 1 + x)
    owners = [x for x in range(len(blocks)) if ref[blocks[x]] == FREED + 1 + x]
    head, count = int(state[0]), int(state[1])
    for i, x in enumerate(owners):
        ref[blocks[x]] = 0
        queue[(head + count + i) % len(queue)] = blocks[x]
    return {"free_queue": queue, "free_state": np.array([head, count + len(owners)], np.int32),
            "ref_cnt": ref}


@pytest.mark.parametrize("seed", range(8))
def test_the_kernels_counting_in_any_order(seed):
    """Shared blocks, rows released twice, blocks that are already free: the
    result is the oracle's whatever order the entries come in."""
    rng = np.random.default_rng(seed)
    R, B, P = 9, 16, 3
    tokens = rng.integers(P * B, 300, R)
    table, ref, queue, state = pool_state(tokens, tokens, B, prefix_blocks=P, sharers=(0, 2, 3, 7),
                                          seed=seed)
    rows = rng.integers(0, R, int(rng.integers(1, 14)))  # with repeats
    want = oracle.release_blocks(table, rows, tokens, queue, state, ref, B)
    n = sum(-(-int(tokens[r]) // B) for r in rows)
    for k in range(4):
        got = kernel_release(table, rows, tokens, queue, state, ref, B,
                             np.random.default_rng(k).permutation(n))
        for name in want:
            assert np.array_equal(got[name], want[name]), name


def test_calls_refuse_tensors_of_another_device(monkeypatch):
    """The library launches on the current device: table calls and scored
    attention name the device of their tensors, and a stream is made for no other."""
    from types import SimpleNamespace

    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0x40 + i, raising=False)
    assert binding._stream(None).value == 0x40 and binding._stream(None, 0).value == 0x40
    with pytest.raises(ValueError, match="current device"):
        binding._stream(None, 1)
    for index, device, fine in ((0, 0, True), (1, 1, False), (1, 0, False), (0, 1, False)):
        stream = SimpleNamespace(cuda_stream=0x80, device=torch.device("cuda", index))
        assert binding._stream(stream).value == 0x80  # plain calls, as ever
        if fine:
            assert binding._stream(stream, device).value == 0x80
        else:
            with pytest.raises(ValueError, match="current device"):
                binding._stream(stream, device)
    # which calls check: those with scores, whatever their other options
    q = SimpleNamespace(device=torch.device("cuda", 1))
    assert binding._scored_device(q, None) is None
    assert binding._scored_device(q, binding._options(4)) is None
    assert binding._scored_device(q, binding._options(4, None, None, binding.pkv_score_options())) == 1
    calls = binding.TableCalls.__new__(binding.TableCalls)
    calls.build_args = calls.release_args = ()
    calls._device = 1
    calls.lib = SimpleNamespace(pkv_build_step_tables=None, pkv_release_blocks=None)  # never reached
    for call in (calls.build, calls.release):
        with pytest.raises(ValueError, match="current device"):
            call()
