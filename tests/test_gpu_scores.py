"""Attention with capped, biased or range-masked scores (pkv_score_options)
against the fp64 oracle on the GPU, through every call that takes the options.
The element-wise bound is the oracle's own (oracle/scored_oracle.py): one bf16
rounding of the weights, one of the output and the fp32 roundings of the
scores.
"""

import numpy as np
import pytest

import oracle
from parity import bits_to_f64, oracle_step
from score_cases import NAN_BITS, SHAPES, batch, key_ranges, slopes_of

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_hkv_gb300 import binding  # noqa: E402
from paged_kv_cache_hkv_gb300.runner import DeviceStep, bf16_to_numpy  # noqa: E402
from paged_kv_cache_hkv_gb300.synth import RequestSpec, make_step  # noqa: E402


@pytest.fixture(autouse=True)
def _clear_errors():
    binding.pkv_get_device_errors(clear=True)
    yield


def expected(step, pool=None, **scores):
    if pool is None:
        slots = oracle.slot_mapping(step.block_table, step.query_start_loc, step.num_computed,
                                    step.block_size)
        pool = oracle.kv_write(step.kv_cache, step.k, step.v, slots)
    kw = dict(softcap=scores.get("softcap", 0.0), slopes=scores.get("alibi_slopes"),
              key_begin=scores.get("key_begin"), key_end=scores.get("key_end"))
    return oracle.scored_attention(step.q, pool, step.block_table, step.seq_lens,
                                   step.query_start_loc, step.num_computed, step.scale, **kw)


def assert_within(bits, ref, bound, what=""):
    g = bits_to_f64(bits)
    err = np.abs(g - ref)
    bad = ~(err <= bound + 1e-30)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what} {int(bad.sum())} of {bad.size} out of bound; first {i}: gpu "
                             f"{g[i]} ref {ref[i]} bound {bound[i]}; worst ratio "
                             f"{np.nanmax(err / (bound + 1e-30)):.2f}")


def run(step, flags=0, write_in_attention=True, decode_splits=None, shared_prefix=None, **scores):
    ds = DeviceStep(step, write_in_attention=write_in_attention, decode_splits=decode_splits,
                    shared_prefix=shared_prefix, **scores)
    ds.out.fill_(7.0)
    ds.run()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == flags
    return ds


MODS = {
    "cap": dict(softcap=20.0),
    "small-cap": dict(softcap=0.5),
    "wide-cap": dict(softcap=1e6),
    "alibi": dict(alibi=True),
    "cap-alibi": dict(softcap=30.0, alibi=True),
    "documents": dict(mask="documents"),
    "prefix": dict(mask="prefix"),
    "window": dict(mask="window"),
    "empty": dict(mask="empty"),
    "random": dict(mask="random"),
    "cap-alibi-random": dict(softcap=10.0, alibi=True, mask="random"),
}


def scores_for(step, mod, seed=0):
    out = {"softcap": mod.get("softcap", 0.0)}
    if mod.get("alibi"):
        out["alibi_slopes"] = slopes_of(step.num_q_heads)
    if "mask" in mod:
        out["key_begin"], out["key_end"] = key_ranges(step, mod["mask"], seed)
    return out


@pytest.mark.parametrize("mod", MODS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_every_shape_and_score(shape, mod):
    hq, hkv, d, B = shape
    step = make_step(batch(seed=hq + d), num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=B,
                     seed=hq * d + B, scale=1.5 / d ** 0.5)
    scores = scores_for(step, MODS[mod])
    ds = run(step, **scores)
    assert_within(ds.out_host(), *expected(step, **scores), what=f"{shape} {mod}")


@pytest.mark.parametrize("mod", ["cap-alibi", "window", "random"])
@pytest.mark.parametrize("splits", [1, 2, 7, 152, 1000])
def test_any_split_of_the_decode_stream(splits, mod):
    specs = [RequestSpec(c, 1) for c in (0, 1, 15, 16, 17, 700, 1499, 31, 2200, 64)]
    step = make_step(specs, num_q_heads=8, num_kv_heads=2, head_dim=128, seed=3)
    scores = scores_for(step, MODS[mod], seed=splits)
    ds = run(step, decode_splits=splits, **scores)
    assert_within(ds.out_host(), *expected(step, **scores))


@pytest.mark.parametrize("mod", MODS)
@pytest.mark.parametrize("B", [8, 16, 32])
def test_shared_prefix_under_scores(B, mod):
    """The prefix attended once for a run of decodes, each row under its own
    bias and range; a prompt chunk and plain decodes around the run."""
    specs = [RequestSpec(40, 30)] + [RequestSpec(192 + s, 1, shares_prefix=True)
                                     for s in (0, 1, 9, 40, 300, 17, 16, 15, 33)] + [RequestSpec(77, 1)]
    step = make_step(specs, num_q_heads=16, num_kv_heads=4, head_dim=64, block_size=B,
                     prefix_tokens=192, seed=B)
    scores = scores_for(step, MODS[mod], seed=B)
    want = expected(step, **scores)
    ds = run(step, shared_prefix=(192, 1, 9), **scores)
    assert_within(ds.out_host(), *want)


def test_long_documents_in_a_chunk_over_a_long_cache():
    step = make_step([RequestSpec(3001, 700), RequestSpec(0, 1500)], num_q_heads=4, num_kv_heads=1,
                     head_dim=128, seed=11)
    for mask in ("documents", "window", "prefix", "random"):
        b, e = key_ranges(step, mask, 5)
        scores = dict(key_begin=b, key_end=e)
        assert_within(run(step, **scores).out_host(), *expected(step, **scores), what=mask)


def test_bias_keeps_its_precision_where_only_far_keys_are_seen():
    """key_end far below the row: the distances are all large, their
    differences decide."""
    specs = [RequestSpec(30000, 1), RequestSpec(9000, 150), RequestSpec(2000, 1)]
    step = make_step(specs, num_q_heads=4, num_kv_heads=2, head_dim=64, seed=4)
    T = step.num_tokens
    scores = dict(alibi_slopes=np.array([0.5, 0.25, 1.0, 0.0039], np.float32),
                  key_begin=np.full(T, 3, np.int32), key_end=np.full(T, 333, np.int32))
    assert_within(run(step, **scores).out_host(), *expected(step, **scores))


@pytest.mark.parametrize("mod", [None, "cap-alibi", "random"])
def test_a_request_of_the_shared_run_with_inconsistent_lengths(mod):
    """It is flagged and its row left as it was; the others of the run keep
    their results. Empty requests stand behind the batch."""
    specs = [RequestSpec(64 + s, 1, shares_prefix=True) for s in (5, 30, 40, 9, 17, 2)]
    specs += [RequestSpec(70, 1), RequestSpec(30, 0), RequestSpec(0, 0)]
    step = make_step(specs, num_q_heads=8, num_kv_heads=2, head_dim=64, prefix_tokens=64, seed=6)
    scores = scores_for(step, MODS[mod], seed=1) if mod else {}
    ref, bound = expected(step, **scores)
    ds = DeviceStep(step, shared_prefix=(64, 0, 6), **scores)
    ds.slot_map()
    ds.write()
    ds.out.fill_(7.0)
    ds.seq_lens[3] += 1
    ds.attend()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == (binding.DEVERR_LENGTHS |
                                                         binding.DEVERR_SHARED)
    out = ds.out_host()
    assert (bits_to_f64(out[3]) == 7.0).all()
    rest = [0, 1, 2, 4, 5, 6]
    assert_within(out[rest], ref[rest], bound[rest])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("poison", ["nan", "inf", "many"])
def test_masked_keys_never_reach_the_output(d, poison):
    """NaN and infinity in the K and V rows of keys that some rows see and
    others do not: a row that does not see them keeps its result, a row that
    does gets what the arithmetic says in those dimensions."""
    specs = [RequestSpec(200, 190), RequestSpec(150, 1), RequestSpec(0, 140), RequestSpec(149, 1)]
    step = make_step(specs, num_q_heads=8, num_kv_heads=2, head_dim=d, seed=9)
    b, e = key_ranges(step, "documents", 2)
    # decodes: one sees the poisoned keys, one starts behind them
    q = step.query_start_loc
    b[q[1]], e[q[1]] = 130, 151
    b[q[3]], e[q[3]] = 0, 150
    scores = dict(key_begin=b, key_end=e, softcap=30.0)
    pool = step.kv_cache.copy()
    bits = NAN_BITS if poison == "nan" else np.uint16(0x7F80)
    keys = {0: [100, 101, 250, 330], 1: [127], 2: [60, 61], 3: [129]}
    if poison == "many":  # more than the kernel lists
        keys = {0: list(range(60, 390, 3)), 1: list(range(0, 130)), 2: list(range(0, 140, 1)), 3: [7]}
    poisoned = np.zeros((step.num_reqs, 400), bool)
    clean = pool.copy()
    for r, js in keys.items():
        for j in js:
            blk, off = step.block_table[r][j // 16], j % 16
            c = step.num_computed[r]
            if j < c:
                pool[blk, 1, off, :, 5] = bits
                if poison != "many":
                    pool[blk, 1, off, :, d - 3] = bits | 0x8000
                else:
                    pool[blk, 1, off, :, 0] = bits
            else:
                t = q[r] + j - c
                step.v[t, :, 5] = bits
                if poison == "many":
                    step.v[t, :, 0] = bits
                else:
                    step.v[t, :, d - 3] = bits | 0x8000
            poisoned[r, j] = True
    dims = [5, 0] if poison == "many" else [5, d - 3]
    finite = step.v.copy()
    finite[(finite & 0x7F80) == 0x7F80] = 0
    step.kv_cache = pool
    ds = run(step, **scores)
    got = bits_to_f64(ds.out_host())
    # the oracle on zeros in the poisoned places: right for every row in every
    # other dimension, and in those of rows that see no poisoned key
    step.kv_cache, step.v = clean, finite
    for r, js in keys.items():
        for j in js:
            if j < step.num_computed[r]:
                step.kv_cache[step.block_table[r][j // 16], 1, j % 16][:, dims] = 0
    ref, bound = expected(step, **scores)
    sees = np.zeros(step.num_tokens, bool)
    for r in range(step.num_reqs):
        for t in range(q[r], q[r + 1]):
            sees[t] = poisoned[r, b[t]:max(b[t], e[t])].any()
    assert sees.any() and (~sees).any()
    for t in range(step.num_tokens):
        cols = [x for x in range(d) if not (sees[t] and x in dims)]
        assert (np.abs(got[t][:, cols] - ref[t][:, cols]) <= bound[t][:, cols] + 1e-30).all(), t
        if sees[t]:
            bad = got[t][:, dims]
            assert np.isnan(bad).all() if poison == "nan" else (~np.isfinite(bad)).all(), t
            if poison == "inf":  # one sign per dimension: no NaN arises
                assert (bad[:, 0] == np.inf).all() and (bad[:, 1] == -np.inf).all(), t


@pytest.mark.parametrize("B", [8, 16, 32])
def test_blocks_outside_every_range_may_be_gone(B):
    """A sliding window whose early blocks went back to the pool: their table
    entries are -1 or ids out of the pool, and are not read."""
    specs = [RequestSpec(700, 1), RequestSpec(650, 70), RequestSpec(900, 1), RequestSpec(260, 1)]
    step = make_step(specs, num_q_heads=8, num_kv_heads=4, head_dim=64, block_size=B, seed=B)
    W = 137
    pos = np.concatenate([np.arange(s.num_computed, s.seq_len) for s in specs])
    scores = dict(key_begin=(pos - W + 1).astype(np.int32))
    want = expected(step, **scores)
    for r, s in enumerate(specs):
        gone = max(0, s.num_computed - W + 1) // B
        step.block_table[r, :gone] = -1
        step.block_table[r, :gone:2] = step.num_blocks + 5
    ds = DeviceStep(step, write_in_attention=True, **scores)
    ds.run()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == 0
    assert_within(ds.out_host(), *want)


def test_rows_behind_the_batch_are_left_and_bad_blocks_are_flagged():
    specs = [RequestSpec(100, 1), RequestSpec(60, 50)]
    step = make_step(specs, num_q_heads=4, num_kv_heads=2, head_dim=64, seed=1)
    pad = 37
    step.q = np.concatenate([step.q, np.full((pad,) + step.q.shape[1:], NAN_BITS)])
    step.k = np.concatenate([step.k, step.k[:pad]])
    step.v = np.concatenate([step.v, step.v[:pad]])
    T = step.num_tokens
    scores = dict(softcap=5.0, key_begin=np.zeros(T + pad, np.int32),
                  key_end=np.full(T + pad, 1 << 30, np.int32))
    want = expected(step, **scores)
    ds = DeviceStep(step, **scores)
    ds.slot_mapping = torch.empty(T + pad, dtype=torch.int64, device="cuda")
    ds.out = torch.full((T + pad, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    ds.run()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == 0
    out = ds.out_host()
    assert_within(out[:T], want[0][:T], want[1][:T])
    assert (out[T:] == out[T, 0, 0]).all()
    assert (bits_to_f64(out[T:]) == 3.0).all()
    # every block of the decode bad: its row is zeros and the flag is set
    ds.block_table[0, :] = -1
    ds.attend()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == binding.DEVERR_BLOCK_RANGE
    assert (bits_to_f64(ds.out_host()[0]) == 0).all()


@pytest.mark.parametrize("mod", ["cap", "small-cap", "cap-alibi", "documents"])
def test_what_masked_keys_and_padding_rows_hold_changes_no_bit(mod):
    specs = [RequestSpec(150, 90), RequestSpec(140, 1), RequestSpec(0, 77)]
    step = make_step(specs, num_q_heads=8, num_kv_heads=2, head_dim=128, seed=31)
    T = step.num_tokens
    begin, end = key_ranges(step, "documents", 4)
    # no row sees the keys 130 and 131 of request 0, nor 60 and 61 of the others
    q = step.query_start_loc
    for r, (a, z) in enumerate(((130, 132), (60, 62), (60, 62))):
        for t in range(q[r], q[r + 1]):
            if begin[t] < z <= end[t]:
                begin[t] = z
            elif begin[t] < z:
                end[t] = min(end[t], a)
    scores = scores_for(step, MODS[mod])
    scores.update(key_begin=begin, key_end=end)
    outs = []
    for fill in (0x0000, 0x7F80, 0xFF80, 0x7FC0, 0x7F7F):
        s = make_step(specs, num_q_heads=8, num_kv_heads=2, head_dim=128, seed=31)
        for r, keys in enumerate(((130, 131), (60, 61), (60, 61))):
            for j in keys:
                c = s.num_computed[r]
                if j < c:
                    s.kv_cache[s.block_table[r][j // 16], :, j % 16] = fill
                else:
                    s.k[q[r] + j - c] = fill
                    s.v[q[r] + j - c] = fill
        # 40 rows behind the batch
        pad = lambda a: np.concatenate([a, np.full((40,) + a.shape[1:], fill, a.dtype)])  # noqa: E731
        s.q, s.k, s.v = pad(s.q), pad(s.k), pad(s.v)
        more = np.zeros(40, np.int32)
        ds = DeviceStep(s, softcap=scores["softcap"], alibi_slopes=scores.get("alibi_slopes"),
                        key_begin=np.concatenate([begin, more]), key_end=np.concatenate([end, more]))
        ds.slot_mapping = torch.empty(T + 40, dtype=torch.int64, device="cuda")
        ds.out = torch.full((T + 40, 8, 128), 2.0, dtype=torch.bfloat16, device="cuda")
        ds.run()
        torch.cuda.synchronize()
        assert binding.pkv_get_device_errors(clear=True) == 0
        outs.append(ds.out_host())
    assert_within(outs[0][:T], *expected(step, **scores))
    for o in outs[1:]:
        assert np.array_equal(o, outs[0])


def test_every_call_takes_the_scores():
    step = make_step(batch(seed=5), num_q_heads=8, num_kv_heads=2, head_dim=64, seed=21)
    scores = scores_for(step, MODS["cap-alibi-random"])
    want = expected(step, **scores)
    outs = []
    for kw in ({}, {"fused_write": True}, {"write_in_attention": True}):
        ds = DeviceStep(step, **kw, **scores)
        ds.run()
        outs.append(ds.out_host())
        assert_within(outs[-1], *want)
    ds.out.zero_()
    ds.attend_with_write()
    assert_within(ds.out_host(), *want)
    ds.out.zero_()
    binding.pkv_paged_attention_static_workspace(
        ds.out, ds.q, ds.kv_cache, ds.block_table, ds.seq_lens, ds.query_start_loc, ds.num_computed,
        max_query_len=step.max_query_len, max_seq_len=step.max_seq_len, scale=step.scale, **ds.scores)
    assert_within(ds.out_host(), *want)
    assert all(np.array_equal(o, outs[0]) for o in outs)
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == 0


def test_graph_replay_another_stream_and_strided_q():
    """Captured once and replayed with other values and ranges in the same
    buffers, on a stream that is not the tensors' own; q, k and v are views of
    one projection's rows."""
    specs = [RequestSpec(300, 1), RequestSpec(20, 45), RequestSpec(511, 1)]
    steps = [make_step(specs, num_q_heads=4, num_kv_heads=2, head_dim=128, seed=s) for s in (1, 2)]
    ranges = [key_ranges(s, "random", i) for i, s in enumerate(steps)]
    T, d = steps[0].num_tokens, 128
    ds = DeviceStep(steps[0], write_in_attention=True, softcap=15.0,
                    alibi_slopes=slopes_of(4), key_begin=ranges[0][0], key_end=ranges[0][1])
    qkv = torch.empty(T, 8 * d, dtype=torch.bfloat16, device="cuda")
    q, k, v = (qkv[:, a * d:b * d].view(T, b - a, d) for a, b in ((0, 4), (4, 6), (6, 8)))
    for view, own in ((q, ds.q), (k, ds.k), (v, ds.v)):
        view.copy_(own)
    ds.q, ds.k, ds.v = q, k, v
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ds.run()  # warm up
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ds.run()
    other = DeviceStep(steps[1])
    for i in (1, 0, 1):
        ds.kv_cache.copy_(torch.from_numpy(steps[i].kv_cache.view(np.int16)).cuda()
                          .view(torch.bfloat16))
        ds.block_table.copy_(torch.from_numpy(steps[i].block_table))
        for view, name in ((q, "q"), (k, "k"), (v, "v")):
            view.copy_(torch.from_numpy(getattr(steps[i], name).view(np.int16)).cuda()
                       .view(torch.bfloat16))
        for name, a in zip(("key_begin", "key_end"), ranges[i]):
            ds.scores[name].copy_(torch.from_numpy(a))
        ds.out.zero_()
        g.replay()
        torch.cuda.synchronize()
        want = expected(steps[i], softcap=15.0, alibi_slopes=slopes_of(4), key_begin=ranges[i][0],
                        key_end=ranges[i][1])
        assert_within(bf16_to_numpy(ds.out), *want)
    del other
    assert binding.pkv_get_device_errors(clear=True) == 0


def test_two_calls_at_once_on_two_streams():
    step = make_step(batch(seed=8), num_q_heads=16, num_kv_heads=2, head_dim=64, seed=2)
    kw = [scores_for(step, MODS[m]) for m in ("cap", "documents")]
    runs = [DeviceStep(step, write_in_attention=True, **k) for k in kw]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(5):
        for ds, s in zip(runs, streams):
            ds.run(s)
    torch.cuda.synchronize()
    for ds, k in zip(runs, kw):
        assert_within(ds.out_host(), *expected(step, **k))
    assert binding.pkv_get_device_errors(clear=True) == 0


def test_runs_are_bit_identical_and_off_means_plain():
    step = make_step(batch(seed=1), num_q_heads=32, num_kv_heads=8, head_dim=128, seed=7)
    scores = scores_for(step, MODS["cap-alibi-random"])
    a, b = run(step, **scores).out_host(), run(step, **scores).out_host()
    assert np.array_equal(a, b)
    plain = DeviceStep(step, write_in_attention=True)
    plain.run()
    off = DeviceStep(step, write_in_attention=True, softcap=0.0)
    off.run()
    assert np.array_equal(plain.out_host(), off.out_host())
    # ranges that say what causal attention says
    p = np.concatenate([np.arange(s.num_computed, s.seq_len) for s in step.specs]).astype(np.int32)
    same = run(step, key_begin=np.full_like(p, -5), key_end=p + 1)
    _, _, ref = oracle_step(step)
    assert np.abs(bits_to_f64(same.out_host()) - ref).max() <= 2e-2


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("softcap,up,down", [(51.0, 32, -30), (60.0, 100, -90)])
@pytest.mark.parametrize("d", [64, 128])
def test_large_and_small_values_under_scores_at_the_cap(d, softcap, up, down, sign):
    """Every score at +softcap or -softcap, V times a power of two: nothing
    overflows or underflows, so the output is the same power of two times the
    output for V of ordinary size, bit for bit."""
    step = make_step(batch(3), num_q_heads=8, num_kv_heads=2, head_dim=d, seed=8)
    step.q[...] = 0x40C0                                # 6
    bits = np.uint16(0x40C0 if sign > 0 else 0xC0C0)    # +-6: |x| >= 288, tanh(x / cap) = +-1
    step.k[...] = bits
    step.kv_cache[:, 0] = bits

    def times(v, k):  # bf16 bits times 2^k (tiny ones to zero)
        e = (v >> 7) & 0xFF
        return np.where((e > 110) & (e < 140), v.astype(np.int32) + k * 128, 0).astype(np.uint16)

    v0, pool0 = step.v.copy(), step.kv_cache[:, 1].copy()
    outs = {}
    for k in (0, up, down):
        step.v[...] = times(v0, k)
        step.kv_cache[:, 1] = times(pool0, k)
        outs[k] = run(step, softcap=softcap).out_host()
        assert_within(outs[k], *expected(step, softcap=softcap), f"2^{k}")
    f0 = bits_to_f64(outs[0])
    for k in (up, down):
        assert np.array_equal(bits_to_f64(outs[k]), np.ldexp(f0, k))
