"""The 8-bit pool's calls on the GPU against the fp64 oracle (oracle/quant_oracle.py):
writes and reads bit for bit, attention within the bound of quant_cases.expected."""

import numpy as np
import pytest

import oracle
from parity import bits_to_f64
from quant_cases import expected, odd_rows, quantised_step, random_slots
from score_cases import SHAPES, batch, key_ranges, slopes_of

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_hkv_gb300 import binding  # noqa: E402
from paged_kv_cache_hkv_gb300.runner import DeviceStep, bf16_to_numpy  # noqa: E402
from paged_kv_cache_hkv_gb300.synth import RequestSpec, make_step  # noqa: E402

E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _clear_errors():
    binding.pkv_get_device_errors(clear=True)
    yield


def bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def pool_of(nb, B, hkv, d, seed):
    """A pool of rows that were written, as (codes, scales) on the host and on the GPU."""
    codes, scales = oracle.quantise_rows(odd_rows(nb * 2 * B, hkv, d, seed).reshape(nb, 2, B, hkv, d))
    return codes, scales, torch.from_numpy(codes).cuda().view(E4M3), torch.from_numpy(scales).cuda()


def host(t):
    return t.view(torch.uint8).cpu().numpy()


ROWS = [(1, 1, 64, 8), (3, 2, 128, 16), (64, 8, 128, 16), (77, 3, 64, 32), (500, 12, 64, 16),
        (33, 40, 128, 8), (2000, 5, 128, 32)]


@pytest.mark.parametrize("T,hkv,d,B", ROWS)
@pytest.mark.parametrize("extra", [0, 24])
def test_write_is_the_definition_bit_for_bit(T, hkv, d, B, extra):
    nb = -(-T // B) + 3
    codes, scales, c, s = pool_of(nb, B, hkv, d, T)
    k, v = odd_rows(T, hkv, d, T + 1), odd_rows(T, hkv, d, T + 2)
    slots = random_slots(T, nb * B, T)
    # rows of k and v side by side in a wider row: their strides are not Hkv * D
    row = hkv * d
    wide = torch.zeros(T, 2 * row + extra, dtype=torch.bfloat16, device="cuda")
    wide[:, :row], wide[:, row:2 * row] = bf16(k).flatten(1), bf16(v).flatten(1)
    binding.pkv_quant_kv_write(c, s, wide[:, :row].view(T, hkv, d), wide[:, row:2 * row].view(T, hkv, d),
                               torch.from_numpy(slots).cuda())
    want = oracle.quant_write(codes, scales, k, v, slots)
    assert np.array_equal(s.cpu().numpy(), want[1])
    assert np.array_equal(host(c), want[0])
    assert binding.pkv_get_device_errors(clear=True) == 0


def test_every_finite_bf16_is_written_as_defined():
    """Every bf16 magnitude as an element under a fixed largest one, and as a row's largest."""
    mags = np.arange(0, 0x7F80, dtype=np.uint16)
    rows = [np.resize(mags, (255, 128))]
    for top in (0x0001, 0x0080, 0x3F80, 0x3FE0, 0x3FE1, 0x4360, 0x7F7F):
        small = np.minimum(rows[0], np.uint16(top))
        small[:, 0] = top
        rows.append(small | np.uint16(0x8000) * (np.arange(128) % 2).astype(np.uint16))
    k = np.concatenate(rows)
    first = np.zeros((len(mags), 128), np.uint16)
    first[:, 3] = mags
    first[:, 7] = mags // 3
    k = np.concatenate([k, first])[:, None, :]
    T = k.shape[0]
    nb = -(-T // 16)
    c = torch.zeros(nb, 2, 16, 1, 128, dtype=torch.uint8, device="cuda").view(E4M3)
    s = torch.zeros(nb, 2, 16, 1, dtype=torch.uint8, device="cuda")
    t = bf16(k)
    binding.pkv_quant_kv_write(c, s, t, t, torch.arange(T, device="cuda"))
    codes, scales = oracle.quantise_rows(k)
    for i in (0, 1):
        assert np.array_equal(host(c)[:, i].reshape(-1, 1, 128)[:T], codes)
        assert np.array_equal(s.cpu().numpy()[:, i].reshape(-1, 1)[:T], scales)


@pytest.mark.parametrize("hq,hkv,d,B", SHAPES + [(40, 40, 128, 16)])
def test_mapped_write_and_the_step_write_equal_the_two_calls(hq, hkv, d, B):
    step = make_step(batch(seed=d), num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=B, seed=B)
    step.k, step.v = odd_rows(step.num_tokens, hkv, d, 1), odd_rows(step.num_tokens, hkv, d, 2)
    codes, scales, _ = quantised_step(step)
    for kw in ({}, {"fused_write": True}, {"write_in_attention": True}):
        ds = DeviceStep(step, quantised=True, **kw)
        ds.run()
        got = ds.quant_pool_host()
        assert np.array_equal(got[1], scales), kw
        assert np.array_equal(got[0], codes), kw
        assert np.array_equal(ds.slots_host(), oracle.slot_mapping(
            step.block_table, step.query_start_loc, step.num_computed, B))
    assert binding.pkv_get_device_errors(clear=True) == 0


@pytest.mark.parametrize("T,hkv,d,B", ROWS)
@pytest.mark.parametrize("gap", [0, 8, 16])  # rows 32-byte aligned, 16-byte aligned, strided
def test_read_is_exact_and_leaves_padding_alone(T, hkv, d, B, gap):
    nb = -(-T // B) + 3
    codes, scales, c, s = pool_of(nb, B, hkv, d, T)
    slots = random_slots(T, nb * B, T)
    slots[T // 2] = slots[0]  # a row read twice
    row = hkv * d
    wide = torch.full((T, 2 * row + gap), 5.0, dtype=torch.bfloat16, device="cuda")
    k, v = wide[:, :row].view(T, hkv, d), wide[:, row + gap:].view(T, hkv, d)
    before = bf16_to_numpy(k.contiguous())
    binding.pkv_quant_kv_read(k, v, c, s, torch.from_numpy(slots).cuda())
    want = oracle.quant_read(before, before.copy(), codes, scales, slots)
    for got, w in zip((k, v), want):
        got = bits_to_f64(bf16_to_numpy(got.contiguous()))
        assert np.array_equal(got, bits_to_f64(w), equal_nan=True)
    assert (wide[:, row:row + gap] == 5.0).all()
    assert binding.pkv_get_device_errors(clear=True) == 0


def test_rows_read_back_and_written_again_keep_their_values():
    T, hkv, d, B = 3000, 4, 128, 16
    codes, scales, c, s = pool_of(-(-T // B), B, hkv, d, 5)
    slots = torch.randperm(c.shape[0] * B, device="cuda")
    k = torch.empty(slots.shape[0], hkv, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    binding.pkv_quant_kv_read(k, v, c, s, slots)
    binding.pkv_quant_kv_write(c, s, k, v, slots)
    assert np.array_equal(oracle.quant_values(host(c), s.cpu().numpy()),
                          oracle.quant_values(codes, scales), equal_nan=True)


def test_slots_out_of_the_pool_are_skipped_and_flagged():
    codes, scales, c, s = pool_of(4, 16, 2, 64, 1)
    k = bf16(odd_rows(3, 2, 64, 2))
    slots = torch.tensor([64, 1 << 40, 3], device="cuda")
    binding.pkv_quant_kv_write(c, s, k, k, slots)
    want = oracle.quant_write(codes, scales, odd_rows(3, 2, 64, 2), odd_rows(3, 2, 64, 2), [-1, -1, 3])
    assert np.array_equal(host(c), want[0]) and np.array_equal(s.cpu().numpy(), want[1])
    assert binding.pkv_get_device_errors(clear=True) == binding.DEVERR_SLOT_RANGE
    out = torch.full_like(k, 2.0)
    binding.pkv_quant_kv_read(out, out.clone(), c, s, slots)
    assert (out[:2] == 2.0).all()
    assert binding.pkv_get_device_errors(clear=True) == binding.DEVERR_SLOT_RANGE


@pytest.mark.parametrize("hkv,d,B", [(1, 64, 8), (3, 128, 16), (8, 128, 32)])
@pytest.mark.parametrize("pinned", [False, True])
def test_copy_blocks(hkv, d, B, pinned):
    codes, scales, c, s = pool_of(9, B, hkv, d, 3)
    dst = torch.zeros(7, 2, B, hkv, d, dtype=torch.uint8)
    dst_s = torch.zeros(7, 2, B, hkv, dtype=torch.uint8)
    dst, dst_s = (dst.pin_memory(), dst_s.pin_memory()) if pinned else (dst.cuda(), dst_s.cuda())
    pairs = torch.tensor([[8, 0], [2, 6], [2, 3], [9, 1], [0, 7]], dtype=torch.int32, device="cuda")
    binding.pkv_quant_copy_blocks(dst.view(E4M3), dst_s, c, s, pairs)
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == binding.DEVERR_BLOCK_RANGE
    for src, d_ in ((8, 0), (2, 6), (2, 3)):
        assert np.array_equal(dst[d_].cpu().numpy(), codes[src])
        assert np.array_equal(dst_s[d_].cpu().numpy(), scales[src])
    for d_ in (1, 2, 4, 5):
        assert not dst[d_].any() and not dst_s[d_].any()


# ------------------------------------------------------------------ attention
def assert_within(bits, ref, bound, what=""):
    g = bits_to_f64(bits)
    err = np.abs(g - ref)
    bad = ~(err <= bound + 1e-30)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what} {int(bad.sum())} of {bad.size} out of bound; first {i}: gpu "
                             f"{g[i]} ref {ref[i]} bound {bound[i]}; worst ratio "
                             f"{np.nanmax(err / (bound + 1e-30)):.2f}")


MODS = {
    "plain": dict(),
    "cap": dict(softcap=20.0),
    "small-cap": dict(softcap=0.5),
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


def check(step, what="", flags=0, decode_splits=None, shared_prefix=None, write=True, few_rows=None,
          **scores):
    ds = DeviceStep(step, quantised=True, write_in_attention=write, decode_splits=decode_splits,
                    shared_prefix=shared_prefix, few_rows=few_rows, **scores)
    ds.out.fill_(7.0)
    ds.run()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == flags
    assert_within(ds.out_host(), *expected(step, quantised_step(step)[2], **scores), what=what)
    return ds


@pytest.mark.parametrize("mod", MODS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_every_shape_and_score(shape, mod):
    """Decodes, requests of a few tokens and chunks in one step."""
    hq, hkv, d, B = shape
    step = make_step(batch(seed=hq + d), num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=B,
                     seed=hq * d + B, scale=1.5 / d ** 0.5)
    check(step, f"{shape} {mod}", **scores_for(step, MODS[mod]))


@pytest.mark.parametrize("mod", ["plain", "cap-alibi", "window", "random"])
@pytest.mark.parametrize("rows", [1, 2, 3, 5, 8, 16, 32, 64])
@pytest.mark.parametrize("hq,hkv,d,B", [(8, 1, 64, 32), (16, 4, 128, 16), (4, 4, 64, 8), (6, 3, 128, 8),
                                        (24, 12, 64, 16)])
def test_requests_of_a_few_tokens(hq, hkv, d, B, rows, mod):
    """Every request of the step has few new tokens: all of them are on the decode
    stream while rows x heads fit it, and behind that some or none."""
    rng = np.random.default_rng(rows * d)
    specs = [RequestSpec(int(c), int(n)) for c, n in zip(
        [0, 1, 15, 16, 17, 300, 811, 40, 1203, 5], rng.integers(1, rows + 1, size=10))]
    specs[4] = RequestSpec(17, rows)
    step = make_step(specs, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=B, seed=rows + B)
    check(step, f"{rows} rows {mod}", **scores_for(step, MODS[mod], seed=rows))


@pytest.mark.parametrize("mod", ["plain", "cap-alibi", "window", "random"])
@pytest.mark.parametrize("splits", [1, 2, 7, 152, 1000])
@pytest.mark.parametrize("rows", [1, 5])
def test_any_split_of_the_decode_stream(splits, mod, rows):
    specs = [RequestSpec(c, 1 + (i % rows)) for i, c in enumerate((0, 1, 15, 16, 17, 700, 1499, 31, 2200, 64))]
    step = make_step(specs, num_q_heads=8, num_kv_heads=2, head_dim=128, seed=3)
    check(step, decode_splits=splits, **scores_for(step, MODS[mod], seed=splits))


@pytest.mark.parametrize("mod", ["plain", "cap-alibi", "random"])
@pytest.mark.parametrize("few", [1, 2, 4, 6, 16])
def test_a_chosen_number_of_rows_beside_long_chunks(few, mod):
    """Requests of up to few_rows new tokens on the decode kernels, the others and a
    shared prefix on the prefill kernel, whatever the longest is."""
    specs = [RequestSpec(70, 20), RequestSpec(33, 1), RequestSpec(400, 5), RequestSpec(200, 90),
             RequestSpec(901, 4), RequestSpec(17, 3), RequestSpec(5, 16)] + [
        RequestSpec(64 + s, 1, shares_prefix=True) for s in (0, 9, 40)] + [RequestSpec(320, 2)]
    step = make_step(specs, num_q_heads=16, num_kv_heads=4, head_dim=128, prefix_tokens=64, seed=few)
    check(step, few_rows=few, shared_prefix="auto", **scores_for(step, MODS[mod], seed=few))
    check(step, few_rows=few, write=False, **scores_for(step, MODS[mod], seed=few))


@pytest.mark.parametrize("mod", MODS)
@pytest.mark.parametrize("B", [8, 16, 32])
def test_shared_prefix(B, mod):
    specs = [RequestSpec(40, 30)] + [RequestSpec(192 + s, 1, shares_prefix=True)
                                     for s in (0, 1, 9, 40, 300, 17, 16, 15, 33)] + [RequestSpec(77, 1)]
    step = make_step(specs, num_q_heads=16, num_kv_heads=4, head_dim=64, block_size=B,
                     prefix_tokens=192, seed=B)
    check(step, shared_prefix="auto", **scores_for(step, MODS[mod], seed=B))


@pytest.mark.parametrize("mod", MODS)
def test_chunks_equal_the_bf16_pool_of_the_same_values(mod):
    """Rows on the prefill kernel are bit for bit those of pkv_paged_attention over
    the pool's values."""
    specs = [RequestSpec(300, 200), RequestSpec(0, 129), RequestSpec(1000, 40)]
    step = make_step(specs, num_q_heads=32, num_kv_heads=8, head_dim=128, seed=9)
    scores = scores_for(step, MODS[mod])
    quant = check(step, **scores)
    plain = DeviceStep(step, **scores)
    pool = quantised_step(step)[2]
    plain.kv_cache.copy_(bf16(pool))
    plain.attend()
    torch.cuda.synchronize()
    assert np.array_equal(quant.out_host(), plain.out_host())


def test_rows_of_nan_reach_the_rows_that_see_them_only():
    """NaN rows of K and V (an infinity in a written row) behind a window, and in it."""
    specs = [RequestSpec(200, 1), RequestSpec(200, 3), RequestSpec(333, 1), RequestSpec(90, 40)]
    step = make_step(specs, num_q_heads=8, num_kv_heads=2, head_dim=64, seed=4)
    T = step.num_tokens
    begin = np.zeros(T, np.int32)
    end = np.zeros(T, np.int32)
    for r, s in enumerate(specs):
        t0 = int(step.query_start_loc[r])
        begin[t0:t0 + s.query_len] = 50
        end[t0:t0 + s.query_len] = s.num_computed - 20
    bad = step.kv_cache.copy()
    for r, s in enumerate(specs):
        for j, what in ((10, 0x7F80), (49, 0x7FC0), (s.num_computed - 20, 0xFF80), (s.num_computed - 1, 0x7FC0)):
            blk = step.block_table[r, j // 16]
            bad[blk, :, j % 16, :, 5] = what
    step.kv_cache = bad
    ds = check(step, key_begin=begin, key_end=end)
    assert np.isfinite(bits_to_f64(ds.out_host())).all()
    # and one that request 0 sees, in head 1 alone
    blk = step.block_table[0, 100 // 16]
    step.kv_cache[blk, 1, 100 % 16, 1, 7] = 0x7F80
    ds = DeviceStep(step, quantised=True, write_in_attention=True, key_begin=begin, key_end=end)
    ds.run()
    got = bits_to_f64(ds.out_host())
    assert np.isnan(got[0, 4:]).all() and np.isfinite(got[0, :4]).all() and np.isfinite(got[1:]).all()


def test_bad_blocks_are_masked_and_flagged():
    specs = [RequestSpec(300, 1), RequestSpec(300, 2), RequestSpec(200, 60)]
    step = make_step(specs, num_q_heads=8, num_kv_heads=2, head_dim=128, seed=6)
    ds = DeviceStep(step, quantised=True, write_in_attention=True)
    ds.block_table[0, 3] = step.num_blocks
    ds.block_table[1, 4] = -1
    ds.block_table[2, 1] = -7
    ds.run()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == binding.DEVERR_BLOCK_RANGE
    begin = np.zeros(step.num_tokens, np.int32)
    got = bits_to_f64(ds.out_host())
    _, _, pool = quantised_step(step)
    for r, e in ((0, 3), (1, 4), (2, 1)):  # as if those sixteen keys were not there
        t0, n, L = int(step.query_start_loc[r]), specs[r].query_len, specs[r].seq_len
        keep = [j for j in range(L) if j // 16 != e]
        for i in range(n):
            seen = [j for j in keep if j <= L - n + i]
            blk = step.block_table[r][np.array(seen) // 16]
            k, v = (bits_to_f64(pool[blk, x, np.array(seen) % 16]) for x in (0, 1))
            q = bits_to_f64(step.q[t0 + i]).reshape(2, 4, 128)
            x = step.scale * np.einsum("hgd,nhd->hgn", q, k)
            w = np.exp(x - x.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            want = np.einsum("hgn,nhd->hgd", w, v).reshape(8, 128)
            assert np.abs(got[t0 + i] - want).max() < 2e-2
    assert (begin == 0).all()


def test_too_small_a_workspace_for_the_chunks_is_flagged():
    specs = [RequestSpec(100, 100), RequestSpec(700, 300), RequestSpec(60, 1)]
    step = make_step(specs, num_q_heads=8, num_kv_heads=2, head_dim=128, seed=6)
    ds = DeviceStep(step, quantised=True, write_in_attention=True)
    size = binding.pkv_quant_attention_workspace_size(
        3, 8, ds.layout, max_blocks_per_req=step.max_blocks_per_req, chunk_keys=208)
    ds.workspace = torch.empty(size, dtype=torch.uint8, device="cuda")
    tail = torch.full_like(ds.workspace, 3)
    ds.run()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) & binding.DEVERR_CHUNK_KEYS
    assert (tail == 3).all()
    ref, bound = expected(step, quantised_step(step)[2])
    keep = np.r_[0:100, 400]  # the first chunk fits, the decode needs no room
    got = ds.out_host()
    assert_within(got[keep], ref[keep], bound[keep])


def test_rows_behind_the_batch_stay_as_they_were():
    step = make_step([RequestSpec(30, 1), RequestSpec(50, 4), RequestSpec(10, 30)], num_q_heads=8,
                     num_kv_heads=2, head_dim=64, seed=1)
    ds = DeviceStep(step, quantised=True)
    T = step.num_tokens
    q = torch.cat([ds.q, torch.full_like(ds.q[:9], float("nan"))])
    out = torch.full_like(q, 3.0)
    ds.slot_map()
    ds.write()
    binding.pkv_quant_paged_attention(
        out, q, ds.kv_cache, ds.kv_scales, ds.block_table, ds.seq_lens, ds.query_start_loc,
        ds.num_computed, max_query_len=step.max_query_len, max_seq_len=step.max_seq_len,
        scale=step.scale, workspace=ds.workspace)
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == 0
    assert (out[T:] == 3.0).all()
    assert_within(bf16_to_numpy(out[:T]), *expected(step, quantised_step(step)[2]))


@pytest.mark.parametrize("specs", [
    [RequestSpec(300, 1), RequestSpec(20, 1)],
    [RequestSpec(300, 5), RequestSpec(20, 2)],
    [RequestSpec(300, 70), RequestSpec(20, 1), RequestSpec(800, 2)]], ids=["decode", "few", "mixed"])
def test_a_step_recorded_into_a_graph(specs):
    step = make_step(specs, num_q_heads=16, num_kv_heads=4, head_dim=128, seed=2)
    ds = DeviceStep(step, quantised=True, write_in_attention=True)
    want = expected(step, quantised_step(step)[2])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ds.run()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ds.run()
    for fill in (1.0, 9.0):
        ds.out.fill_(fill)
        graph.replay()
        torch.cuda.synchronize()
        assert_within(ds.out_host(), *want)
    assert binding.pkv_get_device_errors(clear=True) == 0


def test_empty_calls():
    lay = (4, 2, 16, 2, 64)
    c = torch.zeros(lay, dtype=torch.uint8, device="cuda").view(E4M3)
    s = torch.zeros(lay[:4], dtype=torch.uint8, device="cuda")
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    binding.pkv_quant_kv_write(c, s, none, none, slots)
    binding.pkv_quant_kv_read(none, none, c, s, slots)
    binding.pkv_quant_copy_blocks(c, s, c, s, torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert binding.pkv_get_device_errors(clear=True) == 0
