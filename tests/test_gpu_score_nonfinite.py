"""Infinities and NaN in V under scored attention: what each row must hold, key
by key, where few and where most of the keys are bad; bad blocks among them; and
that a chunk whose V is all NaN takes no longer than a few times a clean one."""

import numpy as np
import pytest

from parity import bits_to_f64
from score_cases import key_ranges, slopes_of

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_hkv_gb300 import binding  # noqa: E402
from paged_kv_cache_hkv_gb300.runner import DeviceStep  # noqa: E402
from paged_kv_cache_hkv_gb300.synth import RequestSpec, make_step  # noqa: E402
from test_gpu_scores import expected  # noqa: E402


@pytest.fixture(autouse=True)
def _clear_errors():
    binding.pkv_get_device_errors(clear=True)
    yield


KINDS = {1: 0x7FC0, 2: 0x7F80, 4: 0xFF80}  # NaN, +infinity, -infinity


def at_key(step, r, j):
    """A view of the V row [Hkv, D] of key j of request r, in the pool or the new rows."""
    c = step.num_computed[r]
    if j >= c:
        return step.v[step.query_start_loc[r] + j - c]
    B = step.block_size
    return step.kv_cache[step.block_table[r][j // B], 1, j % B]


def poison(step, share, rng):
    """Bad values in a share of the keys: kinds[r] uint8 [keys, D], a KINDS bit or 0."""
    kinds = []
    for r, s in enumerate(step.specs):
        k = np.zeros((s.seq_len, step.head_dim), np.uint8)
        for j in np.flatnonzero(rng.random(s.seq_len) < share):
            dims = rng.choice(step.head_dim, size=int(rng.integers(1, 6)), replace=False)
            for d in dims:
                # most dimensions get one kind only, so that infinities stay visible
                k[j, d] = rng.choice([1, 2, 4]) if d % 8 == 0 else (2 if d % 2 else 4)
                at_key(step, r, j)[:, d] = KINDS[int(k[j, d])]
        kinds.append(k)
    return kinds


def check(step, out, kinds, clean, begin, end):
    """`clean`: (reference, bound) with zeros in the bad places."""
    got = bits_to_f64(out)
    ref, bound = clean
    seen_any = 0
    for r, s in enumerate(step.specs):
        for i in range(s.query_len):
            t = step.query_start_loc[r] + i
            lo, hi = max(0, begin[t]), min(end[t], s.seq_len)
            seen = np.bitwise_or.reduce(kinds[r][lo:hi], axis=0) if lo < hi else 0 * kinds[r][0]
            nan = (seen & 1 > 0) | (seen & 6 == 6)
            want = np.where(nan, np.nan, np.where(seen == 2, np.inf, np.where(seen == 4, -np.inf, 0.0)))
            bad = seen > 0
            seen_any += bad.any()
            assert (np.abs(got[t][:, ~bad] - ref[t][:, ~bad]) <= bound[t][:, ~bad] + 1e-30).all(), (r, i)
            assert np.array_equal(got[t][:, bad], np.broadcast_to(want[bad], got[t][:, bad].shape),
                                  equal_nan=True), (r, i)
    assert seen_any > 20


SPECS = [RequestSpec(300, 150), RequestSpec(0, 140), RequestSpec(150, 1), RequestSpec(170, 45)]


@pytest.mark.parametrize("share", [0.02, 0.6])
@pytest.mark.parametrize("form", ["ranges", "cap", "bias"])
@pytest.mark.parametrize("mask", ["documents", "window", "random"])
@pytest.mark.parametrize("d,B", [(64, 8), (128, 16), (128, 8), (64, 32)])
def test_each_row_holds_what_its_keys_say(d, B, mask, form, share):
    scores = {"ranges": {}, "cap": dict(softcap=20.0),
              "bias": dict(alibi_slopes=slopes_of(8) * np.float32(0.1))}[form]
    rng = np.random.default_rng(d + B)
    step = make_step(SPECS, num_q_heads=8, num_kv_heads=2, head_dim=d, block_size=B, seed=3)
    begin, end = key_ranges(step, mask, 6)
    scores.update(key_begin=begin, key_end=end)
    kinds = poison(step, share, rng)
    ds = DeviceStep(step, write_in_attention=True, **scores)
    ds.run()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == 0
    for r, k in enumerate(kinds):
        for j, dim in np.argwhere(k):
            at_key(step, r, j)[:, dim] = 0
    check(step, ds.out_host(), kinds, expected(step, **scores), begin, end)


@pytest.mark.parametrize("share", [0.02, 0.6])
@pytest.mark.parametrize("d", [64, 128])
def test_under_a_shared_prefix(d, share):
    specs = [RequestSpec(160 + s, 1, shares_prefix=True) for s in (0, 3, 70, 9, 31)]
    specs += [RequestSpec(20, 60)]
    rng = np.random.default_rng(d)
    step = make_step(specs, num_q_heads=8, num_kv_heads=2, head_dim=d, prefix_tokens=160, seed=4)
    begin, end = key_ranges(step, "random", 8)
    scores = dict(softcap=20.0, key_begin=begin, key_end=end)
    kinds = poison(step, share, rng)
    for r in range(5):  # the prefix is one: what every sharer's last poison left there
        for j in range(160):
            row = at_key(step, r, j)[0]
            kinds[r][j] = np.where((row & 0x7F80) != 0x7F80, 0,
                                   np.where(row & 0x7F, 1, np.where(row & 0x8000, 4, 2)))
    ds = DeviceStep(step, write_in_attention=True, shared_prefix=(160, 0, 5), **scores)
    ds.run()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == 0
    for r, k in enumerate(kinds):
        for j, dim in np.argwhere(k):
            at_key(step, r, j)[:, dim] = 0
    check(step, ds.out_host(), kinds, expected(step, **scores), begin, end)


def test_a_masked_chunk_gives_nothing_back():
    """Blocks of 8: the other half of a chunk whose one block is out of the pool
    is masked with it, so its infinities do not come back where most keys are
    bad."""
    step = make_step([RequestSpec(200, 60)], num_q_heads=4, num_kv_heads=2, head_dim=64, block_size=8,
                     seed=5)
    T = step.num_tokens
    for j in range(260):
        at_key(step, 0, j)[:, 7] = 0x7F80
    begin, end = np.zeros(T, np.int32), np.zeros(T, np.int32)
    begin[:30], end[:30] = 40, 48      # the masked half (block 5; block 4 is gone)
    begin[30:], end[30:] = 48, 200     # the others see infinities
    ds = DeviceStep(step, key_begin=begin, key_end=end)
    ds.slot_map()
    ds.write()
    ds.block_table[0, 4] = -1
    begin2 = begin.copy()
    begin2[29] = 32                    # one row's range makes block 4 a used one
    ds.scores["key_begin"] = torch.from_numpy(begin2).cuda()
    ds.attend()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == binding.DEVERR_BLOCK_RANGE
    out = bits_to_f64(ds.out_host())
    assert (out[:30] == 0).all()
    assert (out[30:, :, 7] == np.inf).all() and np.isfinite(np.delete(out[30:], 7, axis=2)).all()


@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_a_chunk_of_nan_takes_no_longer_than_a_few_clean_ones(d, alibi):
    """512 rows over 32768 keys; V of the chunk's own keys all NaN, and every
    third of all keys infinite in some elements."""
    n, c, hq, hkv, B = 512, 32768 - 512, 32, 8, 16
    blocks = (n + c) // B
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    kv = torch.empty(blocks, 2, B, hkv, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    q = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
    work = torch.empty(binding.pkv_attention_workspace_size(1, hq, kv), dtype=torch.uint8, device="cuda")
    args = (out, q, kv, torch.arange(blocks, dtype=torch.int32, device="cuda").view(1, -1), i32(n + c),
            i32(0, n), i32(c))
    kw = dict(max_query_len=n, max_seq_len=n + c, scale=d ** -0.5, workspace=work, softcap=50.0,
              alibi_slopes=torch.full((hq,), 1e-4, device="cuda") if alibi else None)

    def best():
        times = []
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            binding.pkv_paged_attention(*args, **kw)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    clean = best()
    v = kv[:, 1]
    own = v[c // B:].clone()
    v[c // B:] = float("nan")
    nan = best()
    assert out.isnan().all(-1).all(-1).all()
    v[c // B:] = own
    v[:, ::3, :, 5] = float("inf")
    inf = best()
    assert (out[:, :, 5] == float("inf")).all()
    assert binding.pkv_get_device_errors(clear=True) == 0
    # (the search itself is some 1000 turns of a warp; before it was shared by
    # the lanes the first was 200 times a clean call)
    assert nan < 8 * clean and inf < 30 * clean, (clean, nan, inf)
