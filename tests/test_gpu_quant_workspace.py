"""The 8-bit calls' workspace: no larger than the partials that a call can leave, and
nothing behind it is written."""

import numpy as np
import pytest

from quant_cases import expected, quantised_step
from test_gpu_quant import assert_within

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_hkv_gb300 import binding  # noqa: E402
from paged_kv_cache_hkv_gb300.runner import DeviceStep  # noqa: E402
from paged_kv_cache_hkv_gb300.synth import RequestSpec, make_step  # noqa: E402

GUARD = 1 << 20


def guarded(size):
    """A workspace of `size` bytes and the filled bytes behind it."""
    buf = torch.full((size + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    assert buf.data_ptr() % 256 == 0
    return buf[:size], buf[size:]


def size_of(ds, chunk_keys, decode_splits=None):
    s = ds.step
    return binding.pkv_quant_attention_workspace_size(
        s.num_reqs, s.num_q_heads, ds.layout, max_blocks_per_req=s.max_blocks_per_req,
        chunk_keys=chunk_keys, decode_splits=decode_splits)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 1, 128), (16, 16, 128), (4, 2, 64), (12, 12, 64),
                                      (64, 8, 128), (40, 40, 128)])
def test_the_size_follows_from_the_ctas_of_a_wave(hq, hkv, d):
    """A CTA holds at most 24 units (three tiles of 8) in each of its eight warps, an
    SM's CTAs of one tile 16 of 8; a CTA leaves two partials of (maximum, sum, O) for
    each of them. With fewer CTAs in a wave than there are slabs of kv heads every slab
    has one: heads x 64 / group rows then."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lay = binding.pkv_cache_layout(1000, 16, hkv, d)
    size = binding.pkv_quant_attention_workspace_size(1, hq, lay, max_blocks_per_req=64, chunk_keys=0)
    few = 2 * max(24 * 8 * sms, hq * (64 // (hq // hkv))) * (d + 2) * 4
    one = (1 + 20 * sms) * hq * (d + 2) * 4  # single tokens: a partial for each CTA and request
    assert size <= few + one + (1 << 20)


@pytest.mark.parametrize("hq,hkv,d,B", [(16, 4, 128, 16), (8, 1, 64, 32), (6, 6, 64, 8), (72, 9, 64, 16)])
def test_nothing_behind_the_workspace_is_written(hq, hkv, d, B):
    """Every number of new tokens on the decode kernels, requests cut by many CTAs."""
    group = hq // hkv
    for rows in sorted({1, 2, 3, 5, 8, 12, 16, 24, 33, 64 // group} & set(range(1, 64 // group + 1))):
        specs = [RequestSpec(c, 1 + (rows - 1) * (i % 2)) for i, c in enumerate((3900, 700, 31, 2000, 5, 900))]
        step = make_step(specs, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=B, seed=rows)
        ds = DeviceStep(step, quantised=True, write_in_attention=True)
        ds.workspace, guard = guarded(size_of(ds, 0))
        ds.run()
        torch.cuda.synchronize()
        assert binding.pkv_get_device_errors(clear=True) == 0
        assert (guard == 0xA5).all()
        if rows in (1, 3, 64 // group):
            assert_within(ds.out_host(), *expected(step, quantised_step(step)[2]), what=rows)


@pytest.mark.parametrize("splits", [1, 500])
def test_nothing_behind_it_with_a_callers_splits(splits):
    step = make_step([RequestSpec(1900, 16), RequestSpec(700, 1), RequestSpec(40, 9)], num_q_heads=16,
                     num_kv_heads=4, head_dim=128, seed=splits)
    ds = DeviceStep(step, quantised=True, write_in_attention=True, decode_splits=splits)
    ds.workspace, guard = guarded(size_of(ds, 0, splits))
    ds.run()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == 0
    assert (guard == 0xA5).all()
    assert_within(ds.out_host(), *expected(step, quantised_step(step)[2]))


def test_nothing_behind_it_where_the_chunks_do_not_fit():
    specs = [RequestSpec(100, 100), RequestSpec(700, 300), RequestSpec(60, 1)]
    step = make_step(specs, num_q_heads=8, num_kv_heads=2, head_dim=128, seed=6)
    ds = DeviceStep(step, quantised=True, write_in_attention=True)
    ds.workspace, guard = guarded(size_of(ds, 208))
    ds.run()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) & binding.DEVERR_CHUNK_KEYS
    assert (guard == 0xA5).all()
    ref, bound = expected(step, quantised_step(step)[2])
    keep = np.r_[0:100, 400]  # the first chunk fits, the decode needs no room
    assert_within(ds.out_host()[keep], ref[keep], bound[keep])
