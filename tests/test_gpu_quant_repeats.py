"""Attention over the 8-bit pool gives the same bits whatever lies in the places of the
pool that hold no key of a request, and in shared memory before the call."""

import numpy as np
import pytest

from quant_cases import expected, quantised_step
from score_cases import key_ranges
from test_gpu_quant import assert_within

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_hkv_gb300 import binding  # noqa: E402
from paged_kv_cache_hkv_gb300.runner import DeviceStep  # noqa: E402
from paged_kv_cache_hkv_gb300.synth import RequestSpec, make_step  # noqa: E402

# (code, scale byte): what rows of the pool can hold
FILLS = [(0, 10), (0x7E, 247), (0xFE, 140), (0, 255), (0x38, 190)]


@pytest.mark.parametrize("mask", [None, "window"])
@pytest.mark.parametrize("rows", [1, 2, 5])
@pytest.mark.parametrize("hq,hkv,d,B", [(12, 12, 64, 8), (6, 6, 128, 16), (4, 2, 64, 32), (16, 4, 128, 16),
                                        (8, 1, 128, 8)])
def test_rows_that_are_no_keys_change_no_bit(hq, hkv, d, B, rows, mask):
    specs = [RequestSpec(c, 1 + i % rows) for i, c in enumerate((0, 3, 17, 40, 300, 811, 1203, 90))]
    step = make_step(specs, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=B, seed=rows + d,
                     scale=3.0 / d ** 0.5)
    scores = dict(zip(("key_begin", "key_end"), key_ranges(step, mask, seed=d))) if mask else {}
    ds = DeviceStep(step, quantised=True, write_in_attention=True, **scores)
    kept = torch.zeros(step.num_blocks * B, dtype=torch.bool)
    for r, s in enumerate(step.specs):
        j = np.arange(s.num_computed)
        kept[torch.from_numpy(step.block_table[r, j // B].astype(np.int64) * B + j % B)] = True
    lost = (~kept).view(-1, 1, B).expand(-1, 2, -1).cuda()
    codes, scales = ds.kv_cache.view(torch.uint8), ds.kv_scales
    first = None
    for code, scale in FILLS:
        codes[lost] = code
        scales[lost] = scale
        ds.out.fill_(7.0)
        ds.run()
        torch.cuda.synchronize()
        got = ds.out_host()
        if first is None:
            first = got
            assert_within(got, *expected(step, quantised_step(step)[2], **scores))
        assert np.array_equal(got, first), (code, scale)
    assert binding.pkv_get_device_errors(clear=True) == 0


@pytest.mark.parametrize("rows", [1, 5])
@pytest.mark.parametrize("hq,hkv,d,B", [(12, 12, 64, 8), (16, 8, 128, 8), (8, 1, 128, 8)])
def test_other_calls_in_between_change_no_bit(hq, hkv, d, B, rows):
    """Half a chunk of a request with 8-token blocks lies in no copy: the stage holds
    what the kernel before left there."""
    rng = np.random.default_rng(rows)
    specs = [RequestSpec(int(c), 1 + i % rows) for i, c in enumerate(rng.integers(100, 1500, 40))]
    step = make_step(specs, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=B, seed=3)
    ds = DeviceStep(step, quantised=True, write_in_attention=True)
    other = make_step([RequestSpec(2000, 1) for _ in range(60)], num_q_heads=32, num_kv_heads=8, head_dim=128,
                      seed=1)
    others = [DeviceStep(other), DeviceStep(other, quantised=True)]
    first = None
    for i in range(12):
        others[i % 2].run()
        others[1].kv_scales.fill_(20 * i)
        ds.run()
        got = ds.out_host()
        first = got if first is None else first
        assert np.array_equal(got, first), i
    assert binding.pkv_get_device_errors(clear=True) == 0
