"""Key ranges that leave holes: keys between those of a request's rows that none of
them sees never reach the output of the 8-bit pool's calls, whatever they hold."""

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


@pytest.mark.parametrize("few_rows", [None, 1])  # the decode kernels, the prefill kernel
@pytest.mark.parametrize("rows", [2, 4, 6])
@pytest.mark.parametrize("hq,hkv,d,B", [(8, 2, 64, 16), (16, 4, 128, 8), (8, 1, 128, 32), (4, 4, 64, 32)])
def test_places_between_the_rows_ranges_hold_anything(hq, hkv, d, B, rows, few_rows):
    specs = [RequestSpec(c, rows) for c in (400, 37, 16, 90)]
    step = make_step(specs, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=B, seed=rows + B)
    rng = np.random.default_rng(rows + d)
    begin, end = np.zeros((2, step.num_tokens), np.int32)
    seen = np.zeros((len(specs), step.max_seq_len), bool)
    for r, s in enumerate(specs):
        for i in range(rows):
            t = int(step.query_start_loc[r]) + i
            a = int(rng.integers(0, s.seq_len - 1))
            begin[t], end[t] = a, min(a + int(rng.integers(1, 12)), s.seq_len)
            seen[r, begin[t]:end[t]] = True
    ds = DeviceStep(step, quantised=True, write_in_attention=True, key_begin=begin, key_end=end,
                    few_rows=few_rows)
    codes, scales = ds.kv_cache.view(torch.uint8), ds.kv_scales
    for r, s in enumerate(specs):  # (the new tokens' rows are written by the call)
        j = np.flatnonzero(~seen[r, :s.num_computed])
        blk = torch.from_numpy(step.block_table[r, j // B].astype(np.int64)).cuda()
        off = torch.from_numpy(j % B).cuda()
        for i in (0, 1):
            codes[blk, i, off] = torch.tensor([0x7F, 0xFF], dtype=torch.uint8, device="cuda").repeat(d // 2)
            scales[blk, i, off] = 255 if i else 254
    ds.run()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == 0
    assert_within(ds.out_host(), *expected(step, quantised_step(step)[2], key_begin=begin, key_end=end))
