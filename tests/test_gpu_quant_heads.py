"""The 8-bit decode with as many kv heads as a stage holds scales of."""

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


@pytest.mark.parametrize("hkv,B,rows", [(1799, 16, 1), (1792, 8, 3), (1024, 32, 20)])
def test_as_many_kv_heads_as_always_fit(hkv, B, rows):
    specs = [RequestSpec(50, rows), RequestSpec(5, 1), RequestSpec(17, 1)]
    step = make_step(specs, num_q_heads=hkv, num_kv_heads=hkv, head_dim=64, block_size=B, seed=rows)
    binding.pkv_get_device_errors(clear=True)
    for splits in (None, 4):
        ds = DeviceStep(step, quantised=True, write_in_attention=True, decode_splits=splits)
        ds.run()
        torch.cuda.synchronize()
        assert binding.pkv_get_device_errors(clear=True) == 0
        assert_within(ds.out_host(), *expected(step, quantised_step(step)[2]))
