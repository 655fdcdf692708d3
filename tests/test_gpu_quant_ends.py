"""The 8-bit pool at the ends of bf16's exponent range: every finite row has finite
values."""

import numpy as np
import pytest

import oracle
from parity import bits_to_f64

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


def top_rows(num_tokens, hkv, d, seed):
    """Rows whose largest magnitude is one of the last bf16 (0x7f60 .. 0x7f7f: 1.75 *
    2^127 and above), their elements of that size or less."""
    rng = np.random.default_rng(seed)
    top = np.resize(np.arange(0x7F60, 0x7F80), (num_tokens, hkv, 1))
    x = np.minimum(rng.integers(0x7E00, 0x7F80, (num_tokens, hkv, d)), top)
    x[..., rng.integers(0, d)] = top[..., 0]
    return (x | rng.integers(0, 2, x.shape) << 15).astype(np.uint16)


@pytest.mark.parametrize("hkv,d,B", [(3, 128, 16), (2, 64, 8), (20, 128, 32)])
def test_the_largest_rows_read_back_as_the_largest_values(hkv, d, B):
    """All three ways to write, and the rows read back: finite, and within 2^-4 of what
    was written."""
    step = make_step([RequestSpec(5, 40), RequestSpec(30, 1), RequestSpec(0, 70)], num_q_heads=hkv,
                     num_kv_heads=hkv, head_dim=d, block_size=B, seed=B)
    step.k, step.v = (top_rows(step.num_tokens, hkv, d, i) for i in (1, 2))
    slots = oracle.slot_mapping(step.block_table, step.query_start_loc, step.num_computed, B)
    codes, scales = oracle.quant_write(*oracle.quantise_rows(step.kv_cache), step.k, step.v, slots)
    for kw in ({}, {"fused_write": True}, {"write_in_attention": True}):
        ds = DeviceStep(step, quantised=True, **kw)
        ds.run()
        assert np.array_equal(ds.quant_pool_host()[0], codes), kw
        assert np.array_equal(ds.quant_pool_host()[1], scales), kw
        k, v = torch.zeros_like(ds.k), torch.zeros_like(ds.v)
        binding.pkv_quant_kv_read(k, v, ds.kv_cache, ds.kv_scales, ds.slot_mapping)
        for got, wrote in ((k, step.k), (v, step.v)):
            got, wrote = bits_to_f64(bf16_to_numpy(got)), bits_to_f64(wrote)
            assert np.isfinite(got).all()
            assert (np.abs(got - wrote) <= 2.0 ** -4 * np.abs(wrote)).all()
