"""The 8-bit pool at both ends of bf16's exponent range: every finite row has finite
values, and attention over rows of any size is right relative to their size."""

import numpy as np
import pytest

import oracle
from parity import bits_to_f64
from quant_cases import expected, quantised_step
from score_cases import key_ranges

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_hkv_gb300 import binding  # noqa: E402
from paged_kv_cache_hkv_gb300.runner import DeviceStep, bf16_to_numpy  # noqa: E402
from paged_kv_cache_hkv_gb300.synth import RequestSpec, f32_to_bf16_bits, make_step  # noqa: E402


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


def sized(step, power):
    """The step's V rows times 2^power (their NaN padding as it is)."""
    for x in (step.v, step.kv_cache[:, 1]):
        x[...] = f32_to_bf16_bits(np.ldexp(bits_to_f64(x), power).astype(np.float32))


def run_within(step, decode_splits, **scores):
    ds = DeviceStep(step, quantised=True, write_in_attention=True, decode_splits=decode_splits, **scores)
    ds.out.fill_(7.0)
    ds.run()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == 0
    ref, bound = expected(step, quantised_step(step)[2], **scores)
    got = bits_to_f64(ds.out_host())
    # numbers below 2^-126 are zeros: the output's, and a weight's product's
    assert (np.abs(got - ref) <= bound + 2.0 ** -126).all(), np.nanmax(np.abs(got - ref) / (bound + 2.0 ** -126))
    return got


def even_step(rows, d, group, seed):
    """Long and short requests whose keys weigh about the same: the sums of the
    softmax are as large as their numbers of keys."""
    specs = [RequestSpec(c, 1 + i % rows) for i, c in enumerate((2300, 40, 1100, 0, 17, 3100))]
    step = make_step(specs, num_q_heads=2 * group, num_kv_heads=2, head_dim=d, seed=seed)
    step.q = f32_to_bf16_bits((bits_to_f64(step.q) / 32).astype(np.float32))
    return step


@pytest.mark.parametrize("mask", [None, "prefix"])
@pytest.mark.parametrize("splits", [None, 1, 3])
@pytest.mark.parametrize("rows,d,group", [(1, 128, 4), (4, 128, 4), (5, 64, 8), (3, 64, 1)])
@pytest.mark.parametrize("power", [-112, -105])
def test_v_rows_of_the_smallest_sizes(power, rows, d, group, splits, mask):
    step = even_step(rows, d, group, seed=rows)
    sized(step, power)
    scores = dict(zip(("key_begin", "key_end"), key_ranges(step, mask, seed=d))) if mask else {}
    got = run_within(step, splits, **scores)
    assert np.abs(got).max() > 0


@pytest.mark.parametrize("mask", [None, "prefix"])
@pytest.mark.parametrize("splits", [None, 1, 3])
@pytest.mark.parametrize("rows,d,group", [(1, 128, 4), (4, 128, 4), (5, 64, 8), (3, 64, 1)])
@pytest.mark.parametrize("power", [70, 118, "top"])
def test_v_rows_of_the_largest_sizes(power, rows, d, group, splits, mask):
    step = even_step(rows, d, group, seed=rows + 50)
    if power == "top":  # one sign a dim: the outputs are as large as the rows
        sign = (np.arange(d) % 3 == 0).astype(np.uint16) << np.uint16(15)
        for x in (step.v, step.kv_cache[:, 1]):
            x[...] = np.where((x & 0x7FFF) > 0x7F80, x, sign | np.uint16(0x7F7F))
    else:
        sized(step, power)
    scores = dict(zip(("key_begin", "key_end"), key_ranges(step, mask, seed=d))) if mask else {}
    assert np.isfinite(run_within(step, splits, **scores)).all()


@pytest.mark.parametrize("splits", [None, 1, 2])
def test_v_rows_of_both_ends_in_one_request(splits):
    """Requests of tiny rows, of huge ones, and of both: where a piece of a request holds
    huge rows, what tiny ones add is beyond the result's bits."""
    step = even_step(1, 128, 4, seed=9)
    tiny = {int(b) for b in step.block_table[0] if b >= 0} | {int(b) for b in step.block_table[2][:30] if b >= 0}
    small = np.array(sorted(tiny))
    big = np.array([b for b in range(step.num_blocks) if b not in tiny])
    for blocks, power in ((small, -112), (big, 110)):
        x = step.kv_cache[blocks, 1]
        step.kv_cache[blocks, 1] = f32_to_bf16_bits(np.ldexp(bits_to_f64(x), power).astype(np.float32))
    step.v = f32_to_bf16_bits(np.ldexp(bits_to_f64(step.v), -112).astype(np.float32))
    run_within(step, splits)
