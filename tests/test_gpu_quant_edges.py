"""The 8-bit pool where a caller's memory and hints are not tidy: places that no
write reached, tables without the blocks in front of a window, a longer maximum than
the step needs, a first call inside a capture."""

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
from paged_kv_cache_hkv_gb300.runner import DeviceStep, bf16_to_numpy  # noqa: E402
from paged_kv_cache_hkv_gb300.synth import RequestSpec, make_step  # noqa: E402

E4M3 = torch.float8_e4m3fn
SPECS = {
    "one": [RequestSpec(c, 1) for c in (0, 1, 7, 8, 15, 16, 17, 300, 811)],
    "few": [RequestSpec(c, 1 + i % 4) for i, c in enumerate((0, 3, 9, 14, 31, 300, 811))],
    "mixed": [RequestSpec(300, 70), RequestSpec(20, 1), RequestSpec(801, 2), RequestSpec(9, 200)],
}


@pytest.fixture(autouse=True)
def _clear_errors():
    binding.pkv_get_device_errors(clear=True)
    yield


@pytest.mark.parametrize("mask", [None, "window"])
@pytest.mark.parametrize("specs", SPECS)
@pytest.mark.parametrize("hq,hkv,d,B", [(8, 2, 64, 16), (16, 4, 128, 8), (8, 1, 128, 32), (6, 6, 64, 8),
                                        (4, 4, 64, 32), (32, 8, 128, 16)])
def test_places_that_no_write_reached_hold_anything(hq, hkv, d, B, specs, mask):
    """NaN codes and NaN scales in every row of the pool but the step's cached keys
    (and of those, with windows, the ones that some row sees; the table has no entry
    for a block wholly in front of them): nothing of it reaches an output."""
    step = make_step(SPECS[specs], num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=B, seed=B + d)
    scores = {}
    if mask:
        scores = dict(zip(("key_begin", "key_end"), key_ranges(step, mask, seed=d)))
    ds = DeviceStep(step, quantised=True, write_in_attention=True, **scores)
    codes, scales = ds.kv_cache.view(torch.uint8), ds.kv_scales
    kept = torch.zeros(step.num_blocks * B, dtype=torch.bool)
    table = ds.block_table.cpu()
    for r, s in enumerate(step.specs):
        t0 = int(step.query_start_loc[r])
        lo = max(0, int(scores["key_begin"][t0:t0 + s.query_len].min())) if mask else 0
        j = torch.arange(lo, s.num_computed)
        kept[table[r].long()[j // B] * B + j % B] = True
        table[r, :lo // B] = -1
    ds.block_table.copy_(table)
    lost = (~kept).view(-1, 1, B).expand(-1, 2, -1).cuda()
    codes[lost] = torch.tensor([0x7F, 0xFF], dtype=torch.uint8, device="cuda").repeat(d // 2)
    scales[lost] = 255
    ds.workspace.fill_(0x7F)
    ds.run()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == 0
    assert_within(ds.out_host(), *expected(step, quantised_step(step)[2], **scores))


@pytest.mark.parametrize("mask", ["window", "random", "documents"])
def test_key_ranges_leave_nothing_behind(mask):
    """Expanded tables have entries for the seen blocks alone: the same bits whatever
    the others hold."""
    for specs in SPECS.values():
        step = make_step(specs, num_q_heads=16, num_kv_heads=4, head_dim=128, seed=3)
        scores = dict(zip(("key_begin", "key_end"), key_ranges(step, mask, seed=5)))
        ds = DeviceStep(step, quantised=True, write_in_attention=True, **scores)
        ds.run()
        first = ds.out_host()
        for fill in (0, 255, 127, 1):
            ds.workspace.fill_(fill)
            ds.out.zero_()
            ds.run()
            assert np.array_equal(ds.out_host(), first)
    assert binding.pkv_get_device_errors(clear=True) == 0


@pytest.mark.parametrize("hint", [5, 16, 17, 600])
def test_a_longer_maximum_than_the_step_needs(hint):
    """max_query_len above every request's new tokens: other kernels, the same results."""
    step = make_step(SPECS["few"], num_q_heads=16, num_kv_heads=4, head_dim=128, seed=6)
    ds = DeviceStep(step, quantised=True)
    ds.slot_map()
    ds.write()
    ws = torch.empty(binding.pkv_quant_attention_workspace_size(
        step.num_reqs, 16, ds.kv_cache, max_blocks_per_req=step.max_blocks_per_req,
        chunk_keys=binding.quant_chunk_keys(step.query_len.tolist(), step.seq_lens.tolist(), 4, 16,
                                            max_query_len=hint)), dtype=torch.uint8, device="cuda")
    out = torch.full_like(ds.out, 5.0)
    binding.pkv_quant_paged_attention(
        out, ds.q, ds.kv_cache, ds.kv_scales, ds.block_table, ds.seq_lens, ds.query_start_loc,
        ds.num_computed, max_query_len=hint, max_seq_len=step.max_seq_len, scale=step.scale, workspace=ws)
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == 0
    assert_within(bf16_to_numpy(out), *expected(step, quantised_step(step)[2]))


@pytest.mark.parametrize("hq,hkv,d,B", [(11, 11, 64, 16), (26, 13, 128, 32), (72, 9, 64, 8)])
@pytest.mark.parametrize("specs", SPECS)
def test_a_first_call_of_a_shape_inside_a_capture(hq, hkv, d, B, specs):
    """Numbers of kv heads that no other test has (odd, more than a CTA's warps):
    what a shape's first call works out is worked out while a graph is recorded."""
    step = make_step(SPECS[specs], num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=B, seed=hq)
    ds = DeviceStep(step, quantised=True, write_in_attention=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ds.run(stream=side)
    for fill in (1.0, 9.0):
        ds.out.fill_(fill)
        graph.replay()
        torch.cuda.synchronize()
        assert_within(ds.out_host(), *expected(step, quantised_step(step)[2]))
    assert binding.pkv_get_device_errors(clear=True) == 0


def test_a_slot_read_many_times():
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(40, 3, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    codes = torch.zeros(5, 2, 8, 3, 64, dtype=torch.uint8, device="cuda").view(E4M3)
    scales = torch.zeros(5, 2, 8, 3, dtype=torch.uint8, device="cuda")
    binding.pkv_quant_kv_write(codes, scales, k, v, torch.arange(40, device="cuda"))
    whole = [torch.empty_like(k) for _ in range(2)]
    binding.pkv_quant_kv_read(*whole, codes, scales, torch.arange(40, device="cuda"))
    slots = torch.tensor([7, 7, 39, 0, 7, 39] * 50, device="cuda")
    back = [torch.empty(300, 3, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    binding.pkv_quant_kv_read(*back, codes, scales, slots)
    for x, y in zip(whole, back):
        assert torch.equal(x[slots], y)
