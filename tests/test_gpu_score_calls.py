"""Calls with scores that their documentation allows and that the other tests
do not make: more prompt chunks than a CTA keeps metadata for, an output on a
16-byte boundary, and two captured steps, one with a shared prefix, that take
turns on one workspace."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_hkv_gb300 import binding  # noqa: E402
from paged_kv_cache_hkv_gb300.runner import DeviceStep  # noqa: E402
from paged_kv_cache_hkv_gb300.synth import RequestSpec, make_step  # noqa: E402
from test_gpu_scores import MODS, assert_within, expected, run, scores_for  # noqa: E402


@pytest.fixture(autouse=True)
def _clear_errors():
    binding.pkv_get_device_errors(clear=True)
    yield


@pytest.mark.parametrize("mod", ["cap", "alibi", "random", "cap-alibi-random"])
@pytest.mark.parametrize("shared", [False, True])
def test_hundreds_of_short_chunks(shared, mod):
    rng = np.random.default_rng(7)
    specs = [RequestSpec(int(rng.integers(0, 90)), int(rng.integers(2, 6))) for _ in range(207)]
    prefix = 32 if shared else 0
    if shared:
        specs[60:60] = [RequestSpec(32 + s, 1, shares_prefix=True) for s in (0, 4, 50, 16, 31)]
    step = make_step(specs, num_q_heads=8, num_kv_heads=2, head_dim=64, prefix_tokens=prefix, seed=12)
    scores = scores_for(step, MODS[mod], seed=2)
    want = expected(step, **scores)
    ds = run(step, shared_prefix=(32, 60, 5) if shared else None, **scores)
    assert_within(ds.out_host(), *want)


@pytest.mark.parametrize("mod", ["cap", "cap-alibi", "documents"])
@pytest.mark.parametrize("d", [64, 128])
def test_output_on_a_16_byte_boundary(d, mod):
    specs = [RequestSpec(90, 40), RequestSpec(0, 131), RequestSpec(70, 1)]
    step = make_step(specs, num_q_heads=8, num_kv_heads=4, head_dim=d, seed=d)
    scores = scores_for(step, MODS[mod], seed=3)
    ds = DeviceStep(step, write_in_attention=True, **scores)
    n = ds.out.numel()
    room = torch.full((n + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    ds.out = room[8:8 + n].view_as(ds.out)
    assert ds.out.data_ptr() % 32 == 16
    ds.run()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == 0
    assert_within(ds.out_host(), *expected(step, **scores))
    assert (room[:8] == 7).all() and (room[8 + n:] == 7).all()


def test_two_captured_steps_on_one_workspace():
    runs = []
    for seed, mod in ((1, "cap-alibi-random"), (2, "cap")):
        specs = [RequestSpec(64 + s, 1, shares_prefix=True) for s in (5, 200, 40, 9)]
        specs += [RequestSpec(17, 60), RequestSpec(300, 1)]
        step = make_step(specs, num_q_heads=8, num_kv_heads=2, head_dim=128, prefix_tokens=64, seed=seed)
        scores = scores_for(step, MODS[mod], seed=seed)
        ds = DeviceStep(step, write_in_attention=True, shared_prefix=(64, 0, 4) if seed == 1 else None,
                        **scores)
        runs.append((ds, expected(step, **scores)))
    work = max((ds.workspace for ds, _ in runs), key=torch.Tensor.numel)
    side = torch.cuda.Stream()
    graphs = []
    for ds, _ in runs:
        ds.workspace = work
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            ds.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            ds.run()
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0):
        runs[i][0].out.zero_()
        graphs[i].replay()
        graphs[1 - i].replay()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == 0
    for ds, want in runs:
        assert_within(ds.out_host(), *want)
