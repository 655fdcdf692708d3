"""DeviceStep without a GPU: when the marshalled calls are made anew."""

import numpy as np
import pytest

from paged_kv_cache_hkv_gb300 import binding
from paged_kv_cache_hkv_gb300.synth import RequestSpec, make_step
from score_cases import key_ranges, slopes_of

torch = pytest.importorskip("torch")

from paged_kv_cache_hkv_gb300.runner import DeviceStep  # noqa: E402


@pytest.fixture
def step_calls(monkeypatch):
    """DeviceStep on the CPU; what each StepCalls was made with, in order."""
    made = []
    monkeypatch.setattr(binding, "pkv_attention_workspace_size", lambda *a, **kw: 512)
    monkeypatch.setattr(binding, "StepCalls", lambda **kw: made.append(kw) or len(made))
    return made


def test_calls_are_made_anew_when_what_they_hold_was_replaced(step_calls):
    step = make_step([RequestSpec(20, 1), RequestSpec(0, 9)], num_q_heads=4, num_kv_heads=2,
                     head_dim=64)
    begin, end = key_ranges(step, "random", 1)
    ds = DeviceStep(step, device="cpu", softcap=3.0, alibi_slopes=slopes_of(4), key_begin=begin,
                    key_end=end)
    first = ds.calls()
    assert ds.calls() is first and len(step_calls) == 1
    for name in ("alibi_slopes", "key_begin", "key_end"):
        ds.scores[name] = ds.scores[name].clone()
        assert ds.calls() != first, name
        first = ds.calls()
        assert step_calls[-1][name] is ds.scores[name]
    ds.scores["softcap"] = 4.0
    ds.calls()
    assert step_calls[-1]["softcap"] == 4.0 and len(step_calls) == 5
    ds.scores["key_begin"] = None
    ds.calls()
    assert step_calls[-1]["key_begin"] is None and len(step_calls) == 6
    ds.out = ds.out.clone()
    ds.write_in_attention = True
    ds.calls()
    assert step_calls[-1]["out"] is ds.out and step_calls[-1]["write_in_attention"]
    for name, value in (("fused_write", True), ("decode_splits", 3), ("shared_prefix", (16, 0, 1))):
        setattr(ds, name, value)
        ds.calls()
        assert step_calls[-1][name] == value
    n = len(step_calls)
    ds.key_begin = np.zeros(3)  # nothing that the calls hold
    ds.calls()
    assert len(step_calls) == n


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
def test_replaced_scores_count_in_the_next_run():
    step = make_step([RequestSpec(200, 1), RequestSpec(30, 70)], num_q_heads=4, num_kv_heads=2,
                     head_dim=64, seed=3)
    ranges = [key_ranges(step, "random", s) for s in (1, 2)]
    ds = DeviceStep(step, softcap=20.0, key_begin=ranges[0][0], key_end=ranges[0][1])
    ds.run()
    ds.scores["key_begin"], ds.scores["key_end"] = (torch.from_numpy(a).cuda() for a in ranges[1])
    ds.scores["softcap"] = 2.0
    ds.run()
    fresh = DeviceStep(step, softcap=2.0, key_begin=ranges[1][0], key_end=ranges[1][1])
    fresh.run()
    assert np.array_equal(ds.out_host(), fresh.out_host())
