"""Requests of a shared-prefix run that attend nothing (bad lengths): they are
flagged, their rows stay as they were and the others keep their results."""

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
from test_gpu_scores import assert_within, expected  # noqa: E402

BAD = binding.DEVERR_LENGTHS | binding.DEVERR_SHARED


def scored(step, on):
    if not on:
        return {}
    begin, end = key_ranges(step, "random", 3)
    return dict(softcap=20.0, alibi_slopes=slopes_of(step.num_q_heads), key_begin=begin, key_end=end)


def prepare(specs, scores_on, B=16):
    binding.pkv_get_device_errors(clear=True)
    step = make_step(specs, num_q_heads=8, num_kv_heads=2, head_dim=64, prefix_tokens=64,
                     block_size=B, seed=7)
    scores = scored(step, scores_on)
    ds = DeviceStep(step, shared_prefix=(64, 0, 6), **scores)
    ds.slot_map()
    ds.write()
    ds.out.fill_(7.0)
    return step, scores, ds


RUN = [RequestSpec(64 + s, 1, shares_prefix=True) for s in (5, 30, 40, 9, 17, 2)]
# (num_computed, seq_lens) of a request that asks for more than its table holds,
# and lengths whose sum wraps
WRONG = {"longer-than-the-table": lambda width: (width, width + 1),
         "far-longer": lambda width: (1 << 30, (1 << 30) + 1),
         "wrapped": lambda width: ((1 << 31) - 1, -(1 << 31))}


@pytest.mark.parametrize("scores_on", [False, True])
@pytest.mark.parametrize("wrong", WRONG)
@pytest.mark.parametrize("bad", [(0,), (3,), (5,), (0, 1, 4), tuple(range(6))])
@pytest.mark.parametrize("others", [True, False])
def test_members_longer_than_their_table(others, bad, wrong, scores_on):
    specs = RUN + ([RequestSpec(70, 1), RequestSpec(20, 9)] if others else [])
    step, scores, ds = prepare(specs, scores_on)
    ref, bound = expected(step, **scores)
    for r in bad:
        c, L = WRONG[wrong](step.block_table.shape[1] * 16)
        ds.num_computed[r], ds.seq_lens[r] = c, L
    ds.attend()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == BAD
    out = ds.out_host()
    rows = np.ones(step.num_tokens, bool)
    rows[list(bad)] = False
    assert (bits_to_f64(out[~rows]) == 7.0).all()
    assert_within(out[rows], ref[rows], bound[rows])


@pytest.mark.parametrize("scores_on", [False, True])
def test_the_first_member_starts_behind_row_zero(scores_on):
    """query_start_loc[0] is 1: request 0 has no place in the batch; the others'
    rows are one further on."""
    step, scores, ds = prepare(RUN, scores_on)
    ref, bound = expected(step, **scores)
    for name in ("q", "out"):
        t = getattr(ds, name)
        setattr(ds, name, torch.cat([t[:1], t]))
    for name in ("key_begin", "key_end"):
        if ds.scores[name] is not None:
            ds.scores[name] = torch.cat([ds.scores[name][:1], ds.scores[name]])
    ds.query_start_loc += 1
    ds.attend()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == BAD
    out = ds.out_host()
    assert (bits_to_f64(out[:2]) == 7.0).all()
    assert_within(out[2:], ref[1:], bound[1:])
