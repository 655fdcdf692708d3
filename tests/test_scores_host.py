"""Capped, biased and range-masked attention without a GPU: the oracle's
formulas against closed forms, and the refusals of the options."""

import ctypes

import numpy as np
import pytest

import oracle
from paged_kv_cache_hkv_gb300 import binding, build
from paged_kv_cache_hkv_gb300.synth import RequestSpec, make_step
from score_cases import batch, key_ranges, slopes_of
from test_abi_host import FAKE, _attn, _layout
from test_abi_host import header_define as E


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return binding.load()


def _opt(**fields):
    s = binding.pkv_score_options()
    for k, v in fields.items():
        if k == "reserved":
            s.reserved[v] = 1
        else:
            setattr(s, k, v)
    o = binding.pkv_attention_options()
    o.reserved[0] = binding.PKV_OPTIONS_SCORES
    o.scores = ctypes.pointer(s)
    o._keep_scores = s
    return ctypes.pointer(o)


# with no GPU a call whose options pass ends at the device check, or at the
# next argument check
@pytest.mark.parametrize("cap", [-1.0, float("nan"), float("inf"), -float("inf"), 1e-31, 2e30])
def test_bad_caps_are_refused(lib, cap):
    assert _attn(lib, opt=_opt(softcap=cap)) == E("PKV_ERR_BAD_SHAPE")


def test_cap_and_scale_together(lib):
    assert _attn(lib, scale=1e-20, opt=_opt(softcap=1e15)) == E("PKV_ERR_BAD_SHAPE")
    assert _attn(lib, scale=1e20, opt=_opt(softcap=1e-15)) == E("PKV_ERR_BAD_SHAPE")
    assert _attn(lib, q=None, opt=_opt(softcap=30.0)) == E("PKV_ERR_NULL_POINTER")


@pytest.mark.parametrize("field", ["alibi_slopes", "key_begin", "key_end"])
def test_misaligned_arrays_are_refused(lib, field):
    assert _attn(lib, opt=_opt(**{field: 0x10002})) == E("PKV_ERR_MISALIGNED")
    assert _attn(lib, q=None, opt=_opt(**{field: 0x10004})) == E("PKV_ERR_NULL_POINTER")


def test_reserved_words(lib):
    for i in range(4):
        assert _attn(lib, opt=_opt(reserved=i)) == E("PKV_ERR_BAD_SHAPE")
    o = _opt(softcap=-1.0)
    o.contents.reserved[0] = 2
    assert _attn(lib, opt=o) == E("PKV_ERR_BAD_SHAPE")
    # reserved[0] 0: a caller built before the field existed; `scores` is not read
    o.contents.reserved[0] = 0
    assert _attn(lib, q=None, opt=o) == E("PKV_ERR_NULL_POINTER")
    o.contents.reserved[1] = 1
    assert lib.pkv_attention_workspace_size(2, 4, _layout(), o) < 0
    n = binding.pkv_attention_options()
    n.reserved[0] = binding.PKV_OPTIONS_SCORES  # scores NULL: plain attention
    assert _attn(lib, q=None, opt=ctypes.pointer(n)) == E("PKV_ERR_NULL_POINTER")
    # an empty batch is checked too
    assert _attn(lib, R=0, opt=_opt(softcap=-1.0)) == E("PKV_ERR_BAD_SHAPE")
    assert FAKE


def test_binding_checks_the_tensors():
    torch = pytest.importorskip("torch")
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    assert binding._scores(q, 0.0, None, None, None) is None
    assert binding._scores(q, None, None, None, None) is None
    assert binding._scores(q, 3.0, None, None, None).softcap == 3.0
    for kw in (dict(alibi_slopes=torch.zeros(4)), dict(key_begin=torch.zeros(5, dtype=torch.int32)),
               dict(key_end=torch.zeros(5, dtype=torch.int32))):
        full = dict(softcap=0.0, alibi_slopes=None, key_begin=None, key_end=None)
        with pytest.raises(ValueError, match="CUDA"):  # host tensors
            binding._scores(q, **{**full, **kw})


def _pool(step):
    slots = oracle.slot_mapping(step.block_table, step.query_start_loc, step.num_computed,
                                step.block_size)
    return oracle.kv_write(step.kv_cache, step.k, step.v, slots)


def _scored(step, **kw):
    return oracle.scored_attention(step.q, _pool(step), step.block_table, step.seq_lens,
                                   step.query_start_loc, step.num_computed, step.scale, **kw)[0]


def test_oracle_with_everything_off_is_plain_attention():
    step = make_step(batch(), num_q_heads=4, num_kv_heads=2, head_dim=64, seed=1)
    plain = oracle.paged_attention(step.q, _pool(step), step.block_table, step.seq_lens,
                                   step.query_start_loc, step.num_computed, step.scale)
    assert np.abs(_scored(step) - plain).max() < 1e-12
    assert np.abs(_scored(step, softcap=1e9) - plain).max() < 1e-9
    assert np.abs(_scored(step, slopes=np.zeros(4)) - plain).max() < 1e-12


def test_oracle_closed_forms():
    step = make_step([RequestSpec(9, 1)], num_q_heads=2, num_kv_heads=1, head_dim=64, seed=2)
    one = np.array([1], np.int32)
    V = oracle.bf16_bits_to_f64(step.kv_cache[step.block_table[0, 0], 1, :, 0])
    # a range of one key gives that key's value; no key gives zeros
    got = _scored(step, key_begin=one * 4, key_end=one * 5)
    assert np.abs(got[0] - V[4]).max() < 1e-12
    assert (_scored(step, key_begin=one * 5, key_end=one * 5) == 0).all()
    # a cap near zero gives the mean; a steep slope gives the nearest key
    mean = _scored(step, softcap=1e-9, key_begin=one * 2, key_end=one * 6)
    assert np.abs(mean[0] - V[2:6].mean(0)).max() < 1e-6
    near = _scored(step, slopes=np.array([1e6, 1e6]), key_end=one * 7)
    assert np.abs(near[0] - V[6]).max() < 1e-12


def test_a_document_is_attended_as_if_it_were_alone():
    step = make_step([RequestSpec(0, 60)], num_q_heads=2, num_kv_heads=1, head_dim=64, seed=3)
    cuts = [0, 13, 40, 60]
    begin = np.concatenate([np.full(z - a, a) for a, z in zip(cuts[:-1], cuts[1:])]).astype(np.int32)
    got = _scored(step, key_begin=begin, slopes=slopes_of(2), softcap=2.0)
    for a, z in zip(cuts[:-1], cuts[1:]):
        alone = make_step([RequestSpec(0, z - a)], num_q_heads=2, num_kv_heads=1, head_dim=64, seed=3)
        alone.q, alone.k, alone.v = step.q[a:z], step.k[a:z], step.v[a:z]
        ref = _scored(alone, slopes=slopes_of(2), softcap=2.0)
        assert np.abs(got[a:z] - ref).max() < 1e-12


def test_the_kernels_clamped_distances_leave_the_softmax():
    """|p - j| and |clamp(p, begin, end - 1) - j| differ by a constant over
    begin <= j < end."""
    for mask in ("random", "documents", "prefix", "window"):
        step = make_step(batch(), num_q_heads=4, num_kv_heads=2, head_dim=64, materialize=False)
        begin, end = key_ranges(step, mask, 1)
        for r, s in enumerate(step.specs):
            for i in range(s.query_len):
                t, p = step.query_start_loc[r] + i, s.num_computed + i
                lo, hi = max(0, begin[t]), min(end[t], s.seq_len)
                if lo < hi:
                    j = np.arange(lo, hi)
                    ref = max(min(p, hi - 1), lo)
                    assert len(set(np.abs(p - j) - np.abs(ref - j))) == 1
