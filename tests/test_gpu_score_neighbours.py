"""What other requests of the batch hold does not reach a request's scored
prefill: a tile's rows behind the request are the next request's queries."""

import numpy as np
import pytest

from score_cases import slopes_of

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_hkv_gb300 import binding  # noqa: E402
from paged_kv_cache_hkv_gb300.synth import RequestSpec, make_step  # noqa: E402
from test_gpu_score_ranges import times_power  # noqa: E402
from test_gpu_scores import assert_within, expected, run  # noqa: E402

FORMS = {"ranges": dict(), "cap": dict(softcap=30.0), "wide-cap": dict(softcap=300.0),
         "bias": dict(alibi=0.02), "falling-bias": dict(alibi=-0.02),
         "cap-bias": dict(softcap=30.0, alibi=0.02)}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hq,hkv,d", [(6, 6, 128), (8, 2, 64), (8, 1, 128)])
def test_the_next_requests_queries_change_no_bit(hq, hkv, d, form):
    """The first request's last tile is mostly the second request's rows, over
    key tiles that its own rows see in full. Queries 64 times as large make
    those rows' maxima jump from tile to tile; the first request's output stays
    as it was, bit for bit."""
    binding.pkv_get_device_errors(clear=True)
    specs = [RequestSpec(1000, 128 * hkv // hq + 3), RequestSpec(20, 140)]
    outs = []
    for power in (0, 6):
        step = make_step(specs, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, seed=5,
                         scale=2.0 / d ** 0.5)
        n = specs[0].query_len
        step.q[n:] = times_power(step.q[n:], power)
        scores = dict(softcap=FORMS[form].get("softcap", 0.0),
                      key_begin=np.zeros(step.num_tokens, np.int32))
        if "alibi" in FORMS[form]:
            scores["alibi_slopes"] = (slopes_of(hq) * FORMS[form]["alibi"]).astype(np.float32)
        outs.append(run(step, **scores).out_host()[:n])
        ref, bound = expected(step, **scores)
        assert_within(outs[-1], ref[:n], bound[:n])
    assert np.array_equal(outs[0], outs[1])
