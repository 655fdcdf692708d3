"""Infinities in V of split decodes: the combine's pieces that hold nothing make
no NaN of them."""

import numpy as np
import pytest

from parity import bits_to_f64
from score_cases import slopes_of

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_hkv_gb300 import binding  # noqa: E402
from paged_kv_cache_hkv_gb300.runner import DeviceStep  # noqa: E402
from paged_kv_cache_hkv_gb300.synth import RequestSpec, make_step  # noqa: E402
from test_gpu_scores import expected  # noqa: E402


@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("splits", [None, 1, 2, 5, 40, 300])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("requests", [1, 9])
def test_an_infinity_stays_one(requests, d, splits, scored):
    """Key 2, in a request's first piece, has an infinity in one element and a
    negative one in another; key 70 a NaN in a third. The other elements keep
    their values."""
    binding.pkv_get_device_errors(clear=True)
    specs = [RequestSpec(90 + 11 * r, 1) for r in range(requests)]
    step = make_step(specs, num_q_heads=8, num_kv_heads=2, head_dim=d, seed=requests)
    scores = dict(softcap=20.0, alibi_slopes=slopes_of(8) * np.float32(0.05)) if scored else {}
    bad = {(2, 3): 0x7F80, (2, 9): 0xFF80, (70, 20): 0x7FC0}
    rows = {j: [step.kv_cache[step.block_table[r][j // 16], 1, j % 16] for r in range(requests)]
            for j, _ in bad}
    for (j, dim), bits in bad.items():
        for row in rows[j]:
            row[:, dim] = bits
    ds = DeviceStep(step, write_in_attention=True, decode_splits=splits, **scores)
    ds.run()
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == 0
    for j, dim in bad:
        for row in rows[j]:
            row[:, dim] = 0
    ref, bound = expected(step, **scores)
    got = bits_to_f64(ds.out_host())
    assert (got[:, :, 3] == np.inf).all() and (got[:, :, 9] == -np.inf).all()
    assert np.isnan(got[:, :, 20]).all()
    rest = [x for x in range(d) if x not in (3, 9, 20)]
    assert (np.abs(got - ref)[:, :, rest] <= bound[:, :, rest] + 1e-30).all()
