"""The 8-bit pool's limits without a GPU."""

import numpy as np
import pytest

import oracle
from test_abi_host import _layout
from test_abi_host import header_define as E
from test_quant_host import _attn, lib  # noqa: F401


@pytest.mark.parametrize("sign", [0, 0x8000])
def test_every_finite_row_has_finite_values(sign):
    """Each of the last bf16 magnitudes as a row's largest, all others beside it: the
    values are bf16, within 2^-4, and held the same when written again."""
    mags = np.arange(0x7F00, 0x7F80, dtype=np.uint16)
    rows = np.minimum(mags[None, :], mags[:, None]) | np.uint16(sign)
    codes, scales = oracle.quantise_rows(rows)
    bits = oracle.quant_pool_bits(codes, scales)
    x, y = oracle.bf16_bits_to_f64(rows), oracle.bf16_bits_to_f64(bits)
    assert np.isfinite(y).all()
    assert (np.abs(x - y) <= 2.0 ** -4 * np.abs(x)).all()
    assert (np.abs(y[:, -1]) == np.abs(y).max(axis=1)).all()
    again = oracle.quantise_rows(bits)
    assert np.array_equal(oracle.quant_values(*again), y)


@pytest.mark.parametrize("write", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_more_kv_heads_than_a_stage_holds_scales_of_are_refused(lib, d, write):  # noqa: F811
    """Before anything is written or launched."""
    lay = _layout(hkv=4096, d=d)
    assert _attn(lib, write, lay=lay, Hq=4096) == E("PKV_ERR_UNSUPPORTED")
    assert _attn(lib, write, lay=lay, Hq=8 * 4096, mq=500) == E("PKV_ERR_UNSUPPORTED")
    if not write:
        assert _attn(lib, lay=_layout(hkv=1799, d=d), Hq=1799) != E("PKV_ERR_UNSUPPORTED")
