"""The 8-bit pool's limits without a GPU."""

import os
import shutil
import subprocess

import numpy as np
import pytest

import oracle
from paged_kv_cache_hkv_gb300 import build
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


def test_the_row_calls_reciprocals_are_exact(tmp_path):
    """row_split as the library has it, compiled for the host: every kind of word number
    below 2^31 for row lengths of every kind."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    rows = [1, 2, 3, 5, 8, 24, 64, 100, 128, 192, 640, 1000, 4096, 5000, 28784, 1 << 20, (1 << 29) + 1]
    src = tmp_path / "split.cc"
    src.write_text("""#include "row_split.h"
#include <cstdio>
#include <cstdlib>
int main(int n, char** v) {
  for (int i = 1; i < n; ++i) {
    const pkv::RowSplit s = pkv::row_split(std::atoi(v[i]));
    std::printf("%u %u %d %d\\n", s.mul, s.shift, s.row_pair, s.vec_per_row);
  }
}
""")
    exe = tmp_path / "split"
    subprocess.run([gxx, "-std=c++17", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe), *map(str, rows)], check=True, capture_output=True, text=True).stdout
    rng = np.random.default_rng(1)
    for vec, line in zip(rows, out.splitlines(), strict=True):
        mul, shift, d, same = map(int, line.split())
        assert d == 2 * vec and same == vec
        near = d * rng.integers(0, (1 << 31) // d + 1, 2000)
        w = np.concatenate([rng.integers(0, 1 << 31, 5000), np.arange(5000), (1 << 31) - 1 - np.arange(5000),
                            near, near - 1, near + 1])
        w = w[(w >= 0) & (w < 1 << 31)].astype(np.uint64)
        total = ((np.uint64(mul) * w) >> np.uint64(32)) + w
        assert (total < 1 << 32).all()  # (the kernel's sum has 32 bits)
        assert np.array_equal(total >> np.uint64(shift), w // np.uint64(d)), vec
