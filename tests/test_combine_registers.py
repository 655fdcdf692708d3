"""The combine's single-row instances, which every split decode launches, keep their
values in registers."""

import os
import re
import subprocess

from paged_kv_cache_hkv_gb300 import build


def test_single_row_combines_spill_nothing(tmp_path):
    src = os.path.join(build.CSRC, "combine.cu")
    r = subprocess.run([build.nvcc(), *build.NVCC_FLAGS, "-Xptxas", "-v", "-c", src, "-o", str(tmp_path / "c.o")],
                       capture_output=True, text=True, check=True)
    found = re.findall(r"entry function '\w*combine_kernelILi(\d+)ELi(\d)ELb([01])ELi(\d+)E\w*'.*?(\d+) bytes spill "
                       r"stores, (\d+) bytes spill loads", r.stderr + r.stdout, re.S)
    single = {f[:3]: (int(f[4]), int(f[5])) for f in found if f[3] == "0"}
    assert len(single) == 12  # head sizes x heads a warp x DEEP
    assert all(spill == (0, 0) for spill in single.values()), single
