"""The block-scaled product copies its scales into LDS four steps at a time, the
last copies behind the contraction's end.  A buffer's range check subtracts a
scalar offset from the size, so an offset larger than a small buffer would put
every lane in range: these copies have none (the assembly is read, nothing runs)."""
import os

import pytest

from combine_ep_get_layout_amd import build
from test_expert_copies import assembly, is_copy


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")
def test_copies_of_scales_have_no_scalar_offset(tmp_path):
    code = assembly(os.path.join(build.CSRC, "ep_block_linear.hip"), tmp_path / "kernels.s")
    seen = 0
    for lines in code.values():
        for line in lines:
            if is_copy(line) and line.startswith("buffer_load_dword "):
                # data goes to LDS: the operands are lane offset, descriptor, scalar offset
                scalar = line.split(",")[-1].split()[0]
                assert scalar == "0", line
                seen += 1
    assert seen >= 100
