"""HIP launches fewer than 2^32 threads: what needs more is refused by name, before
any GPU work (pointers are never dereferenced)."""
import pytest

from combine_ep_get_layout_amd import _abi
from test_block_abi import UNS, cast


@pytest.mark.parametrize("kw", [dict(num=1 << 24, n=8, k=8), dict(num=1 << 23, n=136, k=8),
                                dict(num=1 << 22, n=136, k=136), dict(num=(1 << 31) - 1, n=8, k=8),
                                dict(num=2048, n=1 << 20, k=128),
                                dict(num=(1 << 31) - 1, n=1 << 20, k=1 << 20)])
def test_cast_refuses_blocks_that_no_launch_takes(kw):
    assert cast(**kw) == UNS
    assert cast(**kw, ct=16, st=16) == UNS
    assert _abi.load().ep_status_string(UNS)
