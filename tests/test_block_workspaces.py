"""The workspace queries of the block-scaled product and the gated block, which a
program asks once for its largest batch (host calls, nothing runs)."""
import pytest

from combine_ep_get_layout_amd import _abi

ROWS = [*range(0, 3000, 7), *(r + d for r in (4096, 6000, 16384, 25600, 65536, 1 << 20) for d in (-1, 0, 1)),
        (1 << 31) - 1024]


@pytest.mark.parametrize("n,k", [(8, 128), (8, 8192), (264, 1152), (4096, 7168), (7168, 2048), (2056, 7168),
                                 (1 << 16, 16384)])
def test_product_does_not_ask_more_for_fewer_rows(n, k):
    got = [_abi.load().ep_block_linear_workspace_bytes(r, n, k) for r in ROWS]
    assert got == sorted(got)


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("hidden,inter", [(8, 8), (128, 1792), (512, 512), (1024, 1408), (2048, 1024), (4096, 1024),
                                          (7168, 2048), (8, 4096), (16384, 8192)])
def test_block_does_not_ask_more_for_fewer_tokens(hidden, inter, backward):
    got = [_abi.load().ep_gated_ffn_workspace_bytes(r, hidden, inter, backward) for r in ROWS]
    assert got == sorted(got) and all(got)
    # the rows that a pass keeps, sums of at most 26 and 256 MB, and a line
    room = 256 * (1 + backward) + 256 + 26_214_400 + 256_000_000 * backward
    for r, b in zip(ROWS, got):
        assert 0 <= b - 2 * r * inter * (3 if backward else 1) <= room


@pytest.mark.parametrize("n,k", [(12, 7168), (4096, 7168 + 64), (4, 7168), (4096, 64), (1 << 20, 1 << 11),
                                 ((1 << 20) + 8, 1024), (8, (1 << 20) + 128)])
def test_product_asks_nothing_for_sizes_it_refuses(n, k):
    assert _abi.load().ep_block_linear_workspace_bytes(333, n, k) == 0


@pytest.mark.parametrize("hidden,inter", [(12, 8), (8, 12), (4, 8), (8, 4), (1 << 15, 1 << 14), ((1 << 20) + 8, 8),
                                          (8, (1 << 19) + 8)])
def test_block_asks_nothing_for_sizes_it_refuses(hidden, inter):
    f = _abi.load().ep_gated_ffn_workspace_bytes
    assert f(333, hidden, inter, 0) == f(333, hidden, inter, 1) == 0
