"""Limits of the operators over the paged fp8 cache: what lies just behind them is
refused before any CUDA call, what lies within is not."""
import pytest

from test_fp8_paged_abi import attend

UNSUPPORTED, WORKSPACE = 2, 4


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("blocks,size,status", [
    ((1 << 27) - 1, 16, UNSUPPORTED),                        # the last tokens' positions would be those of missing ones
    ((1 << 18) - 1, 8192, UNSUPPORTED),
    (0x7F000000 // 16 + 1, 16, UNSUPPORTED),
    (0x7F000000 // 16, 16, WORKSPACE),                       # (the next thing that is missing)
])
def test_positions_of_attention(sparse, blocks, size, status):
    assert attend(sparse, batch=1, tokens=1, most=1, h=1, hq=4, mb=blocks, bs=size, nb=100, start=None) == status
