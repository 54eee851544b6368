"""Limits of the operators over the paged fp8 cache: what lies just behind them is
refused before any CUDA call, what lies within is not."""
import ctypes

import pytest

from test_fp8_paged_abi import FAKE, attend

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("blocks,size,status", [
    ((1 << 27) - 1, 16, UNSUPPORTED),                        # the last tokens' positions would be those of missing ones
    ((1 << 18) - 1, 8192, UNSUPPORTED),
    (0x7F000000 // 16 + 1, 16, UNSUPPORTED),
    (0x7F000000 // 16, 16, WORKSPACE),                       # (the next thing that is missing)
])
def test_positions_of_attention(sparse, blocks, size, status):
    assert attend(sparse, batch=1, tokens=1, most=1, h=1, hq=4, mb=blocks, bs=size, nb=100, start=None) == status


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("apart,token,head,status", [        # elements from q to out, strides of both (9 tokens, 8 heads of 128)
    (1024, 2048, 128, WORKSPACE),                            # heads behind heads in a token's row
    (128, 2048, 256, WORKSPACE),                             # head by head
    (128, 256, 2304, WORKSPACE),                             # the same with the tokens of a head together
    (-1024, 2048, 128, WORKSPACE),                           # out in front
    (1023, 2048, 128, INVALID), (1025, 2048, 128, INVALID), (127, 2048, 256, INVALID), (129, 2048, 256, INVALID),
    (2048, 2048, 128, INVALID), (0, 2048, 256, INVALID), (-1, 2048, 128, INVALID),
])
def test_queries_and_outputs_in_one_buffer(sparse, apart, token, head, status):
    kw = dict(qt=token, qh=head, ot=token, oh=head, out=ctypes.c_void_p(FAKE.value + 2 * apart))
    assert attend(sparse, **kw) == status
