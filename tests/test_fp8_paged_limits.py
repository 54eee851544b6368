"""Limits of the operators over the paged fp8 cache: what lies just behind them is
refused before any CUDA call, what lies within is not."""
import ctypes

import pytest

import int8_w8a8_scaled_gb300 as w8
from int8_w8a8_scaled_gb300 import _lib
from test_fp8_paged_abi import ATTEND, FAKE, FAKE2, WRITE, attend

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


@pytest.mark.parametrize("kw", [dict(k=FAKE, v=FAKE2), dict(k=FAKE2, v=FAKE), dict(k=ctypes.c_void_p(FAKE.value + 2 * 1023), v=FAKE2, qt=1280, ot=1280, kt=1280)])
def test_queries_turned_in_place_over_keys_or_values(kw):
    """A key of another token or head would be read before or after its memory is a turned query."""
    a = {**WRITE, "out": FAKE, **kw}
    assert _lib.load().w8a8_fp8_kv_rotate_write(
        a["q"], a["k"], a["v"], a["dtype"], a["tokens"], a["hq"], a["h"], a["d"], a["qt"], a["qh"], a["kt"], a["kh"], a["vt"], a["vh"],
        a["cs"], a["mp"], a["rot"], a["pos"], a["axes"], None, a["inter"], a["kc"], a["vc"], a["nb"], a["bs"], a["slots"], a["ks"],
        a["vs"], a["out"], a["ot"], a["oh"], None) == INVALID


@pytest.mark.parametrize("most,heads,status", [
    ((1 << 31) - 1, 1, UNSUPPORTED), ((1 << 31) - 64, 1, UNSUPPORTED), (0x7F000000 + 1, 1, UNSUPPORTED), ((1 << 28) - 1, 8, UNSUPPORTED),
    (0x7F000000, 1, WORKSPACE), (0x7F000000 // 8, 8, WORKSPACE),
])
def test_rows_of_a_request(most, heads, status):
    """The kernels count a request's rows in 32 bits, a step of rows past the last one."""
    a = {**ATTEND, "tokens": most, "batch": 1, "most": most, "h": 1, "hq": heads, "qt": 0, "qh": 128}
    assert _lib.load().w8a8_fp8_kv_select_blocks(
        a["q"], a["qd"], a["tokens"], a["hq"], a["h"], a["d"], a["qt"], a["qh"], FAKE, FAKE, a["nb"], a["bs"], a["table"], a["mb"],
        a["lens"], a["start"], 1, a["most"], 0, 1, a["budget"], a["sel"], None, 0, None) == status
    kw = {x: a[x] for x in ("tokens", "batch", "most", "h", "hq", "qt", "qh")}
    for sparse in (False, True):
        assert attend(sparse, **kw, ot=128 * heads, oh=128, out=ctypes.c_void_p(FAKE.value + (1 << 44))) == status
    assert (w8.fp8_kv_attention_workspace_size(1, most, heads, 1, 128) > 0) == (status == WORKSPACE)
    assert (w8.fp8_kv_sparse_attention_workspace_size(most, heads, 1, 128, 4, 16) > 0) == (status == WORKSPACE)
