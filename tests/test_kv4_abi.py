"""Refusals of the 4-bit serving step's entry points: every bad argument is a
status, found before any CUDA call."""
import ctypes

import pytest
import torch

import int8_w8a8_scaled_gb300 as w8
from int8_w8a8_scaled_gb300 import _lib

FAKE = ctypes.c_void_p(0x7F0000000000)      # never dereferenced: validation fails first
FAKE2 = ctypes.c_void_p(0x7F0000010000)
ODD = ctypes.c_void_p(0x7F0000000001)
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4


def test_cache_bytes():
    size = _lib.load().w8a8_kv4_cache_bytes
    assert size(10, 8, 32, 128) == 10 * 8 * 2 * 2304
    assert w8.kv4_cache_shape(10, 8, 32, 128) == (10, 8, 2, 2304)
    assert size(1 << 30, 65535, 1 << 20, 128) == 0          # past 2^62 bytes
    for bad in ((0, 8, 16, 128), (1, 0, 16, 128), (1, 1, 24, 128), (1, 1, 0, 128), (1, 1, 16, 96)):
        assert size(*bad) == 0
        with pytest.raises(ValueError):
            w8.kv4_cache_shape(*bad)


CACHE = dict(k=FAKE, v=FAKE, dtype=w8.BF16, tokens=4, heads=2, d=128, kt=256, kh=128, vt=256, vh=128, cache=FAKE, nb=4, bs=16,
             slots=FAKE, ks=FAKE, vs=FAKE, kind=0)
CACHE_BAD = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(cache=None), INVALID), (dict(slots=None), INVALID),
    (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(dtype=w8.FP32), INVALID), (dict(kind=2), INVALID),
    (dict(tokens=0), INVALID), (dict(heads=0), INVALID), (dict(nb=0), INVALID), (dict(bs=0), INVALID), (dict(kt=-1), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(bs=24), UNSUPPORTED), (dict(tokens=1 << 33), UNSUPPORTED), (dict(nb=1 << 31), UNSUPPORTED),
    (dict(cache=ODD), MISALIGNED), (dict(k=ODD), MISALIGNED), (dict(slots=ODD), MISALIGNED), (dict(ks=ODD), MISALIGNED),
]


@pytest.mark.parametrize("kw,status", CACHE_BAD)
def test_cache_calls_refuse(kw, status):
    lib, a = _lib.load(), {**CACHE, **kw}
    strides = (a["kt"], a["kh"], a["vt"], a["vh"])
    assert lib.w8a8_kv4_cache_write(a["k"], a["v"], a["dtype"], a["tokens"], a["heads"], a["d"], *strides, a["cache"], a["nb"],
                                    a["bs"], a["slots"], a["ks"], a["vs"], a["kind"], None) == status
    assert lib.w8a8_last_error()
    assert lib.w8a8_kv4_cache_read(a["cache"], a["nb"], a["bs"], a["slots"], a["ks"], a["vs"], a["kind"], a["k"], a["v"],
                                   a["dtype"], a["tokens"], a["heads"], a["d"], *strides, None) == status


def test_read_refuses_overlapping_outputs():
    a = CACHE
    lib = _lib.load()
    for kt, kh in ((0, 128), (256, 64)):
        assert lib.w8a8_kv4_cache_read(FAKE, 4, 16, FAKE, FAKE, FAKE, 0, FAKE, FAKE, a["dtype"], 4, 2, 128, kt, kh, 256, 128,
                                       None) == INVALID


TABLES = dict(ctx=FAKE, new=FAKE, batch=4, free=FAKE, count=FAKE, cap=10, table=FAKE, mb=8, bs=16, start=FAKE, lens=FAKE,
              slots=FAKE, pos=FAKE, tokens=4, left=FAKE2, after=None)


@pytest.mark.parametrize("kw,status", [
    *[({k: None}, INVALID) for k in ("ctx", "new", "free", "count", "table", "start", "lens", "slots", "pos", "left")],
    (dict(batch=0), INVALID), (dict(mb=0), INVALID), (dict(bs=0), INVALID), (dict(tokens=0), INVALID), (dict(cap=-1), INVALID),
    (dict(left=FAKE), INVALID), (dict(after=FAKE), INVALID), (dict(after=FAKE2), INVALID), (dict(batch=16385), UNSUPPORTED), (dict(mb=1 << 27), UNSUPPORTED),
    (dict(tokens=1 << 31), UNSUPPORTED), (dict(cap=1 << 31), UNSUPPORTED), (dict(slots=ctypes.c_void_p(0x7F0000000004)), MISALIGNED),
    (dict(ctx=ODD), MISALIGNED), (dict(left=ODD), MISALIGNED),
])
def test_block_tables_refuse(kw, status):
    lib, a = _lib.load(), {**TABLES, **kw}
    assert lib.w8a8_build_block_tables(a["ctx"], a["new"], a["batch"], a["free"], a["count"], a["cap"], a["table"], a["mb"],
                                       a["bs"], a["start"], a["lens"], a["slots"], a["pos"], a["tokens"], a["left"], a["after"],
                                       None) == status


ATTEND = dict(q=FAKE, qd=w8.BF16, tokens=4, hq=8, hkv=2, d=128, qt=1024, qh=128, cache=FAKE, nb=4, bs=16, table=FAKE, mb=8,
              lens=FAKE, start=FAKE, batch=4, most=2, ks=FAKE, vs=FAKE, kind=1, out=FAKE, od=w8.BF16, ot=1024, oh=128, ws=FAKE,
              wsb=1 << 40)


@pytest.mark.parametrize("kw,status", [
    *[({k: None}, INVALID) for k in ("q", "cache", "table", "lens", "ks", "vs", "out")],
    (dict(qd=w8.FP32), INVALID), (dict(od=w8.INT8), INVALID), (dict(kind=-1), INVALID), (dict(tokens=0), INVALID),
    (dict(hq=0), INVALID), (dict(hkv=3), INVALID), (dict(mb=0), INVALID), (dict(batch=0), INVALID), (dict(most=0), INVALID),
    (dict(start=None), INVALID), (dict(start=None, most=1, tokens=3), INVALID), (dict(ot=64), INVALID), (dict(oh=64), INVALID),
    (dict(qt=-1), INVALID), (dict(d=32), UNSUPPORTED), (dict(bs=8), UNSUPPORTED), (dict(hq=130), UNSUPPORTED),
    (dict(batch=65536), UNSUPPORTED), (dict(mb=1 << 27), UNSUPPORTED), (dict(tokens=1 << 31), UNSUPPORTED),
    (dict(batch=1 << 13, mb=1 << 16), UNSUPPORTED), (dict(most=1 << 30), UNSUPPORTED), (dict(cache=ODD), MISALIGNED), (dict(q=ODD), MISALIGNED), (dict(table=ODD), MISALIGNED),
    (dict(start=ODD), MISALIGNED), (dict(ws=None), WORKSPACE), (dict(wsb=8), WORKSPACE), (dict(ws=ODD), WORKSPACE),
])
def test_attention_refuses(kw, status):
    lib, a = _lib.load(), {**ATTEND, **kw}
    assert lib.w8a8_kv4_attention(
        a["q"], a["qd"], a["tokens"], a["hq"], a["hkv"], a["d"], a["qt"], a["qh"], a["cache"], a["nb"], a["bs"], a["table"],
        a["mb"], a["lens"], a["start"], a["batch"], a["most"], a["ks"], a["vs"], 0.1, a["kind"], a["out"], a["od"], a["ot"],
        a["oh"], a["ws"], a["wsb"], None) == status


def test_attention_workspace_size():
    assert w8.kv4_attention_workspace_size(4, 1, 32, 8, 128) > 0
    for bad in ((0, 1, 32, 8, 128), (4, 0, 32, 8, 128), (4, 1, 33, 8, 128), (4, 1, 32, 8, 96), (4, 1, 65, 1, 128)):
        assert w8.kv4_attention_workspace_size(*bad) == 0


VERIFY = dict(p=FAKE, q=FAKE, dt=w8.FP32, v=100, pld=100, qld=100, tok=FAKE, start=FAKE, batch=2, rows=4, u=FAKE, s=FAKE,
              out=FAKE, most=3, n=FAKE)


@pytest.mark.parametrize("kw,status", [
    *[({k: None}, INVALID) for k in ("p", "tok", "start", "u", "s", "out", "n")],
    (dict(dt=w8.INT8), INVALID), (dict(v=0), INVALID), (dict(batch=0), INVALID), (dict(rows=-1), INVALID), (dict(most=-1), INVALID),
    (dict(pld=99), INVALID), (dict(qld=99), INVALID), (dict(batch=65536), UNSUPPORTED),
    (dict(v=1 << 30, pld=1 << 30, qld=1 << 30), UNSUPPORTED), (dict(most=1 << 20), UNSUPPORTED), (dict(p=ODD), MISALIGNED),
    (dict(tok=ODD), MISALIGNED), (dict(out=ODD), MISALIGNED),
])
def test_verify_refuses(kw, status):
    lib, a = _lib.load(), {**VERIFY, **kw}
    assert lib.w8a8_verify_drafts(a["p"], a["q"], a["dt"], a["v"], a["pld"], a["qld"], a["tok"], a["start"], a["batch"], a["rows"],
                                  a["u"], a["s"], a["out"], a["most"], a["n"], None) == status


def test_python_layer_refuses_cpu_tensors():
    t = torch.zeros(1)
    with pytest.raises(ValueError, match="CUDA"):
        w8.kv4_cache_write(t, t, t, t, t, t)
    with pytest.raises(ValueError, match="CUDA"):
        w8.build_block_tables(t, t, t, t, t, 16, t, t, t, t, t)
    with pytest.raises(ValueError, match="CUDA"):
        w8.kv4_attention(t, t, t, t, t, t, t)
    with pytest.raises(ValueError, match="CUDA"):
        w8.verify_drafts(t, None, t, t, t, t, t, t)
