"""Refusals of the operators over the paged fp8 cache: every bad argument is a
status, found before any CUDA call."""
import ctypes

import pytest
import torch

import int8_w8a8_scaled_gb300 as w8
from int8_w8a8_scaled_gb300 import _lib

FAKE = ctypes.c_void_p(0x7F0000000000)      # never dereferenced: validation fails first
FAKE2 = ctypes.c_void_p(0x7F1000000000)
ODD = ctypes.c_void_p(0x7F0000000001)
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4

PAGED_BAD = [
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(nb=0), INVALID), (dict(bs=0), INVALID), (dict(mb=0), INVALID),
    (dict(h=0), INVALID), (dict(tokens=0), INVALID), (dict(batch=0), INVALID), (dict(most=0), INVALID),
    (dict(start=None), INVALID),                             # without starts a request has one token
    (dict(d=96), UNSUPPORTED), (dict(bs=24), UNSUPPORTED), (dict(bs=16384), UNSUPPORTED), (dict(h=65536, hq=65536), UNSUPPORTED),
    (dict(nb=1 << 28), UNSUPPORTED), (dict(mb=1 << 28), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED),
    (dict(batch=60000, mb=100000), UNSUPPORTED), (dict(tokens=1 << 31), UNSUPPORTED),
    (dict(table=ODD), MISALIGNED), (dict(lens=ODD), MISALIGNED), (dict(start=ODD), MISALIGNED), (dict(kc=ODD), MISALIGNED),
]
HEADS_BAD = [
    (dict(hq=7), INVALID), (dict(hq=0), INVALID), (dict(hq=65 * 2), UNSUPPORTED), (dict(q=None), INVALID), (dict(qd=w8.FP32), INVALID),
    (dict(qt=-1), INVALID), (dict(qh=-1), INVALID), (dict(qt=1 << 62), INVALID), (dict(q=ODD), MISALIGNED),
]
ATTEND = dict(q=FAKE, qd=w8.BF16, tokens=9, hq=8, h=2, d=128, qt=1024, qh=128, kc=FAKE, vc=FAKE, nb=40, bs=16, table=FAKE, mb=8,
              lens=FAKE, start=FAKE, batch=3, most=5, sel=FAKE, budget=4, ks=FAKE, vs=FAKE, out=FAKE2, od=w8.BF16, ot=1024, oh=128,
              ws=None, wsb=0)
ATTEND_BAD = PAGED_BAD + HEADS_BAD + [
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(out=None), INVALID),
    (dict(od=w8.E4M3), INVALID), (dict(ot=100), INVALID), (dict(oh=64), INVALID), (dict(out=FAKE), INVALID),
    (dict(out=ctypes.c_void_p(FAKE.value + 16)), INVALID),   # over q
    (dict(vc=ODD), MISALIGNED), (dict(ks=ODD), MISALIGNED), (dict(out=ODD), MISALIGNED),
    (dict(), WORKSPACE), (dict(ws=ODD, wsb=1 << 40), WORKSPACE), (dict(ws=FAKE, wsb=8), WORKSPACE),
]


def attend(sparse, **kw):
    a = {**ATTEND, **kw}
    lib = _lib.load()
    head = (a["q"], a["qd"], a["tokens"], a["hq"], a["h"], a["d"], a["qt"], a["qh"], a["kc"], a["vc"], a["nb"], a["bs"], a["table"],
            a["mb"], a["lens"], a["start"], a["batch"], a["most"])
    tail = (a["ks"], a["vs"], 0.1, a["out"], a["od"], a["ot"], a["oh"], a["ws"], a["wsb"], None)
    if sparse:
        return lib.w8a8_fp8_kv_sparse_attention(*head, a["sel"], a["budget"], *tail)
    return lib.w8a8_fp8_kv_paged_attention(*head, *tail)


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("kw,status", ATTEND_BAD)
def test_attention_refuses(sparse, kw, status):
    assert attend(sparse, **kw) == status
    assert _lib.load().w8a8_last_error()


@pytest.mark.parametrize("kw,status", [(dict(sel=None), INVALID), (dict(budget=0), INVALID), (dict(sel=ODD), MISALIGNED),
                                       (dict(budget=1 << 20), UNSUPPORTED), (dict(budget=1 << 40), UNSUPPORTED)])
def test_sparse_attention_refuses(kw, status):
    assert attend(True, **kw) == status


@pytest.mark.parametrize("kw,status", PAGED_BAD + [(dict(means=None), INVALID), (dict(scales=None), INVALID), (dict(kc=None), INVALID),
                                                   (dict(means=ODD), MISALIGNED), (dict(scales=ODD), MISALIGNED)])
def test_block_means_refuse(kw, status):
    a = {**ATTEND, "means": FAKE, "scales": FAKE, **kw}
    assert _lib.load().w8a8_fp8_kv_block_means(a["kc"], a["nb"], a["bs"], a["h"], a["d"], a["table"], a["mb"], a["lens"], a["start"],
                                               a["tokens"], a["batch"], a["most"], a["means"], a["scales"], None) == status


SELECT_BAD = [x for x in PAGED_BAD if "kc" not in x[0]] + HEADS_BAD + [
    (dict(means=None), INVALID), (dict(scales=None), INVALID), (dict(sel=None), INVALID), (dict(first=-1), INVALID),
    (dict(last=0), INVALID), (dict(budget=0), INVALID), (dict(first=3), INVALID), (dict(last=1 << 62), INVALID),
    (dict(mb=50000), UNSUPPORTED), (dict(budget=1 << 31), UNSUPPORTED), (dict(means=ODD), MISALIGNED), (dict(scales=ODD), MISALIGNED),
    (dict(sel=ODD), MISALIGNED), (dict(), WORKSPACE), (dict(ws=ODD, wsb=1 << 40), WORKSPACE), (dict(ws=FAKE, wsb=8), WORKSPACE),
]


@pytest.mark.parametrize("kw,status", SELECT_BAD)
def test_select_blocks_refuses(kw, status):
    a = {**ATTEND, "means": FAKE, "scales": FAKE, "first": 1, "last": 2, **kw}
    assert _lib.load().w8a8_fp8_kv_select_blocks(
        a["q"], a["qd"], a["tokens"], a["hq"], a["h"], a["d"], a["qt"], a["qh"], a["means"], a["scales"], a["nb"], a["bs"], a["table"],
        a["mb"], a["lens"], a["start"], a["batch"], a["most"], a["first"], a["last"], a["budget"], a["sel"], a["ws"], a["wsb"],
        None) == status


WRITE = dict(q=FAKE, k=FAKE, v=FAKE, dtype=w8.BF16, tokens=4, hq=8, h=2, d=128, qt=1024, qh=128, kt=256, kh=128, vt=256, vh=128, cs=FAKE,
             mp=100, rot=128, pos=FAKE, axes=1, sections=None, inter=0, kc=FAKE, vc=FAKE, nb=4, bs=16, slots=FAKE, ks=FAKE, vs=FAKE,
             out=FAKE2, ot=1024, oh=128)
WRITE_BAD = [(dict([(x, None)]), INVALID) for x in ("q", "k", "v", "cs", "pos", "kc", "vc", "slots", "ks", "vs", "out")] + [
    (dict(dtype=w8.FP32), INVALID), (dict(tokens=0), INVALID), (dict(hq=-1), INVALID), (dict(h=0), INVALID), (dict(nb=0), INVALID),
    (dict(bs=0), INVALID), (dict(mp=0), INVALID), (dict(rot=0), INVALID), (dict(rot=130), INVALID), (dict(rot=31), INVALID),
    (dict(axes=0), INVALID), (dict(axes=5), INVALID), (dict(axes=2), INVALID), (dict(axes=2, sections=(32, 31)), INVALID),
    (dict(axes=2, sections=(70, -6)), INVALID), (dict(axes=1, sections=(63,)), INVALID), (dict(kt=-1), INVALID), (dict(vh=-1), INVALID),
    (dict(qt=-1), INVALID), (dict(ot=64), INVALID), (dict(oh=64), INVALID), (dict(kt=1 << 62), INVALID),
    (dict(out=FAKE, ot=2048), INVALID), (dict(out=ctypes.c_void_p(FAKE.value + 2)), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(bs=24), UNSUPPORTED), (dict(nb=1 << 28), UNSUPPORTED), (dict(tokens=1 << 33), UNSUPPORTED),
    (dict(h=65536), UNSUPPORTED), (dict(mp=1 << 31), UNSUPPORTED),
] + [(dict([(x, ODD)]), MISALIGNED) for x in ("q", "k", "v", "cs", "pos", "kc", "vc", "slots", "ks", "vs", "out")]


@pytest.mark.parametrize("kw,status", WRITE_BAD)
def test_rotate_write_refuses(kw, status):
    a = {**WRITE, **kw}
    sections = (ctypes.c_int32 * len(a["sections"]))(*a["sections"]) if a["sections"] else None
    assert _lib.load().w8a8_fp8_kv_rotate_write(
        a["q"], a["k"], a["v"], a["dtype"], a["tokens"], a["hq"], a["h"], a["d"], a["qt"], a["qh"], a["kt"], a["kh"], a["vt"], a["vh"],
        a["cs"], a["mp"], a["rot"], a["pos"], a["axes"], sections, a["inter"], a["kc"], a["vc"], a["nb"], a["bs"], a["slots"], a["ks"],
        a["vs"], a["out"], a["ot"], a["oh"], None) == status
    assert _lib.load().w8a8_last_error()


def test_workspace_sizes():
    assert w8.fp8_kv_attention_workspace_size(4, 5, 8, 2, 128) > 0
    for bad in ((0, 1, 8, 2, 128), (1, 0, 8, 2, 128), (1, 1, 8, 3, 128), (1, 1, 8, 2, 80), (70000, 1, 8, 2, 128), (1, 1, 130, 2, 64)):
        assert w8.fp8_kv_attention_workspace_size(*bad) == 0
    assert w8.fp8_kv_sparse_attention_workspace_size(4, 8, 2, 128, 16, 64) > 0
    for bad in ((0, 8, 2, 128, 16, 64), (4, 8, 2, 96, 16, 64), (4, 8, 2, 128, 0, 64), (4, 8, 2, 128, 1 << 23, 64), (4, 7, 2, 128, 16, 64)):
        assert w8.fp8_kv_sparse_attention_workspace_size(*bad) == 0
    assert w8.fp8_kv_select_blocks_workspace_size(10, 8, 100) == 32000
    assert w8.fp8_kv_select_blocks_workspace_size(1 << 20, 8, 1000) <= 64 << 20
    for bad in ((0, 8, 100), (1, 0, 100), (1, 8, 0), (1, 8, 49153)):
        assert w8.fp8_kv_select_blocks_workspace_size(*bad) == 0


def test_python_layer_refuses():
    """What the marshalling itself finds, on CPU tensors of the right and wrong kinds."""
    q, kc = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 16, 2, 64, dtype=torch.uint8)
    lens, table, one = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 1, dtype=torch.int32), torch.ones(1)
    good = dict(q=q, k_cache=kc, v_cache=kc, seq_lens=lens, block_table=table, k_scale=one, v_scale=one, out=q)
    for change in (dict(q=q[:, :, :32]), dict(out=q[:2]), dict(k_cache=kc.short()), dict(v_cache=kc[:1]), dict(seq_lens=lens.long()),
                   dict(block_table=table[0]), dict(k_scale=torch.ones(2)), dict(query_start=lens), dict(q=q.transpose(1, 2)),
                   dict(k_cache=kc.transpose(1, 2))):
        with pytest.raises((ValueError, TypeError)):
            w8.fp8_kv_attention(**{**good, **change})
    with pytest.raises(ValueError, match="CUDA"):
        w8.fp8_kv_attention(**good)
    sel = torch.zeros(3, 2, 4, dtype=torch.int32)
    for change in (dict(selected=sel[:2]), dict(selected=sel.long()), dict(selected=sel[0])):
        with pytest.raises(ValueError):
            w8.fp8_kv_sparse_attention(**{**good, "selected": sel, **change})
    means, scales = torch.zeros(2, 2, 64, dtype=torch.int8), torch.zeros(2, 2)
    good = dict(q=q, means=means, mean_scales=scales, seq_lens=lens, block_table=table, block_size=16, selected=sel)
    for change in (dict(means=means.short()), dict(mean_scales=scales[0]), dict(selected=sel[:, :1]), dict(q=q[:, :, :32])):
        with pytest.raises(ValueError):
            w8.fp8_kv_select_blocks(**{**good, **change})
    with pytest.raises(ValueError):
        w8.fp8_kv_block_means(kc, lens, table, means[:1], scales[:1])
    k, cs, pos, slots = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(9, 64), lens, torch.zeros(3, dtype=torch.int64)
    good = dict(q=q, k=k, v=k, cos_sin=cs, positions=pos, k_cache=kc, v_cache=kc, slots=slots, k_scale=one, v_scale=one, q_out=q)
    for change in (dict(q=None), dict(q_out=None), dict(v=k.half()), dict(q=q.half()), dict(cos_sin=cs.half()), dict(positions=pos.long()),
                   dict(sections=(10, 22)), dict(sections=()), dict(sections=(1,) * 5), dict(slots=pos), dict(k=k[:2]), dict(q=q[:2])):
        with pytest.raises((ValueError, TypeError)):
            w8.fp8_kv_rotate_write(**{**good, **change})
    with pytest.raises(ValueError, match="CUDA"):
        w8.fp8_kv_rotate_write(**good)


def test_workspace_sizes_say_why():
    lib = _lib.load()
    for size, good, bad in (
            (w8.fp8_kv_attention_workspace_size, (4, 5, 8, 2, 128), (4, 5, 9, 2, 128)),
            (w8.fp8_kv_sparse_attention_workspace_size, (4, 8, 2, 128, 16, 64), (0, 8, 2, 128, 16, 64)),
            (w8.fp8_kv_select_blocks_workspace_size, (10, 8, 100), (0, 8, 100))):
        assert size(*good) > 0 and not lib.w8a8_last_error()
        assert size(*bad) == 0 and lib.w8a8_last_error()
