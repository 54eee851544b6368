"""The serving step over a 4-bit paged KV cache on the GPU, against the oracle.

Whole numbers (codes, scales, tables, slots, tokens) are equal.  Attention's
tolerance, per output element, with r the same weights' mean of |V|:
  * the output's rounding, half a step: 2^-8 |ref| (bf16), 2^-11 |ref| (fp16),
    or half the smallest subnormal number where the output is below the
    normal ones (fp16: 2^-25);
  * the softmax weights' rounding to f16 before the second product, 2^-11 of
    each weight, in its numerator and again in the sum that divides it:
    2^-10 r.  The codes times their group scales are exact in f16;
  * fp32 scores: d products and sums and the scaling, each off by 2^-24 of
    at most B = max_t sum_d |q_d K_td| * sm_scale, move a weight's exponent by
    (d + 8) 2^-24 B, twice as much relative to the maximum; exp2's
    approximation and the sums of 32 bits over the tokens stay below 2^-18.
    Together (2 (d + 8) 2^-24 B + 2^-18) r."""
import numpy as np
import pytest
import torch

import int8_w8a8_scaled_gb300 as w8
from oracle import kv4

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().float().cpu().numpy()


def head_rows(rng, shape, dtype, spikes=True):
    x = rng.standard_normal(shape).astype(np.float32)
    if spikes:
        x[..., 5::37] *= 8
    return torch.from_numpy(x).to(DT[dtype])


# ------------------------------------------------------------------ cache


def view_of(x, layout):
    """The same [T, H, D] values in another memory layout."""
    T, H, D = x.shape
    if layout == "plain":
        return x.contiguous()
    if layout == "merged":                                   # a slice of a wider row
        wide = torch.zeros(T, 3 * H, D, dtype=x.dtype, device=x.device)
        wide[:, H:2 * H] = x
        return wide[:, H:2 * H]
    if layout == "heads_first":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    odd = torch.zeros(T * (H * D + 3) + 1, dtype=x.dtype, device=x.device)   # rows that start at any element
    y = odd[1:].as_strided((T, H, D), (H * D + 3, D, 1))
    y.copy_(x)
    return y


@pytest.mark.parametrize("tokens,heads,d,bs,kind,dtype,layout", [
    (1, 1, 64, 16, "e2m1", "bf16", "plain"),
    (5, 3, 128, 32, "e2m1", "fp16", "merged"),
    (37, 2, 64, 48, "int4", "bf16", "odd"),
    (130, 5, 128, 16, "int4", "fp16", "heads_first"),
    (33, 8, 128, 64, "e2m1", "bf16", "odd"),
])
def test_cache_write_and_read(tokens, heads, d, bs, kind, dtype, layout):
    rng = np.random.default_rng(tokens)
    k, v = head_rows(rng, (tokens, heads, d), dtype), head_rows(rng, (tokens, heads, d), dtype)
    # a group of zeros, a NaN, both infinities, one value alone, the smallest and largest numbers
    k[0, 0, :16] = 0.0
    v[-1, -1, 3] = float("nan")
    v[-1, 0, 17], v[-1, 0, 18] = float("inf"), -float("inf")
    k[-1, 0, 16:32] = 0.0
    k[-1, 0, 20] = 2.0 ** -20
    k[-1, -1, 40] = torch.finfo(DT[dtype]).max
    nb = -(-tokens // bs) + 2
    slots = rng.permutation(nb * bs)[:tokens].astype(np.int64)
    if tokens > 4:
        slots[1], slots[3] = -1, nb * bs                     # outside the cache: skipped
    before = rng.integers(0, 256, w8.kv4_cache_shape(nb, heads, bs, d)).astype(np.uint8)
    kg, vg = 0.0131, 0.0217
    cache = dev(before)
    args = (dev(slots), dev(np.float32([kg])), dev(np.float32([vg])))
    w8.kv4_cache_write(view_of(k.cuda(), layout), view_of(v.cuda(), layout), cache, *args, kind=kind)
    want = kv4.write(before, slots, host(k), host(v), kg, vg, kind)
    assert np.array_equal(cache.cpu().numpy(), want)
    ko, vo = (view_of(torch.full((tokens, heads, d), 7.0, dtype=DT[dtype], device="cuda"), layout) for _ in range(2))
    w8.kv4_cache_read(cache, *args, ko, vo, kind=kind)
    inside = (slots >= 0) & (slots < nb * bs)
    rk, rv = kv4.tokens_of(want, np.where(inside, slots, 0), kg, vg, kind)
    for got, ref in ((ko, rk), (vo, rv)):
        ref = np.where(inside[:, None, None], ref, 0.0).astype(np.float32)  # one fp32 rounding, as the kernel's
        assert np.array_equal(host(got), host(torch.from_numpy(ref).to(DT[dtype])))


def test_cache_of_two_layouts_and_an_empty_call():
    cache = torch.zeros(w8.kv4_cache_shape(2, 1, 16, 64), dtype=torch.uint8, device="cuda")
    none = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    one = torch.ones(1, device="cuda")
    w8.kv4_cache_write(none, none, cache, torch.empty(0, dtype=torch.int64, device="cuda"), one, one)
    assert not cache.any()
    with pytest.raises(ValueError):
        w8.kv4_cache_write(none, none, cache, torch.empty(1, dtype=torch.int64, device="cuda"), one, one)
    with pytest.raises(ValueError):
        w8.kv4_cache_write(none, none, cache, torch.empty(0, dtype=torch.int64, device="cuda"), one, one, kind="fp4")


# ------------------------------------------------------------------ tables


@pytest.mark.parametrize("batch,bs,ctx,new,short,pad", [
    (1, 16, 0, 1, 0, 0), (3, 16, 40, 1, 0, 5), (300, 32, 100, 40, 0, 0), (300, 48, 100, 40, 60, 9), (1000, 16, 64, 3, 500, 1),
    (7, 128, 5, 2000, 0, 300), (16384, 16, 20, 2, 1000, 3), (5, 1, 3, 4, 0, 2),
])
def test_block_tables(batch, bs, ctx, new, short, pad):
    rng = np.random.default_rng(batch)
    c, n = rng.integers(-1, ctx + 1, batch).astype(np.int32), rng.integers(0, new + 1, batch).astype(np.int32)
    n[0] = max(1, n[0])
    mb = -(-(ctx + new) // bs)
    if batch > 4:
        n[3] = mb * bs + 1                                    # does not fit its table
        n[2] = -5
    held = -(-np.maximum(c, 0) // bs)
    need = -(-(np.maximum(c, 0) + np.maximum(n, 0)) // bs) - held
    if batch > 4:
        need[3] = 0
    ids = rng.permutation(int(held.sum() + need.sum()) + 20).astype(np.int32)
    table = np.full((batch, mb), -7, np.int32)
    table[np.arange(mb)[None] < held[:, None]] = ids[:held.sum()]
    if batch > 5 and held[5]:
        table[5, held[5] - 1] = -1
    free = ids[held.sum():]
    count = max(0, int(need.sum()) - short)
    tokens = int(np.maximum(n, 0).sum()) + pad
    out = [torch.full((s,), -9, dtype=t, device="cuda") for s, t in
           ((batch + 1, torch.int32), (batch, torch.int32), (tokens, torch.int64), (tokens, torch.int32), (1, torch.int32), (1, torch.int32))]
    gt = dev(table)
    for _ in range(2):                                        # a call can be repeated
        w8.build_block_tables(dev(c), dev(n), dev(free), dev(np.int32([count])), gt, bs, *out)
    want = kv4.block_tables(c, n, free, count, table, bs, tokens)
    assert np.array_equal(gt.cpu().numpy(), want[0])
    for got, ref in zip(out, want[1:]):
        assert np.array_equal(got.cpu().numpy(), np.atleast_1d(ref))


# ------------------------------------------------------------------ attention


def build(rng, lens, heads, d, bs, kind, kg, vg, dtype="bf16", extra=2):
    """A cache filled with quantised values, and a shuffled block table."""
    blocks = -(-np.maximum(lens, 0) // bs)
    nb = int(blocks.sum()) + extra
    table = np.full((len(lens), max(1, int(blocks.max())) + 1), -1, np.int32)
    table[np.arange(table.shape[1])[None] < blocks[:, None]] = rng.permutation(nb)[:blocks.sum()]
    cache = torch.zeros(w8.kv4_cache_shape(nb, heads, bs, d), dtype=torch.uint8, device="cuda")
    k, v = (head_rows(rng, (nb * bs, heads, d), dtype).cuda() for _ in range(2))
    w8.kv4_cache_write(k, v, cache, torch.arange(nb * bs, device="cuda"), dev(np.float32([kg])), dev(np.float32([vg])), kind=kind)
    return cache, table


def check(out, q, cache, lens, table, start, kg, vg, sm, kind, dtype):
    ref, r, big = kv4.attention(host(q), cache.cpu().numpy(), lens, table, start, np.float32(kg), np.float32(vg), sm, kind)
    d = q.shape[2]
    tol = (HALF_STEP[dtype] * np.abs(ref) + r * (2.0 ** -10 + 2.0 ** -18 + 2 * (d + 8) * 2.0 ** -24 * big[..., None]) +
           torch.finfo(DT[dtype]).smallest_normal * HALF_STEP[dtype])
    err = np.abs(host(out).astype(np.float64) - ref)
    assert np.isfinite(host(out)).all()
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size} outside, worst at {worst}: {host(out)[worst]} for {ref[worst]}"


def run(lens, news, hq, hkv, d, bs, kind, dtype, seed=0, out_dtype=None, layout="plain", edit=None, most=None, sm=None, single=False):
    rng = np.random.default_rng(seed)
    lens, news = np.asarray(lens), np.asarray(news)
    kg, vg = 0.0137, 0.0211
    cache, table = build(rng, lens, hkv, d, bs, kind, kg, vg, dtype)
    if edit is not None:
        edit(table, cache)
    start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    q = head_rows(rng, (int(start[-1]), hq, d), dtype, spikes=False).cuda()
    out = view_of(torch.full_like(q, float("nan"), dtype=DT[out_dtype or dtype]), layout)
    sm = 1.0 / np.sqrt(d) if sm is None else sm
    w8.kv4_attention(view_of(q, layout), cache, dev(lens.astype(np.int32)), dev(table), dev(np.float32([kg])), dev(np.float32([vg])),
                     out, query_start=None if single else dev(start), max_query_len=most or int(news.max()), sm_scale=sm, kind=kind)
    assert w8.device_status() == 0
    check(out, q, cache, lens, table, start, kg, vg, sm, kind, out_dtype or dtype)
    return out


@pytest.mark.parametrize("kind", ["e2m1", "int4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (6, 2), (8, 2), (5, 1), (16, 2), (12, 1), (64, 1)])
def test_attention_single_tokens(hq, hkv, d, kind):
    run([1, 15, 16, 17, 0, 100, 333], [1] * 7, hq, hkv, d, 16, kind, "bf16", single=True)


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp16"), ("fp16", "bf16")])
@pytest.mark.parametrize("bs", [16, 48, 128])
def test_attention_types_and_pages(dtype, out_dtype, bs):
    run([bs - 1, bs, bs + 1, 5 * bs + 7], [1, 2, 1, 3], 8, 2, 128, bs, "e2m1", dtype, out_dtype=out_dtype)


@pytest.mark.parametrize("layout", ["merged", "heads_first", "odd"])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_strides(layout, new):
    run([200, 77, 50], [new] * 3, 4, 2, 64, 16, "int4", "bf16", layout=layout)


@pytest.mark.parametrize("hq,hkv", [(4, 1), (8, 8), (6, 2), (16, 1)])
@pytest.mark.parametrize("news", [(2, 3, 4), (5, 1, 0), (8, 8, 16), (17, 1, 33)])
def test_attention_drafts(hq, hkv, news):
    run([300, 64, 90], news, hq, hkv, 128, 32, "e2m1", "bf16")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["e2m1", "int4"])
@pytest.mark.parametrize("lens,news,hq,hkv", [
    ((130,), (130,), 1, 1), ((500, 140, 3), (200, 140, 3), 4, 2), ((129, 1, 700), (64, 1, 257), 3, 1), ((260, 40), (130, 20), 10, 2),
])
def test_attention_prompts(lens, news, hq, hkv, d, kind):
    run(lens, news, hq, hkv, d, 32, kind, "bf16")


def test_attention_rows_that_see_nothing():
    """More new rows than tokens: the first rows see nothing and are zeros."""
    out = run([3, 0, 5], [6, 2, 5], 4, 2, 64, 16, "e2m1", "bf16")
    assert not out[:3].any() and not out[6:8].any()
    out = run([40, 10], [60, 30], 4, 2, 128, 16, "e2m1", "fp16")
    assert not out[:20].any() and not out[60:80].any()


@pytest.mark.parametrize("news", [(1, 1, 1), (3, 2, 1), (60, 50, 40)])
def test_attention_skips_blocks_outside_the_cache(news):
    """Negative ids, ids past the end, a request with no block at all; the
    skipped blocks' neighbours hold NaN scales, which nothing may read."""
    def edit(table, cache):
        table[0, 1], table[0, 3] = -1, cache.shape[0]
        table[1, :] = -1
        used = set(table[(table >= 0) & (table < cache.shape[0])].tolist())
        for i in range(cache.shape[0]):
            if i not in used:
                cache[i] = 0xFF
    out = run([170, 100, 99], news, 8, 2, 128, 32, "e2m1", "bf16", edit=edit)
    assert not out[news[0]:news[0] + news[1]].any()


@pytest.mark.parametrize("new", [1, 30])
def test_attention_ignores_what_lies_past_a_request(new):
    """The rest of a request's last block holds NaN scales."""
    def edit(table, cache):
        rec = 18 * 64
        for b, n in enumerate((21, 64 + 37)):
            last = table[b, (n - 1) // 64]
            for t in range(n % 64, 64):
                r = cache[last, :, t // 16]
                for at in (8 * 64, 17 * 64):
                    r[:, at + t % 16 * 4:at + t % 16 * 4 + 4] = 0x7F
        assert rec == cache.shape[3]
    run([21, 101], [min(new, 21), new], 4, 2, 64, 64, "e2m1", "bf16", edit=edit)


@pytest.mark.parametrize("sm", [0.0, 3.0, -0.5, 1e-6])
@pytest.mark.parametrize("new", [1, 24])
def test_attention_scales(sm, new):
    """Equal weights, near one-hot weights, a negative scale."""
    run([150, 49], [new] * 2, 8, 2, 128, 16, "e2m1", "fp16", sm=sm)


def test_attention_long_request():
    run([40000, 7], [1, 1], 8, 1, 128, 64, "int4", "fp16")
    run([9000, 130], [3, 4], 4, 1, 64, 16, "e2m1", "bf16")


def test_attention_many_short_requests():
    rng = np.random.default_rng(3)
    run(rng.integers(0, 60, 700), [1] * 700, 4, 2, 64, 16, "e2m1", "bf16")
    run(rng.integers(1, 40, 200), rng.integers(0, 9, 200), 8, 2, 64, 16, "int4", "bf16")


def test_attention_lengths_past_the_table_are_clamped():
    rng = np.random.default_rng(4)
    cache, table = build(rng, np.array([64]), 1, 64, 32, "e2m1", 0.01, 0.01)
    table = np.ascontiguousarray(table[:, :2])
    q = head_rows(rng, (1, 2, 64), "bf16").cuda()
    out = torch.empty_like(q)
    one = dev(np.float32([0.01]))
    w8.kv4_attention(q, cache, dev(np.int32([1000])), dev(table), one, one, out)
    check(out, q, cache, [64], table, [0, 1], 0.01, 0.01, 0.125, "e2m1", "bf16")


def test_attention_leaves_rows_past_max_query_len_and_padding():
    rng = np.random.default_rng(5)
    cache, table = build(rng, np.array([64, 64]), 1, 64, 32, "e2m1", 0.01, 0.01)
    q = head_rows(rng, (12, 2, 64), "bf16").cuda()
    out = torch.full_like(q, 7.0)
    one = dev(np.float32([0.01]))
    w8.kv4_attention(q, cache, dev(np.int32([64, 64])), dev(table), one, one, out, query_start=dev(np.int32([0, 4, 9])), max_query_len=5)
    assert (out[9:] == 7.0).all() and not (out[:9] == 7.0).all(2).any()


@pytest.mark.parametrize("most", [1, 3, 20])
def test_attention_of_the_first_rows_only(most):
    """A max_query_len below a request's new tokens: its first rows, each with
    the tokens that it sees among all of them; the others stay."""
    rng = np.random.default_rng(7)
    lens, start = np.array([90, 200]), np.int32([0, 40, 140])
    cache, table = build(rng, lens, 2, 64, 16, "e2m1", 0.013, 0.013)
    q = head_rows(rng, (140, 8, 64), "bf16").cuda()
    out = torch.full_like(q, 7.0)
    one = dev(np.float32([0.013]))
    w8.kv4_attention(q, cache, dev(lens.astype(np.int32)), dev(table), one, one, out, query_start=dev(start), max_query_len=most)
    rows = np.concatenate([np.arange(most), 40 + np.arange(most)])
    ref, r, big = kv4.attention(host(q), cache.cpu().numpy(), lens, table, start, np.float32(0.013), np.float32(0.013), 0.125, "e2m1")
    # besides the module's bounds: a weight is off by up to 2^-38 of the row's
    # largest (f16's last bit, 2^-25 at half a step, after its scaling by 2^13), on
    # each of 200 values of at most 6 * 448 * 0.013; it shows where a row's other
    # weights meet zeros
    tol = (2.0 ** -8 * np.abs(ref) + r * (2.0 ** -10 + 2.0 ** -18 + 2 * 72 * 2.0 ** -24 * big[..., None]) +
           2.0 ** -38 * 200 * 6 * 448 * 0.013)
    assert (np.abs(host(out).astype(np.float64) - ref)[rows] <= tol[rows]).all()
    rest = np.setdiff1d(np.arange(140), rows)
    assert (out[torch.from_numpy(rest).cuda()] == 7.0).all()


@pytest.mark.parametrize("new", [1, 40])
def test_offsets_past_32_bits(new):
    """Blocks 5 GB into the cache."""
    rng = np.random.default_rng(8)
    lens = np.array([100, 60])
    small, table = build(rng, lens, 1, 64, 16, "int4", 0.013, 0.013)
    nb = 5_000_000_000 // (18 * 64)
    cache = torch.empty(w8.kv4_cache_shape(nb, 1, 16, 64), dtype=torch.uint8, device="cuda")
    far = nb - small.shape[0]
    cache[far:] = small
    q = head_rows(rng, (2 * new, 4, 64), "bf16").cuda()
    start = dev(np.int32([0, new, 2 * new]))
    one, gl = dev(np.float32([0.013])), dev(lens.astype(np.int32))
    out, want = torch.empty_like(q), torch.empty_like(q)
    args = dict(query_start=start, max_query_len=new, kind="int4")
    w8.kv4_attention(q, small, gl, dev(table), one, one, want, **args)
    w8.kv4_attention(q, cache, gl, dev(np.where(table >= 0, table + far, -1).astype(np.int32)), one, one, out, **args)
    assert torch.equal(out, want)
    k, v = (head_rows(rng, (30, 1, 64), "bf16").cuda() for _ in range(2))
    slots = torch.arange(30, device="cuda") * 3
    w8.kv4_cache_write(k, v, small, slots, one, one, kind="int4")
    w8.kv4_cache_write(k, v, cache, slots + far * 16, one, one, kind="int4")
    assert torch.equal(cache[far:], small)
    near, away = ([torch.empty_like(k), torch.empty_like(k)] for _ in range(2))
    w8.kv4_cache_read(small, slots, one, one, *near, kind="int4")
    w8.kv4_cache_read(cache, slots + far * 16, one, one, *away, kind="int4")
    assert torch.equal(near[0], away[0]) and torch.equal(near[1], away[1])


@pytest.mark.parametrize("new", [1, 40])
def test_attention_on_another_stream_in_a_graph_and_repeated(new):
    rng = np.random.default_rng(6)
    lens = np.array([3000, 900, 1700])
    cache, table = build(rng, lens, 2, 128, 16, "e2m1", 0.013, 0.013)
    q = head_rows(rng, (3 * new, 8, 128), "bf16").cuda()
    one, gl, gt = dev(np.float32([0.013])), dev(lens.astype(np.int32)), dev(table)
    start = dev(np.int32([0, new, 2 * new, 3 * new]))
    ws = w8.Workspace(w8.kv4_attention_workspace_size(3, new, 8, 2, 128))
    first = torch.empty_like(q)
    w8.kv4_attention(q, cache, gl, gt, one, one, first, query_start=start, max_query_len=new, workspace=ws)
    check(first, q, cache, lens, table, start.cpu().numpy(), 0.013, 0.013, 128 ** -0.5, "e2m1", "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(q)
    w8.kv4_attention(q, cache, gl, gt, one, one, out, query_start=start, max_query_len=new, stream=s,
                     workspace=w8.Workspace(w8.kv4_attention_workspace_size(3, new, 8, 2, 128)))
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w8.kv4_attention(q, cache, gl, gt, one, one, out, query_start=start, max_query_len=new, workspace=ws)
    for _ in range(3):
        out.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


# ------------------------------------------------------------------ verification


@pytest.mark.parametrize("batch,drafts,vocab,dtype,greedy", [
    (1, 1, 1, "fp32", False), (1, 0, 777, "fp32", False), (3, 2, 33, "fp32", False), (9, 7, 1000, "bf16", False),
    (17, 4, 32001, "fp32", False), (5, 3, 5000, "fp16", True), (6, 5, 40000, "fp32", True), (2, 3, 131072, "bf16", False),
    (200, 3, 2049, "fp32", False),
])
def test_verify(batch, drafts, vocab, dtype, greedy):
    rng = np.random.default_rng(batch * 7 + vocab)
    for trial in range(3):
        counts = rng.integers(0, drafts + 1, batch)
        start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        rows = int(start[-1])
        of = np.repeat(np.arange(batch), counts)
        logits = 2 * rng.standard_normal((rows + batch, vocab))
        soft = lambda x: np.exp(x) / np.exp(x).sum(1, keepdims=True)  # noqa: E731
        target = torch.from_numpy(soft(logits)).to(DT[dtype])
        dl = logits[np.arange(rows) + of] + 0.5 * rng.standard_normal((rows, vocab))
        draft = None if greedy else torch.from_numpy(soft(dl)).to(DT[dtype])
        tokens = (dl.argmax(1) if greedy else np.array([rng.choice(vocab, p=row) for row in soft(dl)])).astype(np.int32).reshape(rows)
        if rows > 3:
            tokens[1] = vocab                                 # outside: not kept
        if rows > 5:
            target[3 + of[3], :vocab // 2] = float("nan")     # no weight
            target[4 + of[4]] = 0.0                           # no distribution at all
        u, s = rng.random(rows).astype(np.float32), rng.random(batch).astype(np.float32)
        s[0] = 0.0
        ld = vocab + 5
        wide = lambda t: torch.zeros(t.shape[0], ld, dtype=t.dtype, device="cuda")[:, :vocab].copy_(t)  # noqa: E731
        out = torch.full((batch, drafts + 1), 99, dtype=torch.int32, device="cuda")
        n = torch.full((batch,), 99, dtype=torch.int32, device="cuda")
        w8.verify_drafts(wide(target), None if draft is None else wide(draft), dev(tokens), dev(start), dev(u), dev(s), out, n)
        want = kv4.verify(host(target), None if draft is None else host(draft), tokens, start, u, s, drafts)
        assert np.array_equal(n.cpu().numpy(), want[1])
        assert np.array_equal(out.cpu().numpy(), want[0])


def test_verify_equal_models_keep_everything():
    p = torch.softmax(torch.randn(6, 500, device="cuda"), 1)
    tokens = torch.multinomial(p[:4], 1).int().squeeze(1)
    target = torch.cat([p[:2], p[4:5], p[2:4], p[5:6]])
    out = torch.empty(2, 3, dtype=torch.int32, device="cuda")
    n = torch.empty(2, dtype=torch.int32, device="cuda")
    w8.verify_drafts(target, p[:4].contiguous(), tokens, dev(np.int32([0, 2, 4])), torch.full((4,), 1 - 2.0 ** -24, device="cuda"),
                     torch.rand(2, device="cuda"), out, n)
    assert n.tolist() == [2, 2] and torch.equal(out[:, :2].flatten(), tokens) and (out >= 0).all()
