"""Long contexts over the paged fp8 cache on the GPU, against the oracle.

Codes, scales, selections and rotated queries are equal: every rounding of
theirs is part of the definition.  Attention's tolerance, per output element,
with r the weights' mean of |V| and w the largest weight of the row:
  * the output's rounding, half a step: 2^-8 |ref| (bf16), 2^-11 |ref| (fp16),
    or half the smallest subnormal number where the output is below the normal
    ones (fp16: 2^-25);
  * the softmax weights' rounding before the second product, 2^-11 of each
    weight, in its numerator and again in the sum that divides it: 2^-10 r; a
    weight below 2^-18 of the row's largest may lose bits down to 2^-28 of that
    one, so that a row of T tokens is off by at most T 2^-28 w max |V|, twice
    with the sum;
  * fp32 scores: d products and sums and the scaling, each off by 2^-24 of at
    most B = max_t sum_d |q_d K_td| * sm_scale, move a weight's exponent by
    (d + 8) 2^-24 B, twice as much relative to the maximum; elements of the
    query that are smaller than 2^-13 of its row's largest may lose bits down
    to 2^-24 of that one: 2^-24 B', with the largest in the place of all;
    exp2's approximation and the sums of 32 bits over the tokens stay below
    2^-18.  Together (2 (d + 8) 2^-24 B + 2^-22 B' + 2^-18) r."""
import numpy as np
import pytest
import torch

import int8_w8a8_scaled_gb300 as w8
from oracle import fp8_paged as fp

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
E4M3 = torch.float8_e4m3fn


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().float().cpu().numpy()


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def head_rows(rng, shape, dtype, spikes=True):
    x = rng.standard_normal(shape).astype(np.float32)
    if spikes:
        x[..., 5::37] *= 8
    return torch.from_numpy(x).to(DT[dtype])


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


# ------------------------------------------------------------------ rotation and write


@pytest.mark.parametrize("tokens,hq,h,d,rot,sections,inter,bs,dtype,layout,in_place", [
    (1, 4, 1, 64, 64, None, False, 16, "bf16", "plain", False),
    (7, 6, 3, 128, 128, None, True, 32, "fp16", "merged", True),
    (37, 8, 2, 64, 32, (4, 6, 6), True, 48, "bf16", "odd", False),
    (130, 5, 5, 128, 64, (8, 24), False, 16, "fp16", "heads_first", True),
    (33, 32, 8, 128, 112, None, False, 64, "bf16", "plain", True),
    (9, 3, 1, 64, 6, (1, 0, 1, 1), False, 16, "bf16", "merged", False),
    (600, 32, 8, 128, 128, (16, 24, 24), False, 64, "bf16", "merged", False),
    (11, 0, 2, 128, 16, None, True, 16, "fp16", "plain", False),
])
def test_rotate_write(tokens, hq, h, d, rot, sections, inter, bs, dtype, layout, in_place):
    rng = np.random.default_rng(tokens)
    q, k, v = (head_rows(rng, (tokens, n, d), dtype) for n in (max(hq, 1), h, h))
    k[0, 0, 0], v[0, 0, 1], v[-1, -1, 2], k[-1, 0, d - 1] = float("nan"), float("inf"), -float("inf"), torch.finfo(DT[dtype]).max
    axes = 1 if sections is None else len(sections)
    angle = rng.uniform(-3, 3, (50, rot // 2))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    pos = rng.integers(0, 50, (axes, tokens)).astype(np.int32)
    if tokens > 4:
        pos[-1, 2], pos[0, 4] = -1, 50                       # outside the table: NaN
    nb = -(-tokens // bs) + 2
    slots = rng.permutation(nb * bs)[:tokens].astype(np.int64)
    if tokens > 4:
        slots[1], slots[3] = -1, nb * bs                     # outside the cache: skipped
    before = [rng.integers(0, 256, (nb, bs, h, d)).astype(np.uint8) for _ in range(2)]
    caches = [dev(x).view(E4M3) for x in before]
    kg, vg = 0.0131, 0.0217
    qg = view_of(q.cuda(), layout)
    q_out = None if hq == 0 else qg if in_place else view_of(torch.full_like(q, 7.0).cuda(), layout)
    w8.fp8_kv_rotate_write(None if hq == 0 else qg, view_of(k.cuda(), layout), view_of(v.cuda(), layout), dev(table),
                           dev(pos if axes > 1 else pos[0]), *caches, dev(slots), dev(np.float32([kg])), dev(np.float32([vg])), q_out,
                           sections=sections, interleaved=inter)
    args = (pos, table, sections, inter)
    if hq:
        want = torch.from_numpy(fp.rotate(q.float().numpy(), *args)).to(DT[dtype])
        assert np.array_equal(host(q_out), host(want), equal_nan=True)
    assert np.array_equal(codes(caches[0]), fp.write(before[0], slots, fp.rotate(k.float().numpy(), *args), kg))
    assert np.array_equal(codes(caches[1]), fp.write(before[1], slots, v.float().numpy(), vg))


def test_rotate_write_of_a_merged_projection_in_place():
    """q, k and v are slices of one buffer, and q is turned where it lies."""
    rng = np.random.default_rng(5)
    rows = head_rows(rng, (19, 12, 64), "bf16")
    angle = rng.uniform(-3, 3, (50, 32))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    pos, slots = rng.integers(0, 50, 19).astype(np.int32), rng.permutation(32)[:19].astype(np.int64)
    caches = [torch.zeros(2, 16, 2, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
    one, buf = torch.ones(1, device="cuda"), rows.cuda()
    q, k, v = buf[:, :8], buf[:, 8:10], buf[:, 10:]
    w8.fp8_kv_rotate_write(q, k, v, dev(table), dev(pos), *caches, dev(slots), one, one, q)
    x = rows.float().numpy()
    assert np.array_equal(host(buf[:, :8]), host(torch.from_numpy(fp.rotate(x[:, :8], pos, table)).bfloat16()))
    assert np.array_equal(host(buf[:, 8:]), x[:, 8:])
    zero = np.zeros((2, 16, 2, 64), np.uint8)
    assert np.array_equal(codes(caches[0]), fp.write(zero, slots, fp.rotate(x[:, 8:10], pos, table), 1.0))
    assert np.array_equal(codes(caches[1]), fp.write(zero, slots, x[:, 10:], 1.0))


# ------------------------------------------------------------------ attention


class Step:
    """A step over random caches: `lens` tokens of each request, the last `new` of them in q."""

    def __init__(self, seed, lens, new, hq, h, d, bs, dtype="bf16", extra_rows=0, spare=2, tail=None):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.new = np.int32(lens), np.int32(new)
        self.d, self.bs, self.h, self.hq, self.dtype = d, bs, h, hq, dtype
        blocks = -(-np.maximum(self.lens, 0) // bs)
        self.nb = int(blocks.sum()) + spare
        self.table = np.full((len(lens), max(1, int(blocks.max()))), -1, np.int32)
        self.table[np.arange(self.table.shape[1])[None] < blocks[:, None]] = rng.permutation(self.nb)[:blocks.sum()]
        x = np.clip(rng.standard_normal((2, self.nb, bs, h, d)) * 20, -448, 448).astype(np.float32)
        self.kc, self.vc = fp.encode(x)
        if tail is not None:                                 # what no request's token has written
            held = np.zeros((self.nb, bs), bool)
            for b, n in enumerate(self.lens):
                for col in range(int(blocks[b])):
                    held[self.table[b, col], :n - col * bs] = True
            self.kc[~held], self.vc[~held] = tail, tail
        self.start = np.concatenate([[0], np.cumsum(np.maximum(self.new, 0))]).astype(np.int32)
        self.tokens = int(self.start[-1]) + extra_rows
        self.q = head_rows(rng, (max(1, self.tokens), hq, d), dtype)
        self.kg, self.vg, self.sm = 0.011, 0.017, 1.0 / d ** 0.5
        self.most = max(1, int(self.new.max()))

    def run(self, layout="plain", selected=None, most=None, out_dtype=None, query_start=True, fill=7.0, **kw):
        q = view_of(self.q.cuda(), layout)
        out = view_of(torch.full(self.q.shape, fill, dtype=DT[out_dtype or self.dtype], device="cuda"), layout)
        args = [q, dev(self.kc).view(E4M3), dev(self.vc).view(E4M3), dev(self.lens), dev(self.table)]
        call = w8.fp8_kv_attention
        if selected is not None:
            args.append(dev(selected))
            call = w8.fp8_kv_sparse_attention
        call(*args, dev(np.float32([self.kg])), dev(np.float32([self.vg])), out, query_start=dev(self.start) if query_start else None,
             max_query_len=most or self.most, sm_scale=self.sm, **kw)
        return out

    def check(self, out, selected=None, most=None, out_dtype=None, query_start=True, fill=7.0):
        q = self.q.float().numpy()
        ref, written, r, reach, far = fp.attention(q, self.kc, self.vc, self.kg, self.vg, self.lens, self.table,
                                                   self.start if query_start else None, most or self.most, self.sm, selected)
        got, dt = host(out).astype(np.float64), out_dtype or self.dtype
        assert (got[~written] == fill).all()
        got, ref, r, reach, far = got[written], ref[written], r[written], reach[written, :, None], far[written, :, None]
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        with np.errstate(all="ignore"):
            top = np.nanmax(np.abs(fp.VALUES[self.vc])) * self.vg
            tol = (HALF_STEP[dt] * np.abs(ref) + 2.0 ** -25 + (2.0 ** -10 + 2 * (self.d + 8) * 2.0 ** -24 * reach + 2.0 ** -22 * far + 2.0 ** -18) * r
                   + 2 * 2.0 ** -28 * self.seen(selected) * top)
            bad = np.abs(got - ref) > tol
        assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5], tol[bad][:5])

    def seen(self, selected):
        return max(1, int(self.lens.max())) if selected is None else selected.shape[2] * self.bs


ATTENTION = [
    # lens, new, hq, h, d, bs, dtype, layout
    ([1], [1], 1, 1, 64, 16, "bf16", "plain"),
    ([17, 300, 0, 64], [1, 1, 1, 1], 8, 2, 128, 16, "fp16", "odd"),
    ([128, 127, 129, 1000], [3, 2, 1, 5], 8, 2, 128, 32, "bf16", "merged"),
    ([40, 2, 777], [5, 2, 7], 12, 4, 64, 48, "fp16", "heads_first"),
    ([200, 90], [9, 0], 16, 2, 128, 16, "bf16", "plain"),            # 72 rows a KV head, and a request without any
    ([700], [33], 5, 5, 64, 64, "fp16", "odd"),
    ([400, 1, 60, 250], [150, 1, 60, 1], 8, 4, 128, 16, "bf16", "merged"),   # prompts with single tokens between
    ([300, 257], [300, 257], 4, 1, 64, 128, "fp16", "plain"),                # whole prompts, two row blocks of 256
    ([1500], [130], 8, 4, 128, 32, "fp16", "plain"),
    ([2000, 1999], [4, 4], 64, 8, 128, 64, "bf16", "plain"),
    ([90, 500], [1, 1], 64, 1, 64, 16, "bf16", "plain"),             # 64 heads to a KV head
]


@pytest.mark.parametrize("lens,new,hq,h,d,bs,dtype,layout", ATTENTION)
def test_attention(lens, new, hq, h, d, bs, dtype, layout):
    s = Step(len(lens) + hq, lens, new, hq, h, d, bs, dtype, extra_rows=2)
    s.check(s.run(layout))


def test_attention_of_single_tokens_without_starts():
    s = Step(3, [50, 1, 0, 33], [1, 1, 1, 1], 8, 2, 128, 16)
    s.check(s.run(query_start=False), query_start=False)


@pytest.mark.parametrize("new", [2, 40])
def test_attention_writes_the_other_type(new):
    s = Step(4, [100, 80], [new, 1], 8, 2, 64, 16, "bf16")
    s.check(s.run(out_dtype="fp16"), out_dtype="fp16")


@pytest.mark.parametrize("new", [[3, 5, 2], [100, 60, 1]])
def test_attention_with_holes_short_requests_and_limits(new):
    """Entries outside the cache, rows in front of the first token, fewer rows looked at than there are."""
    s = Step(5, [200, 170, 2], new, 8, 4, 128, 16)
    s.table[0, 3], s.table[0, 7], s.table[1, 0], s.table[2, 0] = -1, s.nb, -5, 1 << 30
    s.check(s.run())
    s = Step(6, [200, 1, 60], [new[0], 9, new[2]], 4, 2, 64, 16, extra_rows=3)   # 9 rows, of which only the last has a token
    s.check(s.run(most=4), most=4)
    s.check(s.run(most=1 << 20), most=1 << 20)


@pytest.mark.parametrize("lens,new", [([37, 200, 5], [4, 2, 5]), ([137, 300], [70, 90]), ([1000, 33], [1, 1])])
@pytest.mark.parametrize("d", [64, 128])
def test_what_no_token_has_written_may_be_anything(lens, new, d):
    s = Step(7, lens, new, 8, 2, d, 32, tail=0x7F)
    s.check(s.run())
    if len(lens) > 2:
        s.table[1, 2] = -1
        s.check(s.run())


@pytest.mark.parametrize("lens,new", [([60, 200], [6, 3]), ([300, 260], [70, 130]), ([70, 40], [1, 1])])
def test_a_nan_reaches_only_the_rows_that_see_it(lens, new):
    s = Step(8, lens, new, 8, 2, 128, 16)
    for b, back in ((0, 2), (1, 1)):                         # values of late tokens, which earlier rows do not see
        t = lens[b] - back
        s.vc[s.table[b, t // 16], t % 16, 1, 5] = 0xFF
        s.vc[s.table[b, t // 16], t % 16, 0, 77] = 0x7F
    s.kc[s.table[1, (lens[1] - 1) // 16], (lens[1] - 1) % 16, 0, 3] = 0x7F
    s.check(s.run())


@pytest.mark.parametrize("lens,new", [([60, 200], [6, 3]), ([300, 260], [70, 130]), ([70, 40], [1, 1])])
def test_a_nan_or_an_infinity_in_a_query_stays_in_its_row(lens, new):
    s = Step(9, lens, new, 8, 2, 128, 16)
    s.q[0, 0, 3], s.q[0, 5, 9], s.q[-1, 7, 127] = float("nan"), float("inf"), -float("inf")
    s.check(s.run())


@pytest.mark.parametrize("new", [[2, 5], [60, 100]])
def test_far_scores_and_queries_of_every_size(new):
    s = Step(10, [300, 270], new, 8, 2, 128, 16)
    s.q[0] *= 1e4
    s.q[1] *= 2.0 ** -120
    s.q[2, 1] = 0
    if new[0] > 2:
        s.q[3, :, ::2] *= 2.0 ** -20
    s.check(s.run())
    s.kg = -s.kg                                             # the signs of both scales count
    s.check(s.run())
    s.sm = 0.0                                               # all weights equal
    s.check(s.run())


def test_many_equal_weights_below_the_largest():
    """One key far above the others, whose many small weights are together as much."""
    s = Step(11, [6000, 6000], [1, 40], 4, 2, 64, 16)
    s.kc[...] = 0
    s.q[...] = 0
    s.q[:, :, 0] = 1.0
    for b in range(2):
        s.kc[s.table[b, 0], 0, :, 0] = fp.encode(np.float32([128.0]))[0]
    s.kg, s.sm = 1.0, 13 * np.log(2.0) / 128                 # 2^13 times a weight of the rest
    s.check(s.run())


@pytest.mark.parametrize("new", [[4, 1], [70, 3]])
def test_attention_repeats_bit_for_bit_in_a_graph(new):
    s = Step(12, [3000, 900], new, 16, 2, 128, 64)
    first = s.run()
    q, out = s.q.cuda(), torch.zeros(s.q.shape, dtype=torch.bfloat16, device="cuda")
    args = (q, dev(s.kc).view(E4M3), dev(s.vc).view(E4M3), dev(s.lens), dev(s.table), dev(np.float32([s.kg])), dev(np.float32([s.vg])), out)
    kw = dict(query_start=dev(s.start), max_query_len=s.most, sm_scale=s.sm)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        w8.fp8_kv_attention(*args, **kw)
        w8.fp8_kv_attention(*args, **kw)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)
    assert w8.device_status() == 0


# ------------------------------------------------------------------ means, selection


@pytest.mark.parametrize("lens,new,h,d,bs", [
    ([1, 16, 17, 100], [1, 1, 2, 40], 2, 64, 16), ([700, 64, 63], [200, 64, 1], 3, 128, 64), ([500, 0, 3], [500, 0, 7], 1, 128, 48),
    ([2100, 40], [1500, 1], 2, 64, 1024), ([300], [2], 5, 128, 128),
])
def test_block_means(lens, new, h, d, bs):
    s = Step(20, lens, new, h, h, d, bs, tail=0x7F)
    s.kc[s.table[0, 0], 0, 0, :] = 0x7F                      # NaN codes count as 0
    s.kc[s.table[0, -1], :, -1, :] = 0                       # a block of zeros: scale 1
    if len(lens) > 2 and s.table[1, 0] >= 0:
        s.table[1, 0] = s.nb                                 # outside the cache: skipped
    means, scales = s.rng.integers(-127, 128, (s.nb, h, d)).astype(np.int8), s.rng.random((s.nb, h)).astype(np.float32)
    gm, gs = dev(means), dev(scales)
    w8.fp8_kv_block_means(dev(s.kc).view(E4M3), dev(s.lens), dev(s.table), gm, gs, query_start=dev(s.start), max_query_len=s.most)
    wm, ws = fp.block_means(s.kc, s.lens, s.table, s.start, s.most, means, scales)
    assert np.array_equal(gm.cpu().numpy(), wm) and np.array_equal(gs.cpu().numpy(), ws)


SELECT = [
    # lens, new, hq, h, d, bs, budget, first, last, dtype, layout
    ([1, 40, 1000], [1, 1, 1], 4, 2, 64, 16, 5, 1, 2, "bf16", "plain"),
    ([900, 2000], [3, 2], 8, 1, 128, 16, 20, 0, 1, "fp16", "odd"),
    ([5000], [9], 12, 4, 64, 16, 64, 2, 3, "bf16", "merged"),
    ([700, 3, 260], [70, 3, 1], 10, 2, 128, 16, 7, 1, 1, "fp16", "heads_first"),
    ([9000], [5], 16, 16, 64, 16, 300, 0, 1, "bf16", "plain"),
    ([600, 600], [2, 90], 64, 1, 128, 32, 3, 1, 2, "bf16", "plain"),          # no room beside the forced ones
    ([3000], [4], 24, 2, 64, 16, 33, 0, 1, "fp16", "plain"),                  # 12 heads to a KV head: two tiles
]


def selection_of(s, means, scales, budget, first, last, layout="plain", most=None, fill=-9):
    selected = torch.full((s.q.shape[0], s.h, budget), fill, dtype=torch.int32, device="cuda")
    w8.fp8_kv_select_blocks(view_of(s.q.cuda(), layout), dev(means), dev(scales), dev(s.lens), dev(s.table), s.bs, selected,
                            query_start=dev(s.start), max_query_len=most or s.most, first_blocks=first, last_blocks=last)
    return selected.cpu().numpy()


@pytest.mark.parametrize("lens,new,hq,h,d,bs,budget,first,last,dtype,layout", SELECT)
def test_select_blocks(lens, new, hq, h, d, bs, budget, first, last, dtype, layout):
    s = Step(30, lens, new, hq, h, d, bs, dtype, extra_rows=2)
    means, scales = s.rng.integers(-127, 128, (s.nb, h, d)).astype(np.int8), (s.rng.random((s.nb, h)) + 0.1).astype(np.float32)
    before = np.full((s.q.shape[0], h, budget), -9, np.int32)
    want = fp.select(s.q.float().numpy(), means, scales, s.lens, s.table, bs, s.start, s.most, first, last, budget, before)
    assert np.array_equal(selection_of(s, means, scales, budget, first, last, layout), want)


def test_select_blocks_ties_holes_and_odd_numbers():
    s = Step(31, [4000, 2500], [3, 40], 4, 2, 64, 16, extra_rows=1)
    means, scales = s.rng.integers(-2, 3, (s.nb, 2, 64)).astype(np.int8), np.ones((s.nb, 2), np.float32)   # many equal scores
    s.q = torch.from_numpy(s.rng.integers(-1, 2, s.q.shape).astype(np.float32)).bfloat16()
    s.q[0] = 0                                               # all scores equal
    s.q[1, 1, 3], s.q[2, 3, 0], s.q[4, 0, 7] = float("nan"), float("inf"), -float("inf")
    s.table[0, 30], s.table[1, 5], s.table[1, 0] = -1, s.nb, 1 << 30
    scales[s.table[0, 20]], scales[s.table[0, 21]] = float("nan"), float("inf")
    before = np.full((s.q.shape[0], 2, 50), -9, np.int32)
    want = fp.select(s.q.float().numpy(), means, scales, s.lens, s.table, 16, s.start, 30, 1, 2, 50, before)
    assert np.array_equal(selection_of(s, means, scales, 50, 1, 2, most=30), want)


def test_select_blocks_in_several_slabs():
    """More tokens than one pass holds scores of: 64 MB / (heads * columns * 4)."""
    s = Step(32, [60, 40, 900], [60, 40, 300], 2, 2, 64, 16)
    s.table = np.concatenate([s.table, np.full((3, 40000 - s.table.shape[1]), -1, np.int32)], 1)
    assert s.tokens * 2 * 40000 * 4 > (64 << 20)
    means, scales = s.rng.integers(-127, 128, (s.nb, 2, 64)).astype(np.int8), (s.rng.random((s.nb, 2)) + 0.1).astype(np.float32)
    before = np.full((s.q.shape[0], 2, 6), -9, np.int32)
    want = fp.select(s.q.float().numpy(), means, scales, s.lens, s.table, 16, s.start, s.most, 1, 2, 6, before)
    assert np.array_equal(selection_of(s, means, scales, 6, 1, 2), want)


# ------------------------------------------------------------------ sparse attention


def random_columns(s, budget, rng):
    sel = np.full((s.q.shape[0], s.h, budget), -1, np.int32)
    for b, t, pos in fp.requests(s.lens, s.start, s.q.shape[0], s.most, s.table.shape[1] * s.bs):
        n = max(0, pos // s.bs + 1) if pos >= 0 else 0
        for kv in range(s.h):
            cols = np.sort(rng.permutation(n)[:rng.integers(0, budget + 1)])
            sel[t, kv, :len(cols)] = cols
    return sel


SPARSE = [
    # lens, new, hq, h, d, bs, budget, dtype, layout
    ([1], [1], 1, 1, 64, 16, 1, "bf16", "plain"),
    ([1000, 50, 0, 333], [1, 1, 1, 1], 8, 2, 128, 16, 9, "fp16", "odd"),
    ([2000, 900], [5, 3], 16, 2, 128, 32, 30, "bf16", "merged"),
    ([600, 90], [130, 40], 6, 2, 64, 48, 5, "fp16", "heads_first"),
    ([5000], [2], 32, 1, 128, 64, 70, "bf16", "plain"),
    ([400], [3], 64, 1, 64, 16, 12, "bf16", "plain"),
    ([700, 300], [2, 1], 5, 5, 128, 128, 4, "fp16", "plain"),
]


@pytest.mark.parametrize("lens,new,hq,h,d,bs,budget,dtype,layout", SPARSE)
def test_sparse_attention(lens, new, hq, h, d, bs, budget, dtype, layout):
    s = Step(40, lens, new, hq, h, d, bs, dtype, extra_rows=2, tail=0x7F)
    sel = random_columns(s, budget, s.rng)
    s.check(s.run(layout, selected=sel), selected=sel)


def test_sparse_attention_with_odd_selections():
    """No column, the same one twice, ones outside the table, past the token, outside the cache, in any order."""
    s = Step(41, [500, 300], [4, 2], 8, 2, 128, 16, tail=0xFF)
    sel = np.full((s.q.shape[0], 2, 8), -1, np.int32)
    sel[0, 0] = [31, 3, 3, 0, 7, -4, 1 << 30, 2]
    sel[0, 1] = s.table.shape[1]
    sel[1, 0] = [-1, -1, 5, -1, 4, -1, -1, 30]
    sel[2, :, 0] = 31                                        # partly past the token
    sel[4, :, :3] = [[25, 2, 1], [18, 18, 18]]               # past the token; its own block three times
    s.table[0, 7] = -1
    s.vc[s.table[0, 31], 3, 1, 9] = 0x7F                     # token 499: only the last row may see it
    s.check(s.run(selected=sel), selected=sel)


def test_sparse_attention_in_a_graph():
    s = Step(42, [3000, 900], [4, 1], 16, 2, 128, 64)
    sel = random_columns(s, 20, s.rng)
    first = s.run(selected=sel)
    out = torch.zeros(s.q.shape, dtype=torch.bfloat16, device="cuda")
    args = (s.q.cuda(), dev(s.kc).view(E4M3), dev(s.vc).view(E4M3), dev(s.lens), dev(s.table), dev(sel), dev(np.float32([s.kg])),
            dev(np.float32([s.vg])), out)
    kw = dict(query_start=dev(s.start), max_query_len=s.most, sm_scale=s.sm)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        w8.fp8_kv_sparse_attention(*args, **kw)
        w8.fp8_kv_sparse_attention(*args, **kw)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)
    assert w8.device_status() == 0


# ------------------------------------------------------------------ together


def test_steps_together():
    """Tables, write, means, selection and attention of a prompt and of single tokens after it, on one stream without a look
    from the host; with a budget for all blocks the sparse attention is the whole one's."""
    rng = np.random.default_rng(50)
    hq, h, d, bs, mb, nb, batch = 8, 2, 128, 16, 24, 60, 3
    angle = np.arange(400)[:, None] * 100.0 ** (-np.arange(d // 2) / (d // 2))
    table_cs = dev(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32))
    kc, vc = (torch.full((nb, bs, h, d), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    means, scales = torch.zeros(nb, h, d, dtype=torch.int8, device="cuda"), torch.zeros(nb, h, device="cuda")
    ints = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    table, free = torch.full((batch, mb), -1, dtype=torch.int32, device="cuda"), dev(rng.permutation(nb).astype(np.int32))
    count, held, g = ints(1) + nb, ints(batch), torch.full((1,), 0.05, device="cuda")
    for new in ([200, 33, 1], [1, 1, 1], [3, 1, 2]):
        n = sum(new)
        start, lens, pos, slots, left, after = ints(batch + 1), ints(batch), ints(n), torch.zeros(n, dtype=torch.int64, device="cuda"), ints(1), ints(1)
        w8.build_block_tables(held, dev(np.int32(new)), free, count, table, bs, start, lens, slots, pos, left, free_count_out=after)
        rows = head_rows(rng, (n, hq + 2 * h, d), "bf16").cuda()
        q, k, v = rows.split([hq, h, h], 1)
        w8.fp8_kv_rotate_write(q, k, v, table_cs, pos, kc, vc, slots, g, g, q)
        w8.fp8_kv_block_means(kc, lens, table, means, scales, query_start=start, max_query_len=max(new))
        whole, sparse, few = (torch.full((n, hq, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3))
        kw = dict(query_start=start, max_query_len=max(new))
        w8.fp8_kv_attention(q, kc, vc, lens, table, g, g, whole, **kw)
        sel, small = (torch.full((n, h, b), -9, dtype=torch.int32, device="cuda") for b in (mb, 5))
        w8.fp8_kv_select_blocks(q, means, scales, lens, table, bs, sel, **kw)
        w8.fp8_kv_sparse_attention(q, kc, vc, lens, table, sel, g, g, sparse, **kw)
        w8.fp8_kv_select_blocks(q, means, scales, lens, table, bs, small, **kw)
        w8.fp8_kv_sparse_attention(q, kc, vc, lens, table, small, g, g, few, **kw)
        held, count = lens, after
        q32, cpu = q.float().cpu().numpy(), lambda t: t.cpu().numpy()  # noqa: E731
        args = (codes(kc), codes(vc), 0.05, 0.05, cpu(lens), cpu(table), cpu(start), max(new), d ** -0.5)
        want_small = fp.select(q32, cpu(means), cpu(scales), cpu(lens), cpu(table), bs, cpu(start), max(new), 1, 2, 5, cpu(small))
        assert np.array_equal(cpu(small), want_small)
        for out, selected in ((whole, None), (sparse, cpu(sel)), (few, cpu(small))):
            ref = fp.attention(q32, *args, selected)[0]
            err = np.abs(host(out) - ref)
            assert (err <= 2.0 ** -6 * np.abs(ref) + 2.0 ** -7 * np.abs(ref).max()).all()
    assert w8.device_status() == 0
