"""The operators over the paged fp8 cache at the edges of what their documentation
allows (tolerances as in test_gpu_fp8_paged.py)."""
import numpy as np
import pytest
import torch

import int8_w8a8_scaled_gb300 as w8
from oracle import fp8_paged as fp
from test_gpu_fp8_paged import E4M3, Step, codes, dev, head_rows, host, random_columns, selection_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,start,tokens", [
    ([500, 300, 0, 0], [0, 1, 2, 0, 0], 2),                  # a batch padded by zeros
    ([500, 300, 77, 900], [0, 3, 3, 5, 0], 6),               # the last start below the others, a row of nobody
    ([500, 300, 400], [4, 6, 0, 4], 6),                      # the first request's rows behind the last one's
    ([90, 300, 400, 200], [-3, 1, 1 << 30, 1 << 30, 3], 4), # clamped starts: 1, 3, 0 and 0 rows
])
def test_starts_that_do_not_rise(lens, start, tokens):
    s = Step(90, lens, [tokens] + [0] * (len(lens) - 1), 8, 2, 128, 16, extra_rows=1)
    s.start, s.tokens, s.most = np.int32(start), tokens, 4
    s.q = s.q[:tokens]
    owners = [t for _, t, _ in fp.requests(s.lens, s.start, tokens, s.most, s.table.shape[1] * s.bs)]
    assert len(owners) == len(set(owners))                   # no row of two requests
    s.check(s.run())
    sel = random_columns(s, 9, s.rng)
    s.check(s.run(selected=sel), selected=sel)
    means, scales = s.rng.integers(-127, 128, (s.nb, 2, 128)).astype(np.int8), (s.rng.random((s.nb, 2)) + 0.1).astype(np.float32)
    before = np.full((tokens, 2, 5), -9, np.int32)
    want = fp.select(s.q.float().numpy(), means, scales, s.lens, s.table, 16, s.start, s.most, 1, 2, 5, before)
    assert np.array_equal(selection_of(s, means, scales, 5, 1, 2), want)
    s.check(s.run(selected=want), selected=want)


@pytest.mark.parametrize("lens,new,most,bs", [
    ([40], [40], 1, 16), ([700, 64, 63], [200, 64, 1], 3, 64), ([33, 300], [33, 290], 16, 16), ([20], [50], 2, 16),
])
def test_block_means_of_more_tokens_than_are_looked_at(lens, new, most, bs):
    """Every block that got new tokens has new means, whatever max_query_len is."""
    s = Step(91, lens, new, 2, 2, 64, bs, tail=0x7F)
    means, scales = s.rng.integers(-127, 128, (s.nb, 2, 64)).astype(np.int8), s.rng.random((s.nb, 2)).astype(np.float32)
    gm, gs = dev(means), dev(scales)
    w8.fp8_kv_block_means(dev(s.kc).view(E4M3), dev(s.lens), dev(s.table), gm, gs, query_start=dev(s.start), max_query_len=most)
    wm, ws = fp.block_means(s.kc, s.lens, s.table, s.start, max(new), means, scales)
    assert np.array_equal(gm.cpu().numpy(), wm) and np.array_equal(gs.cpu().numpy(), ws)


@pytest.mark.parametrize("most", [64, (1 << 31) - 1])
def test_block_means_of_many_heads_with_a_generous_limit(most):
    """max_query_len may be any number above the new tokens."""
    s = Step(92, [100, 33], [5, 1], 32, 32, 64, 16)
    means, scales = torch.zeros(s.nb, 32, 64, dtype=torch.int8, device="cuda"), torch.zeros(s.nb, 32, device="cuda")
    w8.fp8_kv_block_means(dev(s.kc).view(E4M3), dev(s.lens), dev(s.table), means, scales, query_start=dev(s.start), max_query_len=most)
    zero = np.zeros((s.nb, 32, 64), np.int8), np.zeros((s.nb, 32), np.float32)
    wm, ws = fp.block_means(s.kc, s.lens, s.table, s.start, 5, *zero)
    assert np.array_equal(means.cpu().numpy(), wm) and np.array_equal(scales.cpu().numpy(), ws)


@pytest.mark.parametrize("layout", ["halves", "heads", "dims", "heads_first"])
@pytest.mark.parametrize("new", [[3, 2], [70, 1]])
def test_queries_and_outputs_side_by_side(layout, new):
    """q and out are slices of one buffer that share none of its elements."""
    s = Step(93, [300, 200], new, 8, 2, 64, 16)
    T, H, D = s.q.shape
    if layout == "halves":
        buf = torch.full((T, 2 * H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        q, out = buf[:, :H], buf[:, H:]
    elif layout == "heads":
        buf = torch.full((T, 2 * H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        q, out = buf[:, ::2], buf[:, 1::2]
    elif layout == "dims":
        buf = torch.full((T, H, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
        q, out = buf[:, :, :D], buf[:, :, D:]
    else:
        buf = torch.full((H, T, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
        q, out = buf[:, :, D:], buf[:, :, :D]
    q.copy_(s.q)
    w8.fp8_kv_attention(q, dev(s.kc).view(E4M3), dev(s.vc).view(E4M3), dev(s.lens), dev(s.table), dev(np.float32([s.kg])),
                        dev(np.float32([s.vg])), out, query_start=dev(s.start), max_query_len=s.most, sm_scale=s.sm)
    s.check(out)
    assert torch.equal(q.cpu(), s.q)


def test_rotated_queries_beside_the_projection():
    """q_out is a slice of the buffer that q, k and v are slices of."""
    rng = np.random.default_rng(94)
    x = head_rows(rng, (19, 12, 64), "bf16")
    buf = torch.full((19, 20, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    buf[:, :12] = x.cuda()
    angle = rng.uniform(-3, 3, (50, 32))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    pos, slots = rng.integers(0, 50, 19).astype(np.int32), rng.permutation(32)[:19].astype(np.int64)
    caches = [torch.zeros(2, 16, 2, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
    one = torch.ones(1, device="cuda")
    w8.fp8_kv_rotate_write(buf[:, :8], buf[:, 8:10], buf[:, 10:12], dev(table), dev(pos), *caches, dev(slots), one, one, buf[:, 12:])
    x = x.float().numpy()
    assert np.array_equal(host(buf[:, 12:]), host(torch.from_numpy(fp.rotate(x[:, :8], pos, table)).bfloat16()))
    assert np.array_equal(host(buf[:, :12]), x)
    zero = np.zeros((2, 16, 2, 64), np.uint8)
    assert np.array_equal(codes(caches[0]), fp.write(zero, slots, fp.rotate(x[:, 8:10], pos, table), 1.0))
    assert np.array_equal(codes(caches[1]), fp.write(zero, slots, x[:, 10:], 1.0))


def test_select_blocks_for_the_last_of_two_billion_rows():
    """Rows of q up to the largest number of them: a pass over the scores may not count past 2^31."""
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("a selection of 17 GB")
    tokens = (1 << 31) - 1
    q = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda").expand(tokens, 1, 64)
    means = torch.zeros(3, 1, 64, dtype=torch.int8, device="cuda")
    means[:, 0, 0] = torch.tensor([-3, 5, 1], dtype=torch.int8, device="cuda")
    selected = torch.full((tokens, 1, 2), -9, dtype=torch.int32, device="cuda")
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.zeros(w8.fp8_kv_select_blocks_workspace_size(tokens, 1, 3), dtype=torch.uint8, device="cuda")
    w8.fp8_kv_select_blocks(q, means, torch.ones(3, 1, device="cuda"), ints(48), ints(0, 1, 2).view(1, 3), 16, selected,
                            query_start=ints(tokens - 1, tokens), first_blocks=0, last_blocks=1, workspace=ws)
    assert selected[-1, 0].tolist() == [1, 2]
    assert (selected[:-1] == -9).all()


@pytest.mark.parametrize("lens,new,hq,h", [([60, 300], [6, 3], 8, 2), ([300, 260], [70, 200], 8, 2), ([26, 100], [1, 1], 48, 1), ([500], [300], 2, 1)])
@pytest.mark.parametrize("scale", [None, "k", "sm"])
def test_nan_scores_of_rows_that_see_no_token(lens, new, hq, h, scale):
    """Zeros, whether the tokens lie in blocks outside the cache or behind the row; NaN where one is seen."""
    s = Step(99, lens, new, hq, h, 64, 16, tail=0x7F)
    s.table[0, :(lens[0] - new[0] // 2) // 16] = -1          # the first request's first rows see nothing, or none of its rows
    if len(lens) > 1:
        s.table[1, ::2] = s.nb
    s.q[::3, 0, 3], s.q[1::5, hq - 1, 7] = float("nan"), float("inf")
    if scale == "k":
        s.kg = float("nan")
    elif scale == "sm":
        s.sm = float("nan")
    out = s.run()
    s.check(out)
    if len(lens) > 1:                                        # all of its tokens gone
        s.table[1] = -1
        out = s.run()
        s.check(out)
        assert not out[int(s.start[1]):].any()
    sel = random_columns(s, 9, s.rng)
    s.check(s.run(selected=sel), selected=sel)


# ------------------------------------------------------------------ lengths that they are for


@pytest.mark.parametrize("lens,new,hq,h,bs,budget,first,last", [
    ([60000, 33000], [40, 3], 4, 2, 16, 200, 1, 2),          # 3750 and 2063 columns: the wide kernel
    ([50000], [2100], 2, 1, 16, 64, 2, 3),                   # a prompt chunk of thousands, in several passes and slabs
    ([40000, 39000, 38000], [1, 1, 1], 16, 2, 16, 2400, 0, 1),
    ([34000, 100], [1200, 1], 8, 1, 32, 30, 1, 2),           # 1063 columns: the narrow kernel
])
def test_select_blocks_of_long_contexts(lens, new, hq, h, bs, budget, first, last):
    s = Step(95, lens, new, hq, h, 64, bs)
    means, scales = s.rng.integers(-127, 128, (s.nb, h, 64)).astype(np.int8), (s.rng.random((s.nb, h)) + 0.1).astype(np.float32)
    before = np.full((s.q.shape[0], h, budget), -9, np.int32)
    want = fp.select(s.q.float().numpy(), means, scales, s.lens, s.table, bs, s.start, s.most, first, last, budget, before)
    assert np.array_equal(selection_of(s, means, scales, budget, first, last), want)


def test_select_blocks_of_long_contexts_with_ties():
    s = Step(96, [60000], [70], 2, 1, 64, 16)
    means, scales = s.rng.integers(-1, 2, (s.nb, 1, 64)).astype(np.int8), np.ones((s.nb, 1), np.float32)
    s.q = torch.from_numpy(s.rng.integers(-1, 2, s.q.shape).astype(np.float32)).bfloat16()
    s.q[0] = 0
    s.table[0, 2000:2100] = -1
    before = np.full((70, 1, 3000), -9, np.int32)
    want = fp.select(s.q.float().numpy(), means, scales, s.lens, s.table, 16, s.start, 70, 1, 2, 3000, before)
    assert np.array_equal(selection_of(s, means, scales, 3000, 1, 2), want)


@pytest.mark.parametrize("lens,new,hq,h,d,bs", [
    ([70000, 50], [1, 1], 4, 1, 64, 16), ([40000], [5], 8, 2, 128, 64), ([50000, 20000], [40, 1], 2, 1, 128, 32), ([30000], [50], 4, 2, 64, 16),
])
def test_attention_of_long_contexts(lens, new, hq, h, d, bs):
    s = Step(97, lens, new, hq, h, d, bs, tail=0x7F)
    s.check(s.run())
    sel = random_columns(s, 100, s.rng)
    s.check(s.run(selected=sel), selected=sel)


def test_steps_of_a_long_context():
    """Means of a whole prompt of tens of thousands of tokens, then selection and sparse attention by them."""
    s = Step(98, [45000, 20010], [2, 1], 8, 2, 64, 32, tail=0x7F)
    gm, gs = torch.zeros(s.nb, 2, 64, dtype=torch.int8, device="cuda"), torch.zeros(s.nb, 2, device="cuda")
    w8.fp8_kv_block_means(dev(s.kc).view(E4M3), dev(s.lens), dev(s.table), gm, gs, query_start=dev(np.int32([0, 45000, 65010])),
                          max_query_len=45000)
    zero = np.zeros((s.nb, 2, 64), np.int8), np.zeros((s.nb, 2), np.float32)
    wm, ws = fp.block_means(s.kc, s.lens, s.table, np.int32([0, 45000, 65010]), 45000, *zero)
    assert np.array_equal(gm.cpu().numpy(), wm) and np.array_equal(gs.cpu().numpy(), ws)
    before = np.full((3, 2, 64), -9, np.int32)
    want = fp.select(s.q.float().numpy(), wm, ws, s.lens, s.table, 32, s.start, 2, 1, 2, 64, before)
    got = selection_of(s, wm, ws, 64, 1, 2)
    assert np.array_equal(got, want)
    s.check(s.run(selected=got), selected=got)
