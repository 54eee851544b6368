"""Attention over the 4-bit cache where a CTA or warp goes through many units
and tiles one after the other, against 64 bits on the GPU.

Tolerance, per output element, with r the weights' mean of |V|:
  * the output's rounding, half a step: 2^-8 |ref| (bf16), 2^-11 |ref| (fp16),
    or half the smallest subnormal number below the normal ones;
  * softmax weights of 11 bits (f16) in the numerator and in the sum: 2^-10 r;
    below 2^-27 of the largest they are f16 subnormals, off by up to 2^-38 of
    the largest: 2^-38 sum |V|;
  * fp32 scores: (2 (d + 8) 2^-24 B + 2^-18) r with B = max_t sum_d |q_d K_td|
    |sm_scale|: products, sums and the scaling are each off by 2^-24 of at most
    B, and twice that relative to the maximum; exp2's approximation and the
    32-bit sums stay below 2^-18;
  * raising the maximum rescales the sums and outputs, 2^-23 each time: at most
    one raise a tile, 2^-23 r a tile."""
import numpy as np
import pytest
import torch

import int8_w8a8_scaled_gb300 as w8

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def decoded(records, at, kind):
    """[tokens, d] in 64 bits of K (at 0) or V (at 9 d) of records [n, 18 d]."""
    d = records.shape[1] // 18
    both = records[:, at:at + 8 * d].reshape(-1, d // 2).long()
    code = torch.stack((both & 15, both >> 4), 2).flatten(1)
    if kind == "int4":
        x = torch.where(code >= 8, code - 16, code).double()
    else:
        x = torch.where(code >= 8, -1.0, 1.0).double() * torch.tensor(E2M1, dtype=torch.float64, device="cuda")[code % 8]
    s = records[:, at + 8 * d:at + 9 * d].reshape(-1, d // 16).contiguous().view(torch.float8_e4m3fn).double()
    return x * s.repeat_interleave(16, 1)


def reference(q, cache, lens, news, table, kg, vg, sm, kind):
    """(out, r, B, sum |V|) in 64 bits of every row of q, NaN for a row that sees
    a score of NaN or +infinity."""
    h, d, bs = cache.shape[1], q.shape[2], 16 * cache.shape[2]
    share, first = q.shape[1] // h, 0
    out, r, total = (torch.zeros(q.shape, dtype=torch.float64, device="cuda") for _ in range(3))
    big = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    for b, (length, n) in enumerate(zip(lens, news)):
        blocks = dev(table[b, :-(-length // bs)].astype(np.int64))
        limit = length - n + torch.arange(n, device="cuda")
        seen = (torch.arange(length, device="cuda")[None] <= limit[:, None])[None]
        for j in range(h if n and length else 0):
            records = cache[blocks, j].flatten(0, 1)
            k, v = decoded(records, 0, kind)[:length] * kg, decoded(records, 9 * d, kind)[:length] * vg
            x = q[first:first + n, j * share:(j + 1) * share].double().transpose(0, 1)      # [share, n, d]
            s = (x @ k.T * sm).masked_fill(~seen, -np.inf)
            lost = (s.isnan() | (s == np.inf)).any(2, keepdim=True)
            w = torch.nan_to_num(torch.softmax(s, 2))                                       # rows that see nothing: zeros
            at = slice(j * share, (j + 1) * share)
            out[first:first + n, at] = (w @ v).masked_fill(lost, np.nan).transpose(0, 1)
            r[first:first + n, at] = (w @ v.abs()).transpose(0, 1)
            total[first:first + n, at] = (seen.double() @ v.abs()).transpose(0, 1).expand(n, share, d)
            big[first:first + n, at] = ((x.abs() @ k.abs().T) * abs(sm)).masked_fill(~seen, 0.0).amax(2).T
        first += n
    return out, r, big, total


def close(got, want, lens):
    ref, r, big, total = want
    d, half = got.shape[2], HALF_STEP[got.dtype]
    tiles = -(-int(max(lens)) // 16)
    tol = (half * ref.abs() + r * (2.0 ** -10 + 2.0 ** -18 + tiles * 2.0 ** -23 + 2 * (d + 8) * 2.0 ** -24 * big[..., None]) +
           2.0 ** -38 * total + torch.finfo(got.dtype).smallest_normal * half)
    lost = ref.isnan()
    assert torch.equal(got.isnan(), lost) and torch.isfinite(got[~lost]).all()
    over = torch.where(lost, 0.0, (got.double() - ref).abs() - tol)
    assert (over <= 0).all(), f"{int((over > 0).sum())} of {over.numel()} outside"


def serve(lens, news, hq, hkv, d, kind, dtype, bs=32, seed=0, rise=None, loud=None, spoil=None, only=slice(None), sm=None):
    """One call over requests of these lengths, compared with 64 bits.

    rise: requests (a slice) whose keys point along their queries, further the
    later the token, so that the maximum goes up to the end.  loud: the queries'
    scale for each packed token and head.  spoil: changes the query in place.  only: the heads compared."""
    lens, news = np.asarray(lens), np.asarray(news)
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    blocks = -(-lens // bs)
    nb = int(blocks.sum()) + 2
    table = np.full((len(lens), int(blocks.max())), -1, np.int32)
    table[np.arange(table.shape[1])[None] < blocks[:, None]] = rng.permutation(nb)[:blocks.sum()]
    k, v = (torch.randn(nb * bs, hkv, d, generator=gen, device="cuda") for _ in range(2))
    q = torch.randn(int(news.sum()), hq, d, generator=gen, device="cuda")
    if rise is not None:
        start = np.concatenate([[0], np.cumsum(news)])
        for b in range(len(lens))[rise]:
            q[start[b]:start[b + 1]] += 1.0
            for i, block in enumerate(table[b, :blocks[b]].tolist()):
                k[block * bs:(block + 1) * bs] += 0.5 * i / blocks[b]
    if loud is not None:
        q *= loud
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    if spoil is not None:
        spoil(q)
    kg, vg = 0.0151, 0.0173
    cache = torch.zeros(w8.kv4_cache_shape(nb, hkv, bs, d), dtype=torch.uint8, device="cuda")
    scales = dev(np.float32([kg])), dev(np.float32([vg]))
    w8.kv4_cache_write(k, v, cache, torch.arange(nb * bs, device="cuda"), *scales, kind=kind)
    out = torch.full_like(q, float("nan"))
    start = dev(np.concatenate([[0], np.cumsum(news)]).astype(np.int32))
    sm = 1.0 / d ** 0.5 if sm is None else sm
    w8.kv4_attention(q, cache, dev(lens.astype(np.int32)), dev(table), *scales, out, query_start=start,
                     max_query_len=int(news.max()), kind=kind, sm_scale=sm)
    assert w8.device_status() == 0
    want = reference(q, cache, lens, news, table, float(np.float32(kg)), float(np.float32(vg)), sm, kind)
    close(out[:, only], [x[:, only] for x in want], lens)
    return out


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("kind", ["e2m1", "int4"])
@pytest.mark.parametrize("d", [64, 128])
def test_units_of_one_tile_whose_queries_differ_in_size(d, kind):
    """Fresh chunks of up to 128 tokens: a CTA goes through several units of one
    tile each, and the queries' scales differ by powers of two between them."""
    rng = np.random.default_rng(d)
    news = rng.integers(65, 129, 120)
    assert 8 * len(news) >= 5 * sms()
    loud = 2.0 ** rng.integers(-6, 7, (len(news), 8)).repeat(2, 1).repeat(news, 0)
    for seed in range(3):
        serve(news, news, 16, 8, d, kind, torch.bfloat16, seed=seed, loud=dev(loud[..., None]).float())


@pytest.mark.parametrize("kind", ["e2m1", "int4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,hq", [(1, 4), (3, 4), (5, 8), (40, 4), (40, 16), (300, 8)])
def test_a_query_with_nan_or_infinity_is_seen_in_its_own_row(new, hq, d, kind):
    """NaN for that token and head, whichever kernel the number of rows picks, and
    nothing of it in the others; nothing at all where a row sees no token."""
    lens, news = [700, 2600, max(0, new - 1)], [new] * 3

    def spoil(q):
        q[0, 1, 5] = float("nan")
        q[new + new // 2, 0, d - 1] = float("inf")
        q[2 * new - 1, 2, 17] = -float("inf")
        q[2 * new, 3] = float("nan")                       # the first row of the last request sees nothing
    out = serve(lens, news, hq, 2, d, kind, torch.bfloat16, spoil=spoil)
    assert out[0, 1].isnan().all() and not out[2 * new].any()
    assert int(out.isnan().any(2).sum()) == 3


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("which", ["k_scale", "v_scale", "sm_scale"])
def test_a_scale_of_nan_gives_nan(which, new):
    """And not the mean of the values; rows that see nothing are zeros."""
    cache = torch.zeros(w8.kv4_cache_shape(9, 2, 16, 64), dtype=torch.uint8, device="cuda")
    one, gone = torch.ones(1, device="cuda"), torch.full((1,), float("nan"), device="cuda")
    q = torch.ones(2 * new, 8, 64, dtype=torch.bfloat16, device="cuda")
    out, table = torch.empty_like(q), torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    w8.kv4_attention(q, cache, dev(np.int32([60, 0])), table, gone if which == "k_scale" else one, gone if which == "v_scale" else one, out,
                     query_start=dev(np.int32([0, new, 2 * new])), max_query_len=new,
                     sm_scale=float("nan") if which == "sm_scale" else 0.125)
    assert out[:new].isnan().all() and not out[new:].any()


@pytest.mark.parametrize("size", [2.0 ** 70, 2.0 ** -70, float("inf")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,hq", [(1, 8), (3, 8), (5, 8), (40, 8)])
def test_a_head_of_another_size_leaves_the_others_alone(new, hq, d, size):
    """Each row has a scale of its own: one head far above or below the others of
    its KV head takes no bits of theirs."""
    def spoil(q):
        q[:, ::4] *= size
    serve([900, 2600], [new] * 2, hq, 2, d, "e2m1", torch.bfloat16, spoil=spoil, only=[1, 2, 3, 5, 6, 7])


@pytest.mark.parametrize("new", [1, 5, 40])
def test_a_query_far_below_the_normal_numbers(new):
    """Among heads of ordinary size, one whose scores come out ordinary by the scale alone."""
    def spoil(q):
        q[:, 1] *= 2.0 ** -70
    serve([900, 2600], [new] * 2, 4, 1, 64, "e2m1", torch.bfloat16, spoil=spoil, only=[1], sm=2.0 ** 67)


@pytest.mark.parametrize("power", [10, 17, 26, 28, 40, 70])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,hq", [(1, 4), (5, 4), (40, 8)])
def test_scores_of_any_size(new, hq, d, power):
    """A query along one token's key, larger by powers of two: that token's value
    alone, however far its score (2^26 and more) is above the others."""
    gen = torch.Generator(device="cuda").manual_seed(power)
    length, hkv = 1500, 2
    nb = -(-length // 16)
    k, v = (torch.randn(nb * 16, hkv, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    cache = torch.zeros(w8.kv4_cache_shape(nb, hkv, 16, d), dtype=torch.uint8, device="cuda")
    one = torch.full((1,), 0.0137, device="cuda")
    w8.kv4_cache_write(k, v, cache, torch.arange(nb * 16, device="cuda"), one, one)
    token = torch.randint(0, length - new, (new, hq), generator=gen, device="cuda")
    head = torch.arange(hq, device="cuda") // (hq // hkv)
    q = (k[token, head].float() * 2.0 ** power).bfloat16()
    out = torch.empty_like(q)
    table = torch.arange(nb, dtype=torch.int32, device="cuda")[None]
    w8.kv4_attention(q, cache, dev(np.int32([length])), table, one, one, out, query_start=dev(np.int32([0, new])), max_query_len=new)
    want = torch.stack([decoded(cache[:, j].flatten(0, 1), 9 * d, "e2m1") for j in range(hkv)], 1)[token, head] * 0.0137
    # the output's half step, and one weight of 11 bits
    assert ((out.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -11)).all()


@pytest.mark.parametrize("new", [1, 7, 300])
def test_a_max_query_len_that_means_no_limit(new):
    """The largest number that the sizes allow, for one head and one request."""
    rng = np.random.default_rng(new)
    nb = 40
    cache = torch.zeros(w8.kv4_cache_shape(nb, 1, 16, 64), dtype=torch.uint8, device="cuda")
    k, v = (torch.from_numpy(rng.standard_normal((nb * 16, 1, 64)).astype(np.float32)).cuda().bfloat16() for _ in range(2))
    one = torch.full((1,), 0.0137, device="cuda")
    w8.kv4_cache_write(k, v, cache, torch.arange(nb * 16, device="cuda"), one, one)
    q = torch.from_numpy(rng.standard_normal((new, 1, 64)).astype(np.float32)).cuda().bfloat16()
    table = torch.arange(nb, dtype=torch.int32, device="cuda")[None]
    for most in (2 ** 31 - 1, 1 << 20, new):
        out = torch.full_like(q, float("nan"))
        w8.kv4_attention(q, cache, dev(np.int32([600])), table, one, one, out, query_start=dev(np.int32([0, new])), max_query_len=most)
        close(out, reference(q, cache, [600], [new], np.arange(nb, dtype=np.int32)[None], 0.013700000010430813, 0.013700000010430813,
                             0.125, "e2m1"), [600])


def few_rows_run(lens, news, hq, hkv):
    """Steps of 32 tokens that each warp of the few-rows kernel goes through."""
    rows = int(news.max()) * hq // hkv
    groups = 1 + (news * (hq // hkv) > 16) if rows > 8 else np.ones_like(news)
    steps = (np.maximum(1, -(-lens // 32)) * (news > 0) * groups).sum() * hkv
    return steps / (sms() * 8 * (2 if rows <= 8 else 1))


def many_rows_run(lens, news, hq, hkv):
    """Tiles of 128 tokens that each CTA of the many-rows kernel goes through."""
    share, tiles = hq // hkv, 0
    for length, n in zip(lens, news):
        for row in range(0, n * share, 256):
            last = min(n * share, row + 256) - 1
            tiles += max(1, -(-min(length, max(0, length - n + last // share + 1)) // 128))
    return tiles * hkv / sms()


EVERY_OTHER = slice(0, None, 2)


@pytest.mark.parametrize("kind", ["e2m1", "int4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,hq", [(1, 32), (1, 64), (2, 32), (3, 32), (5, 32)])
def test_few_rows_long_runs(new, hq, d, kind):
    """Ragged requests up to 8000 tokens: a warp's run is longer than the batch of
    16 steps whose places it looks up at once, through several units, with
    maxima that go up to the end in every other request.  4, 8 and 16 rows, and
    20 in two groups."""
    rng = np.random.default_rng(new + d)
    lens = rng.integers(500, 8001, 64)
    news = np.full(64, new) if new == 1 else rng.integers(1, new + 1, 64)
    news[0] = new
    assert few_rows_run(lens, news, hq, 8) > 20
    serve(lens, news, hq, 8, d, kind, torch.bfloat16 if kind == "e2m1" else torch.float16, rise=EVERY_OTHER)


@pytest.mark.parametrize("new,hq", [(1, 32), (3, 32), (5, 32)])
def test_few_rows_many_units_to_a_run(new, hq):
    """Short requests, empty ones and ones without new tokens among them."""
    rng = np.random.default_rng(new)
    lens, news = rng.integers(0, 300, 900), rng.integers(0 if new > 1 else 1, new + 1, 900)
    lens[::7] = 0
    assert few_rows_run(lens, news, hq, 8) > 12
    serve(lens, news, hq, 8, 64, "e2m1", torch.bfloat16, rise=EVERY_OTHER)


@pytest.mark.parametrize("kind", ["e2m1", "int4"])
@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_long_runs(d, kind):
    """Chunks of prompts: dozens of tiles to a CTA, pairs of row slots."""
    lens, news = np.array([2500, 2300]), np.array([1500, 1333])
    assert many_rows_run(lens, news, 32, 8) > 30
    serve(lens, news, 32, 8, d, kind, torch.bfloat16 if kind == "e2m1" else torch.float16, rise=slice(0, 1))


@pytest.mark.parametrize("kind", ["e2m1", "int4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seed", [1, 2])
def test_many_rows_units_of_all_forms_in_a_run(d, kind, seed):
    """Units of up to 128 rows (both slots take the same ones, the tiles in turn)
    and of more (a slot each), of one tile, of two and of many, whole and cut."""
    rng = np.random.default_rng(seed)
    news = rng.choice([0, 1, 9, 20, 32, 33, 40, 64, 65, 100, 200], 90)
    news[:2] = 200, 1
    lens = news + rng.choice([-1, 0, 0, 30, 128, 250, 1000, 6000], 90) * (news > 0)
    lens = np.maximum(lens, 0)
    assert many_rows_run(lens, news, 32, 8) > 30
    serve(lens, news, 32, 8, d, kind, torch.bfloat16, seed=seed, rise=EVERY_OTHER)
