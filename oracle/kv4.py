"""CPU oracle of the serving step over a 4-bit paged KV cache.

TEST INFRASTRUCTURE ONLY (like the rest of ``oracle/``).

What it computes, straight from the definitions of ``include/w8a8.h``:
  * codes and scales of a group of 16 dims: s = e4m3(clamp(absmax / (M g),
    2^-9, 448)), code = round(x / (s g)), half to even, the products and
    quotients rounded to fp32 (numpy's fp32 operations are IEEE's); values
    code * s * g in 64 bits;
  * the cache's layout, records of 16 tokens;
  * attention with causal rows, in 64 bits;
  * block tables, slots and positions, request by request;
  * verification of drafted tokens, in 64 bits.

Pinned by ``tests/test_oracle_kv4.py``.
"""
from __future__ import annotations

import numpy as np

from . import e4m3_value

LARGEST = {"e2m1": np.float32(6.0), "int4": np.float32(7.0)}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([e4m3_value(c) for c in range(127)], dtype=np.float64)  # non-negative, increasing
E4M3_BYTE = np.array([e4m3_value(c) for c in range(256)], dtype=np.float64)
GROUP, TILE = 16, 16


def nearest_even(x: np.ndarray, levels: np.ndarray) -> np.ndarray:
    """Index of the level nearest to each x (levels increasing, x within
    them), the even index of two equally near ones."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(levels, x), 1, len(levels) - 1)
    below, above = x - levels[hi - 1], levels[hi] - x
    down = (below < above) | ((below == above) & ((hi - 1) % 2 == 0))
    return np.where(down, hi - 1, hi)


def quantise(x: np.ndarray, g, kind: str):
    """(codes 0..15 [..., d], scale bytes [..., d / 16]) of fp32 x [..., d]."""
    x = np.asarray(x, dtype=np.float32)
    g = np.float32(g)
    y = x.reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        a = np.max(np.where(np.isnan(y), np.float32(0), np.abs(y)), axis=-1)
        s = nearest_even(np.clip(a / (LARGEST[kind] * g), np.float32(2.0 ** -9), np.float32(448)), E4M3).astype(np.uint8)
        y = y / (E4M3[s].astype(np.float32) * g)[..., None]
    y = np.where(np.isnan(y), np.float32(0), y)
    if kind == "int4":
        codes = np.clip(np.rint(y.astype(np.float64)), -7, 7).astype(np.int64) & 15
    else:
        codes = nearest_even(np.minimum(np.abs(y), 6.0), E2M1) + 8 * np.signbit(y)
    return codes.astype(np.uint8).reshape(x.shape), s


def values(codes: np.ndarray, scales: np.ndarray, g, kind: str) -> np.ndarray:
    """float64 code * s * g."""
    c = codes.astype(np.int64)
    base = np.where(c >= 8, c - 16, c).astype(np.float64) if kind == "int4" else np.where(c >= 8, -1.0, 1.0) * E2M1[c % 8]
    return base * np.repeat(E4M3_BYTE[scales], GROUP, axis=-1) * float(np.float32(g))


def parts(cache: np.ndarray):
    """Views of a cache [blocks, heads, records, 18 d]: K codes, K scales, V
    codes, V scales, each [blocks, heads, records, 16, bytes]."""
    d = cache.shape[-1] // 18
    cut = ((0, 8 * d), (8 * d, 9 * d), (9 * d, 17 * d), (17 * d, 18 * d))
    return [cache[..., i:j].reshape(*cache.shape[:3], TILE, -1) for i, j in cut]


def write(cache: np.ndarray, slots, k, v, kg, vg, kind: str) -> np.ndarray:
    """A copy of the cache with the tokens written at their slots."""
    out = cache.copy()
    nb, _, records, _ = cache.shape
    d, bs = cache.shape[-1] // 18, cache.shape[2] * TILE
    for t, slot in enumerate(np.asarray(slots).tolist()):
        if slot < 0 or slot >= nb * bs:
            continue
        rec = out[slot // bs, :, slot % bs // TILE]
        row = slot % TILE
        for x, g, at in ((k[t], kg, 0), (v[t], vg, 9 * d)):
            codes, scales = quantise(x, g, kind)
            rec[:, at + row * d // 2:at + (row + 1) * d // 2] = codes[:, ::2] | (codes[:, 1::2] << 4)
            rec[:, at + 8 * d + row * d // 16:at + 8 * d + (row + 1) * d // 16] = scales
    return out


def tokens_of(cache: np.ndarray, slots, kg, vg, kind: str):
    """(K, V) float64 [len(slots), heads, d] that the tokens stand for."""
    bs = cache.shape[2] * TILE
    slots = np.asarray(slots, dtype=np.int64)
    kc, ks, vc, vs = (p[slots // bs, :, slots % bs // TILE, slots % TILE] for p in parts(cache))
    both = lambda c: np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], -1)  # noqa: E731
    return values(both(kc), ks, kg, kind), values(both(vc), vs, vg, kind)


def attention(q, cache, seq_lens, block_table, query_start, kg, vg, sm_scale: float, kind: str):
    """(out, weighted |V|, largest sum of |q K| sm_scale) in float64 for q
    [tokens, Hq, d]; the latter two scale a test's tolerance."""
    q = np.asarray(q, dtype=np.float64)
    nb, h, records, _ = cache.shape
    bs, share = records * TILE, q.shape[1] // h
    out, r, big = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:2])
    for b in range(len(seq_lens)):
        first, n = int(query_start[b]), int(query_start[b + 1]) - int(query_start[b])
        length = min(max(int(seq_lens[b]), 0), block_table.shape[1] * bs)
        t = np.arange(length)
        blk = block_table[b, t // bs].astype(np.int64)
        keep = (blk >= 0) & (blk < nb)
        t, blk = t[keep], blk[keep]
        if n <= 0 or len(t) == 0:
            continue
        k, v = tokens_of(cache, blk * bs + t % bs, kg, vg, kind)
        for i in range(n):
            seen = t <= length - n + i
            if not seen.any():
                continue
            for j in range(q.shape[1]):
                kk, vv, qq = k[seen, j // share], v[seen, j // share], q[first + i, j]
                s = kk @ qq * sm_scale
                w = np.exp(s - s.max())
                w /= w.sum()
                out[first + i, j], r[first + i, j] = w @ vv, w @ np.abs(vv)
                big[first + i, j] = (np.abs(kk) @ np.abs(qq)).max() * abs(sm_scale)
    return out, r, big


def block_tables(context_lens, new_lens, free_blocks, free_count: int, table, block_size: int, tokens: int):
    """(table, query_start, seq_lens, slots, positions, free_left,
    free_count_out)."""
    table, free_blocks = np.array(table), list(free_blocks)
    count = min(max(int(free_count), 0), len(free_blocks))
    slots, positions = np.full(tokens, -1, np.int64), np.zeros(tokens, np.int32)
    start, lens, before, left, after = 0, [], 0, count, count
    starts = [0]
    for b in range(len(context_lens)):
        ctx, new = max(0, int(context_lens[b])), max(0, int(new_lens[b]))
        first, last = -(-ctx // block_size), -(-(ctx + new) // block_size)
        fits = ctx + new <= table.shape[1] * block_size
        need = last - first if fits else 0
        ok = fits and (new == 0 or start + new <= tokens) and (need == 0 or before + need <= count)
        for i in range(need if ok else 0):
            table[b, first + i] = free_blocks[count - 1 - before - i]
        if ok:
            left = min(left, count - before - need)
        if ok and need:
            after = count - before - need
        for i in range(new):
            if start + i >= tokens:
                break
            pos = ctx + i
            positions[start + i] = pos
            if ok and table[b, pos // block_size] >= 0:
                slots[start + i] = int(table[b, pos // block_size]) * block_size + pos % block_size
        before += need
        start += new
        starts.append(start)
        lens.append(ctx + new if ok else 0)
    return table, np.array(starts, np.int32), np.array(lens, np.int32), slots, positions, left, after


def verify(target, draft, tokens, start, uniform, sample, max_drafts: int):
    """(out_tokens, num_accepted); target and draft as float arrays."""
    clean = lambda x: np.where(x > 0, x, 0).astype(np.float64)  # noqa: E731
    batch, vocab = len(start) - 1, target.shape[1]
    out = np.full((batch, max_drafts + 1), -1, np.int32)
    accepted = np.zeros(batch, np.int32)
    for b in range(batch):
        first, n = int(start[b]), min(int(start[b + 1]) - int(start[b]), max_drafts)
        i = 0
        while i < n:
            x = int(tokens[first + i])
            if not 0 <= x < vocab:
                break
            p = float(clean(target[first + b + i, x]))
            q = float(clean(draft[first + i, x])) if draft is not None else 1.0
            if not float(np.float32(uniform[first + i])) * q < p:
                break
            out[b, i] = x
            i += 1
        accepted[b] = i
        p = clean(target[first + b + i])
        w = p
        if i < n and draft is not None:
            w = np.maximum(p - clean(draft[first + i]), 0.0)
        elif i < n and 0 <= int(tokens[first + i]) < vocab:
            w = p.copy()
            w[int(tokens[first + i])] = 0.0
        if not w.sum() > 0:
            w = p
        c = np.cumsum(w)
        if c[-1] > 0:
            above = np.nonzero((c > float(np.float32(sample[b])) * c[-1]) & (w > 0))[0]
            out[b, i] = above[0] if len(above) else np.nonzero(w > 0)[0][-1]
    return out, accepted
