"""CPU oracle of the operators of long contexts over the paged fp8 cache.

TEST INFRASTRUCTURE ONLY (like the rest of ``oracle/``).

What it computes, straight from the definitions of ``include/w8a8.h``:
  * rotation by positions, products and sums rounded to fp32 (numpy's fp32
    operations are IEEE's), and e4m3 codes of the fp32 quotients;
  * attention with causal rows, over the whole cache or over selected columns,
    in 64 bits, with the sizes that its tolerance is made of;
  * 8-bit means of blocks, scores and selections.

Pinned by ``tests/test_oracle_fp8_paged.py``.
"""
from __future__ import annotations

import numpy as np

from . import e4m3_value
from .kv4 import nearest_even

LEVELS = np.array([e4m3_value(c) for c in range(127)], dtype=np.float64)   # non-negative, increasing
VALUES = np.array([e4m3_value(c) for c in range(256)], dtype=np.float64)   # NaN for 0x7F / 0xFF


def encode(x: np.ndarray) -> np.ndarray:
    """e4m3 codes of fp32 x: nearest, ties to the even code, saturating, NaN 0x7F."""
    x = np.asarray(x, dtype=np.float32)
    a = np.minimum(np.abs(np.where(np.isnan(x), np.float32(0), x)).astype(np.float64), 448.0)
    code = nearest_even(a, LEVELS).astype(np.uint8) | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), np.uint8(0x7F), code).astype(np.uint8)


def rotate(x, positions, cos_sin, sections=None, interleaved=False) -> np.ndarray:
    """fp32 [tokens, heads, d] of fp32 x, each pair turned by its angle."""
    x = np.asarray(x, dtype=np.float32)
    n, pairs = x.shape[0], cos_sin.shape[1] // 2
    pos = np.asarray(positions).reshape(-1, n)
    axis = np.repeat(np.arange(len(pos)), [pairs] if sections is None else sections)
    y = x.copy()
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        p = pos[axis[i]]
        inside = (p >= 0) & (p < cos_sin.shape[0])
        at = np.where(inside, p, 0)
        c = np.where(inside, cos_sin[at, i], np.float32("nan")).astype(np.float32)[:, None]
        s = np.where(inside, cos_sin[at, pairs + i], np.float32("nan")).astype(np.float32)[:, None]
        with np.errstate(all="ignore"):
            y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
            y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y


def write(cache, slots, x, scale) -> np.ndarray:
    """A copy of the codes [blocks, block_size, heads, d] with the tokens' x / scale at their slots."""
    out = cache.copy()
    flat = out.reshape(-1, *cache.shape[2:])
    with np.errstate(all="ignore"):
        codes = encode(np.asarray(x, np.float32) / np.float32(scale))
    for t, slot in enumerate(np.asarray(slots).tolist()):
        if 0 <= slot < len(flat):
            flat[slot] = codes[t]
    return out


def requests(seq_lens, query_start, tokens, most, room):
    """(request, row of q, position) of each row that is looked at."""
    lens = np.clip(np.asarray(seq_lens, np.int64), 0, room)
    start = np.arange(len(lens) + 1) if query_start is None else np.asarray(query_start, np.int64)
    for b in range(len(lens)):
        first = min(max(int(start[b]), 0), tokens)
        n = max(min(int(start[b + 1]), tokens) - first, 0) if query_start is not None else 1
        for i in range(min(n, most)):
            yield b, first + i, int(lens[b]) - n + i


def attention(q, k_codes, v_codes, k_scale, v_scale, seq_lens, table, query_start, most, sm_scale, selected=None):
    """(out, written, r, reach, far): outputs of the rows that are looked at, and for each row and head the softmax
    weights' mean of |V| per dim, the largest sum of |q K| sm_scale over the tokens seen, and the same sum with the
    row's largest |q| in the place of every element."""
    tokens, hq, d = q.shape
    nb, bs, h, _ = k_codes.shape
    out, r = np.zeros((2, tokens, hq, d))
    reach, far = np.zeros((2, tokens, hq))
    written = np.zeros(tokens, bool)
    for b, t, pos in requests(seq_lens, query_start, tokens, most, table.shape[1] * bs):
        written[t] = True
        for kv in range(h):
            if selected is None:
                at = np.arange(pos + 1)
            else:
                cols = [int(c) for c in selected[t, kv] if 0 <= c < table.shape[1]]
                at = np.concatenate([np.arange(c * bs, (c + 1) * bs) for c in cols] + [np.zeros(0, np.int64)]).astype(np.int64)
                at = at[at <= pos]
            block = table[b, at // bs].astype(np.int64)
            at, block = at[(block >= 0) & (block < nb)], block[(block >= 0) & (block < nb)]
            if len(at) == 0:
                continue
            K = VALUES[k_codes[block, at % bs, kv]] * float(np.float32(k_scale))
            V = VALUES[v_codes[block, at % bs, kv]] * float(np.float32(v_scale))
            for head in range(kv * (hq // h), (kv + 1) * (hq // h)):
                x = q[t, head].astype(np.float64)
                with np.errstate(all="ignore"):
                    s = (K @ x) * sm_scale if np.isfinite(x).all() else np.full(len(at), np.nan)
                    w = np.exp(s - s.max())
                    w = w / w.sum()
                    out[t, head], r[t, head] = w @ V, w @ np.abs(V)
                    reach[t, head] = (np.abs(K) @ np.abs(x)).max() * abs(sm_scale)
                    far[t, head] = np.abs(K).sum(1).max() * np.abs(x).max() * abs(sm_scale)
    return out, written, r, reach, far


def quantise8(x):
    """int8 codes and fp32 scale of the last dimension's fp32 rows."""
    x = np.asarray(x, np.float32)
    top = np.max(np.where(np.isnan(x), np.float32(0), np.abs(x)), axis=-1, keepdims=True)
    with np.errstate(all="ignore"):
        scale = np.where(top > 0, top * (np.float32(1) / np.float32(127)), np.float32(1)).astype(np.float32)
        y = x / scale
    y = np.where(np.isnan(y), np.float32(0), y).astype(np.float64)
    return np.clip(np.rint(y), -128, 127).astype(np.int8), scale[..., 0]


def block_means(k_codes, seq_lens, table, query_start, most, means, scales):
    """Copies of means and scales with the rows of the blocks that got tokens (`most` has no part in it)."""
    means, scales = means.copy(), scales.copy()
    nb, bs = k_codes.shape[:2]
    rows: dict = {}
    for b, _, pos in requests(seq_lens, query_start, 1 << 31, 1 << 31, table.shape[1] * bs):
        rows.setdefault(b, []).append(pos)
    for b, positions in rows.items():
        length = int(np.clip(seq_lens[b], 0, table.shape[1] * bs))
        for col in sorted({p // bs for p in positions if p >= 0}):
            if not 0 <= table[b, col] < nb:
                continue
            v = VALUES[k_codes[table[b, col], :min(bs, length - col * bs)]]
            total = np.where(np.isnan(v), 0.0, v).sum(0).astype(np.float32)          # exact in 64 bits
            mean = total / np.float32(min(bs, length - col * bs))
            means[table[b, col]], scales[table[b, col]] = quantise8(mean)
    return means, scales


def select(q, means, scales, seq_lens, table, bs, query_start, most, first, last, budget, before):
    """A copy of `before` [tokens, heads, budget] with the rows that are looked at."""
    out = before.copy()
    nb, h = means.shape[:2]
    codes, q_scale = quantise8(q)
    share = q.shape[1] // h
    for b, t, pos in requests(seq_lens, query_start, q.shape[0], most, table.shape[1] * bs):
        n = pos // bs + 1 if pos >= 0 else 0
        cols = np.arange(n)
        block = table[b, :n].astype(np.int64)
        inside = (block >= 0) & (block < nb)
        for kv in range(h):
            at = np.where(inside, block, 0)
            dot = codes[t, kv * share:(kv + 1) * share].astype(np.int64) @ means[at, kv].astype(np.int64).T
            with np.errstate(all="ignore"):
                score = dot.astype(np.float32) * q_scale[t, kv * share:(kv + 1) * share, None]
                score = np.where(np.isnan(score), -np.inf, score).max(0).astype(np.float32) * scales[at, kv]
            score = np.where(np.isnan(score) | ~inside, -np.inf, score)
            forced = (cols < first) | (cols >= n - last)
            order = np.lexsort((cols, -score.astype(np.float64), ~forced))[:budget]
            out[t, kv] = -1
            out[t, kv, :len(order)] = np.sort(cols[order])
    return out
