"""Long contexts over the paged fp8 KV cache, as their operators are measured.

A server with an fp8 (e4m3) cache and long contexts runs these in a step:

    write    queries and keys rotated by their positions (one or several axes), keys and values quantised into the cache
    attend   attention of the step's tokens (single ones, drafts, prompt chunks, all of them mixed) over the cache
    select   8-bit means of the keys of the blocks that got tokens, and for each query the blocks that matter most by them
    sparse   attention of each query over its selected blocks alone

Each has a plain form in elementary torch operations (``own`` false) and the library's calls (``own`` true).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
MAX_POSITION = 32768


# ---------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one token of each of 64 requests: the rotation and the cache write of an ordinary decoding step
        dict(name="write_decode_64", op="write", tokens=64, q_heads=32, kv_heads=8, head_dim=128, rot_dim=128, axes=1, interleaved=False,
             block_size=16, dtype="bf16", fused=True),
        # an image and some text: positions with three axes, half of each narrow head rotated, neighbouring dims paired
        dict(name="write_axes_1501_d64", op="write", tokens=1501, q_heads=12, kv_heads=4, head_dim=64, rot_dim=32, axes=3, interleaved=True,
             block_size=48, dtype="fp16", fused=False),
        # a packed batch of prompts
        dict(name="write_prompt_16384", op="write", tokens=16384, q_heads=32, kv_heads=8, head_dim=128, rot_dim=128, axes=1,
             interleaved=False, block_size=64, dtype="bf16", fused=True),
        # one request's check of two drafted tokens: latency
        dict(name="attend_one_3", op="attend", batch=1, ctx=2000, ragged=False, new=3, singles=0.0, q_heads=32, kv_heads=8, head_dim=128,
             block_size=16, dtype="bf16"),
        # five drafted tokens for each of 32 requests
        dict(name="attend_drafts_32x5", op="attend", batch=32, ctx=4096, ragged=True, new=5, singles=0.0, q_heads=32, kv_heads=8,
             head_dim=128, block_size=32, dtype="bf16"),
        # a step that mixes chunks of prompts into a batch of single tokens
        dict(name="attend_mixed_40", op="attend", batch=40, ctx=8192, ragged=True, new=700, singles=0.9, q_heads=32, kv_heads=8,
             head_dim=128, block_size=64, dtype="fp16"),
        # a chunk of a long document after the chunks before it
        dict(name="attend_chunk_2048_after_30000", op="attend", batch=1, ctx=30000, ragged=False, new=2048, singles=0.0, q_heads=32,
             kv_heads=8, head_dim=128, block_size=64, dtype="bf16"),
        # blocks for one token of each of 32 requests
        dict(name="select_decode_32", op="select", batch=32, ctx=32768, ragged=True, new=1, q_heads=32, kv_heads=8, head_dim=128,
             block_size=64, budget=64, first=1, last=2, dtype="bf16"),
        # blocks for a few drafted tokens of long documents, small blocks
        dict(name="select_drafts_4x4_131067", op="select", batch=4, ctx=131067, ragged=False, new=4, q_heads=64, kv_heads=8, head_dim=128,
             block_size=32, budget=256, first=2, last=4, dtype="fp16"),
        # a long document alone: latency
        dict(name="sparse_one_131071", op="sparse", batch=1, ctx=131070, ragged=False, new=1, q_heads=32, kv_heads=8, head_dim=128,
             block_size=64, budget=64, dtype="bf16"),
        # one token of each of 32 requests
        dict(name="sparse_decode_32", op="sparse", batch=32, ctx=32768, ragged=True, new=1, q_heads=32, kv_heads=8, head_dim=128,
             block_size=64, budget=64, dtype="bf16"),
        # a chunk of a prompt, each of its tokens with blocks of its own, narrow heads
        dict(name="sparse_chunk_600_d64", op="sparse", batch=1, ctx=20011, ragged=False, new=600, q_heads=16, kv_heads=4, head_dim=64,
             block_size=32, budget=48, dtype="fp16"),
    ]


def _spread(rng, low, high):
    """A whole number from low to high, even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("write", "attend", "attend", "select", "sparse"))
    kv_heads, share, head_dim = rng.choice((1, 2, 4, 5, 8)), rng.choice((1, 2, 3, 4, 8)), rng.choice((64, 128))
    dtype, block_size = rng.choice(("bf16", "fp16")), rng.choice((16, 32, 48, 64, 128))
    heads = dict(q_heads=kv_heads * share, kv_heads=kv_heads, head_dim=head_dim, block_size=block_size, dtype=dtype)
    if op == "write":
        return dict(op=op, tokens=_spread(rng, 1, 16384 if share < 8 else 9000), rot_dim=head_dim // rng.choice((1, 1, 2, 4)),
                    axes=rng.choice((1, 1, 3)), interleaved=rng.random() < 0.4, fused=rng.random() < 0.5, **heads)
    ragged = rng.random() < 0.5
    if op == "attend":
        new = rng.choice((1, rng.randint(2, 9), _spread(rng, 10, 2000)))
        batch = _spread(rng, 1, 64 if new < 10 else 4)
        ctx = _spread(rng, 1, min(30000, 260000 // batch)) if new < 10 else _spread(rng, 1, 9000)
        return dict(op=op, batch=batch, ctx=ctx, ragged=ragged, new=new, singles=rng.choice((0.0, 0.0, 0.6)), **heads)
    new = rng.choice((1, 1, rng.randint(2, 6), _spread(rng, 7, 300)))
    if op == "select":
        batch = _spread(rng, 1, 32 if new == 1 else 4)
        budget = _spread(rng, 8, 256)
        return dict(op=op, batch=batch, ctx=_spread(rng, 100, min(131000, (1 << 20) // batch) if new < 7 else 30000), ragged=ragged, new=new,
                    budget=budget, first=rng.randint(0, 2), last=rng.randint(1, 4), **heads)
    batch = _spread(rng, 1, 32 if new == 1 else 2)
    return dict(op=op, batch=batch, ctx=_spread(rng, 100, min(131000, (1 << 20) // batch)), ragged=ragged, new=new,
                budget=_spread(rng, 2, 4096 // block_size if new < 7 else 1536 // block_size), **heads)


# ---------------------------------------------------------------------------------------------------- inputs

def _lengths(case):
    """Context and new lengths of a case's requests: the same for every seed, which only changes their order."""
    rng = np.random.default_rng([case["batch"], case["ctx"], 29])
    b = case["batch"]
    ctx, new = np.full(b, case["ctx"], np.int64), np.full(b, case["new"], np.int64)
    if case["ragged"]:
        ctx = rng.integers(max(1, case["ctx"] // 8), case["ctx"] + 1, b)
        new = rng.integers(max(1, case["new"] // 2), case["new"] + 1, b) if case["new"] > 1 else new
        ctx[0] = case["ctx"]
    if case.get("singles"):
        new[rng.random(b) < case["singles"]] = 1
        new[-1] = case["new"]
    return ctx, new


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _head_rows(shape, dtype, gen):
    """Queries, keys or values as projections give them: normal, with a few dims of every head an order larger."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x[..., ::37] *= 8.0
    return x.to(dtype)


def _gpu(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def _pool(num_blocks, case, gen, scale):
    """A filled cache [num_blocks, block_size, heads, head_dim] of e4m3 codes, a part at a time."""
    shape = (num_blocks, case["block_size"], case["kv_heads"], case["head_dim"])
    pool = torch.empty(shape, dtype=E4M3, device="cuda")
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for j in range(0, num_blocks, step):
        part = pool[j:j + step]
        part.copy_((_head_rows(part.shape, torch.float32, gen) / scale).clamp_(-448, 448))
    return pool


def _prepare_write(case, seed):
    gen = _generator(seed)
    n, hq, h, d, bs = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    dtype, rot = DTYPES[case["dtype"]], case["rot_dim"]
    if case["fused"]:
        rows = _head_rows((n, hq + 2 * h, d), dtype, gen)    # the merged projection's rows
        q, k, v = rows[:, :hq], rows[:, hq:hq + h], rows[:, hq + h:]
    else:
        q, k, v = _head_rows((n, hq, d), dtype, gen), _head_rows((n, h, d), dtype, gen), _head_rows((n, h, d), dtype, gen)
    turn = 10000.0 ** (-torch.arange(rot // 2, device="cuda").double() * 2 / rot)
    angle = torch.arange(MAX_POSITION, device="cuda").double()[:, None] * turn
    table = torch.cat([angle.cos(), angle.sin()], 1).float()
    if case["axes"] == 1:
        sections = None
        positions = torch.randint(0, MAX_POSITION, (n,), generator=gen, device="cuda").int()
    else:
        # time, height and width of patches, each with a share of the pairs
        sections = (rot // 8, (rot // 2 - rot // 8) // 2, rot // 2 - rot // 8 - (rot // 2 - rot // 8) // 2)
        grid = torch.arange(n, device="cuda")
        start = torch.randint(0, MAX_POSITION // 2, (1,), generator=gen, device="cuda")
        positions = torch.stack([start + grid // 1024, start + grid // 32 % 32, start + grid % 32]).int()
    num_blocks = -(-n // bs) + 3
    where = torch.randperm((num_blocks - 1) * bs, generator=gen, device="cuda")[:n]
    if n > 40:
        where[-3:] = -1                                      # padding of a captured step
    caches = [torch.zeros(num_blocks, bs, h, d, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    # scales of an earlier calibration, whose largest values are somewhat above these tokens'
    margin = 1.0 + 0.3 * torch.rand(2, generator=gen, device="cuda")
    scale = [(t.float().abs().amax() * m * (1.0 + 0.42 * (t is k)) / 448.0).reshape(1) for t, m in zip((k, v), margin)]
    return dict(op="write", q=q, k=k, v=v, table=table, positions=positions, sections=sections, interleaved=case["interleaved"],
                k_cache=caches[0], v_cache=caches[1], slots=where, k_scale=scale[0], v_scale=scale[1],
                q_out=torch.empty(n, hq, d, dtype=dtype, device="cuda"))


def _prepare_paged(case, seed):
    """What the attention's and the selection's cases share: lengths, block table, caches and queries."""
    gen, rng = _generator(seed), np.random.default_rng([seed, 37])
    ctx, new = _lengths(case)
    order = rng.permutation(case["batch"])
    ctx, new = ctx[order], new[order]
    b, d, bs = case["batch"], case["head_dim"], case["block_size"]
    total = ctx + new
    blocks = -(-total // bs)
    num_blocks = int(blocks.sum()) + 2
    table = np.full((b, int(blocks.max())), -1, np.int32)
    table[np.arange(table.shape[1])[None, :] < blocks[:, None]] = rng.permutation(num_blocks)[:blocks.sum()]
    scale = torch.full((1,), 40.0 / 448.0, device="cuda")
    s = dict(op=case["op"], q=_head_rows((int(new.sum()), case["q_heads"], d), DTYPES[case["dtype"]], gen), seq_lens=_gpu(total), table=_gpu(table),
             query_start=_gpu(np.concatenate([[0], np.cumsum(new)])), most=int(new.max()), block_size=bs, k_scale=scale,
             v_scale=scale.clone(), sm_scale=1.0 / math.sqrt(d), k_cache=_pool(num_blocks, case, gen, scale))
    if case["op"] != "select":
        s["v_cache"], s["out"] = _pool(num_blocks, case, gen, scale), torch.empty_like(s["q"])
    return s, gen, rng, ctx, new


def _prepare_select(case, seed):
    s, gen, _, _, _ = _prepare_paged(case, seed)
    # the means as the steps before have left them
    shape = s["k_cache"].shape
    means, scales = torch.empty(shape[0], *shape[2:], dtype=torch.int8, device="cuda"), torch.empty(shape[0], shape[2], device="cuda")
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for j in range(0, shape[0], step):
        m = s["k_cache"][j:j + step].double().sum(1) / shape[1]
        top = m.abs().amax(2, keepdim=True) / 127.0
        means[j:j + step], scales[j:j + step] = (m / top).round(), top.squeeze(2)
    selected = torch.empty(s["q"].shape[0], shape[2], case["budget"], dtype=torch.int32, device="cuda")
    return dict(s, means=means, mean_scales=scales, selected=selected, first=case["first"], last=case["last"])


def _prepare_sparse(case, seed):
    s, gen, rng, ctx, new = _prepare_paged(case, seed)
    h, bs, k = case["kv_heads"], case["block_size"], case["budget"]
    rows = []
    # a selection: the first block, the token's own and the one before it, and others in their order
    for c, n in zip(ctx, new):
        own_block = (c + np.arange(n)) // bs
        score = rng.random((int(n), h, int(own_block[-1]) + 1), dtype=np.float32)
        col = np.arange(score.shape[2])
        score[:, :, 0] = 2.0
        score = np.where((col >= own_block[:, None] - 1)[:, None], 3.0, score)
        score = np.where((col > own_block[:, None])[:, None], -1.0, score)
        if score.shape[2] > k:
            top = np.argpartition(-score, k - 1, axis=2)[:, :, :k]
            seen = np.take_along_axis(score, top, 2) >= 0
        else:
            top = np.broadcast_to(np.pad(col, (0, k - len(col))), (int(n), h, k))
            seen = np.pad(score, ((0, 0), (0, 0), (0, k - len(col))), constant_values=-1.0) >= 0
        top = np.sort(np.where(seen, top, 1 << 30), 2)
        rows.append(np.where(top == 1 << 30, -1, top).astype(np.int32))
    return dict(s, selected=_gpu(np.concatenate(rows)))


def prepare(case, seed):
    if case["op"] == "attend":
        return _prepare_paged(case, seed)[0]
    return {"write": _prepare_write, "select": _prepare_select, "sparse": _prepare_sparse}[case["op"]](case, seed)


# ---------------------------------------------------------------------------------------------------- plain forms

def _rotated(x, cos, sin, interleaved):
    """x [tokens, heads, d] in 32 bits with its first 2 * pairs dims turned by angles [tokens, pairs]."""
    x = x.float()
    rot, cos, sin = 2 * cos.shape[1], cos[:, None], sin[:, None]
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_write(s):
    pairs, positions = s["table"].shape[1] // 2, s["positions"].long()
    if s["sections"] is not None:
        axis = torch.repeat_interleave(torch.tensor(s["sections"], device=positions.device))
        positions = positions[axis].T                                              # [tokens, pairs]
        pair = torch.arange(pairs, device=positions.device)
        cos, sin = s["table"][positions, pair], s["table"][positions, pairs + pair]
    else:
        cos, sin = s["table"][positions, :pairs], s["table"][positions, pairs:]
    k_cache, v_cache, slots = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1), s["slots"]
    at = torch.where(slots >= 0, slots, k_cache.shape[0] - 1)                      # padding goes to a slot that no token has
    k = _rotated(s["k"], cos, sin, s["interleaved"]) / s["k_scale"]
    v = s["v"].float() / s["v_scale"]
    real = (slots >= 0)[:, None, None]
    k_cache.view(torch.uint8)[at] = torch.where(real, k.clamp(-448, 448), 0.0).to(E4M3).view(torch.uint8)
    v_cache.view(torch.uint8)[at] = torch.where(real, v.clamp(-448, 448), 0.0).to(E4M3).view(torch.uint8)
    return _rotated(s["q"], cos, sin, s["interleaved"]).to(s["q"].dtype), s["k_cache"], s["v_cache"]


def _rows_of(s):
    """The request of each row of q, its index among the request's rows, and the last token that it sees."""
    start, t = s["query_start"].long(), torch.arange(s["q"].shape[0], device=s["q"].device)
    of = torch.searchsorted(start, t, right=True) - 1
    row = t - start[of]
    return of, row, s["seq_lens"].long()[of] - (start[1:] - start[:-1])[of] + row


def _softmax_of(score):
    """Weights that sum to 1 in the last dimension, zeros where nothing is seen; in place."""
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = score.sum(-1, keepdim=True)
    return score.div_(torch.where(total == 0, 1.0, total))


def _plain_attend(s):
    q, table = s["q"], s["table"].clamp(min=0).long()
    b, most, h = table.shape[0], s["most"], s["k_cache"].shape[2]
    of, row, _ = _rows_of(s)
    padded = torch.zeros(b, most, *q.shape[1:], device=q.device)
    padded[of, row] = q.float()
    rows = padded.unflatten(2, (h, -1)).permute(0, 2, 3, 1, 4)                      # [b, h, share, most, d]
    k = s["k_cache"].view(torch.uint8)[table].view(E4M3).flatten(1, 2).transpose(1, 2).float()   # [b, h, tokens, d]
    score = (rows.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, (-1, most)) * (s["sm_scale"] * s["k_scale"])
    del k
    count = s["query_start"].long().diff()
    last = (s["seq_lens"].long() - count)[:, None] + torch.arange(most, device=q.device)[None, :]
    seen = torch.arange(score.shape[-1], device=q.device)[None, None, :] <= last[:, :, None]
    weights = _softmax_of(score.masked_fill_(~seen[:, None, None], -math.inf))
    v = s["v_cache"].view(torch.uint8)[table].view(E4M3).flatten(1, 2).transpose(1, 2).float()
    o = (weights.flatten(2, 3) @ v).unflatten(2, (-1, most)) * s["v_scale"]
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3)[of, row].to(q.dtype)


def _plain_means(s):
    """Means of the touched blocks' keys, one scale for a block and head, in place."""
    bs, table, lens = s["block_size"], s["table"].long(), s["seq_lens"].long()
    count = s["query_start"].long().diff()
    col = ((lens - count) // bs)[:, None] + torch.arange((s["most"] - 1) // bs + 2, device=table.device)[None, :]
    b, j = ((col * bs < lens[:, None]) & (count > 0)[:, None]).nonzero(as_tuple=True)
    col = col[b, j]
    block, held = table[b, col], (lens[b] - col * bs).clamp(max=bs)
    codes = s["k_cache"].view(torch.uint8)[block].view(E4M3).double()               # [touched, tokens, heads, d]
    codes = codes * (torch.arange(bs, device=table.device)[None, :] < held[:, None])[:, :, None, None]
    mean = codes.sum(1).float() / held[:, None, None].float()                       # (the sum is exact in 64 bits)
    top = mean.abs().amax(2, keepdim=True)
    scale = torch.where(top > 0, top / 127.0, 1.0)
    s["means"][block] = (mean / scale).round().to(torch.int8)
    s["mean_scales"][block] = scale.squeeze(2)


def _plain_select(s):
    _plain_means(s)
    q, table, bs = s["q"].float(), s["table"].clamp(min=0).long(), s["block_size"]
    budget, h = s["selected"].shape[2], s["means"].shape[1]
    top = q.abs().amax(2, keepdim=True)
    q_scale = torch.where(top > 0, top / 127.0, 1.0)
    codes = (q / q_scale).round()
    of, row, last = _rows_of(s)
    b, most, n = table.shape[0], s["most"], table.shape[1]
    padded = torch.zeros(b, most, *q.shape[1:], device=q.device)
    padded[of, row] = codes
    scales = torch.zeros(b, most, q.shape[1], device=q.device)
    scales[of, row] = q_scale.squeeze(2)
    means = s["means"][table].permute(0, 2, 3, 1).float()                           # [b, h, d, blocks]
    dot = (padded.unflatten(2, (h, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3) @ means).unflatten(2, (most, -1))
    # whole numbers below 2^24 so far; the largest of the heads that share the keys
    score = (dot * scales.unflatten(2, (h, -1)).permute(0, 2, 1, 3).unsqueeze(-1)).amax(3)
    score = (score * s["mean_scales"][table].permute(0, 2, 1)[:, :, None]).permute(0, 2, 1, 3)[of, row]   # [tokens, h, blocks]
    col, own_block = torch.arange(n, device=q.device), (last // bs)[:, None]
    seen, forced = col <= own_block, (col < s["first"]) | (col > own_block - s["last"])
    score = torch.where(forced[:, None], math.inf, score).masked_fill(~seen[:, None], -math.inf)
    order = torch.sort(score, dim=2, descending=True, stable=True)[1][:, :, :budget]
    order = torch.where(torch.gather(seen[:, None].expand(score.shape), 2, order), order, n)
    order = torch.sort(order, dim=2)[0]
    chosen = torch.full(s["selected"].shape, -1, dtype=torch.int32, device=q.device)
    chosen[:, :, :order.shape[2]] = torch.where(order == n, -1, order).int()
    return s["means"], s["mean_scales"], chosen


def _plain_sparse(s):
    q, bs, h = s["q"], s["block_size"], s["k_cache"].shape[2]
    of, _, last = _rows_of(s)
    col = s["selected"].long()                                                      # [tokens, h, budget]
    block = s["table"].long()[of[:, None, None], col.clamp(min=0)]
    token = torch.arange(bs, device=q.device)
    at = ((block * bs).unsqueeze(-1) + token).flatten(2)
    seen = ((col >= 0)[..., None] & ((col * bs).unsqueeze(-1) + token <= last[:, None, None, None])).flatten(2)
    head = torch.arange(h, device=q.device)[None, :, None]
    k = s["k_cache"].view(torch.uint8).flatten(0, 1)[at, head].view(E4M3).float()   # [tokens, h, budget * bs, d]
    score = (q.float().unflatten(1, (h, -1)) @ k.transpose(2, 3)) * (s["sm_scale"] * s["k_scale"])
    del k
    weights = _softmax_of(score.masked_fill_(~seen[:, :, None], -math.inf))
    v = s["v_cache"].view(torch.uint8).flatten(0, 1)[at, head].view(E4M3).float()
    return ((weights @ v) * s["v_scale"]).flatten(1, 2).to(q.dtype)


# ---------------------------------------------------------------------------------------------------- the library's calls

def _own_run(s):
    import int8_w8a8_scaled_gb300 as w8
    op = s["op"]
    if op == "write":
        w8.fp8_kv_rotate_write(s["q"], s["k"], s["v"], s["table"], s["positions"], s["k_cache"], s["v_cache"], s["slots"], s["k_scale"],
                               s["v_scale"], s["q_out"], sections=s["sections"], interleaved=s["interleaved"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if op == "attend":
        w8.fp8_kv_attention(s["q"], s["k_cache"], s["v_cache"], s["seq_lens"], s["table"], s["k_scale"], s["v_scale"], s["out"],
                            query_start=s["query_start"], max_query_len=s["most"], sm_scale=s["sm_scale"])
        return s["out"]
    if op == "select":
        w8.fp8_kv_block_means(s["k_cache"], s["seq_lens"], s["table"], s["means"], s["mean_scales"], query_start=s["query_start"],
                              max_query_len=s["most"])
        w8.fp8_kv_select_blocks(s["q"], s["means"], s["mean_scales"], s["seq_lens"], s["table"], s["block_size"], s["selected"],
                                query_start=s["query_start"], max_query_len=s["most"], first_blocks=s["first"], last_blocks=s["last"])
        return s["means"], s["mean_scales"], s["selected"]
    w8.fp8_kv_sparse_attention(s["q"], s["k_cache"], s["v_cache"], s["seq_lens"], s["table"], s["selected"], s["k_scale"], s["v_scale"],
                               s["out"], query_start=s["query_start"], max_query_len=s["most"], sm_scale=s["sm_scale"])
    return s["out"]


def run(state):
    if own:
        return _own_run(state)
    return {"write": _plain_write, "attend": _plain_attend, "select": _plain_select, "sparse": _plain_sparse}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------- work

def work(case):
    op, hq, h, d = case["op"], case["q_heads"], case["kv_heads"], case["head_dim"]
    if op == "write":
        n = case["tokens"]
        # queries in and out, keys and values in and as codes, the angles' rows
        return {"bytes": int(n * (4 * hq * d + 2 * h * d * 3 + 4 * case["rot_dim"] + 8 + 4 * case["axes"])), "flops": int(n * 6 * (hq + 2 * h) * d)}
    ctx, new = _lengths(case)
    bs = case["block_size"]
    pairs = int((new * ctx + new * (new + 1) // 2).sum())
    if op == "attend":
        return {"bytes": int((ctx + new).sum() * h * d * 2 + 4 * new.sum() * hq * d + 4 * (ctx + new).sum() / bs), "flops": 4 * pairs * hq * d}
    blocks, touched = -(-(ctx + new) // bs), (ctx + new - 1) // bs - ctx // bs + 1
    if op == "select":
        held = int((ctx + new - ctx // bs * bs).sum())
        return {"bytes": int(held * h * d + touched.sum() * h * (d + 4) + blocks.sum() * (h * (d + 4) + 4)
                             + new.sum() * (2 * hq * d + 4 * h * case["budget"])), "flops": int(2 * (new * blocks).sum() * hq * d)}
    # no more tokens than the request holds are read, and none of a block that nobody selects is there
    seen = np.minimum(np.minimum(new * case["budget"], blocks) * bs, ctx + new)
    attended = int((new * np.minimum(case["budget"] * bs, ctx + new)).sum())
    return {"bytes": int(seen.sum() * h * d * 2 + new.sum() * (4 * hq * d + 4 * h * case["budget"])), "flops": 4 * attended * hq * d}


# ---------------------------------------------------------------------------------------------------- 64 bits

def _codes_to_64(codes):
    """Values of e4m3 codes from their bits."""
    raw = codes.view(torch.uint8).int()
    e, m = raw // 8 % 16, raw % 8
    x = torch.where(e > 0, (8 + m).double() * torch.exp2(e.double() - 10), m.double() * 2.0 ** -9)
    return torch.where(raw >= 128, -x, x)


def _nearest_e4m3(x):
    """Nearest e4m3 value (ties to even) of 64-bit numbers."""
    a = x.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -30))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), x)


def _exact_write(s):
    n, pairs = s["q"].shape[0], s["table"].shape[1] // 2
    pos = s["positions"].reshape(-1, n).tolist()
    axis = [0] * pairs if s["sections"] is None else [a for a, c in enumerate(s["sections"]) for _ in range(c)]
    row = torch.tensor([pos[a] for a in axis], device="cuda")                       # [pairs, tokens]
    c = torch.stack([s["table"][row[i], i] for i in range(pairs)], 1).double()
    z = torch.stack([s["table"][row[i], pairs + i] for i in range(pairs)], 1).double()
    first = torch.arange(pairs, device="cuda") * (2 if s["interleaved"] else 1)
    second = first + (1 if s["interleaved"] else pairs)

    def turn(x):
        x = x.double()
        y = x.clone()
        y[:, :, first] = x[:, :, first] * c[:, None] - x[:, :, second] * z[:, None]
        y[:, :, second] = x[:, :, second] * c[:, None] + x[:, :, first] * z[:, None]
        return y

    real = s["slots"] >= 0
    out = [turn(s["q"])]
    for x, g, cache in ((turn(s["k"]), s["k_scale"], s["k_cache"]), (s["v"].double(), s["v_scale"], s["v_cache"])):
        y = torch.zeros(cache.shape, dtype=torch.float64, device="cuda").flatten(0, 1)
        y[s["slots"][real]] = _nearest_e4m3(x[real] / g.double())
        out.append(y.view(cache.shape))
    return tuple(out)


def _tokens_of(s, cache, b, head, positions):
    """Rows of one request's tokens in 64 bits."""
    block = s["table"][b].long()[positions // s["block_size"]]
    return _codes_to_64(s[cache][block, positions % s["block_size"], head])


def _exact_attend(s):
    h = s["k_cache"].shape[2]
    share, start, out = s["q"].shape[1] // h, s["query_start"].tolist(), torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["seq_lens"].tolist()):
        first, count = start[b], start[b + 1] - start[b]
        at = torch.arange(n, device="cuda")
        for head in range(h):
            k, v = _tokens_of(s, "k_cache", b, head, at) * s["k_scale"].double(), _tokens_of(s, "v_cache", b, head, at) * s["v_scale"].double()
            for i in range(0, count, 512):
                rows = slice(first + i, first + min(i + 512, count))
                score = torch.einsum("igd,td->igt", s["q"][rows, head * share:(head + 1) * share].double(), k) * s["sm_scale"]
                limit = n - count + i + torch.arange(score.shape[0], device="cuda")
                score = score.masked_fill(at > limit[:, None, None], -math.inf)
                out[rows, head * share:(head + 1) * share] = torch.softmax(score, 2) @ v
    return out


def _exact_sparse(s):
    h = s["k_cache"].shape[2]
    share, start, out = s["q"].shape[1] // h, s["query_start"].tolist(), torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    bs, selected = s["block_size"], s["selected"].cpu().numpy()
    for b, n in enumerate(s["seq_lens"].tolist()):
        for t in range(start[b], start[b + 1]):
            last = n - start[b + 1] + t
            for head in range(h):
                at = np.concatenate([np.arange(c * bs, min(c * bs + bs, last + 1)) for c in selected[t, head] if c >= 0])
                at = torch.from_numpy(at).cuda()
                k, v = _tokens_of(s, "k_cache", b, head, at) * s["k_scale"].double(), _tokens_of(s, "v_cache", b, head, at) * s["v_scale"].double()
                score = s["q"][t, head * share:(head + 1) * share].double() @ k.T * s["sm_scale"]
                out[t, head * share:(head + 1) * share] = torch.softmax(score, 1) @ v
    return out


def _exact_select(s):
    """Quotients and products are rounded to 32 bits where the definition says so; all else is exact."""
    f32 = lambda x: x.astype(np.float32).astype(np.float64)  # noqa: E731
    bs, start, lens = s["block_size"], s["query_start"].tolist(), s["seq_lens"].tolist()
    table, means, scales = s["table"].cpu().numpy(), s["means"].cpu().numpy().copy(), s["mean_scales"].double().cpu().numpy()
    for b, n in enumerate(lens):
        for col in range((n - start[b + 1] + start[b]) // bs, -(-n // bs)):
            held = min(bs, n - col * bs)
            mean = f32(f32(_codes_to_64(s["k_cache"][table[b, col], :held]).sum(0).cpu().numpy()) / held)
            top = np.abs(mean).max(1, keepdims=True)
            scale = np.where(top > 0, f32(top / 127.0), 1.0)
            means[table[b, col]], scales[table[b, col]] = np.rint(f32(mean / scale)), scale[:, 0]
    q = s["q"].double().cpu().numpy()
    top = np.abs(q).max(2, keepdims=True)
    q_scale = np.where(top > 0, f32(top / 127.0), 1.0)
    q = np.rint(f32(q / q_scale))
    chosen = np.full(s["selected"].shape, -1, np.int32)
    h, budget = chosen.shape[1:]
    for b, n in enumerate(lens):
        keys, key_scales = means[table[b, :-(-n // bs)]].astype(np.float64), scales[table[b, :-(-n // bs)]]
        for t in range(start[b], start[b + 1]):
            own_block = (n - start[b + 1] + t) // bs
            cols = np.arange(own_block + 1)
            forced = (cols < s["first"]) | (cols > own_block - s["last"])
            for head in range(h):
                g = slice(head * (q.shape[1] // h), (head + 1) * (q.shape[1] // h))
                score = f32(f32((q[t, g] @ keys[:own_block + 1, head].T) * q_scale[t, g]).max(0) * key_scales[:own_block + 1, head])
                order = np.lexsort((cols, np.where(forced, -np.inf, -score)))[:budget]
                chosen[t, head, :len(order)] = np.sort(cols[order])
    return torch.from_numpy(means), torch.from_numpy(scales), torch.from_numpy(chosen)


def exact(case, seed):
    if case["op"] == "attend" and work(case)["flops"] > 2e12:
        return None
    if case["op"] in ("select", "sparse") and int(_lengths(case)[1].sum()) * case["kv_heads"] > 3000:
        return None
    return {"write": _exact_write, "attend": _exact_attend, "select": _exact_select, "sparse": _exact_sparse}[case["op"]](prepare(case, seed))
