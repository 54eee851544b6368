"""The operators of a paged serving step over a 4-bit KV cache, as they are measured.

A step of a server that keeps its keys and values in 4 bits runs four operators:

    tables   block tables, slots and positions of the step's tokens, from the request lengths
    write    new keys and values quantised into the cache at their slots, and read back
    attend   attention of the step's tokens (one, a few drafted ones or a prompt's) over the cache
    verify   drafted tokens accepted or replaced, from both models' probabilities and given random numbers

Each has a plain form in elementary torch operations (``own`` false) and the library's calls (``own`` true).
"""
import math

import numpy as np
import torch

own = False

E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
LARGEST = {"e2m1": 6.0, "int4": 7.0}
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GROUP = 16     # consecutive dims that share a scale
TILE = 16      # tokens of one cache record


# ---------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one new token for each of a few requests: the tables before every token of a small server
        dict(name="tables_decode_8", op="tables", batch=8, ctx=2000, new=1, prompts=0.0, block_size=16, max_blocks=512, short=0.0),
        # a large server's step: most requests add a token, some bring a prompt, and the pool runs out near the end
        dict(name="tables_mixed_1000", op="tables", batch=1000, ctx=9000, new=1500, prompts=0.05, block_size=32, max_blocks=512, short=0.1),
        # keys and values of one token of 32 requests, views of the merged projection
        dict(name="write_decode_32", op="write", tokens=32, heads=8, head_dim=128, block_size=16, kind="e2m1", dtype="bf16", fused=True),
        # a prompt of odd length, narrow heads
        dict(name="write_1111_d64", op="write", tokens=1111, heads=4, head_dim=64, block_size=32, kind="int4", dtype="bf16", fused=False),
        # a packed batch of prompts
        dict(name="write_prompt_16384", op="write", tokens=16384, heads=8, head_dim=128, block_size=64, kind="int4", dtype="fp16", fused=True),
        # one request, one token: latency
        dict(name="attend_one_1023", op="attend", batch=1, ctx=1022, ragged=False, new=1, q_heads=32, kv_heads=8, head_dim=128,
             block_size=16, kind="e2m1", dtype="bf16"),
        # ordinary decoding: a batch of ragged requests, one token each
        dict(name="attend_decode_64", op="attend", batch=64, ctx=8192, ragged=True, new=1, q_heads=32, kv_heads=8, head_dim=128,
             block_size=16, kind="e2m1", dtype="bf16"),
        # two long documents, 8 query heads to a KV head
        dict(name="attend_long_2x131071", op="attend", batch=2, ctx=131070, ragged=False, new=1, q_heads=64, kv_heads=8, head_dim=128,
             block_size=64, kind="int4", dtype="fp16"),
        # five drafted tokens for each request
        dict(name="attend_drafts_32x5", op="attend", batch=32, ctx=4096, ragged=True, new=5, q_heads=32, kv_heads=8, head_dim=128,
             block_size=32, kind="e2m1", dtype="bf16"),
        # prompt chunks after an earlier part of the prompt
        dict(name="attend_prompt_2x4000", op="attend", batch=2, ctx=4200, ragged=False, new=4000, q_heads=32, kv_heads=8, head_dim=128,
             block_size=64, kind="e2m1", dtype="bf16"),
        # a small server's check of a few drafted tokens
        dict(name="verify_4", op="verify", batch=4, drafts=3, vocab=32000, dtype="fp32", greedy=False),
        # a large batch, a large vocabulary
        dict(name="verify_128", op="verify", batch=128, drafts=7, vocab=131072, dtype="fp32", greedy=False),
    ]


def _spread(rng, low, high):
    """A whole number from low to high, even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("tables", "write", "attend", "attend", "attend", "verify"))
    if op == "tables":
        block_size = rng.choice((16, 32, 48, 128))
        return dict(op=op, batch=_spread(rng, 1, 1000), ctx=_spread(rng, 10, 9000), new=_spread(rng, 1, 1500),
                    prompts=rng.choice((0.0, 0.05, 1.0)) if block_size > 16 else 0.0, block_size=block_size,
                    max_blocks=rng.randint(-(-10500 // block_size), 700), short=rng.choice((0.0, 0.1)))
    if op == "write":
        heads, head_dim = rng.choice((1, 2, 4, 5, 8)), rng.choice((64, 128))
        return dict(op=op, tokens=_spread(rng, 1, 16384), heads=heads, head_dim=head_dim, block_size=rng.choice((16, 32, 48, 64)),
                    kind=rng.choice(("e2m1", "int4")), dtype=rng.choice(("bf16", "fp16")), fused=rng.random() < 0.5)
    if op == "attend":
        kv_heads, share = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 5, 8))
        new = rng.choice((1, 1, rng.randint(2, 9), _spread(rng, 10, 1500)))
        batch = _spread(rng, 1, 64 if new == 1 else 32 if new < 10 else 2)
        # prompts stay below the longest listed scores, decoding below the longest listed cache
        ctx = _spread(rng, 1, min(131000, 250000 // batch)) if new < 10 else _spread(rng, 1, 4000)
        return dict(op=op, batch=batch, ctx=ctx, ragged=rng.random() < 0.6, new=new, q_heads=kv_heads * share, kv_heads=kv_heads,
                    head_dim=rng.choice((64, 128)), block_size=rng.choice((16, 32, 48, 64)), kind=rng.choice(("e2m1", "int4")),
                    dtype=rng.choice(("bf16", "fp16")))
    return dict(op=op, batch=_spread(rng, 1, 128), drafts=rng.randint(1, 7), vocab=_spread(rng, 1000, 131072),
                dtype=rng.choice(("fp32", "fp32", "bf16")), greedy=rng.random() < 0.3)


# ---------------------------------------------------------------------------------------------------- inputs

def _lengths(case):
    """Context and new lengths of an attention case's requests: the same for every seed, which only changes their order."""
    rng = np.random.default_rng([case["batch"], case["ctx"], 17])
    b = case["batch"]
    if not case["ragged"]:
        return np.full(b, case["ctx"], np.int64), np.full(b, case["new"], np.int64)
    ctx = rng.integers(max(1, case["ctx"] // 8), case["ctx"] + 1, b)
    new = rng.integers(max(1, case["new"] // 2), case["new"] + 1, b) if case["new"] > 1 else np.ones(b, np.int64)
    ctx[0] = case["ctx"]
    return ctx, new


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _head_rows(shape, dtype, gen):
    """Keys or values as projections give them: normal, with a few dims of every head an order larger."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x[..., ::37] *= 8.0
    return x.to(dtype)


def _new_lengths(case):
    """New tokens of a tables case's requests: the same for every seed, which only changes their order."""
    rng = np.random.default_rng([case["batch"], case["new"], 3])
    new = np.ones(case["batch"], np.int64)
    grow = rng.random(case["batch"]) < case["prompts"]
    new[grow] = rng.integers(1, case["new"] + 1, int(grow.sum()))
    return new


def _prepare_tables(case, seed):
    rng = np.random.default_rng([seed, 5])
    b, bs = case["batch"], case["block_size"]
    ctx = rng.integers(0, case["ctx"] + 1, b)
    new = rng.permutation(_new_lengths(case))
    ctx[(new > 1) & (rng.random(b) < 0.5)] = 0
    held = -(-ctx // bs)
    need = -(-(ctx + new) // bs) - held
    num_blocks = int(held.sum() + need.sum()) + 64
    order = rng.permutation(num_blocks)
    table = np.full((b, case["max_blocks"]), -1, np.int32)
    cols = np.arange(case["max_blocks"])
    table[cols[None, :] < held[:, None]] = order[:held.sum()]
    free = order[held.sum():]
    count = len(free) if case["short"] == 0.0 else int(need.sum() * (1.0 - case["short"]))
    tokens = int(new.sum()) + 7                       # a captured step's padding
    gpu = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", t)  # noqa: E731
    empty = lambda n, t=torch.int32: torch.empty(n, dtype=t, device="cuda")  # noqa: E731
    return dict(op="tables", ctx=gpu(ctx, torch.int32), new=gpu(new, torch.int32), free=gpu(free, torch.int32),
                count=gpu([count], torch.int32), table=gpu(table, torch.int32), block_size=bs,
                query_start=empty(b + 1), seq_lens=empty(b), slots=empty(tokens, torch.int64), positions=empty(tokens),
                free_left=empty(1))


def _prepare_write(case, seed):
    gen = _generator(seed)
    n, h, d, bs = case["tokens"], case["heads"], case["head_dim"], case["block_size"]
    dtype = DTYPES[case["dtype"]]
    if case["fused"]:
        # the merged projection's rows: 4 query heads for each KV head, then keys, then values
        rows = _head_rows((n, 6 * h, d), dtype, gen)
        k, v = rows[:, 4 * h:5 * h], rows[:, 5 * h:]
    else:
        k, v = _head_rows((n, h, d), dtype, gen), _head_rows((n, h, d), dtype, gen)
    num_blocks = -(-n // bs) + 3
    where = torch.randperm((num_blocks - 1) * bs, generator=gen, device="cuda")[:n]
    if n > 40:
        where[-3:] = -1                               # padding of a captured step
    cache = torch.zeros(num_blocks, h, bs // TILE, 18 * d, dtype=torch.uint8, device="cuda")
    # scales of an earlier calibration, whose largest values are somewhat above these tokens'
    margin = 1.0 + 0.3 * torch.rand(2, generator=gen, device="cuda")
    scale = [(t.float().abs().amax() * m / (LARGEST[case["kind"]] * 448.0)).reshape(1) for t, m in zip((k, v), margin)]
    out = [torch.empty(n, h, d, dtype=dtype, device="cuda") for _ in range(2)]
    return dict(op="write", k=k, v=v, cache=cache, slots=where, k_scale=scale[0], v_scale=scale[1], kind=case["kind"],
                k_out=out[0], v_out=out[1])


def _prepare_attend(case, seed):
    gen = _generator(seed)
    rng = np.random.default_rng([seed, 23])
    ctx, new = _lengths(case)
    order = rng.permutation(case["batch"])
    ctx, new = ctx[order], new[order]
    b, h, d, bs = case["batch"], case["kv_heads"], case["head_dim"], case["block_size"]
    dtype = DTYPES[case["dtype"]]
    total = ctx + new
    blocks = -(-total // bs)
    num_blocks = int(blocks.sum()) + 2
    table = np.full((b, int(blocks.max())), -1, np.int32)
    table[np.arange(table.shape[1])[None, :] < blocks[:, None]] = rng.permutation(num_blocks)[:blocks.sum()]
    cache = torch.empty(num_blocks, h, bs // TILE, 18 * d, dtype=torch.uint8, device="cuda")
    largest = LARGEST[case["kind"]]
    scale = torch.full((1,), 40.0 / (largest * 448.0), device="cuda")
    step = max(1, (1 << 27) // (h * bs * d))
    for j in range(0, num_blocks, step):              # the whole pool is filled, a part at a time
        part = cache[j:j + step]
        for at in (0, 9 * d):
            x = _head_rows((part.shape[0], h, bs // TILE, TILE, d), dtype, gen)
            codes, scales = _quantise(x, scale, case["kind"])
            part[..., at:at + 8 * d] = codes.flatten(-2)
            part[..., at + 8 * d:at + 9 * d] = scales.flatten(-2)
    tokens = int(new.sum())
    q = _head_rows((tokens, case["q_heads"], d), dtype, gen)
    start = np.concatenate([[0], np.cumsum(new)])
    gpu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", torch.int32)  # noqa: E731
    return dict(op="attend", q=q, cache=cache, seq_lens=gpu(total), table=gpu(table), query_start=gpu(start), most=int(new.max()),
                k_scale=scale, v_scale=scale.clone(), kind=case["kind"], sm_scale=1.0 / math.sqrt(d), out=torch.empty_like(q))


def _draft_counts(case, seed):
    rng = np.random.default_rng([seed, 31])
    counts = rng.integers(0, case["drafts"] + 1, case["batch"])
    counts[0] = case["drafts"]
    return counts


def _prepare_verify(case, seed):
    gen = _generator(seed)
    counts = _draft_counts(case, seed)
    b, v = case["batch"], case["vocab"]
    start = np.concatenate([[0], np.cumsum(counts)])
    rows = int(start[-1])
    of = np.repeat(np.arange(b), counts)
    at = torch.from_numpy(np.arange(rows) + of).cuda()           # the target's row of each drafted token
    logits = 2.5 * torch.randn(rows + b, v, generator=gen, device="cuda")
    target = torch.softmax(logits, 1).to(DTYPES[case["dtype"]])
    drafted = logits[at].add_(0.7 * torch.randn(rows, v, generator=gen, device="cuda"))
    del logits
    draft = torch.softmax(drafted, 1).to(DTYPES[case["dtype"]])
    del drafted
    if case["greedy"]:
        tokens, draft = draft.float().argmax(1), None            # a draft with no distribution: its tokens alone
    else:
        at = torch.rand(rows, 1, generator=gen, device="cuda").double()
        c = draft.double().cumsum(1)
        tokens = torch.searchsorted(c, at * c[:, -1:]).squeeze(1).clamp_(max=v - 1)
    empty = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(op="verify", target=target, draft=draft, tokens=tokens.int(), start=torch.from_numpy(start).int().cuda(),
                uniform=torch.rand(rows, generator=gen, device="cuda"), sample=torch.rand(b, generator=gen, device="cuda"),
                most=case["drafts"], out_tokens=empty(b, case["drafts"] + 1), accepted=empty(b))


def prepare(case, seed):
    return {"tables": _prepare_tables, "write": _prepare_write, "attend": _prepare_attend,
            "verify": _prepare_verify}[case["op"]](case, seed)


# ---------------------------------------------------------------------------------------------------- plain forms

def _quantise(x, g, kind):
    """Codes (two a byte, the even dim low) and e4m3 scale bytes of x [..., d], one scale for GROUP dims."""
    groups = x.float().unflatten(-1, (-1, GROUP))
    largest = torch.nan_to_num(groups.abs(), nan=0.0, posinf=math.inf).amax(-1, keepdim=True)
    scale = (largest / (LARGEST[kind] * g)).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    y = (groups / (scale.float() * g)).flatten(-2)
    if kind == "int4":
        code = torch.nan_to_num(y.round(), nan=0.0).clamp(-7, 7).to(torch.int8).view(torch.uint8) & 15
    else:
        a = y.abs()
        code = (a > 0.25).to(torch.uint8)
        code += a >= 0.75
        code += a > 1.25
        code += a >= 1.75
        code += a > 2.5
        code += a >= 3.5
        code += a > 5.0
        code += 8 * (torch.signbit(y) & ~torch.isnan(y)).to(torch.uint8)
    return code[..., ::2] | (code[..., 1::2] << 4), scale.squeeze(-1).view(torch.uint8)


def _values(codes, scales, kind):
    """code * group scale in 32 bits (exact) of packed codes [..., d / 2] and scale bytes [..., d / GROUP]."""
    table = torch.tensor(E2M1_VALUES + tuple(-x for x in E2M1_VALUES) if kind == "e2m1" else
                         [float(i) for i in range(8)] + [float(i - 16) for i in range(8, 16)], device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    x = table[both.int()].unflatten(-1, (-1, GROUP)) * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return x.flatten(-2)


def _parts(cache):
    """Views of a cache's key codes, key scales, value codes and value scales [blocks, heads, records, TILE, bytes]."""
    d = cache.shape[-1] // 18
    return [cache[..., i:j].unflatten(-1, (TILE, -1)) for i, j in ((0, 8 * d), (8 * d, 9 * d), (9 * d, 17 * d), (17 * d, 18 * d))]


def _plain_tables(s):
    bs, table = s["block_size"], s["table"]
    ctx, new, free = s["ctx"].long(), s["new"].long(), s["count"].long()
    first, last = (ctx + bs - 1) // bs, (ctx + new + bs - 1) // bs
    fits = ctx + new <= table.shape[1] * bs
    need = torch.where(fits, last - first, 0)
    upto = need.cumsum(0)
    admitted = fits & ((need == 0) | (upto <= free))
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    taken = admitted[:, None] & (col >= first[:, None]) & (col < last[:, None])
    index = (free - 1 - (upto - need)[:, None] - (col - first[:, None])).clamp(0, s["free"].numel() - 1)
    table = torch.where(taken, s["free"][index], table)
    start = torch.cat([torch.zeros_like(free), new.cumsum(0)])
    t = torch.arange(s["slots"].numel(), device=table.device)
    real = t < start[-1]
    b = (torch.searchsorted(start, t, right=True) - 1).clamp(max=ctx.numel() - 1)
    pos = torch.where(real, ctx[b] + t - start[b], 0)
    block = table[b, (pos // bs).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(real & admitted[b] & (block >= 0), block * bs + pos % bs, -1)
    left = free - torch.where(admitted, upto, 0).amax()
    return (table, start.int(), torch.where(admitted, ctx + new, 0).int(), slots, pos.int(), left.int())


def _plain_write(s):
    cache, slots, kind = s["cache"], s["slots"], s["kind"]
    bs = cache.shape[2] * TILE
    real = slots >= 0
    at = torch.where(real, slots, cache.shape[0] * bs - 1)       # padding goes to a slot that no token has
    where = (at // bs, slice(None), at % bs // TILE, at % TILE)
    out = []
    parts = _parts(cache)
    for x, g, codes, scales in ((s["k"], s["k_scale"], parts[0], parts[1]), (s["v"], s["v_scale"], parts[2], parts[3])):
        codes[where], scales[where] = _quantise(x, g, kind)
        y = _values(codes[where], scales[where], kind) * g
        out.append(torch.where(real[:, None, None], y, 0.0).to(x.dtype))
    return tuple(out)


def _plain_attend(s):
    q, cache, table = s["q"], s["cache"], s["table"]
    start, lens = s["query_start"].long(), s["seq_lens"].long()
    b, h, d, most = table.shape[0], cache.shape[1], q.shape[2], s["most"]
    t = torch.arange(q.shape[0], device=q.device)
    of = torch.searchsorted(start, t, right=True) - 1
    row = t - start[of]
    count = start[1:] - start[:-1]
    padded = torch.zeros(b, most, q.shape[1], d, device=q.device)
    padded[of, row] = q.float()
    rows = padded.unflatten(2, (h, -1)).permute(0, 2, 3, 1, 4)                    # [b, h, share, most, d]
    pages = cache[table.clamp(min=0).long()].transpose(1, 2)                      # [b, h, blocks, records, bytes]
    kc, ks, vc, vs = (x.flatten(2, 4) for x in _parts(pages))                     # [b, h, tokens, bytes]
    score = rows.flatten(2, 3) @ (_values(kc, ks, s["kind"]).transpose(2, 3))
    score = score.unflatten(2, (-1, most)) * (s["sm_scale"] * s["k_scale"])
    token = torch.arange(kc.shape[2], device=q.device)
    last = (lens - count)[:, None] + torch.arange(most, device=q.device)[None, :]  # the last token that a row sees
    seen = token[None, None, :] <= last[:, :, None]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = score.sum(-1, keepdim=True)
    o = (score.flatten(2, 3) @ _values(vc, vs, s["kind"])).unflatten(2, (-1, most))
    o = o * s["v_scale"] / torch.where(total == 0, 1.0, total)
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3)[of, row].to(q.dtype)


def _plain_verify(s):
    target, draft, tokens, start, most = s["target"], s["draft"], s["tokens"].long(), s["start"].long(), s["most"]
    b, v = start.numel() - 1, target.shape[1]
    count = start[1:] - start[:-1]
    req = torch.arange(b, device=target.device)
    i = torch.arange(most, device=target.device)[None, :]
    row = (start[:-1, None] + i).clamp(max=max(0, tokens.numel() - 1))            # [b, most]
    token = tokens[row]
    # products of two 24-bit numbers: 64 bits hold them
    p = target[(row + req[:, None]), token].double()
    q = draft[row, token].double() if draft is not None else torch.ones_like(p)
    ok = (s["uniform"][row].double() * q < p) & (i < count[:, None])
    accepted = ok.long().cumprod(1).sum(1)
    at = start[:-1] + accepted
    rest = target[at + req].double()
    if draft is not None:
        last = draft[at.clamp(max=max(0, tokens.numel() - 1))].double()
        rest = torch.where((accepted < count)[:, None], (rest - last).clamp(min=0.0), rest)
    else:
        hit = tokens[at.clamp(max=max(0, tokens.numel() - 1))][:, None] == torch.arange(v, device=target.device)[None, :]
        rest = rest.masked_fill(hit & (accepted < count)[:, None], 0.0)
    rest = torch.where((rest.sum(1, keepdim=True) > 0), rest, target[at + req].double())
    upto = rest.cumsum(1)
    new = (upto <= s["sample"].double()[:, None] * upto[:, -1:]).sum(1).clamp(max=v - 1)
    j = torch.arange(most + 1, device=target.device)[None, :]
    token = torch.cat([token, torch.zeros_like(token[:, :1])], 1)
    out = torch.where(j < accepted[:, None], token, torch.where(j == accepted[:, None], new[:, None], -1))
    return out.int(), accepted.int()


# ---------------------------------------------------------------------------------------------------- the library's calls

def _own_run(s):
    import int8_w8a8_scaled_gb300 as w8
    op = s["op"]
    if op == "tables":
        w8.build_block_tables(s["ctx"], s["new"], s["free"], s["count"], s["table"], s["block_size"], s["query_start"],
                              s["seq_lens"], s["slots"], s["positions"], s["free_left"])
        return s["table"], s["query_start"], s["seq_lens"], s["slots"], s["positions"], s["free_left"]
    if op == "write":
        w8.kv4_cache_write(s["k"], s["v"], s["cache"], s["slots"], s["k_scale"], s["v_scale"], kind=s["kind"])
        w8.kv4_cache_read(s["cache"], s["slots"], s["k_scale"], s["v_scale"], s["k_out"], s["v_out"], kind=s["kind"])
        return s["k_out"], s["v_out"]
    if op == "attend":
        w8.kv4_attention(s["q"], s["cache"], s["seq_lens"], s["table"], s["k_scale"], s["v_scale"], s["out"],
                         query_start=s["query_start"], max_query_len=s["most"], sm_scale=s["sm_scale"], kind=s["kind"])
        return s["out"]
    w8.verify_drafts(s["target"], s["draft"], s["tokens"], s["start"], s["uniform"], s["sample"], s["out_tokens"], s["accepted"])
    return s["out_tokens"], s["accepted"]


def run(state):
    if own:
        return _own_run(state)
    return {"tables": _plain_tables, "write": _plain_write, "attend": _plain_attend, "verify": _plain_verify}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "tables":
        b, tokens = case["batch"], int(_new_lengths(case).sum())
        ids = tokens / case["block_size"]
        return {"bytes": int(16 * b + 12 * tokens + 8 * ids), "flops": int(10 * b + 4 * tokens)}
    if op == "write":
        n = 2 * case["tokens"] * case["heads"] * case["head_dim"]
        # the inputs, the codes and scales written and read, the values
        return {"bytes": int(n * (2 + 2 * 0.5625 + 2) + 16 * case["tokens"]), "flops": 12 * n}
    if op == "attend":
        ctx, new = _lengths(case)
        hq, h, d = case["q_heads"], case["kv_heads"], case["head_dim"]
        pairs = int((new * ctx + new * (new + 1) // 2).sum())
        return {"bytes": int((ctx + new).sum() * h * d * 2 * 0.5625 + 4 * new.sum() * hq * d + 4 * (ctx + new).sum() / case["block_size"]),
                "flops": 4 * pairs * hq * d}
    size = {"fp32": 4, "bf16": 2}[case["dtype"]]
    b, v = case["batch"], case["vocab"]
    # one row of the target for each request, and one of the draft for those with a rejection
    return {"bytes": int(b * v * size * (1 if case["greedy"] else 2)), "flops": 4 * b * v}


# ---------------------------------------------------------------------------------------------------- 64 bits

def _e4m3(x):
    """Nearest e4m3 value (ties to even) of 64-bit numbers in [2^-9, 448]."""
    e = torch.floor(torch.log2(x)).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_write(s):
    out = []
    levels = torch.tensor(E2M1_VALUES, dtype=torch.float64, device="cuda")
    for x, g in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        g = g.double()
        y = x.double().reshape(x.shape[0], x.shape[1], -1, GROUP)
        scale = _e4m3((y.abs().amax(3, keepdim=True) / (LARGEST[s["kind"]] * g)).clamp(2.0 ** -9, 448.0)) * g
        y = y / scale
        if s["kind"] == "int4":
            y = torch.round(y).clamp(-7, 7)
        else:
            far = (y.abs().unsqueeze(-1) - levels).abs()
            # of two equally near levels the one with the even index
            near = (far + 1e-12 * (torch.arange(8, device="cuda") % 2)).argmin(-1)
            y = torch.copysign(levels[near], y)
        y = (y * scale).reshape(x.shape)
        y[s["slots"] < 0] = 0.0
        out.append(y)
    return tuple(out)


def _exact_attend(s):
    q, cache, kind = s["q"], s["cache"], s["kind"]
    h, d, bs = cache.shape[1], q.shape[2], cache.shape[2] * TILE
    share = q.shape[1] // h
    start, lens = s["query_start"].tolist(), s["seq_lens"].tolist()
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    e2m1 = torch.tensor(E2M1_VALUES, dtype=torch.float64, device="cuda")

    def rows(page, at, n):
        """Tokens 0..n-1 of one request and head in 64 bits, from its records [records, 18 d]."""
        raw = page[:, at:at + 8 * d].reshape(-1, d // 2)[:n].int()
        code = torch.stack((raw % 16, raw // 16), 2).reshape(n, d)
        x = (torch.where(code >= 8, code - 16, code).double() if kind == "int4" else
             torch.where(code >= 8, -1.0, 1.0).double() * e2m1[(code % 8).long()])
        byte = page[:, at + 8 * d:at + 9 * d].reshape(-1, d // GROUP)[:n].int()
        e, m = byte // 8 % 16, byte % 8
        scale = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)
        return x * scale.repeat_interleave(GROUP, 1)

    for b, n in enumerate(lens):
        first, count = start[b], start[b + 1] - start[b]
        ids = s["table"][b, :-(-n // bs)].long()
        for head in range(h):
            page = cache[ids, head].reshape(-1, 18 * d)
            k, v = rows(page, 0, n) * s["k_scale"].double(), rows(page, 9 * d, n) * s["v_scale"].double()
            for i in range(0, count, 512):
                part = q[first + i:min(first + i + 512, first + count), head * share:(head + 1) * share].double()
                score = torch.einsum("igd,td->igt", part, k) * s["sm_scale"]
                limit = n - count + i + torch.arange(part.shape[0], device="cuda")
                score = score.masked_fill(torch.arange(n, device="cuda") > limit[:, None, None], -math.inf)
                out[first + i:first + i + part.shape[0], head * share:(head + 1) * share] = torch.softmax(score, 2) @ v
    return out


def _exact_tables(s):
    ctx, new, free = s["ctx"].tolist(), s["new"].tolist(), s["free"].tolist()
    bs, table = s["block_size"], s["table"].cpu().numpy().copy()
    count, upto, left = int(s["count"]), 0, int(s["count"])
    slots, positions = np.full(s["slots"].numel(), -1, np.int64), np.zeros(s["slots"].numel(), np.int32)
    start, lens = [0], []
    for b, (c, n) in enumerate(zip(ctx, new)):
        first, last = -(-c // bs), -(-(c + n) // bs)
        fits = c + n <= table.shape[1] * bs
        need = last - first if fits else 0
        ok = fits and (need == 0 or upto + need <= count)
        if ok:
            table[b, first:last] = [free[count - 1 - upto - i] for i in range(need)]
            left = min(left, count - upto - need)
            t = np.arange(c, c + n)
            slots[start[-1]:start[-1] + n] = table[b, t // bs].astype(np.int64) * bs + t % bs
        positions[start[-1]:start[-1] + n] = np.arange(c, c + n)
        upto += need
        lens.append(c + n if ok else 0)
        start.append(start[-1] + n)
    as32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32)  # noqa: E731
    return as32(table), as32(start), as32(lens), torch.from_numpy(slots), torch.from_numpy(positions), as32([left])


def _exact_verify(s):
    start, tokens = s["start"].tolist(), s["tokens"].tolist()
    uniform, sample = s["uniform"].tolist(), s["sample"].tolist()
    out = np.full((len(start) - 1, s["most"] + 1), -1, np.int32)
    accepted = np.zeros(len(start) - 1, np.int32)
    for b in range(len(start) - 1):
        n, i = start[b + 1] - start[b], 0
        while i < n:
            row, token = start[b] + i, tokens[start[b] + i]
            q = float(s["draft"][row, token]) if s["draft"] is not None else 1.0
            if not uniform[row] * q < float(s["target"][row + b, token]):
                break
            out[b, i] = token
            i += 1
        accepted[b] = i
        p = s["target"][start[b] + b + i].double().cpu().numpy()
        rest = p.copy()
        if i < n and s["draft"] is not None:
            rest = np.maximum(p - s["draft"][start[b] + i].double().cpu().numpy(), 0.0)
        elif i < n:
            rest[tokens[start[b] + i]] = 0.0
        c = np.cumsum(rest if rest.sum() > 0 else p)
        out[b, i] = min(int(np.searchsorted(c, sample[b] * c[-1], side="right")), len(c) - 1)
    return torch.from_numpy(out), torch.from_numpy(accepted)


def exact(case, seed):
    if case["op"] == "attend" and work(case)["flops"] > 2e12:
        return None
    return {"tables": _exact_tables, "write": _exact_write, "attend": _exact_attend,
            "verify": _exact_verify}[case["op"]](prepare(case, seed))
