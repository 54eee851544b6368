"""How the operators over the paged fp8 cache are called: on several streams and
host threads, in graphs, with workspaces of their caller's, with NaN scales, and
with steps of random shapes (tolerances as in test_gpu_fp8_paged.py)."""
import threading

import numpy as np
import pytest
import torch

import int8_w8a8_scaled_gb300 as w8
from int8_w8a8_scaled_gb300 import api
from oracle import fp8_paged as fp
from test_gpu_fp8_paged import E4M3, Step, dev, random_columns

pytestmark = pytest.mark.gpu


@pytest.fixture
def no_workspaces(monkeypatch):
    """No default workspace is there yet, and fresh memory is not zero."""
    monkeypatch.setattr(api, "_default_ws", {})
    torch.cuda.synchronize()
    junk = [torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del junk


def call_of(s, selected=None):
    """A call into `out`, its tensors made."""
    args = [s.q.cuda(), dev(s.kc).view(E4M3), dev(s.vc).view(E4M3), dev(s.lens), dev(s.table)]
    if selected is not None:
        args.append(dev(selected))
    args += [dev(np.float32([s.kg])), dev(np.float32([s.vg]))]
    kw = dict(query_start=dev(s.start), max_query_len=s.most, sm_scale=s.sm)
    op = w8.fp8_kv_attention if selected is None else w8.fp8_kv_sparse_attention
    torch.cuda.synchronize()
    return lambda out, **more: op(*args, out, **kw, **more)


def problem(kind, seed=60):
    """Units that are cut between CTAs, so that the workspace's counters are used."""
    s = Step(seed, [3000, 900, 1700], {"few": [3, 1, 2], "chunk": [60, 1, 80], "sparse": [3, 1, 2]}[kind], 8, 2, 128, 16)
    sel = random_columns(s, 40, s.rng) if kind == "sparse" else None
    return s, sel, call_of(s, sel), torch.empty(s.q.shape, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("kind", ["few", "chunk", "sparse"])
def test_a_streams_first_call(no_workspaces, kind):
    s, sel, call, out = problem(kind)
    stream = torch.cuda.Stream()
    call(out, stream=stream)
    stream.synchronize()
    s.check(out, selected=sel)


@pytest.mark.parametrize("kind", ["few", "chunk", "sparse"])
def test_calls_on_several_streams_at_once(no_workspaces, kind):
    s, sel, call, first = problem(kind)
    call(first)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty_like(first) for _ in streams]
    for _ in range(5):
        for stream, out in zip(streams, outs):
            with torch.cuda.stream(stream):
                call(out)
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, first)
    assert w8.device_status() == 0


@pytest.mark.parametrize("kind", ["few", "chunk", "sparse"])
def test_a_workspace_of_the_callers(kind):
    """One for calls of growing needs, in a graph and beside it, and a plain zeroed buffer."""
    ws = w8.Workspace(256)
    s, sel, call, first = problem(kind)
    call(first)
    out = torch.zeros_like(first)
    call(out, workspace=ws)
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, workspace=ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)
    need = (w8.fp8_kv_sparse_attention_workspace_size(s.tokens, 8, 2, 128, 40, 16) if kind == "sparse" else
            w8.fp8_kv_attention_workspace_size(3, s.most, 8, 2, 128))
    buf = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        out.zero_()
        call(out, workspace=buf)
        assert torch.equal(out, first)
    with pytest.raises(w8.W8A8Error):
        call(out, workspace=buf[:need - 16])


def test_host_threads():
    """Calls of different sizes from several threads, each on a stream of its own."""
    problems = [problem(kind, 61 + i) for i, kind in enumerate(("few", "chunk", "sparse", "few"))]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                problems[i][2](problems[i][3], stream=stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(problems))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for s, sel, _, out in problems:
        s.check(out, selected=sel)
    assert w8.device_status() == 0


@pytest.mark.parametrize("new", [[2, 5], [60, 100]])
@pytest.mark.parametrize("scale", ["k", "v", "sm"])
def test_a_nan_scale_gives_nan(new, scale):
    s = Step(62, [300, 270], new, 8, 2, 128, 16)
    if scale == "k":
        s.kg = float("nan")
    elif scale == "v":
        s.vg = float("nan")
    else:
        s.sm = float("nan")
    assert torch.isnan(s.run()).all()
    if new[0] < 10:
        assert torch.isnan(s.run(selected=random_columns(s, 6, s.rng) * 0)).all()


@pytest.mark.parametrize("seed", range(16))
def test_steps_of_random_shapes(seed):
    rng = np.random.default_rng(1000 + seed)
    h, d, bs = int(rng.choice([1, 2, 3, 8])), int(rng.choice([64, 128])), int(rng.choice([16, 32, 48, 80, 128]))
    hq = h * int(rng.choice([1, 2, 3, 5, 8, 12][:6 if h < 3 else 3]))
    batch = int(rng.integers(1, 5))
    new = rng.choice([0, 1, 1, 2, 5, 9, 40, 70], batch)
    new[0] = max(1, new[0])
    lens = new + rng.integers(0, 700, batch)
    if seed % 4 == 3:
        lens = np.maximum(lens - 20, 0)                      # rows in front of the first token
    s = Step(2000 + seed, lens, new, hq, h, d, bs, str(rng.choice(["bf16", "fp16"])), extra_rows=int(rng.integers(0, 3)), tail=0x7F)
    if seed % 3 == 0:
        s.table[rng.random(s.table.shape) < 0.1] = -1
    layout = str(rng.choice(["plain", "merged", "odd", "heads_first"]))
    s.check(s.run(layout))
    sel = random_columns(s, int(rng.integers(1, 12)), rng)
    s.check(s.run(layout, selected=sel), selected=sel)
    means, scales = rng.integers(-127, 128, (s.nb, h, d)).astype(np.int8), (rng.random((s.nb, h)) + 0.1).astype(np.float32)
    budget = int(rng.integers(2, 9))
    got = torch.full((s.q.shape[0], h, budget), -9, dtype=torch.int32, device="cuda")
    w8.fp8_kv_select_blocks(s.q.cuda(), dev(means), dev(scales), dev(s.lens), dev(s.table), bs, got, query_start=dev(s.start),
                            max_query_len=s.most, first_blocks=1, last_blocks=1)
    want = fp.select(s.q.float().numpy(), means, scales, s.lens, s.table, bs, s.start, s.most, 1, 1, budget,
                     np.full(got.shape, -9, np.int32))
    assert np.array_equal(got.cpu().numpy(), want)
    assert w8.device_status() == 0


def test_blocks_past_four_gigabytes():
    """The same step over a small cache and over the last blocks of one of 4.6 GB each for K and V: the same bits."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("two caches of 4.6 GB")
    hq, h, d, bs, tokens = 16, 8, 128, 64, 75
    rng = np.random.default_rng(70)
    lens, new = np.int32([700, 130]), np.int32([3, 72])
    small, large = 16, 70000                                 # blocks of 64 KB
    table = np.full((2, 11), -1, np.int32)
    table[0], table[1, :3] = rng.permutation(small)[:11], [0, 0, 0]
    table[1, :3] = np.setdiff1d(np.arange(small), table[0])[:3]
    start = dev(np.int32([0, 3, 75]))
    codes = [torch.from_numpy(fp.encode(np.float32(rng.standard_normal((small, bs, h, d)) * 20))).cuda() for _ in range(2)]
    q, k, v = (torch.from_numpy(np.float32(rng.standard_normal((tokens, n, d)))).bfloat16().cuda() for n in (hq, h, h))
    angle = rng.uniform(-3, 3, (700, d // 2))
    cos_sin = dev(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32))
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)]).astype(np.int32)
    row = np.repeat([0, 1], new)
    g = torch.full((1,), 0.02, device="cuda")

    def step(blocks):
        first = blocks - small
        caches = [torch.zeros(blocks, bs, h, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
        for cache, part in zip(caches, codes):
            cache[first:] = part
        ids = np.where(table >= 0, table + first, -1).astype(np.int32)
        slots = ids[row, pos // bs].astype(np.int64) * bs + pos % bs
        means, scales = torch.zeros(blocks, h, d, dtype=torch.int8, device="cuda"), torch.zeros(blocks, h, device="cuda")
        turned, whole, sparse = (torch.zeros_like(q) for _ in range(3))
        few = torch.zeros_like(q[:3])
        sel = torch.zeros(tokens, h, 5, dtype=torch.int32, device="cuda")
        seq, ids = dev(lens), dev(ids)
        w8.fp8_kv_rotate_write(q, k, v, cos_sin, dev(pos), *caches, dev(slots), g, g, turned)
        kw = dict(query_start=start, max_query_len=72)
        w8.fp8_kv_block_means(caches[0], seq, ids, means, scales, query_start=dev(np.int32([0, 700, 830])), max_query_len=700)
        w8.fp8_kv_attention(turned, *caches, seq, ids, g, g, whole, **kw)
        w8.fp8_kv_attention(turned[:3], *caches, seq[:1], ids[:1], g, g, few, query_start=start[:2], max_query_len=3)
        w8.fp8_kv_select_blocks(turned, means, scales, seq, ids, bs, sel, **kw)
        w8.fp8_kv_sparse_attention(turned, *caches, seq, ids, sel, g, g, sparse, **kw)
        assert w8.device_status() == 0
        return [c[first:].clone() for c in (*caches, means, scales)] + [turned, whole, few, sel, sparse]

    for a, b in zip(step(small), step(large)):
        assert a.abs().max() > 0 if a.is_floating_point() else (a != 0).any()
        assert torch.equal(a, b)
