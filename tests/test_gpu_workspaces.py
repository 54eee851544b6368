"""Default workspaces of calls on explicit streams."""
import numpy as np
import pytest
import torch

import int8_w8a8_scaled_gb300 as w8
from int8_w8a8_scaled_gb300 import api

pytestmark = pytest.mark.gpu


def attention_problem(new, seed):
    """Requests that are cut between CTAs, and a call of them into `out`."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens = [3000, 900, 1700]
    blocks = [-(-n // 16) for n in lens]
    nb = sum(blocks)
    cache = torch.zeros(w8.kv4_cache_shape(nb, 2, 16, 128), dtype=torch.uint8, device="cuda")
    k, v = (torch.randn(nb * 16, 2, 128, generator=gen, device="cuda").bfloat16() for _ in range(2))
    scale = torch.full((1,), 0.013, device="cuda")
    w8.kv4_cache_write(k, v, cache, torch.arange(nb * 16, device="cuda"), scale, scale)
    table = torch.full((3, max(blocks)), -1, dtype=torch.int32)
    for b, n in enumerate(blocks):
        table[b, :n] = torch.arange(n) + sum(blocks[:b])
    table, lens = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn(3 * new, 8, 128, generator=gen, device="cuda").bfloat16()
    start = torch.arange(4, dtype=torch.int32, device="cuda") * new

    def call(out, **kw):
        w8.kv4_attention(q, cache, lens, table, scale, scale, out, query_start=start, max_query_len=new, **kw)
    return call, q


def matmul_problem(seed):
    """A matmul with split K, whose parts meet on the workspace's counters."""
    rng = np.random.default_rng(seed)
    M, N, K = 64, 512, 8192
    a, b = (torch.from_numpy(rng.integers(0, 120, (r, K)).astype(np.uint8)).cuda().view(torch.float8_e4m3fn) for r in (M, N))
    one = torch.ones(1, device="cuda")
    cfg = {"swap_ab": 1, "block_n": 64, "split_k": 4, "reduce": w8.REDUCE_GLOBAL}
    assert w8.mm_workspace_size(M, N, K, config=cfg) > 0

    def call(out, **kw):
        w8.scaled_mm(a, b, one, one, out, config=cfg, **kw)
    return call, torch.empty(M, N, device="cuda")


PROBLEMS = {"one": lambda seed: attention_problem(1, seed), "chunk": lambda seed: attention_problem(60, seed), "matmul": matmul_problem}


@pytest.fixture
def no_workspaces(monkeypatch):
    """No default workspace is there yet, and fresh memory is not zero."""
    monkeypatch.setattr(api, "_default_ws", {})
    torch.cuda.synchronize()
    junk = [torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del junk


@pytest.mark.parametrize("problem", PROBLEMS)
def test_two_explicit_streams_with_default_workspaces(problem, no_workspaces):
    calls = [PROBLEMS[problem](seed) for seed in (1, 2)]
    wants = []
    for call, like in calls:
        wants.append(torch.empty_like(like))
        call(wants[-1])
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [[torch.full_like(like, float("nan")) for _ in range(30)] for _, like in calls]
    torch.cuda.synchronize()
    for i in range(30):
        for (call, _), stream, out in zip(calls, streams, outs):
            call(out[i], stream=stream)
    torch.cuda.synchronize()
    for want, out in zip(wants, outs):
        assert all(torch.equal(o, want) for o in out)
    assert w8.device_status() == 0


@pytest.mark.parametrize("problem", PROBLEMS)
def test_graphs_captured_without_a_workspace(problem, no_workspaces):
    """Two graphs, captured one after the other with no call before them, and the
    second one replayed first, with calls outside between."""
    (first, like), (second, _) = (PROBLEMS[problem](seed) for seed in (1, 2))
    outs = [torch.empty_like(like) for _ in range(4)]
    graphs = []
    for call, out in zip((first, second), outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(out)
            call(out)
    with torch.cuda.stream(torch.cuda.graph.default_capture_stream):
        second(outs[3])
    torch.cuda.synchronize()
    second(outs[2])
    torch.cuda.synchronize()
    assert torch.equal(outs[2], outs[3])
    for _ in range(3):
        outs[1].fill_(0)
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[1], outs[2])
    first(outs[2])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2])


def test_a_graph_outlives_the_growth_of_its_default_workspace(no_workspaces):
    call, like = attention_problem(1, 3)
    large, like_large = attention_problem(60, 4)
    out, want = torch.empty_like(like), torch.empty_like(like)
    call(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(out, stream=s)                                 # the stream's workspace, made before the capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(out)
    with torch.cuda.stream(s):
        large(torch.empty_like(like_large))             # it grows
        junk = torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device="cuda")
        for _ in range(3):
            out.fill_(0)
            g.replay()
            assert torch.equal(out, want)
        assert (junk == 0xFF).all()


@pytest.mark.parametrize("problem", PROBLEMS)
def test_a_workspace_of_another_stream_given_up_at_once(problem, no_workspaces):
    """Made on the current stream behind much other work, used on another one, and
    dropped while that call runs."""
    call, like = PROBLEMS[problem](5)
    want = torch.empty_like(like)
    call(want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [torch.empty_like(like) for _ in range(20)]
    for out in outs:
        torch.cuda._sleep(200000)
        call(out, stream=s, workspace=w8.Workspace(64 << 20))
        torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs)
