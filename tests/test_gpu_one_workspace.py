"""One Workspace for the operators of a step, one after the other on a stream: the
arrival counters at its head are zero after each call, and every result is that
of a call with a workspace of its own."""
import numpy as np
import pytest
import torch

import int8_w8a8_scaled_gb300 as w8
from oracle import fp8_paged as fp
from test_gpu_fp8_paged import Step, dev, random_columns
from test_gpu_workspaces import attention_problem, matmul_problem

pytestmark = pytest.mark.gpu
COUNTERS = 65536                                             # bytes at the head of a workspace


def select_into(s, selected, workspace, budget_first=1, last=2):
    rng = np.random.default_rng(7)
    means, scales = rng.integers(-127, 128, (s.nb, s.h, s.d)).astype(np.int8), (rng.random((s.nb, s.h)) + 0.1).astype(np.float32)
    w8.fp8_kv_select_blocks(s.q.cuda(), dev(means), dev(scales), dev(s.lens), dev(s.table), s.bs, selected, query_start=dev(s.start),
                            max_query_len=s.most, first_blocks=budget_first, last_blocks=last, workspace=workspace)
    return means, scales


@pytest.mark.parametrize("lens,new,budget,columns", [
    ([3000, 900, 1700], [3, 1, 2], 20, 0),                   # scores of a few rows
    ([500, 40, 0, 16], [300, 5, 0, 1], 4, 0),                # most of the counters' bytes, and rows with fewer blocks than the budget
    ([60, 40, 900], [60, 40, 300], 6, 40000),                # several slabs of rows of 160 KB
])
def test_a_selection_leaves_the_counters_zero(lens, new, budget, columns):
    s = Step(81, lens, new, 8, 2, 128, 16, extra_rows=2)
    if columns:
        s.table = np.concatenate([s.table, np.full((len(lens), columns - s.table.shape[1]), -1, np.int32)], 1)
    ws = w8.Workspace()
    selected = torch.full((s.q.shape[0], 2, budget), -9, dtype=torch.int32, device="cuda")
    means, scales = select_into(s, selected, ws)
    want = fp.select(s.q.float().numpy(), means, scales, s.lens, s.table, 16, s.start, s.most, 1, 2, budget,
                     np.full(selected.shape, -9, np.int32))
    assert np.array_equal(selected.cpu().numpy(), want)
    assert not ws.buf[:COUNTERS].any()


@pytest.mark.parametrize("kind", ["few", "chunk", "sparse"])
def test_a_selection_and_attention_share_a_workspace(kind):
    """Attention of units that are cut between CTAs, which meet on the counters."""
    s = Step(82, [3000, 900, 1700], [60, 1, 80] if kind == "chunk" else [3, 1, 2], 8, 2, 128, 16)
    ws = w8.Workspace(64 << 20)
    selected = torch.full((s.q.shape[0], 2, 30), -9, dtype=torch.int32, device="cuda")
    select_into(s, selected, ws)
    sel = random_columns(s, 40, s.rng) if kind == "sparse" else None
    out = s.run(selected=sel, workspace=ws)
    s.check(out, selected=sel)
    assert torch.equal(out, s.run(selected=sel))


@pytest.mark.parametrize("kind", ["few", "chunk", "sparse"])
def test_attention_leaves_the_matmuls_counters_zero(kind):
    s = Step(83, [3000, 900, 1700], [60, 1, 80] if kind == "chunk" else [3, 1, 2], 8, 2, 128, 16)
    ws = w8.Workspace(64 << 20)
    sel = random_columns(s, 40, s.rng) if kind == "sparse" else None
    s.check(s.run(selected=sel, workspace=ws), selected=sel)
    assert not ws.buf[:COUNTERS].any()


@pytest.mark.parametrize("batch,tokens,paged", [(1, 5000, False), (4, 700, True), (3, 1, False)])
def test_decode_attention_leaves_the_counters_zero(batch, tokens, paged):
    gen = torch.Generator(device="cuda").manual_seed(85)
    hq, h, bs = 8, 2, 16
    nb = -(-tokens // bs) * batch
    shape = (nb, bs, h, 128) if paged else (batch, tokens, h, 128)
    k, v = (torch.randint(0, 126, shape, generator=gen, device="cuda", dtype=torch.uint8) for _ in range(2))
    table = torch.arange(nb, dtype=torch.int32, device="cuda").view(batch, -1) if paged else None
    q = torch.randn(batch, hq, 128, generator=gen, device="cuda").bfloat16()
    lens = torch.tensor([tokens, tokens // 2, 0, 1][:batch], dtype=torch.int32, device="cuda")
    one = torch.full((1,), 0.02, device="cuda")
    ws = w8.Workspace(64 << 20)
    outs = [torch.empty_like(q) for _ in range(2)]
    for out, workspace in zip(outs, (ws, None)):
        w8.fp8_kv_decode_attention(q, k, v, lens, one, one, out, block_table=table, workspace=workspace)
    assert not ws.buf[:COUNTERS].any()
    assert torch.equal(*outs)


@pytest.mark.parametrize("new", [1, 3, 60])
def test_attention_over_the_4_bit_cache_leaves_the_matmuls_counters_zero(new):
    call, like = attention_problem(new, 84)
    ws = w8.Workspace(64 << 20)
    outs = [torch.empty_like(like) for _ in range(2)]
    call(outs[0], workspace=ws)
    assert not ws.buf[:COUNTERS].any()
    call(outs[1])
    assert torch.equal(*outs)


def test_a_step_on_one_workspace():
    """Matmuls with split K, selection and every attention in turn, three times."""
    s = Step(86, [3000, 900, 1700], [3, 1, 2], 8, 2, 128, 16)
    chunk = Step(87, [3000, 900, 1700], [60, 1, 80], 8, 2, 128, 16)
    sel = random_columns(s, 40, s.rng)
    matmul, product = matmul_problem(88)
    kv4, rows = attention_problem(60, 89)
    selected = [torch.full((s.q.shape[0], 2, 30), -9, dtype=torch.int32, device="cuda") for _ in range(2)]
    products, fours = ([torch.empty_like(x) for _ in range(2)] for x in (product, rows))

    def step(i, ws):
        matmul(products[i], workspace=ws)
        select_into(s, selected[i], ws)
        a = s.run(selected=sel, workspace=ws)
        matmul(products[i], workspace=ws)
        b = chunk.run(workspace=ws)
        kv4(fours[i], workspace=ws)
        matmul(products[i], workspace=ws)
        return a, b, s.run(workspace=ws)

    want = step(0, None)
    ws = w8.Workspace(128 << 20)
    for _ in range(3):
        got = step(1, ws)
        for a, b in zip((*want, products[0], selected[0], fours[0]), (*got, products[1], selected[1], fours[1])):
            assert torch.equal(a, b)
    assert not ws.buf[:COUNTERS].any() and w8.device_status() == 0
