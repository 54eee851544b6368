"""Block tables where the packed tokens are too few for all requests."""
import numpy as np
import pytest
import torch

import int8_w8a8_scaled_gb300 as w8
from oracle import kv4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch", [1, 3, 300, 3000])
@pytest.mark.parametrize("part", [0.0, 0.5, 0.97])
def test_requests_past_the_packed_tokens_are_refused(batch, part):
    """Refused like those that the free list has no blocks for, and nothing of
    their tables is written; requests without new tokens stay admitted."""
    rng = np.random.default_rng(batch)
    bs, mb = 16, 9
    ctx, new = rng.integers(0, 90, batch).astype(np.int32), rng.integers(0, 40, batch).astype(np.int32)
    new[0] = 17
    tokens = max(1, int(part * new.sum()))
    held = -(-ctx // bs)
    ids = rng.permutation(10 * batch).astype(np.int32)
    table = np.full((batch, mb), -7, np.int32)
    table[np.arange(mb)[None] < held[:, None]] = ids[:held.sum()]
    free = ids[held.sum():]
    gpu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    out = [torch.full((n,), -9, dtype=t, device="cuda") for n, t in
           ((batch + 1, torch.int32), (batch, torch.int32), (tokens, torch.int64), (tokens, torch.int32), (1, torch.int32), (1, torch.int32))]
    got = gpu(table)
    w8.build_block_tables(gpu(ctx), gpu(new), gpu(free), gpu(np.int32([len(free)])), got, bs, *out)
    want = kv4.block_tables(ctx, new, free, len(free), table, bs, tokens)
    refused = want[2] == 0
    assert refused[new > 0].any() and not refused[(new == 0) & (ctx > 0)].any()
    # an admitted request's new blocks are all in its table
    for b in np.nonzero(~refused)[0]:
        assert (want[0][b, :-(-(ctx[b] + new[b]) // bs)] >= 0).all()
    assert np.array_equal(got.cpu().numpy(), want[0])
    for x, ref in zip(out, want[1:]):
        assert np.array_equal(x.cpu().numpy(), np.atleast_1d(ref))
