"""The four operators of a serving step together, as examples/paged_step.py
runs them."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def blocks_of(server):
    held = [row[:-(-n // 16)] for row, n in zip(server.table.tolist(), server.held.tolist())]
    rest = [row[-(-n // 16):] for row, n in zip(server.table.tolist(), server.held.tolist())]
    return held, rest, server.free[:int(server.free_count)].tolist()


@pytest.mark.parametrize("kind,drafts", [("e2m1", 3), ("int4", 0), ("e2m1", 5)])
def test_steps_keep_their_books(kind, drafts):
    import paged_step
    server, texts = paged_step.main(["--steps", "10", "--drafts", str(drafts), "--kind", kind])
    assert all(0 <= t < paged_step.VOCAB for text in texts for t in text)
    # the last token of a text is not cached yet
    assert server.held.tolist() == [p + len(t) - 1 for p, t in zip((40, 7, 1, 23), texts)]
    held, rest, free = blocks_of(server)
    assert sorted(sum(held, []) + free) == list(range(64))       # every block once
    assert all(x == -1 for row in rest for x in row)


def test_steps_and_one_prompt_agree():
    """The logits after several steps, with rejections between, against those
    of the same text taken in at once: the same cache up to the noise of
    rounding keys and values to 4 bits."""
    import paged_step
    server = paged_step.Server(4, 64, seed=3)
    prompts = [list(range(1, n + 1)) for n in (30, 12, 5, 17)]
    last = server.prompt(prompts)
    texts = [p + [t] for p, t in zip(prompts, last.tolist())]
    for _ in range(4):
        out, accepted = server.step(last, 3)
        last = out.gather(1, accepted[:, None].long())[:, 0]
        for text, row, n in zip(texts, out.tolist(), accepted.tolist()):
            text += row[:n + 1]
    one = torch.ones(4, dtype=torch.int32, device="cuda")
    stepped, _ = server.forward(last, one, 1)
    again = paged_step.Server(4, 64, seed=3)
    new = torch.tensor([len(t) for t in texts], dtype=torch.int32, device="cuda")
    logits, start = again.forward(torch.cat([torch.tensor(t, dtype=torch.int32) for t in texts]).cuda(), new, max(map(len, texts)))
    whole = logits[start[1:].long() - 1]
    assert torch.equal(server.allocated, again.allocated)
    assert (torch.nn.functional.cosine_similarity(stepped, whole, 1) > 0.98).all()
