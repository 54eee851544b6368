"""Block tables refuse outputs that lie over inputs or over each other, before
any CUDA call."""
import itertools

import pytest

from int8_w8a8_scaled_gb300 import _lib

INVALID = 1
BATCH, BLOCKS, TOKENS, CAPACITY = 5, 8, 12, 30
# name: bytes
READ = {"ctx": 4 * BATCH, "new": 4 * BATCH, "free": 4 * CAPACITY, "count": 4}
WRITTEN = {"table": 4 * BATCH * BLOCKS, "start": 4 * (BATCH + 1), "lens": 4 * BATCH, "slots": 8 * TOKENS, "pos": 4 * TOKENS,
           "left": 4, "after": 4}
PLACE = {name: 0x7F0000000000 + 0x10000 * i for i, name in enumerate([*READ, *WRITTEN])}   # never dereferenced


def call(**edit):
    p = {**PLACE, **edit}
    return _lib.load().w8a8_build_block_tables(p["ctx"], p["new"], BATCH, p["free"], p["count"], CAPACITY, p["table"], BLOCKS, 16,
                                               p["start"], p["lens"], p["slots"], p["pos"], TOKENS, p["left"], p["after"], None)


@pytest.mark.parametrize("name,other", [*itertools.product(WRITTEN, READ), *itertools.combinations(WRITTEN, 2)])
def test_no_output_may_lie_over(name, other):
    size = {**READ, **WRITTEN}
    # at the same place, on its last element, and ending in its first
    for at in (0, (size[other] - 1) // 8 * 8, -(size[name] - 1) // 8 * 8 + 8 if size[name] > 8 else 0):
        assert call(**{name: PLACE[other] + at}) == INVALID
        assert b"over" in _lib.load().w8a8_last_error() or b"different words" in _lib.load().w8a8_last_error()
