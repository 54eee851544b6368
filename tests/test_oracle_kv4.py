"""Pins of the 4-bit serving step's oracle: closed forms and brute force."""
import numpy as np
import pytest

from oracle import kv4


@pytest.mark.parametrize("x,index", [(0.25, 0), (0.2500001, 1), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6),
                                     (5.01, 7), (6.0, 7), (0.0, 0)])
def test_e2m1_halves_go_to_the_even_code(x, index):
    assert kv4.nearest_even(np.array([x]), kv4.E2M1)[0] == index


def test_quantise_closed_forms():
    x = np.array([6.0, -6.0, 3.0, 0.5, 0.25, -0.0, 2.5, 100.0] + [0.0] * 8, np.float32)
    x[7] = 5.0
    codes, s = kv4.quantise(x, 1.0, "e2m1")                  # absmax 6: scale 1 (code 0x38)
    assert s.tolist() == [0x38]
    assert codes[:8].tolist() == [7, 15, 5, 1, 0, 8, 4, 6]
    codes, s = kv4.quantise(x * np.float32(7 / 6), 7 / 6, "int4")
    v = kv4.values(codes, s, 7 / 6, "int4")
    assert np.all(np.abs(v - x * 7 / 6) <= 0.5 * 7 / 6 * kv4.E4M3[s[0]] + 1e-6)


@pytest.mark.parametrize("kind", ["e2m1", "int4"])
def test_zero_nan_and_infinite_groups(kind):
    x = np.zeros((3, 16), np.float32)
    x[1, 3], x[1, 4] = np.nan, 1.0
    x[2, 0], x[2, 1] = -np.inf, 5.0
    codes, s = kv4.quantise(x, 0.01, kind)
    assert s[0, 0] == 1 and not codes[0].any()               # the smallest scale, 2^-9
    assert codes[1, 3] == 0 and codes[1, 4] == 7
    assert s[2, 0] == 126 and codes[2, 0] == (15 if kind == "e2m1" else 9)


def test_layout_holds_every_token():
    rng = np.random.default_rng(0)
    cache = np.zeros((3, 2, 2, 18 * 64), np.uint8)
    k, v = rng.standard_normal((2, 96, 2, 64)).astype(np.float32)
    slots = rng.permutation(96)
    cache = kv4.write(cache, slots, k, v, 0.01, 0.02, "int4")
    gk, gv = kv4.tokens_of(cache, slots, 0.01, 0.02, "int4")
    for t in range(0, 96, 7):
        for got, x, g in ((gk, k, 0.01), (gv, v, 0.02)):
            assert np.array_equal(got[t], kv4.values(*kv4.quantise(x[t], g, "int4"), g, "int4"))


def test_attention_against_scalars():
    rng = np.random.default_rng(1)
    cache = np.zeros((4, 1, 1, 18 * 64), np.uint8)
    k, v = rng.standard_normal((2, 20, 1, 64)).astype(np.float32)
    table = np.array([[2, 0], [1, -1]], np.int32)
    slots = [2 * 16 + t if t < 16 else t - 16 for t in range(20)]
    cache = kv4.write(cache, slots, k, v, 0.003, 0.003, "e2m1")
    q = rng.standard_normal((3, 2, 64))
    out, _, _ = kv4.attention(q, cache, [18, 0], table, [0, 2, 3], 0.003, 0.003, 0.2, "e2m1")
    kk, vv = kv4.tokens_of(cache, slots, 0.003, 0.003, "e2m1")
    for i in range(2):
        for h in range(2):
            s = [0.2 * float(np.dot(q[i, h], kk[t, 0])) for t in range(17 + i)]
            w = [np.exp(x - max(s)) for x in s]
            ref = sum(wi * vv[t, 0] for t, wi in enumerate(w)) / sum(w)
            assert np.allclose(out[i, h], ref, rtol=1e-12)
    assert not out[2].any()                                  # an empty request


def test_block_tables_by_hand():
    table = np.full((4, 3), -1, np.int32)
    table[0, 0] = 9
    t, start, lens, slots, pos, left, after = kv4.block_tables([15, 0, 0, 0], [2, 40, 16, 49], [3, 4, 5, 6, 7], 4, table, 16, 110)
    # request 0 takes block 6, request 1 takes 5, 4, 3; request 2 finds none; request 3 does not fit its table
    assert t[0].tolist() == [9, 6, -1] and t[1].tolist() == [5, 4, 3] and t[2].tolist() == [-1] * 3
    assert start.tolist() == [0, 2, 42, 58, 107] and lens.tolist() == [17, 40, 0, 0] and left == after == 0
    assert slots[:3].tolist() == [9 * 16 + 15, 6 * 16, 5 * 16] and pos[:3].tolist() == [15, 16, 0]
    # a request that needs no block runs behind one that finds none; the balance counts the latter's
    *_, left, after = kv4.block_tables([0, 0, 3], [16, 48, 1], [3, 4, 5], 3, np.full((3, 3), 7, np.int32), 16, 65)
    assert left == -1 and after == 2
    assert (slots[42:] == -1).all() and pos[106] == 48 and pos[107:].tolist() == [0] * 3


def test_verify_by_hand():
    target = np.array([[.5, .5, 0, 0], [0, 0, .25, .75], [.1, .2, .3, .4]])
    draft = np.array([[.5, .25, .25, 0], [.0, .5, .5, 0]])
    # token 1 kept (u q = .1 < .5), token 2: .9 * .5 > .25, rejected; the rest is [0, 0, 0, .75]
    out, n = kv4.verify(target, draft, [1, 2], [0, 2], [.4, .9], [.0], 3)
    assert out.tolist() == [[1, 3, -1, -1]] and n.tolist() == [1]
    # both kept: the extra token from the last row
    out, n = kv4.verify(target, draft, [1, 2], [0, 2], [.4, .4], [.35], 3)
    assert out.tolist() == [[1, 2, 2, -1]] and n.tolist() == [2]
    # tokens alone: u < p
    out, n = kv4.verify(target, None, [2, 3], [0, 2], [.0, .0], [.99], 2)
    assert out.tolist() == [[1, -1, -1]] and n.tolist() == [0]


def test_verify_keeps_the_targets_distribution():
    rng = np.random.default_rng(2)
    p, q = np.array([.1, .2, .3, .4]), np.array([.4, .3, .2, .1])
    n = 20000
    tokens = rng.choice(4, n, p=q)
    target = np.repeat(p[None], 2 * n, 0)
    out, _ = kv4.verify(target, np.repeat(q[None], n, 0), tokens, np.arange(n + 1), rng.random(n), rng.random(n), 1)
    share = np.bincount(out[:, 0], minlength=4) / n
    assert np.all(np.abs(share - p) < 5 * np.sqrt(p * (1 - p) / n))
