"""Pins of the oracle of long contexts over the paged fp8 cache (CPU)."""
import numpy as np
import torch

import oracle
from oracle import attention as decode, fp8_paged as fp


def test_encode_is_the_quantisers():
    x = np.concatenate([np.linspace(-500, 500, 4001), [np.nan, np.inf, -np.inf, -0.0, 1e-30, 2.0 ** -10, 3 * 2.0 ** -10]])
    x = torch.from_numpy(x.astype(np.float32)).bfloat16()
    bits = x.view(torch.int16).numpy().view(np.uint16)
    got = fp.encode(x.float().numpy())
    want = oracle.quant(bits.reshape(1, -1), oracle.BF16, oracle.E4M3, oracle.PER_TENSOR, scale=np.float32([1.0]))[0].reshape(-1)
    assert np.array_equal(got, want)


def test_rotation_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 64)).astype(np.float32)
    angle = rng.uniform(-3, 3, (9, 16))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    pos = np.int32([[0, 3, 8, 2, 9], [1, 1, 4, 4, -1]])
    for inter in (False, True):
        y = fp.rotate(x, pos, table, (10, 6), inter)
        for t in range(4):
            for i in range(16):
                a, b = (2 * i, 2 * i + 1) if inter else (i, 16 + i)
                z = (x[t, :, a] + 1j * x[t, :, b]) * np.exp(1j * angle[pos[0 if i < 10 else 1, t], i])
                assert np.allclose(y[t, :, a] + 1j * y[t, :, b], z, atol=1e-6)
        assert np.isnan(y[4, :, :32]).all() and np.array_equal(y[:, :, 32:], x[:, :, 32:])


def test_attention_of_single_tokens_is_the_decode_oracles():
    rng = np.random.default_rng(1)
    kc, vc = rng.integers(0, 126, (2, 7, 16, 2, 128)).astype(np.uint8)
    table = rng.permutation(7)[:6].reshape(2, 3).astype(np.int32)
    table[1, 1] = -1
    q = torch.from_numpy(rng.standard_normal((2, 4, 128)).astype(np.float32)).bfloat16()
    bits = q.view(torch.int16).numpy().view(np.uint16)
    want = decode.fp8_kv_decode_attention(bits, oracle.BF16, kc, vc, np.int32([33, 40]), float(np.float32(0.01)),
                                          float(np.float32(0.02)), sm_scale=0.1, block_table=table)
    got = fp.attention(q.float().numpy(), kc, vc, 0.01, 0.02, np.int32([33, 40]), table, None, 1, 0.1)[0]
    assert np.allclose(got, want, rtol=1e-12)


def test_selecting_all_columns_changes_nothing():
    rng = np.random.default_rng(2)
    kc, vc = rng.integers(0, 126, (2, 9, 16, 2, 64)).astype(np.uint8)
    table = rng.permutation(9)[:8].reshape(2, 4).astype(np.int32)
    q = rng.standard_normal((6, 2, 64)).astype(np.float32)
    lens, start = np.int32([50, 17]), np.int32([0, 4, 6])
    means, scales = fp.block_means(kc, lens, table, np.int32([0, 50, 67]), 99, np.zeros((9, 2, 64), np.int8), np.zeros((9, 2), np.float32))
    sel = fp.select(q, means, scales, lens, table, 16, start, 4, 1, 1, 5, np.full((6, 2, 5), -9, np.int32))
    assert sel[3].tolist() == [[0, 1, 2, 3, -1]] * 2 and sel[5].tolist() == [[0, 1, -1, -1, -1]] * 2
    a = fp.attention(q, kc, vc, 0.01, 0.02, lens, table, start, 4, 0.1)[0]
    b = fp.attention(q, kc, vc, 0.01, 0.02, lens, table, start, 4, 0.1, selected=sel)[0]
    assert np.allclose(a, b, rtol=1e-12)


def test_selection_by_hand():
    """Blocks of one repeated key: the scores are the products, ties go to the lower column."""
    kc = np.zeros((6, 16, 1, 64), np.uint8)
    one = int(fp.encode(np.float32([1.0]))[0])
    for block, value in enumerate((0.0, 2.0, 1.0, 2.0, -4.0, 1.0)):
        kc[block, :, 0, 3] = fp.encode(np.float32([value]))[0]
    assert fp.VALUES[one] == 1.0
    table, lens = np.arange(6, dtype=np.int32)[None], np.int32([95])
    means, scales = fp.block_means(kc, lens, table, np.int32([0, 95]), 95, np.zeros((6, 1, 64), np.int8), np.zeros((6, 1), np.float32))
    assert means[1, 0, 3] == 127 and np.isclose(scales[1, 0], 2 / 127) and scales[0, 0] == 1.0
    q = np.zeros((1, 2, 64), np.float32)
    q[0, 0, 3] = 1.0
    pick = lambda budget, first, last: fp.select(q, means, scales, lens, table, 16, None, 1, first, last, budget, np.zeros((1, 1, budget), np.int32))  # noqa: E731
    assert pick(2, 0, 1)[0, 0].tolist() == [1, 5]
    assert pick(4, 0, 1)[0, 0].tolist() == [1, 2, 3, 5]
    assert pick(3, 1, 1)[0, 0].tolist() == [0, 1, 5]
    q[0, 1, 3] = -1.0                                        # the second head wants block 4
    assert pick(2, 0, 1)[0, 0].tolist() == [4, 5]
