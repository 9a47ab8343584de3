"""Pins of the serving oracle (CPU): the number formats against torch's own
conversions and rational arithmetic, the tables against a hand-worked step, the
selection and the attention against the training oracle on unpaged documents."""
import math

import numpy as np
import pytest

from oracle import cache_oracle as C
from oracle import msa_oracle as O


def test_e4m3_values_match_torch():
    import torch
    t = torch.arange(0x80, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t[:0x7F], C.E4M3) and math.isnan(t[0x7F]) and math.isnan(C.e4m3_value(0x7F))


@pytest.mark.parametrize("exp", [0, -5, 7])
def test_rounding_matches_rational_arithmetic(exp):
    """Vectorised rounding against exact fractions: random rows, ties of the scale and of the codes, zeros,
    saturation, tiny groups, groups that are not finite."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((24, 128))
    x[1] *= 2.0 ** -9
    x[2] *= 2.0 ** 9
    x[3] = 0
    x[4] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -5.0], 128)   # ties at scale 1
    x[4, ::16] = 6.0
    x[5, ::16] = 6 * 1.0625 * np.array([1, 2, 4, 8, 0.5, 0.25, 16, 32])                 # scale ties
    x[6] = 1e30
    x[7, 3], x[7, 40], x[7, 90] = np.inf, np.nan, -np.inf
    x *= 2.0 ** exp
    bits = O.f64_to_bf16(np.where(np.isfinite(x), x, 0))
    bits[7, 3], bits[7, 40], bits[7, 90] = 0x7F80, 0x7FC1, 0xFF80
    codes, scales, vals = C.round_rows(bits, exp)
    f = O.bf16_to_f64(bits)
    for r in range(len(x)):
        for j in range(8):
            want, pattern = C.round_group(f[r, 16 * j:16 * j + 16], exp)
            assert scales[r, j] == pattern
            if want is None:
                assert np.isnan(vals[r, 16 * j:16 * j + 16]).all()
            else:
                assert codes[r, 16 * j:16 * j + 16].tolist() == want
    # values are exact in bf16
    ok = np.isfinite(vals)
    assert np.array_equal(O.bf16_to_f64(O.f64_to_bf16(vals[ok])), vals[ok])


def test_step_by_hand():
    """Three requests, pages of 64: one grows inside a page, one crosses into a new page, one gives two back."""
    table = np.array([[4, 0, 0], [2, 0, 0], [5, 3, 0]])
    ring = np.array([9, 0, 1, 6, 7, 8, 9, 9])          # free: 1, 6, 7 from entry 2 on
    s = C.step([1, 3, -1], [10, 62, 65], 2, 3, ring, table, 64)
    assert s["cu_tokens"].tolist() == [0, 1, 4, 4]
    assert s["slot_map"].tolist() == [4 * 64 + 10, 2 * 64 + 62, 2 * 64 + 63, 1 * 64 + 0]
    assert s["positions"].tolist() == [10, 62, 63, 64]
    assert s["chunks"].tolist() == [[0, 0, 1, 10], [1, 1, 2, 62], [1, 3, 1, 64]]
    assert s["block_table"].tolist() == [[4, 0, 0], [2, 1, 0], [5, 3, 0]]
    assert s["seq_lens"].tolist() == [11, 65, 0]
    assert (s["head"], s["count"]) == (3, 4)
    assert s["free_ring"].tolist() == [9, 0, 1, 6, 7, 5, 3, 9]


def test_cache_bytes_by_hand():
    """One token's rows at their bytes: plain K codes, XORed V codes, scales by row and by group."""
    k = np.arange(128, dtype=np.uint8) % 16
    ks, vs = np.arange(8, dtype=np.uint8) + 1, np.arange(8, dtype=np.uint8) + 100
    cache = np.zeros((2, 1, 2, C.TILE_BYTES), np.uint8)
    C.write_row(cache, 128 + 64 + 13, 0, 128, k, ks, k, vs)    # page 1, tile 1, token 13
    b = cache[1, 0, 1]
    want = (k[0::2] | (k[1::2] << 4)).tolist()
    assert b[13 * 64:14 * 64].tolist() == want
    assert b[4096 + 13 * 8:4096 + 14 * 8].tolist() == ks.tolist()
    # 13 & 12 = 12: the offset's bits 5 and 6 flip, so the row lies in its neighbour's place with halves swapped
    at = 4608 + 12 * 64
    assert (b[at + 32:at + 64].tolist(), b[at:at + 32].tolist()) == (want[:32], want[32:])
    assert b[8704 + 13:8704 + 512:64].tolist() == vs.tolist()
    assert np.count_nonzero(cache) == np.count_nonzero(b)


@pytest.mark.parametrize("block", [64, 128])
def test_selection_and_attention_match_the_training_oracle(block):
    """One request whose whole document is new is the training forward over the cache's values."""
    rng = np.random.default_rng(3)
    n, H, K = 333, 2, 4
    q, k, v = (O.f64_to_bf16(rng.standard_normal((n, h, 128))) for h in (16 * H, H, H))
    qi, ki = (O.f64_to_bf16(rng.standard_normal((n, H, 128))) for _ in range(2))
    M = -(-n // block)
    s = C.step([n], [0], 0, M, rng.permutation(M), np.zeros((1, M), int), block)
    pool = np.zeros((M, H, 128), np.uint16)
    tail = np.zeros((1, 2, block, H, 128), np.uint16)
    C.index_update(ki, s["cu_tokens"], [0], s["block_table"], tail, pool, block)
    sel = C.select(qi, pool, s["block_table"], s["chunks"], block, K)
    cu = np.array([0, n])
    assert np.array_equal(sel, O.select_topk(qi, ki, cu, block, 8, K))
    kv, vv = C.round_rows(k, 0)[2], C.round_rows(v, 0)[2]
    o, lse = C.attend(q, [kv], [vv], s["chunks"], sel, block, 128 ** -0.5)[:2]
    want_o, want_lse = O.forward_blocked(q, O.f64_to_bf16(kv), O.f64_to_bf16(vv), cu, np.array([0]), sel, block, 8,
                                         128 ** -0.5)
    np.testing.assert_allclose(o, want_o, atol=1e-12)
    np.testing.assert_allclose(lse, want_lse, atol=1e-12)


def test_index_pool_over_several_steps():
    """Means over blocks that fill up over many steps equal the training oracle's pooling of the whole document."""
    rng = np.random.default_rng(4)
    n, H, block = 300, 1, 64
    ki = O.f64_to_bf16(rng.standard_normal((n, H, 128)))
    pool, tail = np.zeros((5, H, 128), np.uint16), np.zeros((1, 2, block, H, 128), np.uint16)
    table = np.array([[3, 1, 4, 0, 2]])
    past = 0
    for m in (1, 62, 3, 130, 1, 59, 44):
        C.index_update(ki[past:past + m], [0, m], [past], table, tail, pool, block)
        past += m
    assert past == n
    want = O.pool_index(ki, np.array([0, n]), block)
    assert np.array_equal(pool[table[0, :4]].transpose(1, 0, 2), want[:, :4])
