"""Pins for the attention oracle: rotations that keep lengths and compose, scores
that depend on the distance of positions alone, the two pair layouts as one
permutation, placement by the page table, and closed forms of the softmax
(uniform and one-hot weights, rows that see nothing)."""
import numpy as np

import gen
from oracle import attention as oa


def test_rotation_keeps_lengths_and_composes():
    rng = np.random.default_rng(1)
    x, f = rng.standard_normal((3, 16)), np.array([1.0, 0.3, 0.05])
    y = oa.rotate(x, 7, f, 1.0, False)
    assert np.allclose(np.linalg.norm(y, axis=1), np.linalg.norm(x, axis=1))
    assert np.array_equal(y[:, 6:], x[:, 6:]) and np.array_equal(oa.rotate(x, 0, f, 1.0, True), x)
    assert np.allclose(oa.rotate(oa.rotate(x, 7, f, 1.0, False), 5, f, 1.0, False),
                       oa.rotate(x, 12, f, 1.0, False))
    assert np.allclose(oa.rotate(x, 9, f, 1.5, False)[:, :6], 1.5 * oa.rotate(x, 9, f, 1.0, False)[:, :6])


def test_rotated_scores_depend_on_the_distance():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 8))
    f = np.array([1.0, 0.1, 0.01, 0.001])
    s = [float((oa.rotate(q, p + 11, f, 1.0, True) @ oa.rotate(k, p, f, 1.0, True).T)[0, 0])
         for p in (0, 5, 1000)]
    assert np.allclose(s, s[0])


def test_pair_layouts_are_one_permutation():
    rng = np.random.default_rng(3)
    x, f = rng.standard_normal((2, 8)), np.array([1.0, 0.2, 0.03, 0.4])
    perm = [0, 4, 1, 5, 2, 6, 3, 7]                  # half -> interleaved
    assert np.allclose(oa.rotate(x[:, perm], 13, f, 1.0, True), oa.rotate(x, 13, f, 1.0, False)[:, perm])


def test_a_quarter_turn_by_hand():
    y = oa.rotate(np.array([[3.0, 4.0]]), 1, np.array([np.pi / 2]), 1.0, False)
    assert np.allclose(y, [[-4.0, 3.0]])


def test_append_places_rows_by_the_table():
    rng = np.random.default_rng(4)
    x = gen.paged_batch(rng, [3, 2], [18, 2], 2, 1, 16, 16, pad_rows=1)
    x.table[0, 0] = 99                               # outside: positions 15 of sequence 0 is dropped
    q, k, v = oa.rope_append(x.qkv, x.k_cache, x.v_cache, x.table, x.cu, x.ctx, [], 2)
    rows = x.qkv.astype(np.float64).reshape(6, 4, 16)
    page = x.table[0, 1]
    assert np.array_equal(k[page, 0, :2], rows[1:3, 2]) and np.array_equal(v[page, 0, :2], rows[1:3, 3])
    assert np.array_equal(k[x.table[1, 0], 0, :2], rows[3:5, 2])
    changed = np.any(k != x.k_cache, axis=(1, 3)).sum()
    assert changed == 4 and np.all(np.isnan(q[5])) and np.array_equal(q[0], rows[0, :2])


def test_attention_closed_forms():
    rng = np.random.default_rng(5)
    x = gen.paged_batch(rng, [4], [3], 2, 1, 8, 16)  # the first row lies before position 0
    x.q[:] = 0                                       # equal scores: the mean of what a row sees
    vals = x.v_cache[x.table[0, 0], 0].astype(np.float64)
    out, spread, _, seen = oa.attention(x.q, x.k_cache, x.v_cache, x.table, x.cu, x.ctx, 1.0)
    assert list(seen) == [0, 1, 2, 3] and np.all(out[0] == 0)
    for r in (1, 2, 3):
        assert np.allclose(out[r], vals[:r].mean(0)) and np.allclose(spread[r], np.abs(vals[:r]).mean(0))
    x.q[:, :, 0] = 100                               # one key far ahead: its value alone
    x.k_cache[:] = 0
    x.k_cache[x.table[0, 0], 0, 1, 0] = 10
    out, _, reach, _ = oa.attention(x.q, x.k_cache, x.v_cache, x.table, x.cu, x.ctx, 1.0)
    assert np.allclose(out[3], vals[1]) and np.allclose(out[1], vals[0]) and reach[3, 0] == 1000


def test_attention_shares_heads_and_skips_bad_pages():
    rng = np.random.default_rng(6)
    x = gen.paged_batch(rng, [2], [40], 4, 2, 8, 16)
    args = (x.k_cache, x.v_cache, x.table, x.cu, x.ctx, 0.3)
    out = oa.attention(x.q, *args)[0]
    for j in range(4):                               # head j alone, on its key head
        one = oa.attention(x.q[:, j:j + 1], x.k_cache[:, j // 2:j // 2 + 1], x.v_cache[:, j // 2:j // 2 + 1],
                           *args[2:])[0]
        assert np.allclose(out[:, j], one[:, 0])
    x.table[0, 1] = -1
    got, _, _, seen = oa.attention(x.q, *args)
    assert list(seen) == [23, 24] and np.all(np.isfinite(got))
    # brute force over the keys that are left
    keep = [p for p in range(39) if p // 16 != 1]
    k = np.stack([x.k_cache[x.table[0, p // 16], 0, p % 16] for p in keep]).astype(np.float64)
    v = np.stack([x.v_cache[x.table[0, p // 16], 0, p % 16] for p in keep]).astype(np.float64)
    w = np.exp(0.3 * k @ x.q[0, 0].astype(np.float64))
    assert np.allclose(got[0, 0], (w / w.sum()) @ v)
