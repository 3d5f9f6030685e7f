"""Pins for the speculative-decoding oracle (CPU only): hand-written tables and trees, chains
against the absorbed-attention oracle, and a math.fsum brute force."""
import math

import numpy as np

from chunked_prefill_attention_ragged_gb300 import workloads as wl
from oracle import (absorbed_attention, bf16_bits_to_f64, cache_write, pack_bits, tree_attention, tree_commit,
                    tree_visibility, update_block_table)


def test_update_by_hand():
    # blocks of 4; request 0: 3 + 2 tokens needs a second block, request 1 gives two of three
    # back (5 tokens become 2), request 2 starts with 6 tokens.
    table = [[7, -1, -1], [1, 2, 3], [-1, -1, -1]]
    qo, kv, slots, t, held, stack, short = update_block_table([3, 2, 0], [2, 0, 6], table, [1, 3, 0], [9, 8], 4, 10, 10)
    assert not short and stack == [9]
    # given back in request order, the first of them on top of the stack
    assert t.tolist() == [[7, 2, -1], [1, -1, -1], [3, 8, -1]] and held.tolist() == [2, 1, 2]
    assert qo.tolist() == [0, 2, 2, 8] and kv.tolist() == [5, 2, 6]
    assert slots.tolist() == [31, 8, 12, 13, 14, 15, 32, 33, -1, -1]


def test_update_out_of_blocks_serves_a_prefix_of_the_requests():
    table = [[-1, -1], [-1, -1], [-1, -1]]
    _, _, slots, t, held, stack, short = update_block_table([0, 0, 0], [4, 8, 4], table, [0, 0, 0], [5, 6], 4, 8, 16)
    assert short and t.tolist() == [[6, -1], [-1, -1], [-1, -1]] and held.tolist() == [1, 0, 0] and stack == [5]
    assert slots.tolist() == [24, 25, 26, 27] + [-1] * 12


def test_reserve_and_roll_back_restores_everything():
    rng = np.random.default_rng(3)
    seq, new = rng.integers(0, 50, 7), rng.integers(0, 30, 7)
    need = -(-seq // 8)
    perm = rng.permutation(100)
    table, at = np.full((7, 12), -1), 0
    for r in range(7):
        table[r, :need[r]] = perm[at:at + need[r]]
        at += need[r]
    stack = perm[at:].tolist()
    _, _, _, t, h, s, short = update_block_table(seq, new, table, need, stack, 8, 100, 0)
    _, _, _, t, h, s, _ = update_block_table(seq, new * 0, t, h, s, 8, 100, 0)
    assert not short and np.array_equal(t, table) and np.array_equal(h, need) and s == stack


def test_visibility_by_hand():
    #  0 -> 1 -> 3;  0 -> 2;  4 is another child of the context
    seen, depth = tree_visibility([-1, 0, 0, 1, -1])
    assert seen.astype(int).tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 1, 0, 1, 0],
                                         [0, 0, 0, 0, 1]]
    assert depth.tolist() == [0, 1, 1, 2, 0]
    assert pack_bits(seen, 1)[:, 0].tolist() == [1, 3, 5, 11, 16]
    wide = np.zeros((1, 130), dtype=bool)
    wide[0, [63, 64, 129]] = True
    assert pack_bits(wide, 3).tolist() == [[-2 ** 63, 1, 2]]


def test_chain_is_causal_absorbed_attention():
    rng = np.random.default_rng(11)
    q = wl.to_bf16_bits(rng.standard_normal((5, 3, 576)).astype(np.float32))
    kv = wl.to_bf16_bits(rng.standard_normal((9, 576)).astype(np.float32))
    for length in (9, 5, 3, 0):
        for cap in (0.0, 5.0):
            want = absorbed_attention(q, kv[:length], causal=True, sm_scale=0.07, logits_soft_cap=cap)
            seen, _ = tree_visibility([-1, 0, 1, 2, 3])
            for vis in (None, seen):
                got = tree_attention(q, kv[:length], vis, sm_scale=0.07, logits_soft_cap=cap)
                np.testing.assert_allclose(got[0], want[0], atol=1e-12)
                np.testing.assert_allclose(got[1], want[1], atol=1e-12)


def test_tree_brute_force_and_empty_row():
    rng = np.random.default_rng(5)
    q = wl.to_bf16_bits(rng.standard_normal((3, 1, 576)).astype(np.float32))
    kv = wl.to_bf16_bits(rng.standard_normal((4, 576)).astype(np.float32))   # one context key, three nodes
    seen = np.array([[1, 0, 0], [0, 1, 0], [1, 0, 1]], dtype=bool)
    o, lse = tree_attention(q, kv, seen, sm_scale=0.05)
    qf, kf = bf16_bits_to_f64(q), bf16_bits_to_f64(kv)
    for i, keys in enumerate([[0, 1], [0, 2], [0, 1, 3]]):
        s = [0.05 * math.fsum(qf[i, 0] * kf[k]) for k in keys]
        e = [math.exp(x) for x in s]
        assert abs(lse[i, 0] - math.log(math.fsum(e))) < 1e-12
        want = sum(w * kf[k, :512] for w, k in zip(e, keys)) / math.fsum(e)
        np.testing.assert_allclose(o[i, 0], want, atol=1e-12)
    o, lse = tree_attention(q, kv[:3], seen & False, sm_scale=0.05)      # no context, nothing seen
    assert np.all(o == 0) and np.all(np.isneginf(lse))


def test_commit_by_hand():
    cache = np.arange(2 * 4 * 2 * 1).reshape(2, 4, 2, 1)
    # positions 1.. of request 0 lie in blocks 3, 0: node 0 at (3, 1), 1 at (0, 0), 2 at (0, 1)
    out = tree_commit(cache, [[3, 0]], [1], [[0, 2]], [2])
    want = cache.copy()
    want[:, 0, 0] = cache[:, 0, 1]
    assert np.array_equal(out, want)
    assert np.array_equal(tree_commit(cache, [[3, 0]], [1], [[1, 2]], [0]), cache)


def test_slots_feed_the_cache_write():
    qo, _, slots, table, *_ = update_block_table([3], [3], [[2, -1]], [1], [0], 4, 4, 5)
    cache = np.zeros((3, 4, 8), dtype=np.uint16)
    rows = np.arange(5 * 8, dtype=np.uint16).reshape(5, 8) + 1
    out = cache_write(cache, rows, slots)
    assert np.array_equal(out[2, 3], rows[0]) and np.array_equal(out[table[0, 1], 0], rows[1])
    assert (out == 0).all(axis=2).sum() == 9
