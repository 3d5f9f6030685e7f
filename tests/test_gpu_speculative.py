"""GPU parity of the speculative-decoding step (block tables, tree masks, tree attention, commit)
against the oracle, each by itself and all together, eager and in a captured graph."""
import numpy as np
import pytest

from chunked_prefill_attention_ragged_gb300 import workloads as wl
from oracle import (bf16_bits_to_f64, pack_bits, tree_attention, tree_commit, tree_visibility, update_block_table)
from gpu_util import Guarded, bits_of, f64_of_bf16, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BAD_INDEX, NO_BLOCKS = 2, 4


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def new_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------ block tables
def run_tables(seq, new, table, held, stack, bs, capacity, num_tokens):
    import chunked_prefill_attention_ragged_gb300 as mla
    free = np.full(capacity, -7, dtype=np.int64)
    free[:len(stack)] = stack
    st = new_status()
    dev = [i32(seq), i32(new), i32(table), i32(held), i32(free), i32([len(stack)])]
    slots = Guarded((num_tokens,), torch.int64)
    qo, kv, slot_map = mla.mla_block_table_update(*dev, bs, num_tokens, slot_mapping=slots.tensor, status=st)
    torch.cuda.synchronize()
    slots.check("slot_mapping")
    count = int(dev[5][0])
    return (qo.cpu().numpy(), kv.cpu().numpy(), slot_map.cpu().numpy(), dev[2].cpu().numpy(), dev[3].cpu().numpy(),
            dev[4].cpu().numpy()[:count].tolist(), int(st))


def random_tables(rng, batch, most, bs, width):
    seq, old = rng.integers(0, most + 1, batch), rng.integers(0, most + 1, batch)
    new = rng.integers(0, most + 1, batch)
    held = -(-old // bs)                      # what an earlier step left: more or fewer than needed
    total = int(held.sum() + (-(-(seq + new) // bs)).sum()) + 3
    perm = rng.permutation(total)
    table, at = np.full((batch, width), -1), 0
    for r in range(batch):
        table[r, :held[r]] = perm[at:at + held[r]]
        at += held[r]
    return seq, new, table, held, perm[at:].tolist(), total


@pytest.mark.parametrize("batch,most,bs,pad", [(1, 1, 1, 0), (1, 700, 64, 3), (3, 40, 16, 0), (33, 100, 7, 1),
                                               (1024, 9, 4, 5), (1025, 30, 16, 0), (8192, 3, 2, 9), (64, 900, 64, 77)])
@pytest.mark.parametrize("scarce", [False, True])
def test_block_table_update(batch, most, bs, pad, scarce):
    rng = np.random.default_rng(batch * 31 + most)
    width = -(-2 * most // bs) + 1
    seq, new, table, held, stack, total = random_tables(rng, batch, most, bs, width)
    if scarce:
        stack = stack[:len(stack) // 3]
    n = int(new.sum()) + pad
    want = update_block_table(seq, new, table, held, stack, bs, total, n)
    got = run_tables(seq, new, table, held, stack, bs, total, n)
    for k, name in enumerate(["qo_indptr", "kv_lens", "slot_mapping", "block_table", "num_held"]):
        np.testing.assert_array_equal(got[k], want[k], err_msg=name)
    assert got[5] == want[5]
    assert got[6] == (NO_BLOCKS if want[6] else 0)


def test_block_table_update_empty_batch_and_bad_values():
    import chunked_prefill_attention_ragged_gb300 as mla
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    free, count = i32([4, 5]), i32([2])
    qo, kv, slots = mla.mla_block_table_update(z, z, torch.zeros((0, 3), dtype=torch.int32, device="cuda"), z, free,
                                               count, 64, 3)
    assert qo.tolist() == [0] and kv.numel() == 0 and slots.tolist() == [-1, -1, -1] and int(count) == 2
    # a request that needs more blocks than its row has changes nothing; the others are served
    got = run_tables([0, 10, 0], [4, 4, 4], [[-1, -1], [2, -1], [-1, -1]], [0, 1, 0], [0, 1], 4, 3, 12)
    assert got[3].tolist() == [[1, -1], [2, -1], [0, -1]] and got[6] == BAD_INDEX
    assert got[2].tolist() == [4, 5, 6, 7, -1, -1, -1, -1, 0, 1, 2, 3]
    # negative lengths count as zero; more new tokens than the slot map holds; a stack that claims
    # more than it holds; a negative id on the stack
    assert run_tables([-5], [3], [[-1]], [0], [0], 4, 2, 3)[6] == BAD_INDEX
    got = run_tables([0], [3], [[-1]], [0], [1], 4, 2, 2)
    assert got[6] == BAD_INDEX and got[2].tolist() == [4, 5]
    got = run_tables([0], [3], [[-1]], [0], [-3], 4, 2, 3)
    assert got[6] == BAD_INDEX and got[3].tolist() == [[-1]] and got[2].tolist() == [-1] * 3
    st, c = new_status(), i32([9])
    mla.mla_block_table_update(i32([0]), i32([0]), i32([[-1]]), i32([0]), i32([1, 0]), c, 4, status=st)
    assert int(st) == BAD_INDEX and int(c) == 2


def test_slots_past_32_bits():
    # blocks of 1 << 20 tokens: flat slots need 64 bits
    got = run_tables([5], [3], [[4000, -1]], [1], [1], 1 << 20, 4096, 3)
    assert got[2].tolist() == [4000 * (1 << 20) + k for k in (5, 6, 7)]


def test_block_table_update_many_tokens_bad_values():
    """As above where the slots come from a grid: a request that does not fit its row, a stack that is
    full, more new tokens than slots."""
    bs, new = 16, [3000, 900, 2500, 0]
    table = np.full((4, 200), -1)
    table[3, :2] = [7, 8]
    got = run_tables([0, 4000, 0, 0], new, table, [0, 0, 0, 2], list(range(100, 500)), bs, 500, sum(new) + 3005)
    assert got[6] == BAD_INDEX and got[4].tolist() == [188, 0, 157, 0]
    want = np.concatenate([[7, 8], np.arange(499, 99, -1)])   # (the ones given back go first)
    assert got[3][0, :188].tolist() == want[:188].tolist() and got[3][2, :157].tolist() == want[188:345].tolist()
    pos = np.arange(3000)
    assert np.array_equal(got[2][:3000], want[pos // bs] * bs + pos % bs) and (got[2][3000:3900] == -1).all()
    assert (got[2][-5:] == -1).all()
    got = run_tables([0], [0], [[3, 4]], [2], [1], bs, 2, 9000)     # two blocks come back, one finds room
    assert got[6] == BAD_INDEX and got[5] == [1, 4] and (got[2] == -1).all()
    got = run_tables([0], [12000], [[-1] * 800], [0], list(range(800)), bs, 800, 9000)
    assert got[6] == BAD_INDEX and got[0].tolist() == [0, 12000]
    assert got[2][-1] == (799 - 8999 // bs) * bs + 8999 % bs


@pytest.mark.parametrize("num_tokens", [300, 9000])
def test_block_table_update_replayed(num_tokens):
    """One captured call, lengths changed between replays: against the oracle each time."""
    import chunked_prefill_attention_ragged_gb300 as mla
    rng = np.random.default_rng(num_tokens)
    batch, bs, width, total = 20, 16, 120, 900
    seq, new, table, held = i32([0] * batch), i32([0] * batch), i32(np.full((batch, width), -1)), i32([0] * batch)
    free, count, st = i32(rng.permutation(total)), i32([total]), new_status()
    mla.mla_block_table_update(seq, new, table, held, free, count, bs, num_tokens, status=st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qo, kv, slots = mla.mla_block_table_update(seq, new, table, held, free, count, bs, num_tokens, status=st)
    h_table, h_held, h_stack = np.full((batch, width), -1), [0] * batch, free.cpu().numpy().tolist()
    for _ in range(6):
        s, m = rng.integers(0, 1000, batch), rng.integers(0, num_tokens // batch, batch)
        seq.copy_(i32(s))
        new.copy_(i32(m))
        g.replay()
        torch.cuda.synchronize()
        want = update_block_table(s, m, h_table, h_held, h_stack, bs, total, num_tokens)
        h_table, h_held, h_stack = want[3], want[4], want[5]
        for k, got in enumerate((qo, kv, slots, table, held)):
            np.testing.assert_array_equal(got.cpu().numpy(), want[k])
        assert free.cpu().numpy()[:int(count)].tolist() == list(h_stack)
        st.zero_()


def test_block_table_update_of_two_streams():
    import chunked_prefill_attention_ragged_gb300 as mla
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for k, s in enumerate(streams):
        with torch.cuda.stream(s):
            args = [i32([5, 9]), i32([k + 1, 6000 * k]), i32([[-1] * 400] * 2), i32([0, 0]), i32(np.arange(800)), i32([800])]
        s.synchronize()
        outs.append((args, [mla.mla_block_table_update(*args, 16, 6002 + 3000 * k, stream=s) for _ in range(3)][-1]))
    torch.cuda.synchronize()
    for k, (args, (qo, kv, slots)) in enumerate(outs):
        assert qo.tolist() == [0, k + 1, k + 1 + 6000 * k] and kv.tolist() == [6 + k, 9 + 6000 * k]
        need = 1 + -(-(9 + 6000 * k) // 16)
        assert args[5].tolist() == [800 - need] and slots[0] == 799 * 16 + 5 and (slots[k + 1 + 6000 * k:] == -1).all()


# ---------------------------------------------------------------------------------- tree mask
def random_parents(rng, n, reach):
    return np.array([-1 if i == 0 else int(rng.integers(max(-1, i - reach), i)) for i in range(n)], dtype=np.int64)


@pytest.mark.parametrize("nodes,words,reach", [([1], 1, 1), ([64, 0, 1, 63], 1, 3), ([65, 200, 7], 4, 5), ([300], 5, 1),
                                               ([3, 130], 3, 200), ([2] * 70, 1, 2), ([600], 10, 4),
                                               ([256, 257, 5, 511], 9, 400), ([1500, 1], 24, 1), ([700, 40], 30, 700)])
def test_tree_mask(nodes, words, reach):
    import chunked_prefill_attention_ragged_gb300 as mla
    rng = np.random.default_rng(sum(nodes) + words)
    trees = [random_parents(rng, n, reach) for n in nodes]
    qo = wl.indptr_from_lengths(nodes)
    kv = rng.integers(0, 50, len(nodes)) + np.asarray(nodes)
    parents = np.concatenate(trees + [np.full(3, 99)])        # three rows of padding behind the last tree
    total = len(parents)
    st = new_status()
    for with_kv in (False, True):
        m, p = Guarded((total, words), torch.int64, fill=-5), Guarded((total,), torch.int32, fill=-6)
        mla.mla_tree_mask(i32(parents), i32(qo), words, kv_lens=i32(kv) if with_kv else None, mask=m.tensor,
                          positions=p.tensor, status=st)
        torch.cuda.synchronize()
        m.check("mask")
        p.check("positions")
        for r, t in enumerate(trees):
            seen, depth = tree_visibility(t)
            np.testing.assert_array_equal(m.tensor[qo[r]:qo[r + 1]].cpu().numpy(), pack_bits(seen, words))
            base = int(kv[r]) - nodes[r] if with_kv else 0
            np.testing.assert_array_equal(p.tensor[qo[r]:qo[r + 1]].cpu().numpy(), depth + base)
        assert (m.tensor[qo[-1]:] == -5).all() and (p.tensor[qo[-1]:] == -6).all()
    assert int(st) == 0


def test_tree_mask_of_a_long_chain():
    """Node i sees 0 .. i: 20000 of them, in time that grows with the size of the mask."""
    import chunked_prefill_attention_ragged_gb300 as mla
    n, words, st = 20000, 313, new_status()
    mask, pos = mla.mla_tree_mask(i32(np.arange(n) - 1), i32([0, n]), words, status=st)
    assert int(st) == 0 and torch.equal(pos, torch.arange(n, dtype=torch.int32, device="cuda"))
    i, w = torch.arange(n, device="cuda")[:, None], torch.arange(words, device="cuda")[None]
    ones = (i + 1 - 64 * w).clamp(0, 64)   # bits set in the word, from the lowest on
    want = torch.where(ones == 64, -1, (torch.ones_like(ones) << ones.clamp(max=63)) - 1)
    assert torch.equal(mask, want)


def test_tree_mask_bad_input():
    import chunked_prefill_attention_ragged_gb300 as mla
    st = new_status()
    # a parent that is the node itself, one above it, one below -1: taken as the context
    mask, pos = mla.mla_tree_mask(i32([-1, 1, 3, -2, 0]), i32([0, 5]), 1, status=st)
    assert int(st) == BAD_INDEX
    assert mask[:, 0].tolist() == [1, 2, 4, 8, 17] and pos.tolist() == [0, 0, 0, 0, 1]
    # more nodes than bits: those that fit are there
    st.zero_()
    mask, _ = mla.mla_tree_mask(i32(np.arange(70) - 1), i32([0, 70]), 1, status=st)
    assert int(st) == BAD_INDEX and mask[63, 0] == -1 and mask[69, 0] == -1
    # rows outside the buffers are not touched
    st.zero_()
    out = torch.full((4, 1), 9, dtype=torch.int64, device="cuda")
    mla.mla_tree_mask(i32([-1, 0, 1, 2]), i32([0, 2, 6]), 1, mask=out, status=st)
    assert int(st) == BAD_INDEX and out[:, 0].tolist() == [1, 3, 9, 9]


# ------------------------------------------------------------------------------ tree attention
def bounds(q, kv, seen, o_ref, *, sm_scale, cap):
    """Element-wise error bounds of (O, LSE) by arithmetic.  Logits: 576 products summed in
    fp32, each step off by at most 2^-23 of the sum of magnitudes (rounding or truncation), a
    few more operations on the result (scale, cap: a tanh made of an exponential and a
    reciprocal, each to 2^-22, times the cap); exponentials and their sum: 2^-21 relative more.
    A logit error d moves a weight by a factor e^d and O by at most 2 d sum p |v|.  P is rounded
    to bf16 before its product (2^-8 each, and the sum is of unrounded ones), O at the end."""
    n, heads, length = q.shape[0], q.shape[1], kv.shape[0]
    d = np.zeros((n, heads))
    for i in range(n):
        d[i] = (576 + 8) * 2.0 ** -23 * sm_scale * (np.abs(q[i]) @ np.abs(kv).T).max(axis=1, initial=0)
    d += 2.0 ** -20 + (16 * cap * 2.0 ** -22 if cap else 0)
    pv = np.zeros_like(o_ref)
    for i in range(n):
        keys = [k for k in range(length)
                if k < length - n or (seen[i, k - (length - n)] if seen is not None else k - (length - n) <= i)]
        if keys:
            x = sm_scale * (q[i] @ kv[keys].T)
            x = cap * np.tanh(x / cap) if cap else x
            p = np.exp(x - x.max(axis=1, keepdims=True))
            pv[i] = (p / p.sum(axis=1, keepdims=True)) @ np.abs(kv[keys][:, :512])
    return 2.0 ** -8 * np.abs(o_ref) + (2.0 ** -8 + 2 * d[..., None]) * pv + 1e-6, d + 2.0 ** -20


class Problem:
    def __init__(self, seed, nodes, kv, heads, bs, tree, cap=0.0, sm_scale=wl.DEFAULT_SM_SCALE, spread=1.0, reach=4):
        self.b = wl.random_absorbed(seed, nodes, kv, heads, block_size=bs, logits_soft_cap=cap, sm_scale=sm_scale)
        if spread != 1.0:
            self.b.q_abs = wl.to_bf16_bits((bf16_bits_to_f64(self.b.q_abs) * spread).astype(np.float32))
        rng = np.random.default_rng(seed + 1)
        self.nodes, self.kv = list(nodes), list(kv)
        self.seen = [tree_visibility(random_parents(rng, n, reach))[0] if tree else None for n in nodes]
        self.words = -(-max(max(nodes), 1) // 64) if tree else 0

    def mask(self):
        if not self.words:
            return None
        return to_dev(np.concatenate([pack_bits(s, self.words) for s in self.seen]))

    def run(self, pad=0, **kw):
        import chunked_prefill_attention_ragged_gb300 as mla
        b = self.b
        t = b.q_abs.shape[0] + pad
        q = torch.zeros((t, b.num_heads, 576), dtype=torch.bfloat16, device="cuda")
        q[:t - pad] = to_dev_bf16(b.q_abs)
        q[t - pad:] = float("nan")
        mask = self.mask()
        if mask is not None and pad:
            mask = torch.cat([mask, torch.full((pad, self.words), -1, dtype=torch.int64, device="cuda")])
        o = Guarded((t, b.num_heads, 512), torch.bfloat16, fill=3.0)
        lse = Guarded((t, b.num_heads), torch.float32, fill=4.0)
        st = new_status()
        mla.mla_tree_attention(q, to_dev_bf16(b.cache), to_dev(b.block_table), i32(b.qo_indptr), i32(self.kv), mask,
                               sm_scale=b.sm_scale, logits_soft_cap=b.logits_soft_cap, o=o.tensor, lse=lse.tensor,
                               status=st, **kw)
        torch.cuda.synchronize()
        o.check("O")
        lse.check("LSE")
        assert (o.tensor[t - pad:] == 3.0).all() and (lse.tensor[t - pad:] == 4.0).all(), "rows behind the last request"
        return o.tensor[:t - pad], lse.tensor[:t - pad], int(st)

    def rows(self, r):
        b, k = self.b, self.kv[r]
        pos = np.arange(k)
        return b.cache[b.block_table[r, pos // b.block_size], pos % b.block_size] if k else b.cache[0, :0]

    def check(self, o, lse, requests=None, heads=None):
        b = self.b
        o, lse = f64_of_bf16(o), lse.double().cpu().numpy()
        hs = slice(None) if heads is None else heads
        for r in range(b.batch) if requests is None else requests:
            rows = slice(int(b.qo_indptr[r]), int(b.qo_indptr[r + 1]))
            if rows.start == rows.stop:
                continue
            q, kv = bf16_bits_to_f64(b.q_abs[rows][:, hs]), bf16_bits_to_f64(self.rows(r))
            want_o, want_l = tree_attention(q, kv, self.seen[r], sm_scale=b.sm_scale,
                                            logits_soft_cap=b.logits_soft_cap)
            tol_o, tol_l = bounds(q, kv, self.seen[r], want_o, sm_scale=b.sm_scale, cap=b.logits_soft_cap)
            got_o, got_l = o[rows][:, hs], lse[rows][:, hs]
            assert np.array_equal(np.isneginf(got_l), np.isneginf(want_l)), f"request {r}: empty rows"
            fin = np.isfinite(want_l)
            assert np.isfinite(got_o).all() and np.isfinite(got_l[fin]).all()
            assert (np.abs(got_o - want_o) <= tol_o).all(), (
                f"request {r}: O off by {np.max(np.abs(got_o - want_o) / tol_o):.2f} of its bound")
            assert (np.abs(got_l[fin] - want_l[fin]) <= tol_l[fin]).all(), f"request {r}: LSE"


ATTENTION = [
    # name, nodes, kv, heads, block size, tree, cap
    ("one_token", [1], [1], 16, 64, False, 0.0),
    ("one_token_long", [1], [2500], 16, 64, False, 0.0),
    ("one_head", [1, 1], [77, 300], 1, 64, False, 0.0),
    ("five_heads_tree", [7, 1, 12], [100, 1, 12], 5, 16, True, 0.0),
    ("heads_128", [1, 3, 2], [130, 257, 512], 128, 64, True, 0.0),
    ("tile_edges", [1] * 9, [63, 64, 65, 127, 128, 129, 255, 256, 257], 8, 64, False, 0.0),
    ("node_tile_edges", [64, 65, 63, 128], [64, 130, 300, 200], 2, 64, True, 0.0),
    ("many_nodes", [200], [333], 2, 32, True, 0.0),
    ("chains", [5, 9, 1], [5, 200, 140], 16, 64, False, 0.0),
    ("block_1", [3, 2], [40, 9], 4, 1, True, 0.0),
    ("block_8", [3], [300], 4, 8, True, 0.0),
    ("block_24", [4, 4], [250, 130], 8, 24, True, 0.0),
    ("block_128", [4, 4], [400, 128], 8, 128, True, 0.0),
    ("block_48", [2], [700], 8, 48, True, 0.0),
    ("fewer_keys_than_nodes", [9, 6], [4, 0], 4, 64, False, 0.0),
    ("fewer_keys_than_nodes_tree", [9, 6, 3], [4, 0, 3], 4, 64, True, 0.0),
    ("empty_requests", [0, 5, 0, 0, 2, 0], [10, 50, 0, 300, 2, 7], 4, 64, True, 0.0),
    ("softcap", [4, 3], [200, 513], 16, 64, True, 30.0),
    ("softcap_small", [4], [300], 16, 64, True, 2.0),
    ("many_requests", [1, 2, 3] * 30, [5, 70, 140] * 30, 3, 16, True, 0.0),
    # about 16, 32, 64 and more (node, head) pairs a request, with units that do not fill and
    # requests of more units than one
    ("pairs_16_ragged", [1, 9, 1, 1], [90, 300, 64, 1], 5, 64, True, 0.0),
    ("pairs_32_ragged", [1, 3, 2, 2], [90, 300, 64, 129], 16, 64, True, 0.0),
    ("pairs_64_ragged", [7, 2, 1, 5], [90, 300, 64, 1000], 16, 64, True, 0.0),
    ("pairs_64_softcap", [4, 3], [200, 513], 16, 16, True, 20.0),
    ("pairs_16_block_1", [1, 2], [70, 200], 8, 1, True, 0.0),
    ("pairs_32_block_8", [2, 2], [200, 131], 16, 8, False, 0.0),
    ("wide_block_1", [3, 2], [40, 150], 64, 1, True, 0.0),
    ("wide_block_8", [3], [300], 64, 8, True, 0.0),
    ("wide_block_16", [2, 2], [130, 300], 64, 16, True, 0.0),
    ("wide_block_24", [2, 4], [250, 130], 48, 24, True, 0.0),
    ("wide_block_128", [2, 2], [400, 128], 48, 128, True, 0.0),
    ("wide_few_keys", [20, 9, 12], [4, 0, 12], 8, 64, True, 0.0),
    ("wide_softcap", [4, 3], [200, 513], 32, 64, True, 30.0),
    ("block_5", [3, 9, 2], [1000, 131, 2], 20, 5, True, 0.0),
    ("softcap_256", [4, 3], [200, 513], 16, 64, True, 256.0),
    ("softcap_300", [4, 3], [200, 513], 16, 64, True, 300.0),
]


@pytest.mark.parametrize("name,nodes,kv,heads,bs,tree,cap", ATTENTION, ids=[c[0] for c in ATTENTION])
def test_tree_attention(name, nodes, kv, heads, bs, tree, cap):
    p = Problem(900 + [c[0] for c in ATTENTION].index(name), nodes, kv, heads, bs, tree, cap)
    o, lse, st = p.run(pad=2)
    assert st == 0
    p.check(o, lse)


@pytest.mark.parametrize("spread", [0.01, 12.0])
@pytest.mark.parametrize("nodes,heads", [([6, 2], 64), ([6, 2], 16), ([2, 2], 16), ([1, 1], 16)])
def test_tree_attention_flat_and_peaked(spread, nodes, heads):
    """Nearly uniform weights, and logits whose maximum moves by hundreds along the keys."""
    p = Problem(77, nodes, [700, 333], heads, 64, True, spread=spread)
    o, lse, st = p.run()
    assert st == 0
    p.check(o, lse)


@pytest.mark.parametrize("batch,ctx,nodes,heads", [(1, 20000, 1, 16), (2, 9000, 5, 128), (150, 600, 1, 16),
                                                   (40, 900, 4, 128), (170, 400, 2, 16), (3, 7000, 4, 16),
                                                   (200, 300, 3, 16), (1, 30000, 3, 64)])
def test_tree_attention_split_and_unsplit(batch, ctx, nodes, heads):
    """A request over the whole GPU, and more requests than it has SMs; sampled."""
    p = Problem(33 + batch, [nodes] * batch, [ctx + 13 * (r % 7) + nodes for r in range(batch)], heads, 64, True)
    o, lse, st = p.run()
    assert st == 0
    some = sorted({0, batch // 2, batch - 1})
    p.check(o, lse, some, None if heads <= 16 else [0, heads // 2, heads - 1])


@pytest.mark.parametrize("spread", [1.0, 3000.0])   # logits far below the cap, and up to it
def test_tree_attention_large_cap(spread):
    """As good as without a cap: the bounds have no term for it (a relative error of 2^-20 of a logit,
    three operations' worth, is inside what they allow for 576 products)."""
    cap = 20000.0
    p = Problem(34, [3, 2], [400, 90], 8, 64, True, cap=cap, spread=spread, sm_scale=0.07)
    o, lse, st = p.run()
    assert st == 0
    b = p.b
    o, lse = f64_of_bf16(o), lse.double().cpu().numpy()
    for r in range(2):
        rows = slice(int(b.qo_indptr[r]), int(b.qo_indptr[r + 1]))
        q, kv = bf16_bits_to_f64(b.q_abs[rows]), bf16_bits_to_f64(p.rows(r))
        want_o, want_l = tree_attention(q, kv, p.seen[r], sm_scale=0.07, logits_soft_cap=cap)
        tol_o, tol_l = bounds(q, kv, p.seen[r], want_o, sm_scale=0.07, cap=0)
        top = np.abs(want_l).max() * 2.0 ** -19   # the exponential form, where logits come near the cap
        assert (np.abs(o[rows] - want_o) <= tol_o + 2 * top * np.abs(kv[:, :512]).max()).all()
        assert (np.abs(lse[rows] - want_l) <= tol_l + top).all()


def test_tree_attention_mask_rows_without_any_node():
    """A node that may not even see itself still sees the context; without context its row is empty."""
    p = Problem(5, [4, 3], [40, 3], 4, 64, True)
    p.seen = [s & np.array([False, True, False, True][:len(s)])[:, None] for s in p.seen]
    o, lse, st = p.run()
    assert st == 0 and torch.isneginf(lse[4]).all() and (o[4] == 0).all()
    p.check(o, lse)


@pytest.mark.parametrize("heads", [3, 7, 12, 40])
def test_tree_attention_repeats_bit_for_bit(heads):
    p = Problem(6, [3, 9, 1], [5000, 700, 64], heads, 64, True)
    a = p.run()
    for _ in range(3):
        b = p.run()
        assert np.array_equal(bits_of(a[0]), bits_of(b[0])) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("heads", [4, 8, 16, 64])
def test_tree_attention_does_not_read_past_the_lengths(heads):
    """NaN everywhere that no request owns: behind the last key of the last block, in other
    blocks, in the rows of the padding."""
    p = Problem(8, [3, 1, 4], [130, 65, 500], heads, 64, True)
    before = p.run(pad=3)   # (as many rows: the kernel is chosen by them)
    own = np.zeros(p.b.cache.shape[:2], dtype=bool)
    for r, k in enumerate(p.kv):
        pos = np.arange(k)
        own[p.b.block_table[r, pos // 64], pos % 64] = True
    p.b.cache[~own] = 0x7FC0
    after = p.run(pad=3)
    assert after[2] == 0 and torch.isfinite(after[0].float()).all()
    assert np.array_equal(bits_of(before[0]), bits_of(after[0])) and torch.equal(before[1], after[1])


@pytest.mark.parametrize("bs", [1, 8, 16, 24, 32, 48, 96, 128])
def test_tree_attention_ends_inside_a_block(bs):
    """NaN behind the last key, at every kind of end and block size."""
    kv = [1, 7, 8, 9, 31, 33, 63, 65, 97, 120, 127, 129, 160, 191, 193, 250]
    p = Problem(18, [1] * len(kv), kv, 6, bs, False)
    own = np.zeros(p.b.cache.shape[:2], dtype=bool)
    for r, k in enumerate(kv):
        pos = np.arange(k)
        own[p.b.block_table[r, pos // bs], pos % bs] = True
    p.b.cache[~own] = 0x7FC0
    o, lse, st = p.run()
    assert st == 0
    p.check(o, lse)


@pytest.mark.parametrize("ctx", [60, 20000])   # in one piece, and joined
def test_tree_attention_passes_nan_on_in_its_row_only(ctx):
    p = Problem(19, [3, 2], [ctx, 70], 4, 64, True)
    p.b.q_abs[1, 2, 570] = 0x7FC0
    o, lse, st = p.run()
    assert st == 0 and torch.isnan(o[1, 2].float()).all() and bool(torch.isnan(lse[1, 2]))
    q = p.b.q_abs.copy()
    q[1, 2] = p.b.q_abs[1, 1]
    p.b.q_abs = q
    o2, lse2, _ = p.run()
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[1, 2] = False
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[keep], lse2[keep])


def test_tree_attention_nodes_past_the_mask_are_not_seen():
    p = Problem(21, [70, 3], [100, 40], 2, 64, True)
    assert p.words == 2
    p.seen = [s * (np.arange(s.shape[1]) < 64) for s in p.seen]
    want = p.run()
    p.seen = [s[:, :64] for s in p.seen]
    p.words = 1
    got = p.run()
    assert np.array_equal(bits_of(got[0]), bits_of(want[0])) and torch.equal(got[1], want[1])
    p.seen = [np.pad(s, ((0, 0), (0, max(0, len(s) - s.shape[1])))) for s in p.seen]
    p.check(got[0], got[1])


@pytest.mark.parametrize("ctx", [70, 20000])
def test_tree_attention_output_on_16_bytes(ctx):
    import chunked_prefill_attention_ragged_gb300 as mla
    p = Problem(22, [2], [ctx], 5, 64, True)
    o, lse, _ = p.run()
    o2 = torch.full((10 * 512 + 16,), 3.0, dtype=torch.bfloat16, device="cuda")
    b = p.b
    mla.mla_tree_attention(to_dev_bf16(b.q_abs), to_dev_bf16(b.cache), to_dev(b.block_table), i32(b.qo_indptr),
                           i32(p.kv), p.mask(), sm_scale=b.sm_scale, o=o2[8:-8].view(2, 5, 512))
    assert np.array_equal(bits_of(o2[8:-8].view(2, 5, 512)), bits_of(o))
    assert (o2[:8] == 3.0).all() and (o2[-8:] == 3.0).all()


@pytest.mark.parametrize("heads", [8, 100])
def test_tree_attention_bad_blocks_read_as_zeros(heads):
    p = Problem(9, [2, 2], [300, 150], heads, 64, True)
    p.b.block_table[0, 1] = -2 ** 31 if heads > 8 else 10 ** 6
    p.b.block_table[1, 0] = -1
    o, lse, st = p.run()
    assert st == BAD_INDEX
    cache = np.concatenate([p.b.cache, np.zeros_like(p.b.cache[:1])])
    p.b.block_table[0, 1] = p.b.block_table[1, 0] = len(cache) - 1
    p.b.cache = cache
    p.check(o, lse)


def test_tree_attention_bad_lengths_are_clamped_or_skipped():
    p = Problem(10, [2, 2, 2], [100, 80, 90], 8, 64, True)
    p.kv[1] = 10 ** 6          # past the table: the keys it can name
    o, lse, st = p.run()
    assert st == BAD_INDEX
    p.check(o, lse, [0, 2])
    p.kv[1] = -3
    o, lse, st = p.run()
    assert st == BAD_INDEX and (o[2:4] == 0).all() and torch.isneginf(lse[2:4]).all()
    p.check(o, lse, [0, 2])
    p.kv[1] = 80
    import chunked_prefill_attention_ragged_gb300 as mla
    st = new_status()
    o = torch.full((6, 8, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    _, lse = mla.mla_tree_attention(to_dev_bf16(p.b.q_abs), to_dev_bf16(p.b.cache), to_dev(p.b.block_table),
                                    i32([0, 2, 4, 9]), i32(p.kv), p.mask(), sm_scale=p.b.sm_scale, o=o, status=st)
    assert int(st) == BAD_INDEX and (o[4:] == 3.0).all()
    p.check(o, lse, [0, 1])


def test_tree_attention_more_requests_than_threads():
    """Several requests to a thread in the search for a worker's piece, empty ones among them."""
    rng = np.random.default_rng(4)
    nodes, kv = rng.integers(0, 3, 700), rng.integers(0, 200, 700)
    p = Problem(15, nodes.tolist(), kv.tolist(), 3, 16, False)
    o, lse, st = p.run(pad=1)
    assert st == 0
    p.check(o, lse, list(range(0, 700, 13)) + [699])


@pytest.mark.parametrize("bs", [1, 16, 64])
def test_tree_attention_forced_timeout(monkeypatch, bs):
    """One wait that nothing satisfies gives up and is reported; the next call is right again."""
    p = Problem(16, [3, 2], [500, 40], 16, bs, True)
    monkeypatch.setenv("MLA_TEST_FORCE_TIMEOUT_NS", "2000000")
    assert p.run()[2] == 1
    monkeypatch.delenv("MLA_TEST_FORCE_TIMEOUT_NS")
    o, lse, st = p.run()
    assert st == 0
    p.check(o, lse)


def test_tree_attention_no_lse_and_own_workspace():
    import chunked_prefill_attention_ragged_gb300 as mla
    p = Problem(12, [3], [5000], 16, 64, True)
    o, lse, _ = p.run()
    b = p.b
    ws = torch.full((mla.mla_tree_workspace(3, 16),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN everywhere
    o2, none = mla.mla_tree_attention(to_dev_bf16(b.q_abs), to_dev_bf16(b.cache), to_dev(b.block_table),
                                      i32(b.qo_indptr), i32(p.kv), p.mask(), sm_scale=b.sm_scale, return_lse=False,
                                      workspace=ws)
    assert none is None and np.array_equal(bits_of(o), bits_of(o2))
    with pytest.raises(mla.MlaError):
        mla.mla_tree_attention(to_dev_bf16(b.q_abs), to_dev_bf16(b.cache), to_dev(b.block_table), i32(b.qo_indptr),
                               i32(p.kv), p.mask(), sm_scale=b.sm_scale, workspace=ws[:-16])
    with pytest.raises(ValueError):
        mla.mla_tree_attention(to_dev_bf16(b.q_abs), to_dev_bf16(b.cache), to_dev(b.block_table), i32(b.qo_indptr),
                               i32([5000, 1]), p.mask(), sm_scale=b.sm_scale)


def test_tree_attention_on_two_streams_at_once():
    ps = [Problem(20 + k, [4, 1], [9000 + k, 300], 16, 64, True) for k in range(2)]
    alone = [p.run() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    import chunked_prefill_attention_ragged_gb300 as mla
    args = [(to_dev_bf16(p.b.q_abs), to_dev_bf16(p.b.cache), to_dev(p.b.block_table), i32(p.b.qo_indptr), i32(p.kv),
             p.mask()) for p in ps]
    torch.cuda.synchronize()
    for _ in range(10):
        outs = [mla.mla_tree_attention(*a, sm_scale=p.b.sm_scale, stream=s) for a, p, s in zip(args, ps, streams)]
    torch.cuda.synchronize()
    for (o, lse), want in zip(outs, alone):
        assert np.array_equal(bits_of(o), bits_of(want[0])) and torch.equal(lse, want[1])


def test_tree_attention_cache_past_32_bit_offsets():
    """Rows whose byte and element offsets both pass 2^32 (a cache of 10 GB)."""
    import chunked_prefill_attention_ragged_gb300 as mla
    blocks = 2 ** 32 // (64 * 576) + 20000
    p = Problem(14, [2], [200], 4, 64, True)
    cache = torch.zeros((blocks, 64, 576), dtype=torch.bfloat16, device="cuda")
    where = np.array([blocks - 1, 3, blocks - 700, 2 ** 32 // (64 * 576) + 5])
    cache[torch.from_numpy(where).cuda()] = to_dev_bf16(p.b.cache[p.b.block_table[0, :4]])
    o, lse = mla.mla_tree_attention(to_dev_bf16(p.b.q_abs), cache, i32(where[None]), i32([0, 2]), i32([200]), p.mask(),
                                    sm_scale=p.b.sm_scale)
    torch.cuda.synchronize()
    p.check(o, lse)


# ------------------------------------------------------------------------------------- commit
@pytest.mark.parametrize("layers,entry,bs,batch,nodes", [(1, 576, 64, 1, 3), (3, 576, 16, 5, 20), (2, 8, 4, 9, 64),
                                                         (60, 576, 64, 4, 9), (1, 64, 1, 2, 300)])
def test_tree_commit(layers, entry, bs, batch, nodes):
    import chunked_prefill_attention_ragged_gb300 as mla
    rng = np.random.default_rng(layers * 7 + nodes)
    seq = rng.integers(0, 40, batch)
    need = -(-(seq + nodes) // bs)
    blocks = int(need.sum()) + 2
    perm = rng.permutation(blocks)
    table, at = np.full((batch, int(need.max())), -1, dtype=np.int32), 0
    for r in range(batch):
        table[r, :need[r]] = perm[at:at + need[r]]
        at += need[r]
    width = nodes
    counts = rng.integers(0, width + 1, batch)
    counts[0] = width if batch > 1 else 2
    paths = np.full((batch, width), -1)
    for r in range(batch):
        paths[r, :counts[r]] = np.sort(rng.permutation(nodes)[:counts[r]])
    bits = rng.integers(0, 1 << 16, (layers, blocks, bs, entry), dtype=np.uint16)   # any bits, NaN among them
    cache, st = to_dev_bf16(bits), new_status()
    mla.mla_tree_commit(cache if layers > 1 else cache[0], to_dev(table), i32(seq), i32(paths), i32(counts), status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    np.testing.assert_array_equal(bits_of(cache), tree_commit(bits, table, seq, paths, counts))


def test_tree_commit_bad_input():
    import chunked_prefill_attention_ragged_gb300 as mla
    rng = np.random.default_rng(2)
    bits = rng.integers(0, 1 << 16, (4, 4, 8), dtype=np.uint16)
    table = np.array([[2, 0], [1, 7]], dtype=np.int32)

    def go(seq, paths, counts):
        cache, st = to_dev_bf16(bits), new_status()
        mla.mla_tree_commit(cache, to_dev(table), i32(seq), i32(paths), i32(counts), status=st)
        torch.cuda.synchronize()
        return bits_of(cache), int(st)

    want = bits.copy()
    want[2, 1] = bits[2, 3]
    # the same node twice: the path ends before it; a count beyond the row; a block that is not there
    got, st = go([1, 0], [[2, 2, 3], [0, 1, 2]], [3, 3])
    assert st == BAD_INDEX and np.array_equal(got, want)
    got, st = go([1, 0], [[2, 1, 3], [0, 1, 2]], [2, 9])
    assert st == BAD_INDEX and np.array_equal(got, want)
    got, st = go([1, 0], [[2, 90, 91], [6, -1, -1]], [2, 1])
    assert st == BAD_INDEX and np.array_equal(got, want)
    got, st = go([1, -4], [[2, -1, -1], [1, 2, 3]], [1, 3])
    assert st == BAD_INDEX and np.array_equal(got, want)


# --------------------------------------------------------------------------- all of it, as used
class Serving:
    """Requests that grow by accepted drafts, step after step, on the GPU and in the oracle."""

    def __init__(self, seed, batch, heads, bs, most_nodes, steps):
        self.rng = np.random.default_rng(seed)
        self.batch, self.heads, self.bs, self.most = batch, heads, bs, most_nodes
        self.width = -(-(60 + steps * most_nodes + most_nodes) // bs)
        self.blocks = batch * self.width + 2
        self.tokens = batch * most_nodes
        self.words = -(-most_nodes // 64)
        self.seq = self.rng.integers(1, 60, batch)
        seq = self.seq
        stack = self.rng.permutation(self.blocks).tolist()
        self.table, self.held = np.full((batch, self.width), -1), np.zeros(batch, dtype=np.int64)
        _, _, slots, self.table, self.held, self.stack, _ = update_block_table(
            np.zeros(batch, int), seq, self.table, self.held, stack, bs, self.blocks, int(seq.sum()))
        self.cache = np.full((self.blocks, bs, 576), 0x7FC0, dtype=np.uint16)    # NaN where nothing is stored
        self.cache.reshape(-1, 576)[slots] = wl.to_bf16_bits(self.rng.standard_normal((len(slots), 576)).astype(np.float32))
        free = np.full(self.blocks, -1)
        free[:len(self.stack)] = self.stack
        # the program's state on the device
        self.d = dict(seq=i32(seq), new=i32(np.zeros(batch)), table=i32(self.table), held=i32(self.held), free=i32(free),
                      count=i32([len(self.stack)]), cache=to_dev_bf16(self.cache), status=new_status(),
                      parents=i32(np.full(self.tokens, -1)), paths=i32(np.full((batch, most_nodes), -1)),
                      counts=i32(np.zeros(batch)),
                      q=torch.zeros((self.tokens, heads, 576), dtype=torch.bfloat16, device="cuda"),
                      latent=torch.zeros((self.tokens, 576), dtype=torch.bfloat16, device="cuda"),
                      qo=i32(np.zeros(batch + 1)), kv=i32(np.zeros(batch)),
                      slots=torch.zeros(self.tokens, dtype=torch.int64, device="cuda"),
                      mask=torch.zeros((self.tokens, self.words), dtype=torch.int64, device="cuda"),
                      pos=i32(np.zeros(self.tokens)),
                      o=torch.zeros((self.tokens, heads, 512), dtype=torch.bfloat16, device="cuda"),
                      lse=torch.zeros((self.tokens, heads), dtype=torch.float32, device="cuda"))

    def draw(self):
        """The next drafts, into the device buffers; the accepted path is a chain of the tree."""
        r, d = self.rng, self.d
        self.nodes = r.integers(1, self.most + 1, self.batch)
        self.trees = [random_parents(r, int(n), 4) for n in self.nodes]
        self.accepted = []
        for t in self.trees:
            chain, at = [], int(r.integers(0, len(t)))
            while at >= 0:
                chain.append(at)
                at = int(t[at])
            self.accepted.append(chain[::-1])
        n = int(self.nodes.sum())
        self.q = wl.to_bf16_bits(r.standard_normal((n, self.heads, 576)).astype(np.float32))
        self.latent = wl.to_bf16_bits(r.standard_normal((n, 576)).astype(np.float32))
        paths = np.full((self.batch, self.most), -1)
        for k, c in enumerate(self.accepted):
            paths[k, :len(c)] = c
        d["new"].copy_(i32(self.nodes))
        d["parents"][:n] = i32(np.concatenate(self.trees))
        d["q"][:n] = to_dev_bf16(self.q)
        d["latent"][:n] = to_dev_bf16(self.latent)
        d["paths"].copy_(i32(paths))
        d["counts"].copy_(i32([len(c) for c in self.accepted]))

    def step_gpu(self):
        """What a server runs for one step: every length stays on the device."""
        import chunked_prefill_attention_ragged_gb300 as mla
        d = self.d
        mla.mla_block_table_update(d["seq"], d["new"], d["table"], d["held"], d["free"], d["count"], self.bs,
                                   self.tokens, d["qo"], d["kv"], d["slots"], d["status"])
        mla.mla_cache_write(d["cache"], d["latent"], d["slots"], d["status"])
        mla.mla_tree_mask(d["parents"], d["qo"], self.words, d["kv"], d["mask"], d["pos"], d["status"])
        mla.mla_tree_attention(d["q"], d["cache"], d["table"], d["qo"], d["kv"], d["mask"], sm_scale=wl.DEFAULT_SM_SCALE,
                               o=d["o"], lse=d["lse"], status=d["status"])
        mla.mla_tree_commit(d["cache"], d["table"], d["seq"], d["paths"], d["counts"], d["status"])
        d["seq"] += d["counts"]

    def step_oracle_and_check(self):
        d = self.d
        qo, kv, slots, self.table, self.held, self.stack, short = update_block_table(
            self.seq, self.nodes, self.table, self.held, self.stack, self.bs, self.blocks, self.tokens)
        assert not short and int(d["status"]) == 0
        np.testing.assert_array_equal(d["qo"].cpu().numpy(), qo)
        np.testing.assert_array_equal(d["kv"].cpu().numpy(), kv)
        np.testing.assert_array_equal(d["slots"].cpu().numpy(), slots)
        np.testing.assert_array_equal(d["table"].cpu().numpy(), self.table)
        assert d["free"].cpu().numpy()[:int(d["count"])].tolist() == self.stack
        n = int(qo[-1])
        self.cache.reshape(-1, 576)[slots[:n]] = self.latent
        o, lse = f64_of_bf16(d["o"]), d["lse"].double().cpu().numpy()
        for r in range(self.batch):
            rows = slice(int(qo[r]), int(qo[r + 1]))
            seen, depth = tree_visibility(self.trees[r])
            np.testing.assert_array_equal(d["pos"][rows].cpu().numpy(), self.seq[r] + depth)
            p = np.arange(int(kv[r]))
            keys = bf16_bits_to_f64(self.cache[self.table[r, p // self.bs], p % self.bs])
            q = bf16_bits_to_f64(self.q[rows])
            want_o, want_l = tree_attention(q, keys, seen, sm_scale=wl.DEFAULT_SM_SCALE)
            tol_o, tol_l = bounds(q, keys, seen, want_o, sm_scale=wl.DEFAULT_SM_SCALE, cap=0.0)
            assert (np.abs(o[rows] - want_o) <= tol_o).all() and (np.abs(lse[rows] - want_l) <= tol_l).all()
        paths = d["paths"].cpu().numpy()
        self.cache = tree_commit(self.cache[None], self.table, self.seq, paths, [len(c) for c in self.accepted])[0]
        self.seq = self.seq + np.array([len(c) for c in self.accepted])
        np.testing.assert_array_equal(d["seq"].cpu().numpy(), self.seq)
        np.testing.assert_array_equal(bits_of(d["cache"]), self.cache)


@pytest.mark.parametrize("batch,heads,bs,most", [(3, 4, 16, 9), (5, 16, 64, 20)])
def test_serving_steps(batch, heads, bs, most):
    s = Serving(batch, batch, heads, bs, most, 4)
    for _ in range(4):
        s.draw()
        s.step_gpu()
        torch.cuda.synchronize()
        s.step_oracle_and_check()


def test_serving_steps_replayed_from_one_graph():
    """The step captured once; replays follow the lengths, tables and trees on the device."""
    s = Serving(9, 4, 8, 16, 12, 5)
    s.draw()
    s.step_gpu()           # one-time set-up happens outside the capture
    torch.cuda.synchronize()
    s.step_oracle_and_check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step_gpu()
    torch.cuda.synchronize()
    for _ in range(4):
        s.draw()
        graph.replay()
        torch.cuda.synchronize()
        s.step_oracle_and_check()


# ----------------------------------------------------------------------------------- refusals
def test_python_refusals():
    import chunked_prefill_attention_ragged_gb300 as mla
    p = Problem(40, [3, 2], [100, 40], 4, 64, True)
    b = p.b
    q, cache, table, qo, kv, mask = (to_dev_bf16(b.q_abs), to_dev_bf16(b.cache), to_dev(b.block_table),
                                     i32(b.qo_indptr), i32(p.kv), p.mask())

    def attention(**kw):
        a = dict(q=q, cache=cache, table=table, qo=qo, kv=kv, mask=mask, extra={})
        a.update(kw)
        mla.mla_tree_attention(a["q"], a["cache"], a["table"], a["qo"], a["kv"], a["mask"], sm_scale=0.1, **a["extra"])

    attention()
    for kw, err in [(dict(q=q.float()), TypeError), (dict(q=q.transpose(0, 1)), ValueError), (dict(q=q[:, :, :512]), ValueError),
                    (dict(cache=cache.half()), TypeError), (dict(cache=cache[:, ::2]), ValueError),
                    (dict(table=table.long()), TypeError), (dict(table=table[0]), ValueError),
                    (dict(qo=qo[:-1]), ValueError), (dict(kv=kv.cpu()), TypeError), (dict(mask=mask[:-1]), ValueError),
                    (dict(mask=mask.int()), TypeError), (dict(extra=dict(o=torch.empty_like(q))), ValueError),
                    (dict(extra=dict(lse=torch.zeros(5, 5, device="cuda"))), ValueError),
                    (dict(extra=dict(workspace=torch.zeros(1 << 20, device="cuda"))), TypeError),
                    (dict(extra=dict(status=torch.zeros(1, device="cuda"))), TypeError),
                    (dict(extra=dict(logits_soft_cap=float("nan"))), mla.MlaError)]:
        with pytest.raises(err):
            attention(**kw)
    with pytest.raises(ValueError):
        mla.mla_tree_mask(i32([[-1]]), i32([0, 1]), 1)
    with pytest.raises(ValueError):
        mla.mla_tree_mask(i32([-1]), i32([0, 1]), 0)
    with pytest.raises(ValueError):
        mla.mla_tree_mask(i32([-1]), i32([0, 1]), 1, mask=torch.zeros(1, 2, dtype=torch.int64, device="cuda"))
    seq = i32([3])
    with pytest.raises(mla.MlaError):   # in place over the lengths that are read again
        mla.mla_block_table_update(seq, i32([1]), i32([[-1]]), i32([0]), i32([0]), i32([1]), 4, 1, kv_lens=seq)
    with pytest.raises(ValueError):
        mla.mla_block_table_update(seq, i32([1, 2]), i32([[-1]]), i32([0]), i32([0]), i32([1]), 4)
    with pytest.raises(mla.MlaError):
        mla.mla_block_table_update(seq, i32([1]), i32([[-1]]), i32([0]), i32([0]), i32([1]), 0)
    with pytest.raises(ValueError):
        mla.mla_tree_commit(cache[0], table, kv, i32([[0], [0]]), i32([0, 0]))
    with pytest.raises(mla.MlaError):   # rows of no multiple of 16 bytes
        mla.mla_tree_commit(torch.zeros(2, 4, 12, dtype=torch.bfloat16, device="cuda"), table, kv, i32([[0], [0]]), i32([0, 0]))
    torch.cuda.synchronize()
