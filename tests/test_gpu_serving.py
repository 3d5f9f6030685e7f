"""Decoding steps as a server runs them: requests grow, rest, finish and are replaced, and some find no room."""
import numpy as np
import pytest

from chunked_prefill_attention_ragged_gb300 import workloads as wl
from gpu_util import bits_of, f64_of_bf16, to_dev, to_dev_bf16
from oracle import bf16_bits_to_f64, tree_attention, tree_commit, tree_visibility, update_block_table
from test_gpu_speculative import BAD_INDEX, NO_BLOCKS, Serving, bounds, i32, new_status, random_parents

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


class Server(Serving):
    """Slots that are empty, decode, rest for a step, accept nothing, finish, and take a new prompt."""

    def turn_over(self):
        """Between two steps: some requests finish, some empty slots take a prompt (blocks given back and taken
        by one call, its rows stored).  Returns what happened, for the tests to know that all of it did."""
        import chunked_prefill_attention_ragged_gb300 as mla
        r, d = self.rng, self.d
        new = np.zeros(self.batch, dtype=np.int64)
        done = r.random(self.batch) < 0.3
        taken = (done | (self.seq == 0)) & (r.random(self.batch) < 0.6)
        new[taken] = r.integers(1, 60, int(taken.sum()))
        seq = np.where(done | taken, 0, self.seq)
        n = int(new.sum())
        rows = wl.to_bf16_bits(r.standard_normal((n, 576)).astype(np.float32))
        status = new_status()
        _, _, slots = mla.mla_block_table_update(i32(seq), i32(new), d["table"], d["held"], d["free"], d["count"], self.bs,
                                                 n, status=status)
        if n:
            mla.mla_cache_write(d["cache"], to_dev_bf16(rows), slots, status)
        self.seq = seq + new
        d["seq"].copy_(i32(self.seq))
        _, _, want, self.table, self.held, self.stack, short = update_block_table(
            seq, new, self.table, self.held, self.stack, self.bs, self.blocks, n)
        assert not short and int(status) == 0
        np.testing.assert_array_equal(slots.cpu().numpy(), want)
        self.cache.reshape(-1, 576)[want] = rows
        return bool((done & ~taken).any()), bool((done & taken).any())

    def draw(self):
        r, d = self.rng, self.d
        self.nodes = np.where((self.seq == 0) | (r.random(self.batch) < 0.25), 0, r.integers(1, self.most + 1, self.batch))
        self.trees = [random_parents(r, int(n), 4) for n in self.nodes]
        self.accepted = []
        for t in self.trees:
            chain, at = [], int(r.integers(-1, len(t))) if len(t) else -1
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
        if n:
            d["parents"][:n] = i32(np.concatenate(self.trees))
            d["q"][:n] = to_dev_bf16(self.q)
            d["latent"][:n] = to_dev_bf16(self.latent)
        d["paths"].copy_(i32(paths))
        d["counts"].copy_(i32([len(c) for c in self.accepted]))
        return bool(((self.seq > 0) & (self.nodes == 0)).any()), any(len(t) and not c for t, c in zip(self.trees, self.accepted))


@pytest.mark.parametrize("replayed", [False, True])
@pytest.mark.parametrize("batch,heads,bs,most", [(6, 4, 16, 9), (9, 3, 5, 12), (5, 16, 64, 20)])
def test_requests_grow_rest_finish_and_are_replaced(batch, heads, bs, most, replayed):
    s = Server(50 + batch, batch, heads, bs, most, 12)
    seen, graph = [], None
    for step in range(12):
        what = s.turn_over() if step else (False, False)
        seen.append(what + s.draw())
        if graph is None:
            s.step_gpu()
        else:
            graph.replay()
        torch.cuda.synchronize()
        s.step_oracle_and_check()
        if replayed and step == 0:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                s.step_gpu()
            torch.cuda.synchronize()
    assert np.array(seen).any(axis=0).all(), "every kind of step is among them"


@pytest.mark.parametrize("pad", [0, 9000])   # block tables by one CTA, and from a grid
@pytest.mark.parametrize("why", ["stack", "row"])
def test_a_request_without_room_leaves_the_others_alone(pad, why):
    """The whole step with one request that is not served, nothing looked at in between, its drafts
    "accepted": unused entries of its row name blocks of the others."""
    import chunked_prefill_attention_ragged_gb300 as mla
    rng = np.random.default_rng(61)
    bs, heads, width = 16, 4, 4
    seq, nodes = np.array([30, 30, 15]), [5, 9, 40] if why == "row" else [5, 9, 20]
    if why == "row":
        seq[2] = 30
    held = -(-seq // bs)
    table = np.zeros((3, width), dtype=np.int64)
    ids = rng.permutation(12)
    ids = np.concatenate([[0], ids[ids != 0]])       # block 0 is request 0's first
    at = 0
    for r in range(3):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    stack = ids[at:at + (2 if why == "stack" else 6)].tolist()
    trees = [random_parents(rng, n, 4) for n in nodes]
    tokens = sum(nodes) + pad
    cache = wl.to_bf16_bits(rng.standard_normal((12, bs, 576)).astype(np.float32))
    latent = wl.to_bf16_bits(rng.standard_normal((tokens, 576)).astype(np.float32))
    q = wl.to_bf16_bits(rng.standard_normal((tokens, heads, 576)).astype(np.float32))
    paths, counts = np.array([[1, 3, -1], [0, 4, 8], [2, 17, 19]]), [2, 3, 3]
    want = update_block_table(seq, nodes, table, held, stack, bs, 12, tokens)
    d_cache, d_table, st = to_dev_bf16(cache), i32(table), new_status()
    qo, kv, slots = mla.mla_block_table_update(i32(seq), i32(nodes), d_table, i32(held), i32(stack + [-1] * 4), i32([len(stack)]),
                                               bs, tokens, status=st)
    assert int(st) == (NO_BLOCKS if why == "stack" else BAD_INDEX)
    mla.mla_cache_write(d_cache, to_dev_bf16(latent), slots)
    parents = np.concatenate(trees + [np.full(pad, -1)])
    mask, _ = mla.mla_tree_mask(i32(parents), qo, 1, kv_lens=kv)
    d_q = to_dev_bf16(q)
    o, lse = mla.mla_tree_attention(d_q, d_cache, d_table, qo, kv, mask, sm_scale=wl.DEFAULT_SM_SCALE)
    stored = bits_of(d_cache)
    mla.mla_tree_commit(d_cache, d_table, i32(seq), i32(paths), i32(counts))
    torch.cuda.synchronize()
    np.testing.assert_array_equal(slots.cpu().numpy(), want[2])
    live = want[2] >= 0
    cache.reshape(-1, 576)[want[2][live]] = latent[live]
    np.testing.assert_array_equal(stored, cache)
    o, lse, qo = f64_of_bf16(o), lse.double().cpu().numpy(), want[0]
    for r in range(2):
        rows, pos = slice(int(qo[r]), int(qo[r + 1])), np.arange(seq[r] + nodes[r])
        keys, qr = bf16_bits_to_f64(cache[want[3][r, pos // bs], pos % bs]), bf16_bits_to_f64(q[rows])
        seen = tree_visibility(trees[r])[0]
        want_o, want_l = tree_attention(qr, keys, seen, sm_scale=wl.DEFAULT_SM_SCALE)
        tol_o, tol_l = bounds(qr, keys, seen, want_o, sm_scale=wl.DEFAULT_SM_SCALE, cap=0.0)
        assert (np.abs(o[rows] - want_o) <= tol_o).all() and (np.abs(lse[rows] - want_l) <= tol_l).all()
    moved = tree_commit(cache[None], want[3], seq, paths, counts[:2] + [0])[0]
    others = np.ones(12, dtype=bool)
    others[want[3][2, :held[2]]] = False         # (its own rows are its own affair)
    np.testing.assert_array_equal(bits_of(d_cache)[others], moved[others])
