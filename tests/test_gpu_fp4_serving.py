"""A server's step over a cache of 4-bit entries: blocks and slots, trees, new tokens appended (with their queries), tree
attention, drafts verified, accepted entries moved; step after step, call by call and from one graph."""
import numpy as np
import pytest

from chunked_prefill_attention_ragged_gb300 import workloads as wl
from gpu_util import bits_of, f64_of_bf16, to_dev, to_dev_bf16
from oracle import (bf16_bits_to_f64, fp4_values, rotate, tree_attention, tree_commit, tree_visibility, update_block_table,
                    verify_tree)
from test_gpu_fp4_attention import fast_entries
from test_gpu_fp4_cache import Tokens, angles
from test_gpu_speculative import bounds, i32, new_status

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


class Server:
    def __init__(self, seed, batch, heads, bs, most, steps, vocab, drawn):
        r = self.r = np.random.default_rng(seed)
        self.batch, self.heads, self.bs, self.most, self.vocab, self.drawn = batch, heads, bs, most, vocab, drawn
        self.width = -(-(60 + (steps + 1) * most) // bs)
        self.blocks, self.tokens, self.words = batch * self.width + 2, batch * most, -(-most // 64)
        self.seq = r.integers(1, 60, batch)
        stack = r.permutation(self.blocks).tolist()
        self.table, self.held = np.full((batch, self.width), -1), np.zeros(batch, dtype=np.int64)
        _, _, slots, self.table, self.held, self.stack, _ = update_block_table(
            np.zeros(batch, int), self.seq, self.table, self.held, stack, bs, self.blocks, int(self.seq.sum()))
        self.cache = np.full((self.blocks, bs, 400), 0xFF, dtype=np.uint8)   # NaN where nothing is stored
        self.cache.reshape(-1, 400)[slots] = fast_entries(wl.to_bf16_bits(r.standard_normal((len(slots), 576)).astype(np.float32)))
        free = np.full(self.blocks, -1)
        free[:len(self.stack)] = self.stack
        self.angles, self.root = angles(60 + (steps + 1) * most), r.integers(0, vocab, batch)
        self.weight = wl.to_bf16_bits((1 + r.standard_normal(512) / 8).astype(np.float32))
        t = self.tokens
        zeros = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        self.d = dict(seq=i32(self.seq), new=i32(np.zeros(batch)), table=i32(self.table), held=i32(self.held), free=i32(free),
                      count=i32([len(self.stack)]), cache=to_dev(self.cache), status=new_status(), parents=i32(np.full(t, -1)),
                      drafts=i32(np.zeros(t)), ids=i32(np.zeros(t)), next=i32(self.root), paths=i32(np.full((batch, most), -1)),
                      counts=i32(np.zeros(batch)), q=zeros(t, heads, 576, dtype=torch.bfloat16),
                      latent=zeros(t, 640, dtype=torch.bfloat16), qo=i32(np.zeros(batch + 1)), kv=i32(np.zeros(batch)),
                      slots=zeros(t, dtype=torch.int64), mask=zeros(t, self.words, dtype=torch.int64), pos=i32(np.zeros(t)),
                      o=zeros(t, heads, 512, dtype=torch.bfloat16), lse=zeros(t, heads), u=zeros(t), last=zeros(batch),
                      target=zeros(t, vocab), draft=torch.full((t, vocab), 1 / vocab, device="cuda"),
                      weight=to_dev_bf16(self.weight), angles=to_dev(self.angles),
                      head=torch.from_numpy(r.standard_normal((512, vocab)).astype(np.float32)).cuda())

    def draw(self):
        r, d = self.r, self.d
        self.nodes = r.integers(1, self.most + 1, self.batch)
        self.trees = [np.array([-1] + [int(r.integers(max(0, i - 4), i)) for i in range(1, n)]) for n in self.nodes]
        n = int(self.nodes.sum())
        self.n, self.latent = n, wl.to_bf16_bits(r.standard_normal((n, 576)).astype(np.float32))
        self.q = wl.to_bf16_bits(r.standard_normal((n, self.heads, 576)).astype(np.float32))
        self.drafts, self.u, self.last = r.integers(0, self.vocab, n), r.random(n, dtype=np.float32), r.random(self.batch, dtype=np.float32)
        d["new"].copy_(i32(self.nodes))
        d["parents"][:n] = i32(np.concatenate(self.trees))
        d["drafts"][:n] = i32(self.drafts)
        d["q"][:n] = to_dev_bf16(self.q)
        d["latent"][:n, :576] = to_dev_bf16(self.latent)
        d["u"][:n] = torch.from_numpy(self.u).cuda()
        d["last"].copy_(torch.from_numpy(self.last))

    def step_gpu(self):
        """Every length stays on the device; the last step's token is the root of this step's tree."""
        import chunked_prefill_attention_ragged_gb300 as mla
        d = self.d
        mla.mla_block_table_update(d["seq"], d["new"], d["table"], d["held"], d["free"], d["count"], self.bs, self.tokens,
                                   d["qo"], d["kv"], d["slots"], d["status"])
        mla.mla_tree_mask(d["parents"], d["qo"], self.words, d["kv"], d["mask"], d["pos"], d["status"])
        mla.mla_cache_append(d["cache"], d["latent"][:, :576], d["slots"], d["pos"], d["angles"], norm_weight=d["weight"],
                             q_rope=d["q"][..., 512:], status=d["status"])
        mla.mla_tree_attention_fp4(d["q"], d["cache"], d["table"], d["qo"], d["kv"], d["mask"], sm_scale=wl.DEFAULT_SM_SCALE,
                                   o=d["o"], lse=d["lse"], status=d["status"])
        d["target"].copy_(torch.softmax(d["o"].float().sum(1) @ d["head"], -1))
        d["ids"].copy_(d["drafts"]).index_copy_(0, d["qo"][:-1].long(), d["next"])
        mla.mla_tree_verify(d["target"], d["ids"], d["qo"], d["u"], d["last"], self.most, d["parents"],
                            d["draft"] if self.drawn else None, d["paths"], d["counts"], d["next"], d["status"])
        mla.mla_tree_commit(d["cache"].view(torch.bfloat16), d["table"], d["seq"], d["paths"], d["counts"], d["status"])
        d["seq"] += d["counts"]

    def step_oracle_and_check(self):
        d, n = self.d, self.n
        qo, kv, slots, self.table, self.held, self.stack, short = update_block_table(
            self.seq, self.nodes, self.table, self.held, self.stack, self.bs, self.blocks, self.tokens)
        assert not short and int(d["status"]) == 0
        np.testing.assert_array_equal(d["table"].cpu().numpy(), self.table)
        np.testing.assert_array_equal(d["slots"].cpu().numpy(), slots)
        got = d["cache"].cpu().numpy()
        paths, counts, following = d["paths"].cpu().numpy(), d["counts"].cpu().numpy(), d["next"].cpu().numpy()
        # the entries as they were before they moved: a moved one is where its position was
        rows = got.reshape(-1, 400)[slots[:n]]
        pos = np.concatenate([self.seq[r] + tree_visibility(t)[1] for r, t in enumerate(self.trees)])
        np.testing.assert_array_equal(d["pos"][:n].cpu().numpy(), pos)
        for r in range(self.batch):
            for i, k in enumerate(paths[r, :counts[r]]):
                rows[qo[r] + k] = got[self.table[r, (self.seq[r] + i) // self.bs], (self.seq[r] + i) % self.bs]
        moved = {int(qo[r]) + i for r in range(self.batch) for i in range(counts[r])}
        kept = {int(qo[r]) + int(k) for r in range(self.batch) for k in paths[r, :counts[r]]}
        known = np.array([i in kept or i not in moved for i in range(n)])   # the others were overwritten by a move
        c = Tokens.__new__(Tokens)
        c.kind, c.latent, c.weight, c.pos, c.table, c.interleaved, c.t = ("fp4", self.latent[known], self.weight, pos[known],
                                                                         self.angles, True, int(known.sum()))
        c.check_rows(rows[known])
        want = rotate(bf16_bits_to_f64(self.q)[..., 512:], pos, self.angles, True)
        q = f64_of_bf16(d["q"][:n])
        assert (np.abs(q[..., 512:] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * 8).all()
        np.testing.assert_array_equal(bits_of(d["q"][:n])[..., :512], self.q[..., :512])
        before = self.cache.copy()
        before.reshape(-1, 400)[slots[:n]] = rows
        o, lse, target = f64_of_bf16(d["o"]), d["lse"].double().cpu().numpy(), d["target"].double().cpu().numpy()
        for r, tree in enumerate(self.trees):
            mine = slice(int(qo[r]), int(qo[r + 1]))
            seen, _ = tree_visibility(tree)
            # an entry that a move overwrote is not known any more: rows that do not see one are compared
            whole = ~(seen & ~known[mine]).any(1)
            p = np.arange(int(kv[r]))
            keys = fp4_values(before[self.table[r, p // self.bs], p % self.bs])
            want_o, want_l = tree_attention(q[mine], keys, seen, sm_scale=wl.DEFAULT_SM_SCALE)
            tol_o, tol_l = bounds(q[mine], keys, seen, want_o, sm_scale=wl.DEFAULT_SM_SCALE, cap=0.0)
            assert whole.any() and (np.abs(o[mine] - want_o) <= tol_o)[whole].all() and (np.abs(lse[mine] - want_l) <= tol_l)[whole].all()
            ids = self.drafts[mine].copy()
            ids[0] = self.root[r]
            path, token = verify_tree(target[mine], ids, tree, self.u[mine], self.last[r], self.most,
                                      np.full((len(ids), self.vocab), np.float32(1 / self.vocab)) if self.drawn else None)
            assert paths[r, :counts[r]].tolist() == path and (paths[r, counts[r]:] == -1).all() and following[r] == token
        self.cache = tree_commit(before[None], self.table, self.seq, paths, counts)[0]
        np.testing.assert_array_equal(got, self.cache)
        self.seq, self.root = self.seq + counts, following
        np.testing.assert_array_equal(d["seq"].cpu().numpy(), self.seq)
        return int(counts.sum()) - self.batch


@pytest.mark.parametrize("batch,heads,bs,most,vocab,drawn", [(3, 4, 16, 9, 11, True), (5, 16, 64, 20, 5, False), (2, 33, 7, 12, 7, True)])
def test_steps(batch, heads, bs, most, vocab, drawn):
    s = Server(batch, batch, heads, bs, most, 4, vocab, drawn)
    for _ in range(4):
        s.draw()
        s.step_gpu()
        torch.cuda.synchronize()
        s.step_oracle_and_check()


def test_steps_replayed_from_one_graph():
    s = Server(9, 4, 8, 16, 12, 5, 6, True)
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
