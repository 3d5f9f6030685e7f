"""Drafts verified against the target's probabilities: the same path and token as the oracle's."""
import numpy as np
import pytest

from gpu_util import Guarded, to_dev
from oracle import bf16_bits_to_f64, verify_tree
from chunked_prefill_attention_ragged_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BAD_INDEX = 2


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f32(x):
    return torch.tensor(np.asarray(x), dtype=torch.float32, device="cuda")


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


class Drafts:
    def __init__(self, seed, nodes, vocab, tree=True, drawn=True, bf16=False, close=0.5, peak=2.0, reach=3):
        r = np.random.default_rng(seed)
        self.nodes, self.vocab, self.bf16, self.tree, self.drawn = list(nodes), vocab, bf16, tree, drawn
        t = int(sum(nodes))
        logits = r.standard_normal((t, vocab)) * peak
        draft = softmax(logits + close * r.standard_normal((t, vocab)))
        target = softmax(logits)
        self.qo = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int64)
        self.parents, self.tokens = np.full(t, -1), np.zeros(t, dtype=np.int64)
        for k, n in enumerate(nodes):
            for i in range(n):
                at = self.qo[k] + i
                self.parents[at] = i - 1 if not tree else -1 if i == 0 else int(r.integers(max(0, i - reach), i))
                up = self.qo[k] + max(self.parents[at], 0)
                self.tokens[at] = r.choice(vocab, p=draft[up]) if drawn else np.argsort(-draft[up])[int(r.integers(0, min(3, vocab)))]
        kind = (lambda x: bf16_bits_to_f64(wl.to_bf16_bits(x.astype(np.float32)))) if bf16 else (lambda x: x.astype(np.float32).astype(np.float64))
        self.target, self.draft = kind(target), kind(draft) if drawn else None
        self.u, self.last = r.random(t, dtype=np.float32), r.random(len(nodes), dtype=np.float32)

    def dev(self, x):
        return None if x is None else torch.from_numpy(x.astype(np.float32)).cuda().to(torch.bfloat16 if self.bf16 else torch.float32)

    def run(self, most, pad=0, **kw):
        import chunked_prefill_attention_ragged_gb300 as mla
        b = len(self.nodes)
        acc, cnt, nxt = Guarded((b, most), torch.int32), Guarded((b,), torch.int32), Guarded((b,), torch.int32)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        more = lambda x, v: np.concatenate([x, np.full(pad, v)])  # noqa: E731
        rows = lambda x: None if x is None else np.concatenate([x, np.full((pad, self.vocab), np.nan)])  # noqa: E731
        a = dict(parents=i32(more(self.parents, 99)) if self.tree else None, draft_probs=self.dev(rows(self.draft)))
        a.update(kw)
        mla.mla_tree_verify(self.dev(rows(self.target)), i32(more(self.tokens, -9)), i32(self.qo), f32(more(self.u, np.nan)), f32(self.last),
                            most, accepted=acc.tensor, accepted_counts=cnt.tensor, next_tokens=nxt.tensor, status=st, **a)
        torch.cuda.synchronize()
        for g in (acc, cnt, nxt):
            g.check("outputs")
        return acc.tensor.cpu().numpy(), cnt.tensor.cpu().numpy(), nxt.tensor.cpu().numpy(), int(st)

    def want(self, most):
        b = len(self.nodes)
        acc, cnt, nxt = np.full((b, most), -1), np.zeros(b, dtype=int), np.full(b, -1)
        for r, n in enumerate(self.nodes):
            if not n:
                continue
            s = slice(int(self.qo[r]), int(self.qo[r + 1]))
            path, nxt[r] = verify_tree(self.target[s], self.tokens[s], self.parents[s], self.u[s], self.last[r], most,
                                       None if self.draft is None else self.draft[s])
            acc[r, :len(path)], cnt[r] = path, len(path)
        return acc, cnt, nxt

    def check(self, most, pad=0):
        got, want = self.run(most, pad), self.want(most)
        assert got[3] == 0
        for g, w, name in zip(got, want, ("accepted", "counts", "next")):
            np.testing.assert_array_equal(g, w, err_msg=name)
        return got


CASES = [([1], 2, False), ([1, 1, 1], 7, True), ([5], 1000, False), ([5, 0, 3, 1], 129, True), ([16] * 8, 1003, True),
         ([40, 7, 33], 515, True), ([6, 2], 16385, True), ([9, 12], 32768, True), ([4, 3], 70001, True), ([3, 5], 131072, False),
         ([70, 64, 65], 90, True)]


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("nodes,vocab,tree", CASES)
def test_verify(nodes, vocab, tree, bf16, drawn):
    p = Drafts(sum(nodes) + vocab, nodes, vocab, tree, drawn, bf16, peak=2.0 if vocab < 1000 else 3.5)
    p.check(max(nodes), pad=2)


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("seed", range(4))
def test_wide_trees_with_many_refusals(seed, drawn):
    """Bushy trees over a draft far from the target, over few tokens: children are refused one after another, some with
    the token of a sibling, until nothing may be left."""
    p = Drafts(seed, [30] * 40, [3, 5, 9, 700][seed], True, drawn, close=3.0, reach=30)
    got = p.check(30)
    assert got[1].min() == 1             # (somewhere all are refused)


@pytest.mark.parametrize("drawn", [True, False])
def test_a_path_that_is_full(drawn):
    p = Drafts(5, [12] * 20, 50, True, drawn, close=0.05)
    for most in (1, 2, 3):
        assert min(most, 2) <= p.check(most)[1].max() <= most


def test_more_nodes_than_are_held_at_once():
    p = Drafts(6, [700, 600], 30, True, True, close=0.02, reach=2)
    p.check(700)
    p = Drafts(7, [600, 550], 40, False, False, close=0.0, peak=9.0)
    p.check(600)


def test_nothing_left_of_the_target():
    """Target and draft alike where the draft's token is refused by its uniform of 1 (what is left has no mass), and a
    given token that has all of it."""
    p = Drafts(8, [2, 2], 600, False, True, close=0.0)
    p.draft = p.target.copy()
    p.u[:] = 1.0
    got = p.check(2)
    assert got[1].tolist() == [1, 1]
    p = Drafts(9, [2], 600, False, False)
    p.target[:] = 0
    p.target[:, 17] = 1
    p.tokens[:] = 17
    p.u[:] = 1.0
    got = p.check(2)
    assert got[1].tolist() == [1] and got[2].tolist() == [17]
    p.target[:] = 0
    assert p.run(2)[2].tolist() == [-1]


@pytest.mark.parametrize("last", [0.0, 0.9999999, 1.0, 2.0, float("nan")])
def test_ends_of_the_uniform(last):
    p = Drafts(10, [1, 1], 2000, False, False)
    p.target[:, :5] = 0
    p.target[:, 1990:] = 0
    p.last[:] = last
    got = p.run(1)
    assert got[2].tolist() == ([5, 5] if not last > 0 else [1989, 1989])


def test_probabilities_out_of_range():
    """Into [0, 1], a NaN as 0."""
    p = Drafts(11, [1], 64, False, False)
    p.target[0] = 0
    p.target[0, [3, 9, 20]] = [np.nan, -4.0, 7.0]
    assert p.run(1)[2].tolist() == [20]


def test_rows_that_are_no_probabilities():
    """Sums far past one: some token of the vocabulary, or -1; what was in the output does not stay."""
    d = Drafts(31, [4, 3], 70001, tree=True, drawn=False)
    d.target = np.full_like(d.target, 1e30)
    for value in (1e30, np.nan):
        d.target[:] = value
        acc, cnt, nxt, st = d.run(3)
        assert st == 0 and ((nxt >= -1) & (nxt < 70001)).all() and ((cnt >= 1) & (cnt <= 3)).all() and (acc[:, 0] == 0).all()
    assert (nxt == -1).all()


def test_bad_tokens_parents_and_rows():
    p = Drafts(12, [6, 4], 100, True, True, close=0.0)
    p.u[:] = 0
    p.parents[:] = [-1, 0, 1, 2, 0, 0, -1, 0, 1, 2]
    base = p.run(6)
    assert base[3] == 0 and base[0][0].tolist() == [0, 1, 2, 3, -1, -1]
    tokens = p.tokens.copy()
    for bad in (-1, 100, 1 << 30):
        p.tokens = tokens.copy()
        p.tokens[1] = bad
        got = p.run(6)
        assert got[3] == BAD_INDEX and got[0][0, 1] == 4
    p.tokens = tokens.copy()
    p.tokens[0] = -5                             # node 0's is not looked at
    assert p.run(6)[3] == 0
    p.tokens = tokens
    for bad in (2, 7, -2):
        q = p.parents.copy()
        q[2] = bad
        got = p.run(6, parents=i32(q))
        assert got[3] == BAD_INDEX and got[0][0].tolist() == [0, 1, -1, -1, -1, -1]
    q = p.parents.copy()
    q[1] = -1                                    # another root: never kept
    got = p.run(6, parents=i32(q))
    assert got[3] == 0 and got[0][0, 1] == 4
    p.qo = np.array([0, 6, 11])
    got = p.run(6)
    assert got[3] == BAD_INDEX and got[1].tolist()[1] == 0 and got[2][1] == -1 and (got[0][1] == -1).all()
    np.testing.assert_array_equal(got[0][0], base[0][0])


def test_the_kept_tokens_have_the_targets_distribution():
    """20000 requests of one node with two drawn children: the next token's counts, by chi-square (99.9999%: 15 tokens, 14
    degrees of freedom, 54)."""
    r = np.random.default_rng(13)
    n, v = 20000, 15
    p = Drafts(14, [3], v, True, True, close=1.0)
    target, draft = p.target[0], p.draft[0]
    p.nodes, p.qo = [3] * n, 3 * np.arange(n + 1)
    p.parents = np.tile([-1, 0, 0], n)
    p.tokens = r.choice(v, size=3 * n, p=draft / draft.sum())
    p.target, p.draft = np.tile(target, (3 * n, 1)), np.tile(draft, (3 * n, 1))
    p.u, p.last = r.random(3 * n, dtype=np.float32), r.random(n, dtype=np.float32)
    acc, cnt, nxt, st = p.run(3)
    first = np.where(cnt > 1, p.tokens[3 * np.arange(n) + np.maximum(acc[:, 1], 0)], nxt)
    seen, hope = np.bincount(first, minlength=v), n * target / target.sum()
    assert st == 0 and ((seen - hope) ** 2 / hope).sum() < 54


def test_refusals():
    import chunked_prefill_attention_ragged_gb300 as mla
    p = torch.full((2, 9), 1 / 9, device="cuda")
    ok = (i32([1, 2]), i32([0, 2]), f32([0, 0]), f32([0]), 2)
    mla.mla_tree_verify(p, *ok)
    with pytest.raises(TypeError):
        mla.mla_tree_verify(p.double(), *ok)
    with pytest.raises(TypeError):
        mla.mla_tree_verify(p, *ok, draft_probs=p.bfloat16())
    with pytest.raises(ValueError):
        mla.mla_tree_verify(p, *ok, draft_probs=p[:1])
    with pytest.raises(ValueError):
        mla.mla_tree_verify(p, *ok[:4], 0)
    with pytest.raises(ValueError):
        mla.mla_tree_verify(p[:, :8], *ok)
    with pytest.raises(ValueError):
        mla.mla_tree_verify(p, ok[0][:1], *ok[1:])
    with pytest.raises(ValueError, match="status"):
        mla.mla_tree_verify(p, *ok, status=torch.zeros(0, dtype=torch.int32, device="cuda"))


def test_replayed_and_on_another_stream():
    import chunked_prefill_attention_ragged_gb300 as mla
    a = Drafts(15, [7, 9, 4], 40000)
    b = Drafts(16, [7, 9, 4], 40000)
    d = dict(target=a.dev(a.target), draft=a.dev(a.draft), tokens=i32(a.tokens), parents=i32(a.parents), u=f32(a.u), last=f32(a.last))
    qo, graph, stream = i32(a.qo), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        out = mla.mla_tree_verify(d["target"], d["tokens"], qo, d["u"], d["last"], 9, d["parents"], d["draft"])
    for x in (b, a):
        for k, v in dict(target=x.dev(x.target), draft=x.dev(x.draft), tokens=i32(x.tokens), parents=i32(x.parents), u=f32(x.u),
                         last=f32(x.last)).items():
            d[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(out, x.want(9)):
            np.testing.assert_array_equal(g.cpu().numpy(), w)
    other = mla.mla_tree_verify(d["target"], d["tokens"], qo, d["u"], d["last"], 9, d["parents"], d["draft"], stream=stream)
    torch.cuda.synchronize()
    for g, w in zip(other, out):
        assert torch.equal(g, w)


def test_rows_past_32_bits():
    """More than 2^32 bytes of probabilities: the last request's."""
    import chunked_prefill_attention_ragged_gb300 as mla
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    p = Drafts(17, [3], 131072, False, False)
    t = 9000
    target = torch.zeros((t, 131072), device="cuda")
    target[-3:] = p.dev(p.target)
    tokens, u = np.zeros(t, dtype=np.int64), np.zeros(t, dtype=np.float32)
    tokens[-3:], u[-3:] = p.tokens, p.u
    acc, cnt, nxt = mla.mla_tree_verify(target, i32(tokens), i32([0, t - 3, t]), f32(u), f32([0.5, p.last[0]]), 5)
    want = p.want(5)
    assert acc[1].tolist() == want[0][0].tolist() and int(cnt[1]) == want[1][0] and int(nxt[1]) == want[2][0]
