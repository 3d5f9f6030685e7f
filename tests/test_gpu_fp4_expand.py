"""Tree attention over a 4-bit cache with a workspace that has room for bf16 rows: the same answers as without, and the
oracle's."""
import numpy as np
import pytest

from gpu_util import to_dev, to_dev_bf16
from test_gpu_fp4_attention import Problem4
from test_gpu_speculative import BAD_INDEX, i32

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

GUARD = 4096


def workspaces(p):
    """(any call's, one with room for the rows), what does not matter in them NaN, and a guard behind."""
    import chunked_prefill_attention_ragged_gb300 as mla
    b = p.b
    t, (nb, bs) = b.q_abs.shape[0], b.cache.shape[:2]
    sizes = mla.mla_tree_workspace(t, b.num_heads), mla.mla_tree_workspace_fp4(t, b.num_heads, b.batch, nb, bs)
    assert sizes[1] >= sizes[0] + nb * bs * 1152, "a problem for which it pays"
    return [torch.full((n + GUARD,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes]


def both(p, **kw):
    out = []
    for w in workspaces(p):
        n = w.numel() - GUARD
        out.append(p.run(workspace=w[:n], **kw))
        assert bool((w[n:] == 0xFF).all()), "behind the workspace"
    return out


CASES = [("block_64", [16, 9], [700, 1029], 64, 64, True, 0.0), ("block_32_cap", [30, 1, 40], [65, 300, 40], 40, 32, True, 20.0),
         ("block_16", [37, 12, 25], [500, 131, 25], 17, 16, True, 0.0), ("block_8", [8, 5], [260, 129], 128, 8, False, 0.0),
         ("block_7", [33, 40], [200, 77], 13, 7, True, 0.0), ("block_1", [12], [150], 33, 1, True, 0.0),
         ("no_nodes", [4, 0, 9], [4, 50, 300], 128, 64, True, 0.0)]


@pytest.mark.parametrize("name,nodes,kv,heads,bs,tree,cap", CASES, ids=[c[0] for c in CASES])
def test_against_the_oracle(name, nodes, kv, heads, bs, tree, cap):
    p = Problem4(41, nodes, kv, heads, bs, tree, cap)
    for o, lse, st in both(p, pad=3):
        assert st == 0
        p.check(o, lse)


@pytest.mark.parametrize("batch,ctx,nodes,heads", [(2, 9000, 5, 128), (40, 900, 4, 128), (1, 20000, 9, 16), (90, 200, 10, 16)])
def test_units_in_many_pieces(batch, ctx, nodes, heads):
    p = Problem4(45 + batch, [nodes] * batch, [ctx + 13 * (r % 7) + nodes for r in range(batch)], heads, 64, True)
    for o, lse, st in both(p):
        assert st == 0
        p.check(o, lse, sorted({0, batch // 2, batch - 1}), None if heads <= 16 else [0, heads // 2, heads - 1])


def test_rows_that_are_nan():
    """A scale byte above 252 in a context row makes its request NaN, in a node's row those that see the node."""
    p = Problem4(42, [24, 24, 24], [90, 200, 100], 16, 16, True)
    p.entries[p.at(0, 12)][384 + 3] = 255
    node = 5
    p.entries[p.at(1, 200 - 24 + node)][384 + 15] = 253
    seen = np.asarray(p.seen[1], bool)[:, node]
    p.refresh()
    for o, lse, st in both(p):
        assert st == 0 and torch.isnan(o[:24]).all() and torch.isnan(lse[:24]).all()
        mine = torch.from_numpy(seen).cuda()
        assert torch.isnan(o[24:48][mine]).all() and torch.isfinite(o[24:48][~mine]).all() and torch.isfinite(lse[24:48][~mine]).all()
        assert torch.isfinite(o[48:]).all()


def test_bad_tables_and_lengths():
    """Blocks outside the cache, lengths past the table or negative, rows that are not there: reported, and the same rows."""
    p = Problem4(43, [20, 20, 20, 20], [300, 200, 150, 64], 24, 16, True)
    p.b.block_table[1, 2], p.b.block_table[1, 3] = p.b.cache.shape[0] + 5, -7
    good = list(p.kv)
    p.kv[2], p.kv[3] = 1 << 30, -4
    (a, la, sa), (b, lb, sb) = both(p)
    assert sa == sb == BAD_INDEX
    p.kv = good
    tol = 2.0 ** -6
    for x, y in ((a, b), (la, lb)):   # (request 2: positions without a block are zeros in both)
        assert torch.equal(torch.isfinite(x.float()), torch.isfinite(y.float()))
        fin = torch.isfinite(x.float())
        assert (x.float()[fin] - y.float()[fin]).abs().max() <= tol * max(1.0, float(x.float()[fin].abs().max()))
    p.check(b, lb, [0])


def test_chosen_without_a_workspace_and_replayed():
    import chunked_prefill_attention_ragged_gb300 as mla
    p = Problem4(44, [30, 26], [600, 333], 16, 64, True)
    b = p.b
    q, cache, table, qo, mask = to_dev_bf16(b.q_abs), to_dev(p.entries), to_dev(b.block_table), i32(b.qo_indptr), p.mask()
    kv = i32(p.kv)
    large = both(p)[1]
    call = lambda **kw: mla.mla_tree_attention_fp4(q, cache, table, qo, kv, mask, sm_scale=b.sm_scale, **kw)  # noqa: E731
    o, lse = call()
    torch.cuda.synchronize()
    assert torch.equal(o, large[0]) and torch.equal(lse, large[1])
    work = workspaces(p)[1]
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(o=o2, lse=lse2, workspace=work)
    for lens in ([600, 333], [30, 26], [417, 300]):
        kv.copy_(i32(lens))
        work.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        p.kv = lens
        p.check(o2, lse2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [call(stream=side) for _ in range(3)] + [call() for _ in range(3)]   # two streams at once, a workspace each
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, o2) and torch.equal(y, lse2)


@pytest.mark.parametrize("nodes,heads,rows", [(16, 64, True), (16, 64, False), (1, 128, False), (1, 16, False)])
def test_a_wait_that_gives_up(monkeypatch, nodes, heads, rows):
    """In the test mode each of the kernels reports that a wait ran out, and the next call is as ever."""
    import chunked_prefill_attention_ragged_gb300 as mla
    p = Problem4(46, [nodes], [300], heads, 64, True)
    nb, bs = p.b.cache.shape[:2]
    n = mla.mla_tree_workspace_fp4(nodes, heads, 1, nb, bs) if rows else mla.mla_tree_workspace(nodes, heads)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    monkeypatch.setenv("MLA_TEST_FORCE_TIMEOUT_NS", "2000000")
    assert p.run(workspace=work)[2] == 1
    monkeypatch.delenv("MLA_TEST_FORCE_TIMEOUT_NS")
    o, lse, st = p.run(workspace=work)
    assert st == 0
    p.check(o, lse)


def test_sizes():
    import chunked_prefill_attention_ragged_gb300 as mla
    base = mla.mla_tree_workspace(64, 128)
    f = mla.mla_tree_workspace_fp4
    assert f(32, 128, 32, 100, 64) == base                       # 128 pairs a request: a unit
    assert f(96, 128, 32, 0, 64) == base and f(0, 128, 0, 10, 64) == base
    large = f(33, 128, 32, 100, 64)
    assert base + 6400 * 1152 <= large <= base + 6400 * 1152 + 1024
    assert f(96, 128, 32, 1 << 16, 64) == base                   # 4.8 GB of rows
