"""What is in the cached rows of nodes that a node does not see does not reach it: NaN and infinities too."""
import numpy as np
import pytest

from gpu_util import bits_of, f64_of_bf16
from oracle import tree_attention, bf16_bits_to_f64
from test_gpu_speculative import Problem, bounds

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

NAN, INF, NINF = 0x7FC0, 0x7F80, 0xFF80


def spoil(p, r, node, bits, columns):
    pos = p.kv[r] - p.nodes[r] + node
    p.b.cache[p.b.block_table[r, pos // p.b.block_size], pos % p.b.block_size, columns] = bits


@pytest.mark.parametrize("bs", [1, 5, 8, 16, 24, 32, 64, 128])
@pytest.mark.parametrize("ctx", [0, 50, 61, 126, 900])
def test_unseen_rows_do_not_matter(bs, ctx):
    """Two branches below the context; one holds NaN and infinities in every kind of column."""
    n = 70
    p = Problem(300 + bs, [n, 3], [ctx + n, 40], 4, bs, True)
    side = np.arange(n) % 2          # node i is in branch side[i], under node i - 2
    p.seen[0] = (side[:, None] == side[None]) & (np.arange(n)[None] <= np.arange(n)[:, None])
    clean = p.run()
    assert clean[2] == 0
    p.check(clean[0], clean[1])
    for node in range(1, n, 2):      # branch 1
        spoil(p, 0, node, [NAN, INF, NINF, NAN][node // 2 % 4], [(37 * node) % 512, 300, 511, 5][:1 + node % 3])
    o, lse, st = p.run()
    assert st == 0
    keep = np.ones(n + 3, dtype=bool)
    keep[1:n:2] = False
    k = torch.from_numpy(keep).cuda()
    assert np.array_equal(bits_of(o[k]), bits_of(clean[0][k])) and torch.equal(lse[k], clean[1][k])
    # (node 1 holds NaN, so all of its branch does)
    assert torch.isnan(o[1:n:2].float()).all() and torch.isnan(lse[1:n:2]).all()


@pytest.mark.parametrize("bs", [1, 16, 64])
def test_later_nodes_of_a_chain_do_not_matter(bs):
    p = Problem(310 + bs, [5, 200], [130, 260], 3, bs, False)
    clean = p.run()
    spoil(p, 0, 3, NAN, slice(None))
    spoil(p, 1, 150, INF, slice(0, 600, 2))
    o, lse, st = p.run()
    keep = torch.tensor([i < 3 or 5 <= i < 155 for i in range(205)], device="cuda")
    assert st == 0 and np.array_equal(bits_of(o[keep]), bits_of(clean[0][keep])) and torch.equal(lse[keep], clean[1][keep])
    assert torch.isnan(o[3:5].float()).all() and torch.isnan(lse[155:]).all()


def test_a_node_that_may_not_see_itself():
    p = Problem(320, [1], [30], 5, 64, True)
    p.seen[0][:] = False
    clean = p.run()
    spoil(p, 0, 0, NAN, slice(None))
    o, lse, st = p.run()
    assert st == 0 and np.array_equal(bits_of(o), bits_of(clean[0])) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("bs", [1, 64])
def test_an_infinite_value_that_is_seen(bs):
    """Under a cap its weight is finite: it counts as the largest finite value, in its column only."""
    p = Problem(330, [2], [20], 2, bs, True, cap=5.0)
    p.seen[0] = np.array([[True, False], [True, True]])
    p.b.q_abs[:, :, 9] = 0x3F80
    spoil(p, 0, 1, INF, 9)
    o, lse, st = p.run()
    b = p.b
    rows = p.rows(0).copy()
    rows[19, 9] = 0x7F7F
    q, kv = bf16_bits_to_f64(b.q_abs[0:2]), bf16_bits_to_f64(rows)
    want_o, want_l = tree_attention(q, kv, p.seen[0], sm_scale=b.sm_scale, logits_soft_cap=5.0)
    o = f64_of_bf16(o)
    assert st == 0 and (o[1, :, 9] > 1e36).all()
    kv[19, 9] = 1e3          # (for the bounds: large enough for the cap)
    tol_o, tol_l = bounds(q, kv, p.seen[0], want_o, sm_scale=b.sm_scale, cap=5.0)
    others = np.arange(512) != 9
    assert (np.abs(o - want_o) <= tol_o)[:, :, others].all() and (np.abs(o - want_o) <= tol_o)[0].all()
    assert (np.abs(lse.double().cpu().numpy() - want_l) <= tol_l).all()
