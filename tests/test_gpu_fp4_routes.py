"""The three ways of tree attention over 4-bit entries, each with the entries, masks and requests where it can go wrong:
units of 16 pairs ("few"), units of 128 ("pairs") and rows made bf16 first ("rows").  Which of them a call takes follows from
the pairs a request, on average, and the workspace; every problem here says which it is meant for."""
import numpy as np
import pytest

from chunked_prefill_attention_ragged_gb300 import workloads as wl
from gpu_util import bits_of, f64_of_bf16, to_dev_bf16
from oracle import bf16_bits_to_f64
from oracle.fp8_cache import f64_to_bf16_bits
from test_gpu_fp4_attention import Problem4, fast_entries

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# (nodes, kv, heads) with pairs a request of 16 at most; of 17 to 128; of more
FEW, PAIRS, ROWS = "few", "pairs", "rows"
ROUTES = [FEW, PAIRS, ROWS]


def run(p, route, **kw):
    """One call on a workspace of the route's size, NaN before it."""
    import chunked_prefill_attention_ragged_gb300 as mla
    b = p.b
    t, (nb, bs) = b.q_abs.shape[0], b.cache.shape[:2]
    small = mla.mla_tree_workspace(t, b.num_heads)
    large = mla.mla_tree_workspace_fp4(t, b.num_heads, b.batch, nb, bs)
    pairs = -(-t * b.num_heads // b.batch)
    assert (pairs <= 16) == (route == FEW) and (pairs > 128 and large > small or route != ROWS), "a problem of this route"
    work = torch.full((large if route == ROWS else small,), 0xFF, dtype=torch.uint8, device="cuda")
    return p.run(workspace=work, **kw)


def problem(seed, route, nodes, kv, bs=64, tree=True, cap=0.0, **kw):
    """Requests of these nodes; heads so that they take the route."""
    heads = {FEW: 1, PAIRS: 5, ROWS: 40}[route]
    return Problem4(seed, nodes, kv, heads, bs, tree, cap, **kw)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("scale", [20, 60, 110, 129, 140, 185, 230])
def test_scales_of_every_size(route, scale):
    """Bytes on both sides of 128, from which on a value takes two products.  (The reference is scaled back to values about 1,
    which bounds() is made for; powers of two change no rounding.)"""
    by = 2.0 ** (127 - scale)
    p = problem(401, route, [2, 18, 7], [90, 700, 333], entries=lambda bits: fast_entries(
        wl.to_bf16_bits((bf16_bits_to_f64(bits) / by).astype(np.float32)), scale), sm_scale=float(wl.DEFAULT_SM_SCALE * by))
    o, lse, st = run(p, route)
    assert st == 0 and torch.isfinite(o.float()).all()
    o = f64_to_bf16_bits(f64_of_bf16(o) * by)
    p.b.cache = f64_to_bf16_bits(bf16_bits_to_f64(p.b.cache) * by)
    p.b.sm_scale = wl.DEFAULT_SM_SCALE
    p.check(to_dev_bf16(o), lse)


@pytest.mark.parametrize("route", ROUTES)
def test_a_scale_of_each_size_in_one_tile(route):
    """Rows with one scale byte above 128 among rows without: of a key's 16 groups one is larger by 2^k, and the queries
    are smaller there by as much."""
    p = problem(402, route, [3, 20, 5], [65, 260, 130])
    flat = p.entries.reshape(-1, 400)
    rng = np.random.default_rng(9)
    big = rng.random(len(flat)) < 0.2
    flat[big, 384 + 4] = rng.integers(129, 140, int(big.sum()))
    q = bf16_bits_to_f64(p.b.q_abs)
    q[..., 128:160] *= 2.0 ** -14
    p.b.q_abs = wl.to_bf16_bits(q.astype(np.float32))
    p.refresh()
    o, lse, st = run(p, route)
    assert st == 0
    p.check(o, lse)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("bs", [1, 16, 24, 64])
@pytest.mark.parametrize("ctx", [0, 50, 61, 126, 900])
def test_unseen_rows_do_not_matter(route, bs, ctx):
    """Two branches below the context; one holds NaN scales, scales past 252, NaN and infinite ropes."""
    n = 40
    p = problem(403 + bs, route, [n, 3, 1], [ctx + n, 40, 7], bs)
    side = np.arange(n) % 2
    p.seen[0] = (side[:, None] == side[None]) & (np.arange(n)[None] <= np.arange(n)[:, None])
    clean = run(p, route)
    assert clean[2] == 0
    p.check(clean[0], clean[1], heads=None if p.b.num_heads < 16 else [0, p.b.num_heads - 1])
    for node in range(1, n, 2):
        e = p.entries[p.at(0, ctx + node)]
        if node % 4 == 1:
            e[384 + node % 16] = [255, 253, 254][node // 4 % 3]
        else:
            e[256:384].view("<u2")[node % 64] = [0x7FC0, 0x7F80, 0xFF80][node // 4 % 3]
    o, lse, st = run(p, route)
    assert st == 0
    k = torch.arange(n + 4, device="cuda")
    k = (k >= n) | (k % 2 == 0)
    assert np.array_equal(bits_of(o[k]), bits_of(clean[0][k])) and torch.equal(lse[k], clean[1][k])
    assert torch.isnan(o[1:n:2].float()).all() and torch.isnan(lse[1:n:2]).all()      # (node 1 holds a NaN)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("byte", [253, 254, 255])
@pytest.mark.parametrize("at", [0, 63, 64, 150, 299])
def test_a_nan_in_the_context_reaches_every_row_of_its_request(route, byte, at):
    p = problem(404, route, [2, 20], [320, 300])
    if at == 299:
        at = 320 - 3
    clean = run(p, route)
    p.entries[p.at(0, at)][384 + at % 16] = byte
    o, lse, st = run(p, route)
    assert st == 0 and torch.isnan(o[:2].float()).all() and torch.isnan(lse[:2]).all()
    assert np.array_equal(bits_of(o[2:]), bits_of(clean[0][2:])) and torch.equal(lse[2:], clean[1][2:])


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("cap", [0.5, 30.0, 3000.0])
@pytest.mark.parametrize("spread", [1.0, 12.0])
def test_capped_logits_over_several_tiles(route, cap, spread):
    p = problem(405, route, [1, 20, 9], [700, 333, 64], tree=True, cap=cap, spread=spread)
    o, lse, st = run(p, route)
    assert st == 0
    p.check(o, lse)


@pytest.mark.parametrize("route", ROUTES)
def test_mask_rows_without_any_node_and_without_keys(route):
    p = problem(406, route, [18, 3, 16], [90, 3, 16])
    p.seen = [s & (np.arange(len(s)) % 2 == 1)[:, None] for s in p.seen]
    o, lse, st = run(p, route)
    assert st == 0
    empty = torch.tensor([18, 20] + list(range(21, 37, 2)), device="cuda")      # no context, and nothing of the mask
    assert torch.isneginf(lse[empty]).all() and (o[empty] == 0).all()
    p.check(o, lse)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("bs", [1, 7, 24, 64])
def test_does_not_read_past_the_lengths(route, bs):
    """NaN in every row that no request owns, and in the workspace."""
    kv = [20, 9, 33, 63, 65, 127, 129, 193, 250]
    p = problem(407, route, [17] + [9] * 8 if route != FEW else [17] + [1] * 8, kv, bs)
    before = run(p, route)
    own = np.zeros(p.b.cache.shape[:2], dtype=bool)
    for r, k in enumerate(kv):
        own[p.at(r, np.arange(k))] = True
    p.entries[~own] = 0xFF
    after = run(p, route)
    assert after[2] == 0 and np.array_equal(bits_of(before[0]), bits_of(after[0])) and torch.equal(before[1], after[1])
    p.check(*after[:2])


@pytest.mark.parametrize("route", ROUTES)
def test_one_large_request_among_empty_ones(route):
    """The average counts the empty requests of a padded batch: a request of 60 nodes and 4 heads, 15 units of 16 pairs."""
    empty = {FEW: 30, PAIRS: 3, ROWS: 0}[route]
    p = Problem4(408, [60] + [0] * empty, [700] + [0] * empty, 4, 64, True)
    o, lse, st = run(p, route)
    assert st == 0
    p.check(o, lse)


@pytest.mark.parametrize("route", ROUTES)
def test_a_prefix_that_requests_share(route):
    """Blocks of one request in the tables of others."""
    p = problem(409, route, [12, 5, 20], [300, 260, 280])
    for r in (1, 2):
        p.b.block_table[r, :4] = p.b.block_table[0, :4]
    o, lse, st = run(p, route)
    assert st == 0
    p.check(o, lse)
