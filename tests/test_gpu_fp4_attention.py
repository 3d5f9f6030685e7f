"""Tree attention over a 4-bit cache against the oracle over the entries' values."""
import os

import numpy as np
import pytest

from chunked_prefill_attention_ragged_gb300 import workloads as wl
from gpu_util import Guarded, bits_of, f64_of_bf16, to_dev, to_dev_bf16
from oracle import bf16_bits_to_f64, fp4_values, pack_fp4, quantize, tree_attention
from oracle.fp8_cache import f64_to_bf16_bits
from test_gpu_speculative import ATTENTION, BAD_INDEX, Problem, bounds, i32, new_status

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def fast_entries(rows_bits, scale=126):
    """Entries of bf16 rows [N, 576]: codes by nearest value under one scale byte a row (the oracle's quantizer is slow)."""
    x = bf16_bits_to_f64(rows_bits)
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    s = np.full((len(x), 16), scale, dtype=np.uint8)
    s[:, ::3] += 1
    y = x[:, :512] / np.repeat(2.0 ** (s.astype(float) - 127), 32, axis=-1)
    code = np.searchsorted((grid[1:] + grid[:-1]) / 2, np.abs(y)) | np.where(y < 0, 8, 0)
    return pack_fp4(code.astype(np.uint8), rows_bits[:, 512:], s)


class Problem4(Problem):
    """A Problem whose cache is one of entries; the oracle sees their values."""

    def __init__(self, *a, entries=fast_entries, **kw):
        super().__init__(*a, **kw)
        shape = self.b.cache.shape[:2]
        self.entries = entries(self.b.cache.reshape(-1, 576)).reshape(shape + (400,))
        self.refresh()

    def refresh(self):
        v = fp4_values(self.entries)
        self.b.cache = f64_to_bf16_bits(v)
        self.b.cache[..., 512:] = np.ascontiguousarray(self.entries[..., 256:384]).view("<u2")

    def at(self, r, pos):
        bs = self.b.block_size
        return self.b.block_table[r, pos // bs], pos % bs

    def run(self, pad=0, cache=None, **kw):
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
        mla.mla_tree_attention_fp4(q, to_dev(self.entries) if cache is None else cache, to_dev(b.block_table), i32(b.qo_indptr),
                                   i32(self.kv), mask, sm_scale=b.sm_scale, logits_soft_cap=b.logits_soft_cap, o=o.tensor,
                                   lse=lse.tensor, status=st, **kw)
        torch.cuda.synchronize()
        o.check("O")
        lse.check("LSE")
        assert (o.tensor[t - pad:] == 3.0).all() and (lse.tensor[t - pad:] == 4.0).all(), "rows behind the last request"
        return o.tensor[:t - pad], lse.tensor[:t - pad], int(st)


MORE = [
    ("block_7", [3, 9, 2], [500, 131, 2], 20, 7, True, 0.0),
    ("pairs_17", [17], [300], 1, 64, True, 0.0),
    ("pairs_33_65", [3, 5], [300, 400], 13, 64, True, 0.0),
    ("pairs_128_129", [8, 3], [300, 400], 43, 16, False, 0.0),
    ("one_key", [1, 1], [1, 2], 16, 64, False, 0.0),
]


@pytest.mark.parametrize("name,nodes,kv,heads,bs,tree,cap", ATTENTION + MORE, ids=[c[0] for c in ATTENTION + MORE])
def test_attention(name, nodes, kv, heads, bs, tree, cap):
    p = Problem4(700 + [c[0] for c in ATTENTION + MORE].index(name), nodes, kv, heads, bs, tree, cap)
    o, lse, st = p.run(pad=2)
    assert st == 0
    p.check(o, lse)


def test_entries_as_the_append_makes_them():
    def entries(bits):
        codes, scales = quantize(bf16_bits_to_f64(bits[:, :512]), "fp4")
        return pack_fp4(codes, bits[:, 512:], scales)
    p = Problem4(3, [2, 1], [90, 130], 16, 16, True, entries=entries)
    o, lse, st = p.run()
    assert st == 0
    p.check(o, lse)


@pytest.mark.parametrize("scale", [60, 110, 140, 185])
def test_small_and_large_scales(scale):
    """Scales on both sides of those that one product by a power of two can make."""
    p = Problem4(4, [2, 6], [90, 700], 16, 64, True, entries=lambda bits: fast_entries(
        wl.to_bf16_bits((bf16_bits_to_f64(bits) * 2.0 ** (scale - 127)).astype(np.float32)), scale),
        sm_scale=float(wl.DEFAULT_SM_SCALE * 2.0 ** (127 - scale)))
    o, lse, st = p.run()
    assert st == 0 and torch.isfinite(o.float()).all()
    o = f64_of_bf16(o) * 2.0 ** (127 - scale)    # (bounds() has a constant for values about 1)
    p.b.cache = f64_to_bf16_bits(bf16_bits_to_f64(p.b.cache) * 2.0 ** (127 - scale))
    p.b.sm_scale = wl.DEFAULT_SM_SCALE
    p.check(to_dev_bf16(f64_to_bf16_bits(o)), lse)


@pytest.mark.parametrize("spread", [0.01, 12.0])
@pytest.mark.parametrize("nodes,heads", [([6, 2], 64), ([6, 2], 16), ([2, 2], 16), ([1, 1], 16)])
def test_flat_and_peaked(spread, nodes, heads):
    p = Problem4(77, nodes, [700, 333], heads, 64, True, spread=spread)
    o, lse, st = p.run()
    assert st == 0
    p.check(o, lse)


@pytest.mark.parametrize("batch,ctx,nodes,heads", [(1, 20000, 1, 16), (2, 9000, 5, 128), (150, 600, 1, 16), (40, 900, 4, 128),
                                                   (170, 400, 2, 16), (3, 7000, 4, 16), (1, 30000, 3, 64), (300, 200, 1, 5)])
def test_split_and_unsplit(batch, ctx, nodes, heads):
    p = Problem4(33 + batch, [nodes] * batch, [ctx + 13 * (r % 7) + nodes for r in range(batch)], heads, 64, True)
    o, lse, st = p.run()
    assert st == 0
    some = sorted({0, batch // 2, batch - 1})
    p.check(o, lse, some, None if heads <= 16 else [0, heads // 2, heads - 1])


def test_mask_rows_without_any_node():
    p = Problem4(5, [4, 3], [40, 3], 4, 64, True)
    p.seen = [s & np.array([False, True, False, True][:len(s)])[:, None] for s in p.seen]
    o, lse, st = p.run()
    assert st == 0 and torch.isneginf(lse[4]).all() and (o[4] == 0).all()
    p.check(o, lse)


@pytest.mark.parametrize("heads", [3, 12, 40, 128])
def test_repeats_bit_for_bit(heads):
    p = Problem4(6, [3, 9, 1], [5000, 700, 64], heads, 64, True)
    a = p.run()
    for _ in range(3):
        b = p.run()
        assert np.array_equal(bits_of(a[0]), bits_of(b[0])) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("bs", [1, 5, 16, 24, 64, 128])
@pytest.mark.parametrize("heads", [6, 64])
def test_does_not_read_past_the_lengths(bs, heads):
    """NaN in every row that no request owns."""
    kv = [1, 7, 9, 33, 63, 65, 127, 129, 193, 250]
    p = Problem4(18, [1] * len(kv), kv, heads, bs, False)
    before = p.run(pad=3)
    own = np.zeros(p.b.cache.shape[:2], dtype=bool)
    for r, k in enumerate(kv):
        own[p.at(r, np.arange(k))] = True
    p.entries[~own] = 0xFF
    after = p.run(pad=3)
    assert after[2] == 0 and np.array_equal(bits_of(before[0]), bits_of(after[0])) and torch.equal(before[1], after[1])
    p.check(*after[:2])


@pytest.mark.parametrize("ctx", [60, 20000])
def test_passes_nan_of_a_query_on_in_its_row_only(ctx):
    p = Problem4(19, [3, 2], [ctx, 70], 4, 64, True)
    p.b.q_abs[1, 2, 570] = 0x7FC0
    o, lse, st = p.run()
    assert st == 0 and torch.isnan(o[1, 2].float()).all() and bool(torch.isnan(lse[1, 2]))
    p.b.q_abs[1, 2] = p.b.q_abs[1, 1]
    o2, lse2, _ = p.run()
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[1, 2] = False
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[keep], lse2[keep])


@pytest.mark.parametrize("bs", [1, 16, 24, 64])
@pytest.mark.parametrize("ctx", [0, 50, 61, 126, 900])
@pytest.mark.parametrize("heads", [4, 64])
def test_unseen_rows_do_not_matter(bs, ctx, heads):
    """Two branches below the context; one holds NaN scales, scales past 252, NaN and infinite ropes."""
    n = 70
    p = Problem4(300 + bs, [n, 3], [ctx + n, 40], heads, bs, True)
    side = np.arange(n) % 2
    p.seen[0] = (side[:, None] == side[None]) & (np.arange(n)[None] <= np.arange(n)[:, None])
    clean = p.run()
    assert clean[2] == 0
    p.check(clean[0], clean[1], heads=None if heads < 16 else [0, heads - 1])
    for node in range(1, n, 2):
        e = p.entries[p.at(0, ctx + node)]
        if node % 4 == 1:
            e[384 + node % 16] = [255, 253, 254][node // 4 % 3]
        else:
            e[256:].view("<u2")[node % 64] = [0x7FC0, 0x7F80, 0xFF80][node // 4 % 3]
    o, lse, st = p.run()
    assert st == 0
    k = torch.arange(n + 3, device="cuda")
    k = (k >= n) | (k % 2 == 0)
    assert np.array_equal(bits_of(o[k]), bits_of(clean[0][k])) and torch.equal(lse[k], clean[1][k])
    assert torch.isnan(o[1:n:2].float()).all() and torch.isnan(lse[1:n:2]).all()      # (node 1 holds a NaN)


def test_a_nan_in_the_context_reaches_every_row_of_its_request():
    p = Problem4(11, [2, 2], [300, 300], 16, 64, True)
    clean = p.run()
    p.entries[p.at(0, 150)][390] = 255
    o, lse, st = p.run()
    assert st == 0 and torch.isnan(o[:2].float()).all() and torch.isnan(lse[:2]).all()
    assert torch.equal(o[2:], clean[0][2:]) and torch.equal(lse[2:], clean[1][2:])


def test_nodes_past_the_mask_are_not_seen():
    p = Problem4(21, [70, 3], [100, 40], 2, 64, True)
    p.seen = [s * (np.arange(s.shape[1]) < 64) for s in p.seen]
    want = p.run()
    p.seen = [s[:, :64] for s in p.seen]
    p.words = 1
    got = p.run()
    assert np.array_equal(bits_of(got[0]), bits_of(want[0])) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("heads", [4, 64])
@pytest.mark.parametrize("bs", [5, 16, 64])
def test_bad_blocks_lengths_and_rows(heads, bs):
    """Rows of a block that is not there read as zeros, lengths are clamped, requests outside the rows skipped."""
    p = Problem4(22, [2, 2, 1], [200, 150, 30], heads, bs, False)
    table = p.b.block_table.copy()
    for bad in (-1, p.b.cache.shape[0], 1 << 30, -(1 << 31)):
        p.b.block_table = table.copy()
        p.b.block_table[0, 1] = bad
        o, lse, st = p.run()
        assert st == BAD_INDEX
        p.b.block_table = table
        saved = p.entries.copy()
        p.entries[table[0, 1]] = 0
        p.refresh()
        want = p.run()
        assert want[2] == 0 and np.array_equal(bits_of(o), bits_of(want[0])) and torch.equal(lse, want[1])
        p.entries = saved
        p.refresh()
    import chunked_prefill_attention_ragged_gb300 as mla
    b, st = p.b, new_status()
    cache, q = to_dev(p.entries), to_dev_bf16(b.q_abs)
    o = torch.full((5, heads, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    mla.mla_tree_attention_fp4(q, cache, to_dev(table), i32([0, 2, 9, 5]), i32(p.kv), sm_scale=b.sm_scale, o=o, status=st)
    assert int(st) == BAD_INDEX and (o[2:] == 3.0).all() and torch.isfinite(o[:2].float()).all()
    st.zero_()
    o, lse = mla.mla_tree_attention_fp4(q, cache, to_dev(table), i32(b.qo_indptr), i32([-3, 1 << 30, 30]), sm_scale=b.sm_scale,
                                        status=st)
    assert int(st) == BAD_INDEX and (o[:2] == 0).all() and torch.isneginf(lse[:2]).all()


def test_empty_batch_and_no_cache():
    import chunked_prefill_attention_ragged_gb300 as mla
    q = torch.zeros((2, 4, 576), dtype=torch.bfloat16, device="cuda")
    none = torch.zeros((0, 64, 400), dtype=torch.uint8, device="cuda")
    st = new_status()
    o, lse = mla.mla_tree_attention_fp4(q, none, torch.zeros((2, 0), dtype=torch.int32, device="cuda"), i32([0, 1, 2]), i32([0, 0]),
                                        sm_scale=0.1, status=st)
    assert int(st) == 0 and (o == 0).all() and torch.isneginf(lse).all()
    o = torch.full((2, 4, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    mla.mla_tree_attention_fp4(q, none, torch.zeros((0, 0), dtype=torch.int32, device="cuda"), i32([0]), i32([]), sm_scale=0.1, o=o)
    assert (o == 3.0).all()
    with pytest.raises(ValueError):
        mla.mla_tree_attention_fp4(q, torch.zeros((1, 64, 576), dtype=torch.bfloat16, device="cuda"), i32([[0]]), i32([0, 2]), i32([3]),
                                   sm_scale=0.1)
    with pytest.raises(TypeError):
        mla.mla_tree_attention_fp4(q, torch.zeros((1, 64, 400), dtype=torch.int8, device="cuda"), i32([[0]]), i32([0, 2]), i32([3]),
                                   sm_scale=0.1)
    with pytest.raises(mla.MlaError):
        mla.mla_tree_attention_fp4(q, torch.zeros((1, 64, 400), dtype=torch.uint8, device="cuda"), i32([[0]]), i32([0, 2]), i32([3]),
                                   sm_scale=0.1, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("heads", [4, 64])
def test_replayed_with_other_lengths_and_on_two_streams(heads):
    import chunked_prefill_attention_ragged_gb300 as mla
    p = Problem4(23, [1, 1, 1], [900, 300, 60], heads, 16, False)
    b = p.b
    q, cache, table, kv = to_dev_bf16(b.q_abs), to_dev(p.entries), to_dev(b.block_table), i32([1, 1, 1])
    o = torch.zeros((3, heads, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((3, heads), dtype=torch.float32, device="cuda")
    qo, work = i32(b.qo_indptr), torch.empty(mla.mla_tree_workspace(3, heads), dtype=torch.uint8, device="cuda")
    call = lambda **kw: mla.mla_tree_attention_fp4(q, cache, table, qo, kv, sm_scale=b.sm_scale, **kw)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(o=o, lse=lse, workspace=work)
    for lens in ([900, 300, 60], [5, 17, 0], [333, 12, 59]):
        kv.copy_(i32(lens))
        work.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        p.kv = lens
        p.check(o, lse)
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for k in range(6):
        outs.append(call(stream=streams[k % 2]))
    torch.cuda.synchronize()
    for a, c in outs:
        assert torch.equal(a, o) and torch.equal(c, lse)


def test_rows_past_32_bits():
    """A cache of more than 2^32 bytes, its used blocks at the end."""
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    p = Problem4(24, [2, 1], [200, 77], 16, 64, False)
    n, k = 200000, p.b.cache.shape[0]
    cache = torch.zeros((n, 64, 400), dtype=torch.uint8, device="cuda")
    cache[n - k:] = to_dev(p.entries)
    p.b.block_table = np.where(p.b.block_table >= 0, p.b.block_table + n - k, -1).astype(np.int32)
    table = p.b.block_table
    o, lse, st = p.run(cache=cache)
    assert st == 0
    p.b.block_table = np.where(table >= 0, table - (n - k), -1)
    p.check(o, lse)


@pytest.mark.parametrize("cap", [0.5, 30.0, 20000.0])
def test_capped_logit(cap):
    """One key and one nonzero product a row: a capped logit is off by less than 2^-19 of itself (the bf16 cache's test has
    the count of roundings)."""
    import chunked_prefill_attention_ragged_gb300 as mla
    for heads in (16, 128):
        x = np.concatenate([s * 2.0 ** np.linspace(-20, 11.5, heads // 2) for s in (1, -1)])
        q = torch.zeros((1, heads, 576), dtype=torch.bfloat16, device="cuda")
        q[0, :, 70] = torch.from_numpy(x).to(torch.bfloat16).cuda()
        codes = np.zeros((1, 512), dtype=np.uint8)
        codes[0, 70], codes[0, 3] = 2, 12                # 1 and -2
        cache = torch.zeros((2, 64, 400), dtype=torch.uint8, device="cuda")
        cache[1, 0] = to_dev(pack_fp4(codes, np.zeros((1, 64), np.uint16), np.full((1, 16), 127, np.uint8)))[0]
        o, lse = mla.mla_tree_attention_fp4(q, cache, i32([[1]]), i32([0, 1]), i32([1]), sm_scale=0.0721687824, logits_soft_cap=cap)
        assert (o[0, :, 70] == 1).all() and (o[0, :, 3] == -2).all() and int((o != 0).sum()) == 2 * heads
        c = float(np.float32(cap))
        want = c * np.tanh(float(np.float32(0.0721687824)) * q[0, :, 70].double().cpu().numpy() / c)
        assert (np.abs(lse[0].double().cpu().numpy() - want) <= 2.0 ** -19 * np.abs(want)).all()


def test_a_wait_that_gives_up(monkeypatch):
    """In the test mode a kernel with waits reports that one ran out, and the next call is as ever."""
    p = Problem4(25, [16], [300], 64, 64, True)
    monkeypatch.setenv("MLA_TEST_FORCE_TIMEOUT_NS", "2000000")
    _, _, st = p.run()
    assert st in (0, 1)
    monkeypatch.delenv("MLA_TEST_FORCE_TIMEOUT_NS")
    assert "MLA_TEST_FORCE_TIMEOUT_NS" not in os.environ
    o, lse, st = p.run()
    assert st == 0
    p.check(o, lse)
