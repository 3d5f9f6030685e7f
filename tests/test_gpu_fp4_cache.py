"""New tokens into caches of every entry, 4-bit rows out of them, and prefill over them, against the oracle."""
import numpy as np
import pytest

from chunked_prefill_attention_ragged_gb300 import workloads as wl
from gpu_util import Guarded, bits_of, check_attention, f64_of_bf16, to_dev, to_dev_bf16
from oracle import (bf16_bits_to_f64, e2m1_to_f64, e4m3_to_f64, fp4_codes, gather_latent_fp4, normalise, pack_fp4, pack_fp8,
                    quantize, rotate)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BAD_INDEX = 2
BYTES = {"bf16": 1152, "fp8": 648, "fp4": 400}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def i64(x):
    return torch.tensor(np.asarray(x), dtype=torch.int64, device="cuda")


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def angles(n):
    f = 10000.0 ** (-np.arange(32) / 32)
    a = np.arange(n)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)


class Tokens:
    def __init__(self, seed, t, heads, kind, bs=16, norm=True, interleaved=True, spread=1.0, reach=5000):
        r = np.random.default_rng(seed)
        self.t, self.heads, self.kind, self.bs, self.interleaved = t, heads, kind, bs, interleaved
        self.nb = -(-(t + 7) // bs) + 1
        wide = r.integers(-12, 12, (t, 9)).repeat(64, axis=-1) if spread != 1.0 else 0
        self.latent = wl.to_bf16_bits((r.standard_normal((t, 576)) * 2.0 ** wide * spread).astype(np.float32))
        self.weight = wl.to_bf16_bits((1 + r.standard_normal(512) / 8).astype(np.float32)) if norm else None
        self.pos = r.integers(0, reach, t)
        self.table = angles(reach)
        self.slots = r.permutation(self.nb * bs)[:t]
        self.q = wl.to_bf16_bits(r.standard_normal((t, heads, 192)).astype(np.float32))

    def cache(self):
        shape = (self.nb, self.bs, 576 if self.kind == "bf16" else BYTES[self.kind])
        g = Guarded(shape, torch.bfloat16 if self.kind == "bf16" else torch.uint8)
        g.tensor.view(torch.uint8).fill_(0x5A)
        return g

    def run(self, cache, q=None, q_out=None, **kw):
        import chunked_prefill_attention_ragged_gb300 as mla
        a = dict(latent=to_dev_bf16(self.latent), slots=i64(self.slots), pos=i32(self.pos))
        a.update(kw)
        st = status()
        mla.mla_cache_append(cache, a["latent"], a["slots"], a["pos"], to_dev(self.table),
                             norm_weight=None if self.weight is None else to_dev_bf16(self.weight), norm_eps=1e-6,
                             interleaved=self.interleaved, q_rope=q, q_out=q_out, status=st)
        torch.cuda.synchronize()
        return int(st)

    def want(self):
        """fp64 latents and ropes before they are rounded."""
        x = bf16_bits_to_f64(self.latent)
        lat = normalise(x[:, :512], None if self.weight is None else bf16_bits_to_f64(self.weight), 1e-6)
        return lat, rotate(x[:, 512:], self.pos, self.table, self.interleaved)

    def check_rows(self, rows):
        """Rows [t, bytes] of the cache.  A bf16 value is off by half a step (2^-8) and by what fp32 loses before:
        the norm's sum of 512 squares (at most 21 roundings one behind the other, halved by the root), root, quotient
        and two products, 2^-24 each: below 2^-19; a rotation's two products and sum, 2^-22 of the sum of magnitudes."""
        lat, rope = self.want()
        size = 2 * np.abs(bf16_bits_to_f64(self.latent)[:, 512:]).max(-1)[:, None]
        raw = rows[:, 1024:] if self.kind == "bf16" else rows[:, 512:640] if self.kind == "fp8" else rows[:, 256:384]
        got = bf16_bits_to_f64(np.ascontiguousarray(raw).view("<u2"))
        assert (np.abs(got - rope) <= 2.0 ** -8 * np.abs(rope) + 2.0 ** -22 * size).all(), "rope"
        loose = 0 if self.weight is None else 2.0 ** -19
        if self.kind == "bf16":
            got = bf16_bits_to_f64(np.ascontiguousarray(rows[:, :1024]).view("<u2"))
            assert (np.abs(got - lat) <= (2.0 ** -8 + loose) * np.abs(lat)).all(), "latent"
            return
        group, reach, at = (64, 448.0, 640) if self.kind == "fp8" else (32, 7.0, 384)
        scales = rows[:, at:]
        if self.weight is None:      # bit for bit
            codes, want = quantize(lat, self.kind)
            rope_bits = np.ascontiguousarray(raw).view("<u2")
            np.testing.assert_array_equal(rows, (pack_fp8 if self.kind == "fp8" else pack_fp4)(codes, rope_bits, want))
            return
        # a group whose largest value is as good as at what a scale reaches may have either scale
        s = np.repeat(2.0 ** (scales.astype(np.float64) - 127), group, axis=-1)
        top = np.abs(lat).reshape(self.t, -1, group).max(-1).repeat(group, axis=-1)
        assert (top <= reach * s * (1 + loose)).all() and (top >= reach * s / 2 * (1 - loose)).all(), "scales"
        values = (e4m3_to_f64(rows[:, :512]) if self.kind == "fp8" else e2m1_to_f64(fp4_codes(rows))) * s
        y = np.abs(lat) / s
        if self.kind == "fp8":
            half = 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 4)
        else:
            half = np.where(y < 2, 0.25, np.where(y < 4, 0.5, 1.0))
        assert (np.abs(values - lat) <= half * s + loose * np.abs(lat)).all(), "latent"


APPEND = [(1, 1, 16, True, True), (3, 0, 1, True, False), (5, 4, 7, False, True), (64, 16, 64, True, True), (33, 5, 24, True, False),
          (130, 33, 16, False, False), (17, 128, 64, True, False)]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("t,heads,bs,norm,interleaved", APPEND)
def test_append(kind, t, heads, bs, norm, interleaved):
    c = Tokens(40 + t, t, heads, kind, bs, norm, interleaved)
    g, q = c.cache(), to_dev_bf16(c.q)
    out = Guarded((t, heads, 192), torch.bfloat16, fill=2.0)
    assert c.run(g.tensor, q[..., 128:] if heads else None, out.tensor[..., 128:] if heads else None) == 0
    g.check("cache")
    out.check("queries")
    rows = g.tensor.view(torch.uint8).reshape(c.nb * bs, -1).cpu().numpy()
    c.check_rows(rows[c.slots])
    others = np.ones(c.nb * bs, dtype=bool)
    others[c.slots] = False
    assert (rows[others] == 0x5A).all()
    if heads:
        x = bf16_bits_to_f64(c.q)[..., 128:]
        want = rotate(x, c.pos, c.table, interleaved)
        got = f64_of_bf16(out.tensor)
        assert (np.abs(got[..., 128:] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * np.abs(x).max()).all()
        assert (got[..., :128] == 2.0).all()
        assert np.array_equal(bits_of(q), c.q), "the queries themselves"
        mine = q[..., 128:]
        assert c.run(g.tensor, mine) == 0        # in place
        assert torch.equal(q[..., 128:], out.tensor[..., 128:]) and np.array_equal(bits_of(q[..., :128]), c.q[..., :128])


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_append_of_every_magnitude(kind):
    """Groups from 2^-140 to 2^110, zeros, ties, what a scale just reaches and just does not: bit for bit."""
    c = Tokens(3, 60, 0, kind, norm=False)
    r = np.random.default_rng(4)
    x = r.standard_normal((60, 576)) * 2.0 ** r.integers(-130, 110, (60, 18)).repeat(32, axis=-1)
    x[0, :512] = 0
    x[1, :512] = -0.0
    x[2, :512] = np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0], 64)
    x[3, :512] = np.tile([7.0625, -5.0, 2.5, 448, 450, 0, -464, 1], 64)
    x[4, :512] = 2.0 ** -133
    c.latent = wl.to_bf16_bits(x.astype(np.float32))
    g = c.cache()
    assert c.run(g.tensor) == 0
    c.check_rows(g.tensor.reshape(c.nb * c.bs, -1).cpu().numpy()[c.slots])


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_append_of_values_that_are_not_finite(kind, norm):
    c = Tokens(5, 6, 0, kind, norm=norm)
    c.latent[1, 40], c.latent[2, 500], c.latent[3, 0], c.latent[4, 520] = 0x7FC0, 0x7F80, 0x7F7F, 0x7FC0
    g = c.cache()
    assert c.run(g.tensor) == 0
    rows = g.tensor.reshape(c.nb * c.bs, -1).cpu().numpy()[c.slots]
    group, at = (64, 640) if kind == "fp8" else (32, 384)
    bad = rows[:, at:] == 255
    want = np.zeros_like(bad)
    want[1, slice(None) if norm else 40 // group] = True
    want[2, 500 // group] = True                # (under a norm infinity times zero; the others are zeros)
    want[3, 0] = kind == "fp4" and not norm     # (its square is infinite, so under a norm it is zero)
    np.testing.assert_array_equal(bad, want)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_append_skips_padding_and_reports_what_is_out_of_range(kind):
    c = Tokens(6, 9, 3, kind)
    slots, pos = c.slots.copy(), c.pos.copy()
    slots[2], pos[2] = -1, 1 << 30               # padding: not looked at
    slots[8], pos[8] = -(1 << 40), -5
    g, q = c.cache(), to_dev_bf16(c.q)
    out = torch.full((9, 3, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    assert c.run(g.tensor, q[..., 128:], out, slots=i64(slots), pos=i32(pos)) == 0
    full = c.cache()
    c.run(full.tensor, q[..., 128:], torch.empty_like(out))
    a, b = (x.tensor.view(torch.uint8).reshape(c.nb * c.bs, -1) for x in (g, full))
    keep = torch.ones(c.nb * c.bs, dtype=torch.bool, device="cuda")
    keep[i64(c.slots[[2, 8]])] = False
    assert torch.equal(a[keep], b[keep]) and (a[~keep] == 0x5A).all()
    assert (out[[2, 8]] == 2.0).all() and not (out[[0, 1, 3, 7]] == 2.0).all(-1).any()
    for bad in (dict(slot=c.nb * c.bs), dict(slot=1 << 62), dict(pos=-1), dict(pos=5000)):
        slots, pos = c.slots.copy(), c.pos.copy()
        slots[4], pos[4] = bad.get("slot", slots[4]), bad.get("pos", pos[4])
        g, out = c.cache(), torch.full((9, 3, 64), 2.0, dtype=torch.bfloat16, device="cuda")
        assert c.run(g.tensor, q[..., 128:], out, slots=i64(slots), pos=i32(pos)) == BAD_INDEX
        g.check("cache")
        a = g.tensor.view(torch.uint8).reshape(c.nb * c.bs, -1)
        keep = torch.ones(c.nb * c.bs, dtype=torch.bool, device="cuda")
        keep[c.slots[4]] = False
        assert torch.equal(a[keep], b[keep]) and (a[~keep] == 0x5A).all() and (out[4] == 2.0).all() and not (out[5] == 2.0).all()


def test_append_of_strided_rows_and_no_tokens():
    import chunked_prefill_attention_ragged_gb300 as mla
    c = Tokens(7, 20, 2, "fp4")
    wide = torch.zeros((20, 640), dtype=torch.bfloat16, device="cuda")
    wide[:, 64:] = to_dev_bf16(c.latent)
    a, b = c.cache(), c.cache()
    q = to_dev_bf16(c.q)
    heads_first = torch.zeros((2, 20, 64), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    out = torch.zeros((20, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert c.run(a.tensor, q[..., 128:], out) == 0
    assert c.run(b.tensor, q[..., 128:], heads_first, latent=wide[:, 64:]) == 0
    assert torch.equal(a.tensor, b.tensor) and torch.equal(out, heads_first)
    # one row of queries for both heads
    assert c.run(b.tensor, q[:, :1, 128:].expand(20, 2, 64), out) == 0 and torch.equal(out[:, 0], out[:, 1])
    none = torch.zeros((0, 576), dtype=torch.bfloat16, device="cuda")
    mla.mla_cache_append(a.tensor, none, i64([]), i32([]), to_dev(c.table), q_rope=q[:0, :, 128:])
    assert torch.equal(a.tensor, b.tensor)
    with pytest.raises(mla.MlaError):
        c.run(b.tensor, latent=wide[:, 60:636])      # not on 16 bytes
    with pytest.raises(ValueError):
        c.run(b.tensor, latent=torch.zeros((20, 1152), dtype=torch.bfloat16, device="cuda")[:, ::2])
    with pytest.raises(mla.MlaError):
        c.run(b.tensor, q[..., 128:], torch.zeros((20, 1, 64), dtype=torch.bfloat16, device="cuda").expand(20, 2, 64))
    with pytest.raises(ValueError):
        c.run(b.tensor, q[:5, :, 128:])
    with pytest.raises(TypeError):
        c.run(b.tensor, pos=i64(c.pos))


def test_append_replayed_on_another_stream():
    import chunked_prefill_attention_ragged_gb300 as mla
    c = Tokens(8, 12, 4, "fp4")
    g, table, w, q = c.cache(), to_dev(c.table), to_dev_bf16(c.weight), to_dev_bf16(c.q)
    lat, slots, pos = to_dev_bf16(c.latent), i64(c.slots), i32(c.pos)
    out = torch.zeros((12, 4, 64), dtype=torch.bfloat16, device="cuda")
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        mla.mla_cache_append(g.tensor, lat, slots, pos, table, norm_weight=w, q_rope=q[..., 128:], q_out=out)
    for seed in (9, 10):
        d = Tokens(seed, 12, 4, "fp4")
        lat.copy_(to_dev_bf16(d.latent))
        slots.copy_(i64(d.slots))
        pos.copy_(i32(d.pos))
        g.tensor.fill_(0x5A)
        graph.replay()
        want, w_out = d.cache(), torch.zeros_like(out)
        mla.mla_cache_append(want.tensor, lat, slots, pos, table, norm_weight=w, q_rope=q[..., 128:], q_out=w_out)
        torch.cuda.synchronize()
        assert torch.equal(g.tensor, want.tensor) and torch.equal(out, w_out)


# ------------------------------------------------------------------------------------- gather
@pytest.mark.parametrize("bs", [1, 5, 16, 64])
@pytest.mark.parametrize("batch", [1, 3, 40])
def test_gather(batch, bs):
    """Every code under every scale byte, NaN and overflow included."""
    import chunked_prefill_attention_ragged_gb300 as mla
    r = np.random.default_rng(batch + bs)
    lens, starts = r.integers(0, 60, batch), r.integers(0, 30, batch)
    lens[0] = 60
    width = -(-90 // bs)
    nb = batch * width + 1
    cache = r.integers(0, 256, (nb, bs, 400)).astype(np.uint8)
    table = r.permutation(nb)[:batch * width].reshape(batch, width)
    cu = np.concatenate([[0], np.cumsum(lens)])
    out, st = Guarded((int(cu[-1]), 576), torch.bfloat16), status()
    mla.mla_gather_latent_fp4(to_dev(cache), i32(table), i32(cu), i32(starts), int(cu[-1]), out.tensor, st)
    torch.cuda.synchronize()
    out.check("rows")
    got, want = bits_of(out.tensor), gather_latent_fp4(cache, table, cu, starts)
    nan = np.isnan(bf16_bits_to_f64(want))
    nan[:, 512:] = False
    assert np.isnan(bf16_bits_to_f64(got)[nan]).all()
    np.testing.assert_array_equal(got[~nan], want[~nan])
    assert int(st) == 0
    table[0, 0], table[0, 1 % width] = -1, nb
    if lens[0]:
        mla.mla_gather_latent_fp4(to_dev(cache), i32(table), i32(cu), i32(np.zeros(batch)), int(cu[-1]), out.tensor, st)
        assert int(st) == BAD_INDEX and (out.tensor[:min(60, bs)] == 0).all()


def test_scale_bytes_all():
    import chunked_prefill_attention_ragged_gb300 as mla
    r = np.random.default_rng(0)
    cache = np.zeros((1, 256, 400), dtype=np.uint8)
    cache[0, :, :256] = np.tile(r.permutation(256), (256, 1))
    cache[0, :, 384:] = np.arange(256)[:, None]
    got = bf16_bits_to_f64(bits_of(mla.mla_gather_latent_fp4(to_dev(cache), i32([[0]]), i32([0, 256]), i32([0]), 256)))
    codes = fp4_codes(cache[0])
    with np.errstate(over="ignore"):
        want = e2m1_to_f64(codes) * 2.0 ** (np.arange(256.0) - 127)[:, None]
        want[np.abs(want) > 3.4e38] *= np.inf
    want[255] = np.nan
    np.testing.assert_array_equal(got[:, :512], want)


def test_prefill_over_a_4_bit_cache():
    """Rows appended, then the pipeline over them, against the unchunked oracle over the rows' values."""
    import chunked_prefill_attention_ragged_gb300 as mla
    from chunked_prefill_attention_ragged_gb300.pipeline import ChunkedPrefill
    from oracle import chunked_prefill_attention
    from oracle.fp8_cache import f64_to_bf16_bits
    from oracle import fp4_values
    cb = wl.random_chunked_prefix(23, [130, 5, 260], [300, 0, 1000], 4, num_blocks=64, block_size=64, chunk_tokens=256)
    b = cb.new
    cache = torch.zeros((64, 64, 400), dtype=torch.uint8, device="cuda")
    slots, pos = [], []
    for r, n in enumerate([300, 0, 1000]):
        p = np.arange(n)
        slots.append(cb.block_table[r, p // 64].astype(np.int64) * 64 + p % 64)
        pos.append(p)
    slots, pos = np.concatenate(slots), np.concatenate(pos)
    latent = to_dev_bf16(cb.cache).view(-1, 576)[i64(slots)]
    mla.mla_cache_append(cache, latent, i64(slots), i32(pos), to_dev(angles(1000)))
    pipe = ChunkedPrefill(b.qo_indptr, cb.layout.cu_seq_lens, cb.layout.chunk_starts, b.num_heads, sm_scale=b.sm_scale,
                          cache_fp4=True)
    o, lse = pipe.run(to_dev_bf16(b.q), to_dev_bf16(b.k), to_dev_bf16(b.v), cache, to_dev(cb.block_table), to_dev_bf16(cb.w_kvb))
    torch.cuda.synchronize()
    pipe.check_status()
    values = f64_to_bf16_bits(fp4_values(cache.cpu().numpy().reshape(-1, 400))).reshape(64, 64, 576)
    o_ref, lse_ref = chunked_prefill_attention(b.q, b.k, b.v, b.qo_indptr, values, cb.block_table, cb.prefix_lens, cb.w_kvb,
                                               sm_scale=b.sm_scale)
    check_attention(f64_of_bf16(o), lse.double().cpu().numpy(), o_ref, lse_ref, "4-bit cache pipeline")
