"""mla_cache_append refuses outputs that share memory with anything but, in place, the queries.  Without a GPU: what is not
refused ends at the launch, which fails here."""
import numpy as np
import pytest

import chunked_prefill_attention_ragged_gb300 as mla

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that nothing may follow")
FAR = 1 << 32                      # between arrays that have nothing to do with one another
NAMES = ["cache", "latent", "w", "pos", "cs", "slots", "q", "out", "status"]
INVALID = -1


def append(n=3, heads=2, qt=384, qh=192, ot=1152, oh=576, stride=576, entry=2, nb=8, bs=64, most=100, **at):
    a = {name: (k + 1) * FAR for k, name in enumerate(NAMES)}
    a.update(at)
    return mla.library().mla_cache_append(a["cache"], entry, nb, bs, a["latent"], stride, a["w"], 1e-6, a["pos"], a["cs"], most, 1,
                                          a["slots"], n, a["q"], qt, qh, heads, a["out"], ot, oh, a["status"], None)


def test_apart_is_not_refused():
    assert append() not in (0, INVALID) and append(status=None, w=None) not in (0, INVALID)


SIZES = {"cache": 8 * 64 * 400, "latent": 3 * 1152, "w": 1024, "pos": 12, "cs": 25600, "slots": 24,
         "q": (2 * 384 + 192 + 64) * 2, "out": (2 * 1152 + 576 + 64) * 2, "status": 4}


@pytest.mark.parametrize("written,other", [(w, o) for w in ("cache", "out", "status") for o in NAMES if o != w])
def test_each_output_against_each_array(written, other):
    """The last bytes of one on the first of the other, and just apart."""
    at = 20 * FAR
    for first, second in ((written, other), (other, written)):
        room = -(-SIZES[first] // 16) * 16
        assert append(**{first: at, second: at + room}) != INVALID
        last = (SIZES[first] - 1) // 16 * 16      # (the first of these bytes is inside)
        assert append(**{first: at, second: at + last}) == INVALID


def test_in_place():
    q = 30 * FAR
    assert append(q=q, out=q, ot=384, oh=192) != INVALID
    assert append(q=q, out=q, ot=384, oh=200) == INVALID and append(q=q, out=q, ot=400, oh=192) == INVALID
    assert append(q=q, out=q, ot=384, oh=192, latent=q) == INVALID


@pytest.mark.parametrize("by", [-128, -112, -16, 16, 64, 112, 128, 256, 384 - 128, 384, 400, 768, -768])
def test_views_of_the_same_rows(by):
    """q[..., a:a + 64] and q[..., b:b + 64] of q [T, H, 192]: apart, or part of each other."""
    q = 30 * FAR
    want = any(abs(by + 768 * t + 384 * h) < 128 for t in range(-2, 3) for h in range(-1, 2))
    assert (append(q=q, out=q + by, ot=384, oh=192) == INVALID) == want


def test_queries_and_absorbed_queries_of_one_buffer():
    """A token's row: H x 192 of queries, H x 576 of absorbed ones, the latent."""
    for heads, n in ((16, 5), (128, 2048)):
        row, base = heads * 768 + 576, 40 * FAR
        q, out, lat = base + 2 * 128, base + 2 * (heads * 192 + 512), base + 2 * heads * 768
        kw = dict(n=n, heads=heads, qt=row, qh=192, ot=row, oh=576, stride=row)
        assert append(q=q, out=out, latent=lat, **kw) != INVALID
        assert append(q=q, out=out - 2 * heads * 192, latent=lat, **kw) == INVALID
        assert append(q=q, out=out, latent=lat - 16, **kw) == INVALID
        # heads before tokens
        kw = dict(n=n, heads=heads, qt=192, qh=192 * n, ot=192, oh=192 * n)
        assert append(q=q, out=q - 256, **kw) != INVALID and append(q=q, out=q - 112, **kw) == INVALID


def test_against_every_piece():
    rng = np.random.default_rng(5)
    base, seen = 50 * FAR, [0, 0, 0]
    for _ in range(4000):
        n, heads = int(rng.integers(1, 5)), int(rng.integers(1, 5))
        step = lambda: int(rng.integers(8, 60)) * 8  # noqa: E731
        qt, qh = step(), step()
        ot, oh = [(qt, qh), (qt, step()), (step(), qh), (step(), step())][int(rng.integers(0, 4))]
        by = int(rng.integers(-150, 150)) * 16
        mine = [2 * (t * ot + h * oh) + by for t in range(n) for h in range(heads)]
        if any(abs(x - y) < 128 for i, x in enumerate(mine) for y in mine[:i]):
            continue   # (rows of q_out that share memory are refused for that)
        theirs = [2 * (t * qt + h * qh) for t in range(n) for h in range(heads)]
        hit = any(abs(x - y) < 128 for x in mine for y in theirs)
        place = by == 0 and (ot, oh) == (qt, qh)
        got = append(n=n, heads=heads, qt=qt, qh=qh, ot=ot, oh=oh, q=base, out=base + by) == INVALID
        common = n == 1 or heads == 1 or qt == ot or qh == oh
        ranges = min(mine) < max(theirs) + 128 and min(theirs) < max(mine) + 128
        # (heads that interleave with tokens in ways that the row test takes for shared memory: refused all the same)
        heads_reach, tokens_reach = (heads - 1) * oh + 64, (n - 1) * ot + 64
        crossed = heads > 1 and n > 1 and ot < heads_reach and oh < tokens_reach
        want = crossed or (not place and (hit if common else ranges))
        assert got == want, (n, heads, qt, qh, ot, oh, by)
        seen[0] += hit and not place
        seen[1] += common and ranges and not hit
        seen[2] += not common
    assert min(seen) > 50
