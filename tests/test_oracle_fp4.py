"""Pins of the oracle's 4-bit entries, of the append and of verified drafts, without a GPU."""
import itertools

import numpy as np
import pytest

from oracle import (bf16_bits_to_f64, e2m1_to_f64, e4m3_to_f64, fp4_codes, fp4_values, gather_latent_fp4, normalise, pack_fp4,
                    pack_fp8, quantize, rotate, verify_children, verify_tree)
from oracle.fp8_cache import dequant_fp8_entries


def test_codes_by_hand():
    # sign, two exponent bits, one mantissa bit
    want = {0b0000: 0, 0b0001: 0.5, 0b0010: 1, 0b0011: 1.5, 0b0100: 2, 0b0101: 3, 0b0110: 4, 0b0111: 6, 0b1001: -0.5, 0b1111: -6}
    for code, value in want.items():
        assert e2m1_to_f64(code) == value


def test_an_entry_by_hand():
    e = np.zeros((1, 400), dtype=np.uint8)
    # word 0: value 0 is 1 (2), 2 is 6 (7), 7 is -0.5 (9); word 63 (values 504 ..): value 505 is 3 (5)
    e[0, 0], e[0, 3], e[0, 254] = 0x72, 0x90, 0x05
    e[0, 256:258] = [0x80, 0x3F]                     # the first rope value is 1.0
    e[0, 384:] = 127
    e[0, 399] = 129                                  # the last 32 values count four times
    v = fp4_values(e)[0]
    assert v[0] == 1 and v[2] == 6 and v[7] == -0.5 and v[505] == 12 and v[512] == 1
    assert np.count_nonzero(v) == 5


def test_pack_and_unpack():
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 16, (7, 512)).astype(np.uint8)
    rope, scales = rng.integers(0, 1 << 16, (7, 64)).astype(np.uint16), rng.integers(0, 253, (7, 16)).astype(np.uint8)
    e = pack_fp4(codes, rope, scales)
    assert e.shape == (7, 400) and np.array_equal(fp4_codes(e), codes) and np.array_equal(e[:, 384:], scales)
    cache = e.reshape(7, 1, 400)
    got = gather_latent_fp4(cache, np.array([[3, 1, 2]]), [0, 2], [1])
    assert np.array_equal(bf16_bits_to_f64(got[:, :512]), fp4_values(e[[1, 2]])[:, :512]) and np.array_equal(got[:, 512:], rope[[1, 2]])


@pytest.mark.parametrize("kind,group,reach", [("fp4", 32, 7), ("fp8", 64, 448)])
def test_quantize(kind, group, reach):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 512)) * 2.0 ** rng.integers(-20, 20, (5, 512 // group)).repeat(group, axis=-1)
    x[0, :group] = 0
    x[1, 0] = reach * 2.0 ** 3                       # exactly what the scale 2^3 reaches
    x[1, 1:group] = 0
    codes, scales = quantize(x, kind)
    assert scales[0, 0] == 0 and scales[1, 0] == 130
    values = (e2m1_to_f64(codes) if kind == "fp4" else e4m3_to_f64(codes)) * 2.0 ** (scales.astype(float) - 127).repeat(group, axis=-1)
    grid = np.unique(e2m1_to_f64(np.arange(16)) if kind == "fp4" else e4m3_to_f64(np.delete(np.arange(256), [127, 255]).astype(np.uint8)))
    for t in range(5):
        for i in range(512):
            s = 2.0 ** (float(scales[t, i // group]) - 127)
            assert abs(values[t, i] - x[t, i]) == np.abs(grid * s - x[t, i]).min()
    for t, g in itertools.product(range(5), range(512 // group)):
        top = np.abs(x[t, g * group:(g + 1) * group]).max()
        s = 2.0 ** (float(scales[t, g]) - 127)
        assert top <= reach * s and (scales[t, g] == 0 or top > reach * s / 2)


def test_quantize_ties_and_values_that_do_not_fit():
    x = np.zeros((1, 512))
    x[0, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0]
    x[0, 32], x[0, 64], x[0, 96] = np.nan, np.inf, 7.5 * 2.0 ** 125
    codes, scales = quantize(x, "fp4")
    assert e2m1_to_f64(codes[0, :8]).tolist() == [0, 1, 1, 2, 2, 4, 4, 6]
    assert scales[0, 0] == 127 and scales[0, 1:4].tolist() == [255] * 3 and (codes[0, 32:128] == 0).all()
    e = pack_fp8(*[quantize(x, "fp8")[0], np.zeros((1, 64), np.uint16), quantize(x, "fp8")[1]])
    assert dequant_fp8_entries(e).shape == (1, 576)


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotation(interleaved):
    """A quarter turn by hand, and lengths and relative angles kept."""
    table = np.zeros((3, 64))
    table[0, :32] = 1
    table[1, 32:] = 1                                # 90 degrees
    x = np.arange(64.0)[None].repeat(2, 0)
    y = rotate(x, [0, 1], table, interleaved)
    assert np.array_equal(y[0], x[0])
    if interleaved:
        assert y[1, :4].tolist() == [-1, 0, -3, 2]
    else:
        assert y[1, :2].tolist() == [-32, -33] and y[1, 32:34].tolist() == [0, 1]
    rng = np.random.default_rng(2)
    f = 10000.0 ** (-np.arange(32) / 32)
    angles = np.arange(40)[:, None] * f
    table = np.concatenate([np.cos(angles), np.sin(angles)], axis=1)
    q, k = rng.standard_normal((1, 3, 64)), rng.standard_normal((1, 3, 64))
    a = (rotate(q, [30], table, interleaved) * rotate(k, [21], table, interleaved)).sum(-1)
    b = (rotate(q, [9], table, interleaved) * k).sum(-1)
    np.testing.assert_allclose(a, b, rtol=1e-12)


def test_norm():
    y = normalise(np.full((1, 512), 3.0), np.arange(512), 0.0)
    np.testing.assert_allclose(y[0], np.arange(512))
    assert np.array_equal(normalise([[1.0, 2.0]], None, 0.5), [[1.0, 2.0]])


# ------------------------------------------------------------------------------------- verify
def chances(below):
    """Chance of each test to be the first that passes, and of none to pass."""
    out, rest = [], 1.0
    for b in below:
        b = min(b, 1.0)
        out.append(rest * b)
        rest *= 1 - b
    return out, rest


@pytest.mark.parametrize("children", [1, 2, 3])
def test_drawn_children_leave_the_target_as_it_is(children):
    """Summed over every draw of the children, the kept (or, where none is, the next) token has the target's chances."""
    rng = np.random.default_rng(children)
    for _ in range(4):
        p, q = rng.dirichlet(np.ones(4) * 0.7), rng.dirichlet(np.ones(4) * 0.7)
        total = np.zeros(4)
        for draw in itertools.product(range(4), repeat=children):
            weight = np.prod(q[list(draw)])
            below, left = verify_children(p, draw, q)
            first, none = chances(below)
            for x, c in zip(draw, first):
                total[x] += weight * c
            if none > 1e-12:
                total += weight * none * (left / left.sum())
        np.testing.assert_allclose(total, p, atol=1e-12)


def test_given_children_leave_the_target_as_it_is():
    rng = np.random.default_rng(9)
    for tokens in ([2], [0, 3], [1, 1, 4], [4, 3, 2, 1, 0]):
        p = rng.dirichlet(np.ones(5))
        below, left = verify_children(p, tokens)
        first, none = chances(below)
        total = np.zeros(5)
        for x, c in zip(tokens, first):
            if c:
                total[x] += c
        if none > 1e-12:
            total += none * left / left.sum()
        np.testing.assert_allclose(total, p, atol=1e-12)


def test_a_walk_by_hand():
    # node 0 -> {1: token 2, 2: token 0}, 1 -> {3: token 1}
    target = np.array([[0.5, 0.1, 0.4], [0.2, 0.7, 0.1], [1.0, 0.0, 0.0], [0.0, 0.25, 0.75]])
    tokens, parents = [9, 2, 0, 1], [-1, 0, 0, 1]
    u = [0.0, 0.39, 0.0, 0.69]
    assert verify_tree(target, tokens, parents, u, 0.2, 4) == ([0, 1, 3], 1)
    assert verify_tree(target, tokens, parents, u, 0.25, 4) == ([0, 1, 3], 2)
    assert verify_tree(target, tokens, parents, [0, 0.39, 0, 0.71], 0.99, 4) == ([0, 1], 2)      # 0.2, 0, 0.1 are left
    assert verify_tree(target, tokens, parents, [0, 0.41, 0.83, 0], 0.5, 4) == ([0, 2], 0)       # 0.5 of 0.6
    assert verify_tree(target, tokens, parents, [0, 0.41, 0.84, 0], 0.0, 4) == ([0], 1)          # only token 1 is left
    assert verify_tree(target, tokens, parents, u, 0.0, 2) == ([0, 1], 0)                        # a full path: p itself
    assert verify_tree(np.array([[0.0, 1.0]]), [3], [-1], [0.5], 0.999, 3) == ([0], 1)
    assert verify_tree(np.array([[0.0, 0.0]]), [3], [-1], [0.5], 0.5, 3) == ([0], -1)
