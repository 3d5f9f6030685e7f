"""The 4-bit latent cache entry (MLA_ENTRY_FP4 of include/mla_prefill.h) and the append of new tokens.

An entry of 400 bytes: 512 e2m1 codes, eight to a 32-bit little-endian word (values 8 w + 0, 2, 4, 6
of word w in its nibbles 0 .. 3, values 8 w + 1, 3, 5, 7 in nibbles 4 .. 7), 64 bf16 of rope, 16 scale
bytes 2^(b - 127) for 32 values each.  vLLM ``vllm/models/deepseek_v4/sparse_mla.py`` has the same
three parts with an 8-bit latent.  A group's scale is the least power of two, not below 2^-127, with
|value| <= reach * scale, where reach is 7 for e2m1 and 448 for e4m3.
"""
import numpy as np

from .bf16 import bf16_bits_to_f64
from .fp8_cache import e4m3_to_f64, f64_to_bf16_bits, ue8m0_to_f64
from .gather import gather_latent

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# where the nibble of value i of a word's eight starts
SHIFT = np.array([0, 16, 4, 20, 8, 24, 12, 28])


def e2m1_to_f64(codes) -> np.ndarray:
    c = np.asarray(codes, dtype=np.int64)
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]


def fp4_codes(entries: np.ndarray) -> np.ndarray:
    """The 512 codes of each entry (uint8 [..., 400])."""
    words = np.ascontiguousarray(entries[..., :256]).view("<u4")
    return ((words[..., None] >> SHIFT.astype(np.uint32)) & 15).reshape(entries.shape[:-1] + (512,))


def fp4_values(entries: np.ndarray) -> np.ndarray:
    """fp64 [..., 576] of entries."""
    scale = np.repeat(ue8m0_to_f64(entries[..., 384:]), 32, axis=-1)
    with np.errstate(invalid="ignore"):
        lat = e2m1_to_f64(fp4_codes(entries)) * scale
    rope = bf16_bits_to_f64(np.ascontiguousarray(entries[..., 256:384]).view("<u2"))
    return np.concatenate([lat, rope], axis=-1)


def gather_latent_fp4(cache: np.ndarray, block_table, cu_seq_lens, chunk_starts) -> np.ndarray:
    """bf16 bits [T, 576] of the rows that the slot rule names."""
    rows = gather_latent(cache, block_table, cu_seq_lens, chunk_starts)
    out = f64_to_bf16_bits(fp4_values(rows))
    out[:, 512:] = np.ascontiguousarray(rows[:, 256:384]).view("<u2")
    return out


# ------------------------------------------------------------------------------------ append
def rotate(x, positions, cos_sin, interleaved) -> np.ndarray:
    """x [T, ..., 64] turned, token t by the angles of row positions[t] of cos_sin [P, 64]."""
    x = np.asarray(x, dtype=np.float64)
    out = np.empty_like(x)
    for t, pos in enumerate(positions):
        for i in range(32):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
            c, s = float(cos_sin[pos, i]), float(cos_sin[pos, 32 + i])
            out[t, ..., a] = x[t, ..., a] * c - x[t, ..., b] * s
            out[t, ..., b] = x[t, ..., b] * c + x[t, ..., a] * s
    return out


def normalise(x, weight, eps) -> np.ndarray:
    """x [T, 512] / sqrt(mean(x^2) + eps) * weight; weight None: x."""
    x = np.asarray(x, dtype=np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def group_scales(x, group, reach, most=254) -> np.ndarray:
    """Scale bytes [T, 512 / group] of values x [T, 512]."""
    out = np.zeros((x.shape[0], x.shape[1] // group), dtype=np.uint8)
    for t in range(x.shape[0]):
        for g in range(out.shape[1]):
            v = np.abs(x[t, g * group:(g + 1) * group])
            b = 0
            while b <= most and not (v <= reach * 2.0 ** (b - 127)).all():
                b += 1
            out[t, g] = b if b <= most else 255
    return out


def nearest_codes(y, grid) -> np.ndarray:
    """Index into `grid` (ascending magnitudes) nearest to |y|, ties to the even index."""
    a = np.abs(y)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    up = (a - grid[lo] > grid[hi] - a) | ((a - grid[lo] == grid[hi] - a) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def quantize(x, kind):
    """Codes and scale bytes of values x [T, 512]: kind "fp4" (codes 0 .. 15) or "fp8" (e4m3 bytes)."""
    x = np.asarray(x, dtype=np.float64)
    group, reach, most, sign = (32, 7.0, 252, 8) if kind == "fp4" else (64, 448.0, 254, 128)
    grid = E2M1 if kind == "fp4" else e4m3_to_f64(np.arange(127, dtype=np.uint8))
    scales = group_scales(x, group, reach, most)
    bad = np.repeat(scales == 255, group, axis=-1)
    y = np.where(bad, 0.0, x) / np.where(bad, 1.0, 2.0 ** (np.repeat(scales, group, axis=-1).astype(np.float64) - 127))
    return (nearest_codes(y, grid) | np.where(np.signbit(y), sign, 0)).astype(np.uint8), scales


def pack_fp4(codes, rope_bits, scales) -> np.ndarray:
    """Entries uint8 [T, 400]."""
    words = np.zeros((codes.shape[0], 64), dtype=np.uint32)
    for i in range(8):
        words |= codes[:, i::8].astype(np.uint32) << np.uint32(SHIFT[i])
    rope = np.ascontiguousarray(rope_bits.astype("<u2")).view(np.uint8)
    return np.concatenate([words.astype("<u4").view(np.uint8), rope, scales], axis=-1)


def pack_fp8(codes, rope_bits, scales) -> np.ndarray:
    """Entries uint8 [T, 648]."""
    return np.concatenate([codes, np.ascontiguousarray(rope_bits.astype("<u2")).view(np.uint8), scales], axis=-1)
