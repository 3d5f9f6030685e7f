"""The append's norm over all of bf16's range: squares of a row's values may leave fp32's."""
import numpy as np
import pytest

from chunked_prefill_attention_ragged_gb300 import workloads as wl
from gpu_util import to_dev, to_dev_bf16
from oracle import bf16_bits_to_f64, normalise
from test_gpu_fp4_cache import angles, i32, i64, status

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

POWERS = [-130, -120, -100, -76, -71, -66, -63, -31, -30, -29, -10, 0, 30, 54, 55, 56, 57, 60, 63, 64, 90, 120, 125]


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-12, 1e-6])
@pytest.mark.parametrize("peaked", [False, True])
def test_every_magnitude(eps, peaked):
    """Rows of about 2^k, and rows of one such value among values about 1.  A value is off by half a step of bf16 and by what
    fp32 loses before it (below 2^-19, see check_rows); by half a step of bf16's least numbers (2^-134) where it is one of
    them; and values 2^110 times smaller than their row's largest by what is left of them in fp32 (2^-149 beside 2^-70
    times the row's root mean square, which is 2^50 at least: 2^-129 of the quotient) and the weight, below 2."""
    import chunked_prefill_attention_ragged_gb300 as mla
    rng = np.random.default_rng(81)
    t = len(POWERS)
    x = rng.uniform(0.5, 2.0, (t, 576)) * rng.choice([-1.0, 1.0], (t, 576))
    if peaked:
        x[:, 77] *= 2.0 ** np.array(POWERS)
    else:
        x *= 2.0 ** np.array(POWERS)[:, None]
    bits = wl.to_bf16_bits(x.astype(np.float32))
    weight = wl.to_bf16_bits((1 + rng.uniform(-0.5, 0.9, 512)).astype(np.float32))
    cache = torch.zeros((t, 1, 576), dtype=torch.bfloat16, device="cuda")
    st = status()
    mla.mla_cache_append(cache, to_dev_bf16(bits), i64(np.arange(t)), i32(np.zeros(t)), to_dev(angles(1)),
                         norm_weight=to_dev_bf16(weight), norm_eps=eps, status=st)
    assert int(st) == 0
    want = normalise(bf16_bits_to_f64(bits)[:, :512], bf16_bits_to_f64(weight), float(np.float32(eps)))
    got = cache[:, 0, :512].double().cpu().numpy()
    assert np.isfinite(got).all()
    off = np.abs(got - want) - ((2.0 ** -8 + 2.0 ** -19) * np.abs(want) + 2.0 ** -134 + 2.0 ** -128)
    assert (off <= 0).all(), [POWERS[i] for i in np.nonzero((off > 0).any(1))[0]]


def test_rows_without_a_finite_norm():
    """x / sqrt(mean(x^2)): an infinity makes itself NaN and the others 0, a NaN the whole row NaN; so does 0 / 0."""
    import chunked_prefill_attention_ragged_gb300 as mla
    x = np.ones((3, 576), dtype=np.float32)
    x[0, 5], x[1, 6], x[2] = np.inf, np.nan, 0
    cache = torch.zeros((3, 1, 576), dtype=torch.bfloat16, device="cuda")
    mla.mla_cache_append(cache, to_dev_bf16(wl.to_bf16_bits(x)), i64([0, 1, 2]), i32([0, 0, 0]), to_dev(angles(1)),
                         norm_weight=torch.ones(512, dtype=torch.bfloat16, device="cuda"), norm_eps=0.0)
    got = cache[:, 0, :512].float()
    want = torch.zeros(512, device="cuda")
    want[5] = float("nan")
    assert torch.equal(torch.isnan(got[0]), torch.isnan(want)) and (got[0][~torch.isnan(want)] == 0).all()
    assert torch.isnan(got[1:]).all()
