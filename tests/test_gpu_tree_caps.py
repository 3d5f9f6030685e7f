"""Soft caps: a capped logit is good to a fraction of itself, not of the cap, and caps up to the largest
finite one leave small logits as they are."""
import numpy as np
import pytest

from test_gpu_speculative import i32, new_status

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("sm_scale", [0.0721687824, 1.0])
@pytest.mark.parametrize("cap", [1e-30, 0.5, 2.0, 30.0, 256.0, 300.0, 20000.0, 1e30, 3.4e38])
def test_capped_logit(cap, sm_scale):
    """One key and one nonzero product a row, so that the LSE is the logit.  What may be off: the product
    with sm_scale and the cap's factors, six roundings (6 * 2^-24 of the logit); where |x / cap| >= 1/4 tanh
    as 1 - 2 / (e^(2y) + 1): the exponential to 2^-22, sum, reciprocal 2^-23, together 2^-22 of 1, where tanh
    is at least 0.244: 2^-19.9 of the logit; below, a series whose next term is 2^-21.4 of it.  2^-19 covers
    them, and the way into and out of log2 units (2 * 2^-24)."""
    import chunked_prefill_attention_ragged_gb300 as mla
    heads = 128
    x = np.concatenate([s * 2.0 ** np.linspace(-20, 11.5, heads // 2) for s in (1, -1)])
    q = torch.zeros((1, heads, 576), dtype=torch.bfloat16, device="cuda")
    q[0, :, 70] = torch.from_numpy(x).to(torch.bfloat16).cuda()
    cache = torch.zeros((2, 64, 576), dtype=torch.bfloat16, device="cuda")
    cache[1, 0, 70], cache[1, 0, 3] = 1.0, -2.0
    st = new_status()
    o, lse = mla.mla_tree_attention(q, cache, i32([[1]]), i32([0, 1]), i32([1]), sm_scale=sm_scale, logits_soft_cap=cap,
                                    status=st)
    assert int(st) == 0 and torch.equal(o, cache[1, 0, :512].expand(1, heads, 512))
    c = float(np.float32(cap))
    want = c * np.tanh(float(np.float32(sm_scale)) * q[0, :, 70].double().cpu().numpy() / c)
    err = np.abs(lse[0].double().cpu().numpy() - want)
    assert (err <= 2.0 ** -19 * np.abs(want)).all(), np.max(err / np.abs(want)) * 2 ** 19


@pytest.mark.parametrize("cap", [2.0, 300.0])
def test_nan_and_infinite_logits_under_a_cap(cap):
    """A NaN in a query makes its row NaN; an infinite logit is the cap, of either sign."""
    import chunked_prefill_attention_ragged_gb300 as mla
    q = torch.zeros((1, 4, 576), dtype=torch.bfloat16, device="cuda")
    q[0, :, 70] = torch.tensor([float("nan"), float("inf"), float("-inf"), 0.5])
    cache = torch.zeros((1, 64, 576), dtype=torch.bfloat16, device="cuda")
    cache[0, :40, 70] = 1.0
    o, lse = mla.mla_tree_attention(q, cache, i32([[0]]), i32([0, 1]), i32([40]), sm_scale=1.0, logits_soft_cap=cap)
    assert torch.isnan(o[0, 0].float()).all() and bool(torch.isnan(lse[0, 0]))
    want = np.array([cap, -cap, cap * np.tanh(0.5 / cap)]) + np.log(40)
    assert (np.abs(lse[0, 1:].double().cpu().numpy() - want) <= 2.0 ** -19 * (cap + 4)).all()
    assert (o[0, 1:, 70] == 1.0).all()
