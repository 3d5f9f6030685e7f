"""Views of one token or one head given to mla_cache_append: torch lets such a dimension have any stride."""
import numpy as np
import pytest

from gpu_util import bits_of, to_dev, to_dev_bf16
from test_gpu_fp4_cache import Tokens, i32, i64, status

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("t,heads", [(1, 5), (6, 1), (1, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_strides_of_single_elements(t, heads, in_place):
    import chunked_prefill_attention_ragged_gb300 as mla
    k = Tokens(71, t, heads, "fp4")
    q = to_dev_bf16(k.q)[..., 128:].contiguous()

    def odd(fill):
        flat = torch.full((t * heads * 64 + 999,), 9.0, dtype=torch.bfloat16, device="cuda")
        at = (323 if t == 1 else 64 * heads, 77 if heads == 1 else 64, 1)
        view = torch.as_strided(flat, (t, heads, 64), at)
        if fill is not None:
            view.copy_(fill)
        return view, flat

    def run(q_rope, q_out):
        cache, st = k.cache(), status()
        mla.mla_cache_append(cache.tensor, to_dev_bf16(k.latent), i64(k.slots), i32(k.pos), to_dev(k.table),
                             norm_weight=to_dev_bf16(k.weight), q_rope=q_rope, q_out=q_out, status=st)
        torch.cuda.synchronize()
        cache.check("cache")
        assert int(st) == 0
        return cache.tensor

    want = torch.zeros_like(q)
    rows = run(q, want)
    view, flat = odd(q)
    out, out_flat = (view, flat) if in_place else odd(None)
    got = run(view, None if in_place else out)
    assert np.array_equal(bits_of(out), bits_of(want)) and torch.equal(got, rows)
    out.fill_(9.0)
    assert bool((out_flat == 9.0).all()), "beside the heads"
