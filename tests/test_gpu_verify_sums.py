"""Draft verification over rows whose sum is not 1, up to the largest that the header allows (below 2^21)."""
import numpy as np
import pytest

from test_gpu_speculative import i32, new_status

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("vocab", [5, 2048, 4099, 131072, (1 << 21) - 8])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_rows_of_ones(vocab, kind):
    """The next token is floor(u V): u V is exact in 64 bits, as are the sums."""
    import chunked_prefill_attention_ragged_gb300 as mla
    u = np.array([0.0, 0.1, 0.5, 0.75, 0.9999, 1 - 2.0 ** -24], dtype=np.float32)
    p = torch.ones((len(u), vocab), dtype=kind, device="cuda")
    st = new_status()
    path, counts, token = mla.mla_tree_verify(p, i32(np.zeros(len(u))), i32(np.arange(len(u) + 1)),
                                              torch.zeros(len(u), device="cuda"), torch.from_numpy(u).cuda(), 2, status=st)
    assert int(st) == 0 and counts.tolist() == [1] * len(u) and path.tolist() == [[0, -1]] * len(u)
    assert token.tolist() == np.floor(u.astype(np.float64) * vocab).astype(int).tolist()
