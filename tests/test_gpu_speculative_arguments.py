"""Arguments of the speculative-decoding calls that the Python side looks at."""
import pytest

from test_gpu_speculative import i32

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_a_status_without_an_element_is_refused():
    """It has no address, and would pass for "no status"."""
    import chunked_prefill_attention_ragged_gb300 as mla
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    qo, kv, table = i32([0, 1]), i32([1]), i32([[0]])
    cache = torch.zeros((1, 4, 576), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((1, 2, 576), dtype=torch.bfloat16, device="cuda")
    for call in (lambda st: mla.mla_block_table_update(i32([1]), i32([1]), table, i32([1]), i32([0]), i32([0]), 4, status=st),
                 lambda st: mla.mla_tree_mask(i32([-1]), qo, 1, status=st),
                 lambda st: mla.mla_tree_attention(q, cache, table, qo, kv, sm_scale=0.1, status=st),
                 lambda st: mla.mla_tree_commit(cache, table, kv, i32([[0]]), i32([1]), status=st)):
        for empty in (none, torch.zeros(3, dtype=torch.int32, device="cuda")[3:]):
            with pytest.raises(ValueError, match="status"):
                call(empty)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(st)
        assert int(st) == 0
