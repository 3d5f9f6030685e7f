"""Tree attention over a 4-bit cache without a workspace, where memory for the cache's rows in bf16 is not to be had."""
import numpy as np
import pytest

from gpu_util import bits_of, to_dev, to_dev_bf16
from test_gpu_fp4_attention import Problem4
from test_gpu_speculative import i32, new_status

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_short_of_memory():
    """The limit is this process's own, on what torch's allocator may take: 1.4 GB of rows do not fit under it."""
    import chunked_prefill_attention_ragged_gb300 as mla
    p = Problem4(51, [9, 4], [200, 77], 64, 64, True)
    b, blocks = p.b, 19000
    cache = torch.zeros((blocks, 64, 400), dtype=torch.uint8, device="cuda")
    cache[:len(p.entries)] = to_dev(p.entries)
    args = to_dev_bf16(b.q_abs), cache, to_dev(b.block_table), i32(b.qo_indptr), i32(p.kv), p.mask()
    small = torch.empty(mla.mla_tree_workspace(13, 64), dtype=torch.uint8, device="cuda")
    want = mla.mla_tree_attention_fp4(*args, sm_scale=b.sm_scale, workspace=small)
    need = mla.mla_tree_workspace_fp4(13, 64, 2, blocks, 64)
    assert need > small.numel() + (1 << 30)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    st = new_status()
    try:
        torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + small.numel() + (1 << 28)) / total)
        o, lse = mla.mla_tree_attention_fp4(*args, sm_scale=b.sm_scale, status=st)
        torch.cuda.synchronize()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert int(st) == 0 and np.array_equal(bits_of(o), bits_of(want[0])) and torch.equal(lse, want[1])
    p.check(o, lse)
    o, lse = mla.mla_tree_attention_fp4(*args, sm_scale=b.sm_scale, status=st)
    p.check(o, lse)
