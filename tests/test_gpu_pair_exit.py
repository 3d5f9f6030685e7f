"""Kernels of CTA pairs that are over at once: of 76 pairs all but a few have nothing to do, or one tile, and leave while
the other CTA's last arrivals are on their way.  Call after call, the same answers and no status."""
import numpy as np
import pytest

from chunked_prefill_attention_ragged_gb300 import workloads as wl
from gpu_util import bits_of, to_dev, to_dev_bf16
from test_gpu_fp4_attention import Problem4
from test_gpu_speculative import Problem, i32, new_status

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("bs", [64, 5])
@pytest.mark.parametrize("kind", [Problem, Problem4])
def test_tree_attention(kind, bs):
    import chunked_prefill_attention_ragged_gb300 as mla
    p = kind(61, [2, 0, 1], [70, 9, 300], 40, bs, False)
    b = p.b
    call = mla.mla_tree_attention_fp4 if kind is Problem4 else mla.mla_tree_attention
    cache = to_dev(p.entries) if kind is Problem4 else to_dev_bf16(b.cache)
    st = new_status()
    args = to_dev_bf16(b.q_abs), cache, to_dev(b.block_table), i32(b.qo_indptr), i32(p.kv)
    o, lse = call(*args, sm_scale=b.sm_scale, status=st)
    p.check(o, lse)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(50):
            call(*args, sm_scale=b.sm_scale, o=o2, lse=lse2, status=st)
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    assert int(st) == 0 and np.array_equal(bits_of(o), bits_of(o2)) and torch.equal(lse, lse2)


def test_prefill(monkeypatch):
    import chunked_prefill_attention_ragged_gb300 as mla
    monkeypatch.setenv("MLA_PLAN_CTA_PAIRS", "1")
    b = wl.random_ragged(62, [3, 130], [65, 130], 2)
    plan = mla.mla_prefill_plan(b.qo_indptr, b.kv_indptr, 2, sm_scale=b.sm_scale)
    assert plan.cta_pairs
    q, k, v = (to_dev_bf16(x) for x in (b.q, b.k, b.v))
    o, lse = plan.run(q, k, v)
    for _ in range(1000):
        o2, lse2 = plan.run(q, k, v)
    torch.cuda.synchronize()
    assert plan.status() == 0 and np.array_equal(bits_of(o), bits_of(o2)) and torch.equal(lse, lse2)
