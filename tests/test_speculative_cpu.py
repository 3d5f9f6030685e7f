"""Refusals of the speculative-decoding entry points, without a GPU: nothing reaches the device."""
import pytest

import chunked_prefill_attention_ragged_gb300 as mla

torch = pytest.importorskip("torch")
A = 4096   # an aligned address that is never followed


def tables(**kw):
    a = dict(seq=3 * A, new=4 * A, batch=2, bs=64, table=A, m=4, held=A, free=A, cap=8, count=A, qo=A, kv=A, slots=A, n=3,
             status=None)
    a.update(kw)
    return mla.library().mla_block_table_update(a["seq"], a["new"], a["batch"], a["bs"], a["table"], a["m"], a["held"],
                                                a["free"], a["cap"], a["count"], a["qo"], a["kv"], a["slots"], a["n"],
                                                a["status"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(batch=-1), -1), (dict(bs=0), -1), (dict(m=-1), -1), (dict(cap=-1), -1), (dict(n=-1), -1),
    (dict(batch=8193), -3), (dict(batch=8000, m=1 << 20), -3), (dict(n=1 << 31), -3),
    (dict(seq=None), -1), (dict(new=None), -1), (dict(table=None), -1), (dict(held=None), -1), (dict(free=None), -1),
    (dict(count=None), -1), (dict(slots=None), -1), (dict(slots=A + 4), -1), (dict(seq=A + 2), -1),
    (dict(status=A + 1), -1),
    (dict(kv=A, seq=A, new=2 * A), -1), (dict(qo=A, new=A, seq=2 * A), -1), (dict(held=A, seq=A, new=2 * A), -1),
])
def test_block_table_update_refuses(kw, rc):
    assert tables(**kw) == rc


def mask(**kw):
    a = dict(parents=A, qo=A, kv=None, batch=2, rows=5, words=1, mask=A, pos=None, status=None)
    a.update(kw)
    return mla.library().mla_tree_mask(a["parents"], a["qo"], a["kv"], a["batch"], a["rows"], a["words"], a["mask"],
                                       a["pos"], a["status"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(batch=-1), -1), (dict(rows=-1), -1), (dict(words=0), -1), (dict(words=1025), -3), (dict(rows=1 << 31), -3),
    (dict(parents=None), -1), (dict(qo=None), -1), (dict(mask=None), -1), (dict(mask=A + 4), -1),
    (dict(pos=A + 2), -1), (dict(batch=0), 0), (dict(rows=0), 0),
])
def test_tree_mask_refuses(kw, rc):
    assert mask(**kw) == rc


def attention(**kw):
    a = dict(q=A, cache=A, nb=8, bs=64, table=A, m=4, qo=A, kv=A, mask=None, words=0, batch=2, rows=5, heads=16,
             scale=0.07, cap=0.0, o=A, lse=A, ws=A, ws_bytes=1 << 40, status=None)
    a.update(kw)
    return mla.library().mla_tree_attention(a["q"], a["cache"], a["nb"], a["bs"], a["table"], a["m"], a["qo"], a["kv"],
                                            a["mask"], a["words"], a["batch"], a["rows"], a["heads"], a["scale"],
                                            a["cap"], a["o"], a["lse"], a["ws"], a["ws_bytes"], a["status"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(batch=-1), -1), (dict(rows=-1), -1), (dict(nb=-1), -1), (dict(bs=0), -1), (dict(m=-1), -1),
    (dict(heads=0), -1), (dict(heads=65536), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(cap=float("inf")), -1),
    (dict(words=1), -1), (dict(mask=A, words=0), -1), (dict(mask=A, words=1025), -3), (dict(mask=A + 4, words=1), -1),
    (dict(nb=1 << 25, bs=64), -3), (dict(rows=1 << 27, heads=16), -3), (dict(rows=1 << 62, heads=16), -3),
    (dict(m=1 << 26, bs=64), -3),
    (dict(q=None), -1), (dict(cache=None), -1), (dict(table=None), -1), (dict(qo=None), -1), (dict(kv=None), -1),
    (dict(o=None), -1), (dict(ws=None), -1), (dict(q=A + 8), -1), (dict(cache=A + 8), -1), (dict(o=A + 8), -1),
    (dict(ws=A + 8), -1), (dict(lse=A + 2), -1), (dict(status=A + 2), -1),
    (dict(batch=0), 0), (dict(rows=0), 0),
])
def test_tree_attention_refuses(kw, rc):
    assert attention(**kw) == rc


def commit(**kw):
    a = dict(cache=A, layers=2, stride=8 * 64 * 576, nb=8, bs=64, e=576, table=A, m=4, seq=A, acc=A, counts=A, batch=2,
             width=3, status=None)
    a.update(kw)
    return mla.library().mla_tree_commit(a["cache"], a["layers"], a["stride"], a["nb"], a["bs"], a["e"], a["table"],
                                         a["m"], a["seq"], a["acc"], a["counts"], a["batch"], a["width"], a["status"],
                                         None)


@pytest.mark.parametrize("kw,rc", [
    (dict(layers=-1), -1), (dict(nb=-1), -1), (dict(bs=0), -1), (dict(e=572), -1), (dict(e=0), -1), (dict(m=-1), -1),
    (dict(batch=-1), -1), (dict(width=-1), -1), (dict(stride=8 * 64 * 576 - 8), -1), (dict(stride=8 * 64 * 576 + 4), -1),
    (dict(batch=65536), -3), (dict(cache=None), -1), (dict(seq=None), -1), (dict(acc=None), -1),
    (dict(counts=None), -1), (dict(table=None), -1), (dict(cache=A + 8), -1), (dict(counts=A + 2), -1),
    (dict(batch=0), 0), (dict(layers=0), 0), (dict(width=0), 0),
])
def test_tree_commit_refuses(kw, rc):
    assert commit(**kw) == rc


def test_workspace_refuses():
    lib = mla.library()
    assert lib.mla_tree_workspace(4, 16, None) == -1
    with pytest.raises(mla.MlaError):
        mla.mla_tree_workspace(-1, 16)
    with pytest.raises(mla.MlaError):
        mla.mla_tree_workspace(1 << 40, 16)
    with pytest.raises(mla.MlaError):
        mla.mla_tree_workspace(1 << 62, 16)   # (times the heads: 0 in 64 bits)


def test_python_wants_cuda_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(TypeError):
        mla.mla_block_table_update(i, i, t, i, i, i[:1], 64)
    with pytest.raises(TypeError):
        mla.mla_tree_mask(i, i, 1)
    with pytest.raises(TypeError):
        mla.mla_tree_attention(torch.zeros(1, 1, 576), torch.zeros(1, 1, 576), t, i, i, sm_scale=1.0)
    with pytest.raises(TypeError):
        mla.mla_tree_commit(torch.zeros(1, 1, 576), t, i, t, i)


@pytest.mark.parametrize("kw", [
    dict(seq=A + 4, kv=A), dict(seq=A, kv=A + 4), dict(new=A + 8, qo=A), dict(seq=A - 4, held=A), dict(new=A + 20, slots=A),
    dict(new=A + 28, table=A), dict(seq=A + 28, free=A), dict(new=A, count=A + 4), dict(seq=A, status=A + 4),
])
def test_block_table_update_refuses_overlap(kw):
    """The lengths beside, not the same as, what is written: elsewhere everything is apart."""
    a = dict(seq=3 * A, new=4 * A, table=5 * A, held=6 * A, free=7 * A, count=8 * A, qo=9 * A, kv=10 * A, slots=11 * A)
    a.update(kw)
    assert tables(**a) == -1
