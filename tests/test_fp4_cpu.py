"""Refusals of the 4-bit cache's, the append's and the verification's entry points, without a GPU."""
import ctypes

import numpy as np
import pytest

import chunked_prefill_attention_ragged_gb300 as mla

torch = pytest.importorskip("torch")
A = 4096   # an aligned address that is never followed


def append(**kw):
    a = dict(cache=A, entry=2, nb=8, bs=64, latent=A, stride=576, w=A, eps=1e-6, pos=A, cs=A, most=100, inter=1, slots=A, n=3,
             q=A, qt=192, qh=192, heads=1, out=A, ot=192, oh=192, status=None)
    a.update(kw)
    return mla.library().mla_cache_append(a["cache"], a["entry"], a["nb"], a["bs"], a["latent"], a["stride"], a["w"], a["eps"],
                                          a["pos"], a["cs"], a["most"], a["inter"], a["slots"], a["n"], a["q"], a["qt"],
                                          a["qh"], a["heads"], a["out"], a["ot"], a["oh"], a["status"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(entry=-1), -1), (dict(entry=3), -1), (dict(nb=-1), -1), (dict(bs=0), -1), (dict(n=-1), -1), (dict(most=-1), -1),
    (dict(heads=-1), -1), (dict(stride=568), -1), (dict(stride=580), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(eps=float("inf")), -1), (dict(qt=190), -1), (dict(qh=100), -1), (dict(ot=196), -1), (dict(oh=-192), -1),
    (dict(n=1 << 31), -3), (dict(heads=65536), -3), (dict(nb=1 << 50, bs=64), -3), (dict(stride=1 << 60), -3),
    (dict(cache=None), -1), (dict(latent=None), -1), (dict(pos=None), -1), (dict(cs=None), -1), (dict(slots=None), -1),
    (dict(q=None), -1), (dict(out=None), -1), (dict(cache=A + 8), -1), (dict(latent=A + 8), -1), (dict(w=A + 2), -1),
    (dict(cs=A + 4), -1), (dict(pos=A + 2), -1), (dict(slots=A + 4), -1), (dict(q=A + 8), -1), (dict(out=A + 8), -1),
    (dict(status=A + 2), -1), (dict(entry=1, cache=A + 4), -1),
    (dict(ot=256), -1),                                                  # in place with other strides
    (dict(out=2 * A, ot=56), -1), (dict(out=2 * A, oh=0, heads=2), -1),  # rows that share memory
    (dict(out=2 * A, ot=64, oh=64, heads=2), -1), (dict(out=2 * A, ot=64, oh=128, heads=2), -1),
    (dict(n=0), 0),
])
def test_append_refuses(kw, rc):
    assert append(**kw) == rc


def gather(**kw):
    a = dict(cache=A, nb=8, bs=64, e=400, table=A, m=4, cu=A, starts=A, batch=2, n=5, out=A, status=None)
    a.update(kw)
    return mla.library().mla_gather_latent_fp4(a["cache"], a["nb"], a["bs"], a["e"], a["table"], a["m"], a["cu"], a["starts"],
                                               a["batch"], a["n"], a["out"], a["status"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(n=-1), -1), (dict(batch=-1), -1), (dict(nb=-1), -1), (dict(bs=0), -1), (dict(m=-1), -1), (dict(e=648), -3),
    (dict(batch=0), -2), (dict(cache=None), -1), (dict(table=None), -1), (dict(cu=None), -1), (dict(starts=None), -1),
    (dict(out=None), -1), (dict(out=A + 8), -1), (dict(cache=A + 8), -1), (dict(status=A + 2), -1), (dict(n=0), 0),
])
def test_gather_refuses(kw, rc):
    assert gather(**kw) == rc


def attention(**kw):
    a = dict(q=A, cache=A, nb=8, bs=64, table=A, m=4, qo=A, kv=A, mask=None, words=0, batch=2, rows=5, heads=16,
             scale=0.07, cap=0.0, o=A, lse=A, ws=A, ws_bytes=1 << 40, status=None)
    a.update(kw)
    return mla.library().mla_tree_attention_fp4(a["q"], a["cache"], a["nb"], a["bs"], a["table"], a["m"], a["qo"], a["kv"],
                                                a["mask"], a["words"], a["batch"], a["rows"], a["heads"], a["scale"],
                                                a["cap"], a["o"], a["lse"], a["ws"], a["ws_bytes"], a["status"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(batch=-1), -1), (dict(rows=-1), -1), (dict(nb=-1), -1), (dict(bs=0), -1), (dict(heads=0), -1),
    (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(cap=float("inf")), -1), (dict(words=1), -1),
    (dict(mask=A, words=0), -1), (dict(mask=A, words=1025), -3), (dict(nb=1 << 25, bs=64), -3),
    (dict(rows=1 << 27, heads=16), -3), (dict(q=None), -1), (dict(cache=None), -1), (dict(o=None), -1), (dict(ws=None), -1),
    (dict(cache=A + 8), -1), (dict(ws=A + 8), -1), (dict(status=A + 2), -1), (dict(batch=0), 0), (dict(rows=0), 0),
])
def test_attention_refuses(kw, rc):
    assert attention(**kw) == rc


def verify(**kw):
    a = dict(p=A, q=A, kind=0, vocab=1000, tok=A, par=A, qo=A, batch=2, rows=5, u=A, ul=A, acc=A, most=4, cnt=A, nxt=A, status=None)
    a.update(kw)
    return mla.library().mla_tree_verify(a["p"], a["q"], a["kind"], a["vocab"], a["tok"], a["par"], a["qo"], a["batch"],
                                         a["rows"], a["u"], a["ul"], a["acc"], a["most"], a["cnt"], a["nxt"], a["status"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(kind=2), -1), (dict(kind=-1), -1), (dict(vocab=0), -1), (dict(batch=-1), -1), (dict(rows=-1), -1), (dict(most=0), -1),
    (dict(vocab=(1 << 24) + 1), -3), (dict(rows=1 << 31), -3), (dict(batch=1 << 30, vocab=1 << 20), -3),
    (dict(p=None), -1), (dict(tok=None), -1), (dict(qo=None), -1), (dict(u=None), -1), (dict(ul=None), -1), (dict(acc=None), -1),
    (dict(cnt=None), -1), (dict(nxt=None), -1), (dict(p=A + 2), -1), (dict(q=A + 2), -1), (dict(kind=1, p=A + 1), -1),
    (dict(tok=A + 2), -1), (dict(status=A + 2), -1), (dict(batch=0), 0),
])
def test_verify_refuses(kw, rc):
    assert verify(**kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(rows=-1), -1), (dict(heads=0), -1), (dict(heads=65536), -1), (dict(batch=-1), -1), (dict(nb=-1), -1), (dict(bs=0), -1),
    (dict(rows=1 << 40), -3), (dict(nb=1 << 31), -3), (dict(nb=1 << 26, bs=64), -3),
])
def test_workspace_refuses(kw, rc):
    a = dict(rows=96, heads=128, batch=4, nb=10, bs=64)
    a.update(kw)
    lib, n = mla.library(), ctypes.c_int64(7)
    assert lib.mla_tree_workspace_fp4(a["rows"], a["heads"], a["batch"], a["nb"], a["bs"], ctypes.byref(n)) == rc and n.value == 7
    assert lib.mla_tree_workspace_fp4(4, 16, 1, 1, 1, None) == -1
    with pytest.raises(mla.MlaError):
        mla.mla_tree_workspace_fp4(a["rows"], a["heads"], a["batch"], a["nb"], a["bs"])


def test_python_wants_cuda_tensors():
    i, f = torch.zeros(2, dtype=torch.int32), torch.zeros(2)
    t = torch.zeros((2, 4), dtype=torch.int32)
    cache = torch.zeros((1, 4, 400), dtype=torch.uint8)
    with pytest.raises(TypeError):
        mla.mla_cache_append(cache, torch.zeros((2, 576), dtype=torch.bfloat16), i.long(), i, torch.zeros(5, 64))
    with pytest.raises(TypeError):
        mla.mla_gather_latent_fp4(cache, t, i, i, 3)
    with pytest.raises(TypeError):
        mla.mla_tree_attention_fp4(torch.zeros(1, 1, 576), cache, t, i, i, sm_scale=1.0)
    with pytest.raises(TypeError):
        mla.mla_tree_verify(torch.zeros(2, 9), i, i, f, f, 3)


def test_the_pipeline_wants_one_format():
    from chunked_prefill_attention_ragged_gb300.pipeline import ChunkedPrefill
    with pytest.raises(ValueError, match="one format"):
        ChunkedPrefill(np.array([0]), np.zeros((1, 1)), np.zeros((1, 0)), 1, sm_scale=1.0, cache_fp8=True, cache_fp4=True)
