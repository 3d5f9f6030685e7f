"""mla_tree_verify refuses outputs that share memory with its inputs or one another.  Without a GPU: what is not refused
ends at the launch, which fails here."""
import pytest

import chunked_prefill_attention_ragged_gb300 as mla

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that nothing may follow")
FAR, INVALID = 1 << 32, -1
SIZES = {"target": 5 * 1000 * 4, "draft": 5 * 1000 * 4, "tokens": 20, "parents": 20, "qo": 12, "u": 20, "u_last": 8, "accepted": 32,
         "counts": 8, "next": 8, "status": 4}
NAMES = list(SIZES)


def verify(kind=0, vocab=1000, batch=2, rows=5, most=4, **at):
    a = {name: (k + 1) * FAR for k, name in enumerate(NAMES)}
    a.update(at)
    return mla.library().mla_tree_verify(a["target"], a["draft"], kind, vocab, a["tokens"], a["parents"], a["qo"], batch, rows, a["u"],
                                         a["u_last"], a["accepted"], most, a["counts"], a["next"], a["status"], None)


def test_apart_is_not_refused():
    assert verify() not in (0, INVALID) and verify(draft=None, parents=None, status=None) not in (0, INVALID)
    # the inputs may be one another's: a draft that is the target
    assert verify(draft=FAR) != INVALID and verify(u_last=NAMES.index("u") * FAR + FAR) != INVALID


@pytest.mark.parametrize("written,other", [(w, o) for w in ("accepted", "counts", "next", "status") for o in NAMES if o != w])
def test_each_output_against_each_array(written, other):
    at = 20 * FAR
    for first, second in ((written, other), (other, written)):
        assert verify(**{first: at, second: at + SIZES[first]}) != INVALID
        assert verify(**{first: at, second: at + SIZES[first] - 4}) == INVALID


def test_rows_of_two_bytes():
    at = 20 * FAR
    assert verify(kind=1, target=at, counts=at + 10000) != INVALID and verify(kind=1, target=at, counts=at + 9996) == INVALID


def test_no_rows():
    assert verify(rows=0, target=None, tokens=None, u=None) not in (0, INVALID)
    assert verify(rows=0, target=None, tokens=None, u=None, counts=5 * FAR) == INVALID     # the indptr's
