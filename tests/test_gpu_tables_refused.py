"""Block tables whose rows hold anything behind the entries in use: requests that are not served get no
slot in a block that they do not hold, and name none for the calls that read the table next."""
import numpy as np
import pytest

from oracle import update_block_table
from test_gpu_speculative import BAD_INDEX, NO_BLOCKS, i32, new_status, random_tables, run_tables

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("num_tokens", [12, 9000])   # slots by the one CTA, and from a grid
def test_requests_that_are_not_served_get_no_slots(num_tokens):
    # request 0 holds a block and needs three, in a row of two; request 1 is served from the stack; request
    # 2 finds the stack empty.  Block 0, which request 1 gets, is what unused entries say.
    got = run_tables([2, 0, 0], [8, 4, 3], [[5, 0], [0, 0], [0, 0]], [1, 0, 0], [0], 4, 6, num_tokens)
    assert got[6] == BAD_INDEX | NO_BLOCKS
    assert got[4].tolist() == [1, 1, 0]
    assert got[2][:12].tolist() == [22, 23] + [-1] * 6 + [0, 1, 2, 3]
    assert (got[2][12:] == -1).all()
    # what a request would have needed and does not hold is named no more; other entries stay as they were
    assert got[3].tolist() == [[5, -1], [0, 0], [-1, 0]]


@pytest.mark.parametrize("batch,most,bs", [(1, 40, 4), (3, 40, 16), (33, 100, 7), (300, 30, 4), (1025, 12, 4), (8192, 3, 2)])
@pytest.mark.parametrize("grid", [False, True])
def test_anything_behind_the_entries_in_use(batch, most, bs, grid):
    rng = np.random.default_rng(batch + most)
    width = -(-3 * most // (2 * bs))        # some requests need more
    seq, new, table, held, stack, total = random_tables(rng, batch, most, bs, -(-2 * most // bs) + 1)
    held = np.minimum(held, width)
    table = table[:, :width]
    table = np.where(np.arange(width)[None] < held[:, None], table, rng.integers(0, total, table.shape))
    stack = stack[:len(stack) * 2 // 3]
    n = max(int(new.sum()), 8193 if grid else 0) if grid else min(int(new.sum()), 8192)
    want = update_block_table(seq, new, table, held, stack, bs, total, n)
    got = run_tables(seq, new, table, held, stack, bs, total, n)
    for k, name in enumerate(["qo_indptr", "kv_lens", "slot_mapping", "block_table", "num_held"]):
        np.testing.assert_array_equal(got[k], want[k], err_msg=name)
    assert got[5] == want[5]
    unfit = bool((-(-(seq + new) // bs) > width).any())
    assert got[6] == (NO_BLOCKS if want[6] else 0) | (BAD_INDEX if unfit or int(new.sum()) > n else 0)


@pytest.mark.parametrize("num_tokens", [0, 9000])
def test_a_row_that_gives_back_no_block_is_reported(num_tokens):
    """An entry in use without a block (its id was negative on the stack, or the caller's own) is reported by
    the call that gives it back, also when it goes to another row at once."""
    got = run_tables([0, 0], [0, 0], [[3, -1], [4, 5]], [2, 2], [], 4, 4, num_tokens)
    assert got[6] == BAD_INDEX and got[4].tolist() == [0, 0]
    assert got[5] == [5, 4, -1, 3] and (got[3] == -1).all()
    got = run_tables([0, 0], [0, 4], [[-1], [-1]], [1, 0], [9], 4, 4, num_tokens)
    assert got[6] & BAD_INDEX and got[3].tolist() == [[-1], [-1]] and got[5] == [9]


@pytest.mark.parametrize("num_tokens", [5, 9000])
def test_lengths_past_32_bits(num_tokens):
    """Blocks of 2^20 tokens: the row has room for a length that kv_lens cannot say."""
    got = run_tables([2 ** 31 - 4], [5], [[7] * 2049], [2048], [8], 1 << 20, 4, num_tokens)
    assert got[6] == BAD_INDEX and got[1].tolist() == [2 ** 31 - 1]
    assert got[4].tolist() == [2049] and got[3][0, 2048] == 8
    assert got[2][:5].tolist() == [8 * 2 ** 20 + k for k in (-4, -3, -2, -1, 0)]   # the end of 7, the first of 8
    got = run_tables([2 ** 31 - 4], [3], [[7] * 2049], [2048], [8], 1 << 20, 4, num_tokens)
    assert got[6] == 0 and got[1].tolist() == [2 ** 31 - 1]
