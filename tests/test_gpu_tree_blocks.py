"""Tree attention with every kind of block over several tiles a worker: buffers filled again, rows looked up
a tile ahead, workers that cross units and requests, last tiles mended more than once a worker, parts joined."""
import numpy as np
import pytest

from test_gpu_speculative import Problem

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BLOCKS = [1, 4, 5, 8, 16, 24, 32, 48, 64, 96, 128]


@pytest.mark.parametrize("bs", BLOCKS)
def test_many_ragged_requests(bs):
    """40 requests over about 900 keys, 320 tiles and more: a worker has four tiles and meets one or two ends."""
    rng = np.random.default_rng(bs)
    kv = [int(x) for x in rng.integers(760, 1050, 40)]
    p = Problem(400 + bs, [3 + r % 3 for r in range(40)], kv, 16, bs, True, spread=4.0)
    o, lse, st = p.run(pad=1)
    assert st == 0
    p.check(o, lse, [0, 1, 13, 21, 38, 39], [0, 7, 15])


@pytest.mark.parametrize("bs", BLOCKS)
def test_many_short_requests(bs):
    """Several whole requests to a worker, each of one or two tiles that end anywhere."""
    rng = np.random.default_rng(bs + 50)
    kv = [int(x) for x in rng.integers(1, 200, 310)]
    p = Problem(430 + bs, [1] * 310, kv, 5, bs, False)
    o, lse, st = p.run()
    assert st == 0
    p.check(o, lse, list(range(0, 310, 9)) + [309])


@pytest.mark.parametrize("bs", BLOCKS)
def test_one_long_request(bs):
    """About 235 tiles, three a worker, every worker's part joined."""
    p = Problem(460 + bs, [2], [30011], 16, bs, True, spread=3.0)
    o, lse, st = p.run()
    assert st == 0
    p.check(o, lse, None, [0, 9])


@pytest.mark.parametrize("bs", [1, 8, 24, 32, 64])
def test_units_of_two_long_requests(bs):
    """More units than one a request, each cut by workers, so that a worker ends one unit and begins another."""
    p = Problem(490 + bs, [20, 11], [7003, 5120], 32, bs, True)
    o, lse, st = p.run()
    assert st == 0
    p.check(o, lse, None, [0, 31])
