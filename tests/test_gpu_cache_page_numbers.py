"""Fork and compaction: page numbers and lengths outside the cache are recorded wherever they stand."""
import pytest
import torch

from test_gpu_cache_pages import BF, F8, Pool, _compact, _fork_plain, _i32, _status, q_  # noqa: F401 (q_ is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 100])
@pytest.mark.parametrize("at", [0, 1, 299])
@pytest.mark.parametrize("number", [2000, 2 ** 31 - 1])
@pytest.mark.parametrize("rest", [0, 1, 15])
def test_fork_of_a_sequence_with_a_full_page_outside(q_, page, at, number, rest):
    """Nothing of that child is written, whether or not it has rows to copy; the child beside it is done."""
    table = torch.zeros((5, 310), dtype=torch.int32)
    table[0] = torch.arange(310) + 100
    table[1] = torch.arange(310) + 500
    table[0, at] = number
    table[0, 40] = -3  # a page given up is none outside
    pool = Pool(q_, 2000, 2, page, 64, BF, table)
    ws = q_.workspace(q_.qerl_kv_fork_workspace_size())
    good = [1, 4, 7 * page + 5, 7]
    args = [_i32([a, b]) for a, b in zip([0, 3, 300 * page + rest, 6], good)]
    q_.check(q_.qerl_kv_fork(pool.cache, *args, ws))
    assert _status(q_, ws) == "QERL_ERR_RANGE"
    _fork_plain(pool, *[[x] for x in good])
    pool.same()
    # a child of the rows in front of that page is done
    short = [[0], [3], [at * page], [6]]
    q_.check(q_.qerl_kv_fork(pool.cache, *map(_i32, short), ws))
    assert _status(q_, ws) == "QERL_OK"
    _fork_plain(pool, *short)
    pool.same()


@pytest.mark.parametrize("lengths", [[0, 5, 0], [-1, 0, 0], [0, 0, 2 ** 31 - 1]])
def test_compact_records_lengths_of_a_cache_without_entries(q_, lengths):
    for pages in (0, 7, 200000):
        pool = Pool(q_, pages, 1, 4, 64, F8, torch.zeros((3, 0), dtype=torch.int32))
        assert _compact(q_, pool, lengths) == (0, "QERL_ERR_RANGE")
        assert _compact(q_, pool, [0, 0, 0]) == (0, "QERL_OK")


@pytest.mark.parametrize("n,most", [(3, 5), (300, 40)])
def test_compact_records_entries_and_lengths_of_a_cache_without_pages(q_, n, most):
    table = torch.full((n, most), -2, dtype=torch.int32)
    pool = Pool(q_, 0, 1, 4, 64, F8, table.clone())
    assert _compact(q_, pool, [4] * n) == (0, "QERL_OK")  # pages given up
    assert _compact(q_, pool, [4] * (n - 1) + [4 * most + 1]) == (0, "QERL_ERR_RANGE")
    table[n - 1, 0] = 0
    pool = Pool(q_, 0, 1, 4, 64, F8, table)
    assert _compact(q_, pool, [4] * n) == (0, "QERL_ERR_RANGE")
    assert _compact(q_, pool, [4] * (n - 1) + [0]) == (0, "QERL_OK")
