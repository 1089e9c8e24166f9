"""Forking sequences and compacting the pool of a paged cache: every page and entry against a plain form on the CPU."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def q_():
    import nvfp4_weight_quantized_03_gb300 as mod
    mod.lib()
    return mod


class Pool:
    """Pages of random bytes (every NaN pattern among them) and a table of shuffled page numbers."""

    def __init__(self, q_, num_pages, hk, page, dim, dtype, table, seed=0, pad=0):
        g = torch.Generator().manual_seed(seed)
        size = (num_pages, hk, page, dim * (1 if dtype == F8 else 2))
        self.k, self.v = (torch.randint(0, 256, size, generator=g, dtype=torch.uint8) for _ in range(2))
        self.table = table.to(torch.int32)
        self.dev = [x.cuda() for x in (self.k, self.v)]
        wide = torch.full((table.shape[0], table.shape[1] + pad), 77, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = self.table.cuda()
        self.wide, self.dev_table = wide, wide[:, :table.shape[1]]
        self.page = page
        self.cache = q_.kv_cache(*[x.view(dtype) for x in self.dev], self.dev_table)

    def same(self):
        for mine, dev in zip((self.k, self.v), self.dev):
            assert torch.equal(mine, dev.cpu())
        assert torch.equal(self.table, self.dev_table.cpu())
        assert (self.wide[:, self.table.shape[1]:] == 77).all()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _status(q_, ws):
    return q_.STATUS_NAMES[q_.qerl_read_status(ws)]


def _fork_plain(pool, parents, children, lengths, new):
    page = pool.page
    for a, b, n, fresh in zip(parents, children, lengths, new):
        full, rest = divmod(n, page)
        pool.table[b, :full] = pool.table[a, :full]
        if rest:
            old = int(pool.table[a, full])
            pool.table[b, full] = fresh
            for x in (pool.k, pool.v):
                x[fresh, :, :rest] = x[old, :, :rest]


@pytest.mark.parametrize("hk,page,dim,dtype", [(8, 64, 128, BF), (2, 16, 128, F8), (1, 1, 64, F8), (3, 100, 64, BF),
                                               (4, 24, 128, BF), (1, 700, 128, BF), (2, 8, 64, F8)])
def test_fork(q_, hk, page, dim, dtype):
    r = random.Random(page)
    lens = [1, page, page + 1, 3 * page - 1, 2 * page, 3 * page + (page + 1) // 2, 0]
    used = [-(-m // page) for m in lens]
    kids = [(a, n) for a, m in enumerate(lens) for n in {m, m // 2, max(0, m - 1), 0}]
    num = sum(used) + len(kids) + 3
    order = r.sample(range(num), num)
    table = torch.full((len(lens) + len(kids) + 1, max(used) + 2), -7, dtype=torch.int32)
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = torch.tensor(order[at:at + n])
        at += n
    pool = Pool(q_, num, hk, page, dim, dtype, table, pad=3)
    parents, lengths = [a for a, _ in kids], [n for _, n in kids]
    children = r.sample(range(len(lens), len(lens) + len(kids) + 1), len(kids))
    new = order[at:at + len(kids)]
    ws = q_.workspace(q_.qerl_kv_fork_workspace_size())
    q_.check(q_.qerl_kv_fork(pool.cache, _i32(parents), _i32(children), _i32(lengths), _i32(new), ws))
    assert _status(q_, ws) == "QERL_OK"
    _fork_plain(pool, parents, children, lengths, new)
    pool.same()


def test_fork_many_children_and_a_captured_call(q_):
    """Groups of children; a captured call takes the lengths that stand there when it is replayed."""
    page, groups, per = 16, 40, 16
    r = random.Random(1)
    lens = [r.randint(1, 900) for _ in range(groups)]
    used = [-(-m // page) for m in lens]
    num = sum(used) + groups * per
    order = r.sample(range(num), num)
    table = torch.zeros((groups * (per + 1), max(used)), dtype=torch.int32)
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = torch.tensor(order[at:at + n])
        at += n
    pool = Pool(q_, num, 4, page, 128, BF, table)
    parents = [i // per for i in range(groups * per)]
    children = list(range(groups, groups * (per + 1)))
    lengths = _i32([lens[a] for a in parents])
    args = _i32(parents), _i32(children), lengths, _i32(order[at:])
    ws = q_.workspace(q_.qerl_kv_fork_workspace_size())
    q_.check(q_.qerl_kv_fork(pool.cache, *args, ws))
    _fork_plain(pool, parents, children, lengths.tolist(), order[at:])
    pool.same()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        q_.check(q_.qerl_kv_fork(pool.cache, *args, ws))
    shorter = [max(0, n - r.randint(0, 40)) for n in lengths.tolist()]
    lengths.copy_(_i32(shorter))
    graph.replay()
    torch.cuda.synchronize()
    _fork_plain(pool, parents, children, shorter, order[at:])
    pool.same()
    assert _status(q_, ws) == "QERL_OK"


@pytest.mark.parametrize("item", [(9, 3, 20, 6), (-1, 3, 20, 6), (0, 9, 20, 6), (0, -1, 20, 6), (0, 3, 81, 6),
                                  (0, 3, -1, 6), (0, 3, 20, 40), (0, 3, 20, -1), (1, 3, 20, 6), (2, 3, 20, 6),
                                  (0, 0, 20, 6), (0, 3, 2 ** 31 - 1, 6)])
def test_fork_leaves_a_bad_item_alone(q_, item):
    """Sequence, length or page outside the cache (sequences 1 and 2 have a last page outside), its own parent: the
    item beside it is done."""
    table = torch.tensor([[4, 5, 0, 0, 0], [1, 40, 0, 0, 0], [1, -3, 0, 0, 0], [0] * 5, [0] * 5], dtype=torch.int32)
    pool = Pool(q_, 8, 2, 16, 64, BF, table)
    good = (0, 4, 21, 7)
    args = [_i32([a, b]) for a, b in zip(item, good)]
    ws = q_.workspace(q_.qerl_kv_fork_workspace_size())
    q_.check(q_.qerl_kv_fork(pool.cache, *args, ws))
    assert _status(q_, ws) == "QERL_ERR_RANGE"
    _fork_plain(pool, *[[x] for x in good])
    pool.same()


def test_fork_shares_entries_it_does_not_copy(q_):
    """Full pages are entries alone: one given up (negative) is passed on."""
    table = torch.tensor([[-1, -1, 3, 2], [0, 0, 0, 0]], dtype=torch.int32)
    pool = Pool(q_, 6, 1, 8, 64, BF, table)
    ws = q_.workspace(q_.qerl_kv_fork_workspace_size())
    q_.check(q_.qerl_kv_fork(pool.cache, _i32([0]), _i32([1]), _i32([29]), _i32([5]), ws))
    assert _status(q_, ws) == "QERL_OK"
    _fork_plain(pool, [0], [1], [29], [5])
    pool.same()


# ---- compaction ---------------------------------------------------------------


def _compact_plain(pool, lengths):
    """The live count; moves pool's pages and returns the new table."""
    num, (n, most) = pool.k.shape[0], pool.table.shape
    held = [min(max(m, 0), most * pool.page) for m in lengths]
    held = [-(-m // pool.page) for m in held]
    used = sorted({int(x) for i in range(n) for x in pool.table[i, :held[i]] if 0 <= x < num})
    live = len(used)
    gone = [x for x in used if x >= live]
    room = [x for x in range(live) if x not in set(used)]
    number = {x: x for x in used} | dict(zip(gone, room))
    for a, b in zip(gone, room):
        for x in (pool.k, pool.v):
            x[b] = x[a]
    new = pool.table.clone()
    for i in range(n):
        for j in range(held[i]):
            new[i, j] = number.get(int(new[i, j]), int(new[i, j]))
    return live, new


def _compact(q_, pool, lengths, in_place=False, ws=None, stream=None):
    n, most = pool.table.shape
    wide = torch.full((n, most + 2), 55, dtype=torch.int32, device="cuda")
    new = pool.dev_table if in_place else wide[:, :most]
    live = _i32([-9])
    ws = q_.workspace(q_.qerl_kv_compact_workspace_size(pool.k.shape[0])) if ws is None else ws
    torch.cuda.synchronize()
    q_.check(q_.qerl_kv_compact(pool.cache, _i32(lengths), new, live, ws, stream=stream))
    torch.cuda.synchronize()
    count, want = _compact_plain(pool, lengths)
    if in_place:
        pool.table = want
    assert live.item() == count
    assert torch.equal(new.cpu(), want)
    assert (wide[:, most:] == 55).all()
    pool.same()
    return count, _status(q_, ws)


def _random_pool(q_, r, num, n, most, hk, page, dim, dtype, dense=0.5):
    """n sequences of random lengths over a share of the pool's pages, some shared, some given up."""
    pages = r.sample(range(num), max(1, int(num * dense))) if num else []
    table = torch.full((n, most), 2 ** 30, dtype=torch.int32)
    lengths = []
    for i in range(n):
        m = r.choice([0, 1, r.randint(0, most * page), most * page])
        lengths.append(m if pages else 0)
        for j in range(-(-lengths[-1] // page)):
            table[i, j] = r.choice(pages) if r.random() < 0.9 else -r.randint(1, 5)
    return Pool(q_, num, hk, page, dim, dtype, table, seed=num, pad=1), lengths


@pytest.mark.parametrize("num", [0, 1, 2, 15, 16, 17, 33, 500, 1023, 1025, 20011])
@pytest.mark.parametrize("dense", [0.05, 0.5, 1.0])
def test_compact(q_, num, dense):
    r = random.Random(num)
    pool, lengths = _random_pool(q_, r, num, r.choice([1, 5, 40]), r.choice([1, 7, 60]), 1, 2, 64, F8, dense)
    _, status = _compact(q_, pool, lengths)
    assert status == "QERL_OK"


@pytest.mark.parametrize("hk,page,dim,dtype", [(8, 64, 128, BF), (2, 16, 128, F8), (1, 1, 64, F8), (3, 100, 64, BF),
                                               (1, 700, 128, BF)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_pages_of_every_size(q_, hk, page, dim, dtype, in_place):
    r = random.Random(page)
    pool, lengths = _random_pool(q_, r, 90, 6, 9, hk, page, dim, dtype)
    _, status = _compact(q_, pool, lengths, in_place)
    assert status == "QERL_OK"
    if in_place:  # nothing is left to move
        before = pool.table.clone()
        _compact(q_, pool, lengths, in_place)
        assert torch.equal(before, pool.table)


@pytest.mark.parametrize("n,most", [(64, 64), (65, 64), (4097, 1), (1, 5000), (300, 40)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_tables_of_every_size(q_, n, most, in_place):
    """Around the size from which the marks have a launch of their own, and past it."""
    r = random.Random(n)
    pool, lengths = _random_pool(q_, r, 3001, n, most, 1, 2, 64, BF)
    _, status = _compact(q_, pool, lengths, in_place)
    assert status == "QERL_OK"


def test_compact_long_rows(q_):
    """More entries in a row than a block takes at a time, and more rows."""
    r = random.Random(8)
    pool, lengths = _random_pool(q_, r, 6000, 30, 2500, 1, 1, 64, F8)
    _, status = _compact(q_, pool, lengths)
    assert status == "QERL_OK"


def test_compact_one_workspace_for_pools_of_any_size_and_another_stream(q_):
    r = random.Random(5)
    ws = q_.workspace(q_.qerl_kv_compact_workspace_size(5000))
    ws[256:] = 0xAB  # only the header is zero-filled
    for num in (300, 5000, 17, 4000, 300):
        pool, lengths = _random_pool(q_, r, num, 9, 30, 1, 4, 64, BF)
        _compact(q_, pool, lengths, ws=ws, stream=torch.cuda.Stream() if num == 17 else None)


def test_compact_records_what_lies_outside(q_):
    table = torch.tensor([[9, 100, 3, 2], [8, 7, 6, 5], [1, 0, 0, 0]], dtype=torch.int32)
    for lengths in ([16, 0, 0], [0, 17, 0], [0, 0, -1]):
        pool = Pool(q_, 12, 1, 4, 64, BF, table.clone())
        _, status = _compact(q_, pool, lengths)
        assert status == "QERL_ERR_RANGE"
    pool = Pool(q_, 12, 1, 4, 64, BF, table.clone())
    live, status = _compact(q_, pool, [4, 16, 0])  # entry 100 lies past the length
    assert status == "QERL_OK" and live == 5


def test_compact_without_sequences(q_):
    pool = Pool(q_, 12, 1, 4, 64, BF, torch.zeros((0, 3), dtype=torch.int32))
    assert _compact(q_, pool, []) == (0, "QERL_OK")


def test_compact_captured(q_):
    r = random.Random(3)
    pool, lengths = _random_pool(q_, r, 200, 8, 20, 2, 8, 64, BF)
    dev_lengths = _i32(lengths)
    new, live = torch.empty_like(pool.dev_table).contiguous(), _i32([0])
    ws = q_.workspace(q_.qerl_kv_compact_workspace_size(200))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        q_.check(q_.qerl_kv_compact(pool.cache, dev_lengths, new, live, ws))
    for _ in range(3):
        lengths = [m // 2 for m in lengths]
        dev_lengths.copy_(_i32(lengths))
        graph.replay()
        torch.cuda.synchronize()
        count, want = _compact_plain(pool, lengths)
        assert live.item() == count and torch.equal(new.cpu(), want)
        pool.table = want  # the next replay starts from the new table
        pool.dev_table.copy_(new)
        pool.same()


def test_pages_past_32_bits(q_):
    """Byte and element offsets past 2^32: a copy to a far page, and the far pages moved to the front."""
    num, hk, page, dim = 2 ** 20 + 9, 2, 16, 128
    pages = [torch.zeros((num, hk, page, dim), dtype=BF, device="cuda") for _ in range(2)]
    a, b = num - 1, num - 3
    for x in pages:
        x[a] = torch.randn((hk, page, dim), device="cuda").to(BF)
    want = [x[a].clone() for x in pages]
    table = _i32([[a], [0]])
    cache = q_.kv_cache(*pages, table)
    ws = q_.workspace(q_.qerl_kv_fork_workspace_size())
    q_.kv_fork(cache, _i32([0]), _i32([1]), _i32([11]), _i32([b]), ws)
    assert _status(q_, ws) == "QERL_OK" and table.tolist() == [[a], [b]]
    for x, w in zip(pages, want):
        assert torch.equal(x[b, :, :11], w[:, :11]) and (x[b, :, 11:] == 0).all()
    ws = q_.workspace(q_.qerl_kv_compact_workspace_size(num))
    new, live = q_.kv_compact(cache, _i32([16, 11]), ws)
    assert _status(q_, ws) == "QERL_OK" and new.tolist() == [[1], [0]] and live.item() == 2
    for x, w in zip(pages, want):
        assert torch.equal(x[1], w) and torch.equal(x[0, :, :11], w[:, :11])


def test_two_forks_and_compactions_at_once(q_):
    """On two streams, each with pools and workspaces of its own."""
    r = random.Random(7)
    streams = [torch.cuda.Stream() for _ in range(2)]
    pools = [_random_pool(q_, r, 4000, 50, 200, 2, 8, 128, BF) for _ in streams]
    made = [(_i32(lengths), torch.empty_like(pool.dev_table).contiguous(), _i32([0]),
             q_.workspace(q_.qerl_kv_compact_workspace_size(4000))) for pool, lengths in pools]
    torch.cuda.synchronize()
    for _ in range(3):
        for (pool, _), (lengths, new, live, ws), s in zip(pools, made, streams):
            q_.check(q_.qerl_kv_compact(pool.cache, lengths, new, live, ws, stream=s))
    torch.cuda.synchronize()
    for (pool, lengths), (_, new, live, ws) in zip(pools, made):
        count, want = _compact_plain(pool, lengths)
        assert live.item() == count and torch.equal(new.cpu(), want) and _status(q_, ws) == "QERL_OK"
        pool.same()
