"""What the page calls refuse, on the host and before any work is enqueued."""
import pytest
import torch

import nvfp4_weight_quantized_03_gb300 as q

INVALID, SHAPE, ALIGN, WS = ("QERL_ERR_INVALID_ARGUMENT", "QERL_ERR_UNSUPPORTED_SHAPE", "QERL_ERR_MISALIGNED",
                             "QERL_ERR_WORKSPACE")

# Pointers that are no memory: only calls that are refused (or have nothing to do) may be made with them.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer calls run only without a GPU")


@pytest.fixture(scope="module")
def L():
    from nvfp4_weight_quantized_03_gb300 import build
    build.build()
    return q.lib()


def _cache(**kw):
    a = dict(k=0x10000, v=0x20000, dtype=q.QERL_BF16, num_kv_heads=4, head_dim=128, page_size=16, num_pages=10,
             k_scale=None, v_scale=None, page_table=0x30000, num_seqs=3, max_pages=5, ld_table=5)
    a.update(kw)
    c = q.KvCache()
    for name, value in a.items():
        setattr(c, name, value)
    return c


def _fork(L, cache, **kw):
    a = dict(parents=0x1000, children=0x2000, lengths=0x3000, new=0x4000, count=2, ws=0x8000, wsb=256)
    a.update(kw)
    return q.STATUS_NAMES[L.qerl_kv_fork(cache, a["parents"], a["children"], a["lengths"], a["new"], a["count"], a["ws"],
                                         a["wsb"], None)]


def _compact(L, cache, **kw):
    a = dict(lengths=0x1000, table=0x2000, ld=5, live=0x4000, ws=0x8000, wsb=1 << 20)
    a.update(kw)
    return q.STATUS_NAMES[L.qerl_kv_compact(cache, a["lengths"], a["table"], a["ld"], a["live"], a["ws"], a["wsb"],
                                            None)]


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=q.QERL_F32), INVALID), (dict(page_size=0), INVALID), (dict(num_pages=-1), INVALID),
    (dict(ld_table=4), INVALID), (dict(num_pages=2 ** 31), SHAPE), (dict(head_dim=96), SHAPE),
    (dict(num_kv_heads=0), INVALID), (dict(k=None), INVALID), (dict(page_table=None), INVALID), (dict(k=0x10008), ALIGN)])
def test_bad_caches(L, kw, want):
    assert _fork(L, _cache(**kw)) == want
    assert _compact(L, _cache(**kw)) == want


def test_fork(L):
    assert _fork(L, None) == INVALID and _fork(L, _cache(), count=-1) == INVALID
    for name in ("parents", "children", "lengths", "new"):
        assert _fork(L, _cache(), **{name: None}) == INVALID
        assert _fork(L, _cache(), **{name: 0x1002}) == ALIGN
    assert _fork(L, _cache(), count=2 ** 31) == SHAPE
    assert _fork(L, _cache(), wsb=255) == WS and _fork(L, _cache(), ws=None) == WS
    assert _fork(L, _cache(), ws=0x8010) == ALIGN
    assert _fork(L, _cache(), count=0, parents=None, ws=None) == "QERL_OK"


def test_compact(L):
    assert _compact(L, None) == INVALID and _compact(L, _cache(), live=None) == INVALID
    assert _compact(L, _cache(), lengths=None) == INVALID and _compact(L, _cache(), table=None) == INVALID
    assert _compact(L, _cache(), ld=4) == INVALID
    assert _compact(L, _cache(), table=0x30000, ld=6) == INVALID  # in place with another stride
    for name in ("lengths", "table", "live"):
        assert _compact(L, _cache(), **{name: 0x1002}) == ALIGN
    assert _compact(L, _cache(), wsb=q.qerl_kv_compact_workspace_size(10) - 1) == WS
    assert _compact(L, _cache(), ws=0x8010) == ALIGN


def test_workspace_sizes(L):
    assert q.qerl_kv_fork_workspace_size() == 256
    assert q.qerl_kv_compact_workspace_size(-1) == 0 and q.qerl_kv_compact_workspace_size(2 ** 31) == 0
    sizes = [q.qerl_kv_compact_workspace_size(n) for n in (0, 1, 1000, 10 ** 6, 2 ** 31 - 1)]
    assert sizes == sorted(sizes) and sizes[0] >= 256 and sizes[-1] >= 9 * (2 ** 31 - 1)
