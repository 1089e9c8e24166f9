"""What the tree attention call refuses, on the host and before any work is enqueued."""
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


def _call(L, cache=None, **kw):
    c = q.KvCache()
    fields = dict(k=0x10000, v=0x20000, dtype=q.QERL_BF16, num_kv_heads=4, head_dim=128, page_size=16, num_pages=10,
                  page_table=0x30000, num_seqs=3, max_pages=5, ld_table=5)
    fields.update(cache or {})
    for name, value in fields.items():
        setattr(c, name, value)
    a = dict(q=0x1000, ldq=3584, k=0x2000, ldk=512, v=0x3000, ldv=512, tokens=12, heads=28, cu=0x4000, lens=0x5000,
             mask=0x6000, words=1, scale=0.1, out=0x7000, ldo=3584, lse=0x8000, ws=0x10000, wsb=1 << 30, none=False)
    a.update(kw)
    return q.STATUS_NAMES[L.qerl_tree_attention(None if a["none"] else c, a["q"], a["ldq"], a["k"], a["ldk"], a["v"],
                                                a["ldv"], a["tokens"], a["heads"], a["cu"], a["lens"], a["mask"],
                                                a["words"], a["scale"], a["out"], a["ldo"], a["lse"], a["ws"], a["wsb"],
                                                None)]


@pytest.mark.parametrize("kw,want", [
    (dict(none=True), INVALID), (dict(tokens=-1), INVALID), (dict(heads=0), INVALID), (dict(heads=27), INVALID),
    (dict(heads=1028), SHAPE), (dict(scale=float("inf")), INVALID), (dict(words=0), INVALID), (dict(words=-1), INVALID),
    (dict(words=2 ** 14 + 1), SHAPE), (dict(tokens=2 ** 30 + 1), SHAPE), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(out=None), INVALID), (dict(cu=None), INVALID), (dict(lens=None), INVALID),
    (dict(ldq=3583), INVALID), (dict(ldk=511), INVALID), (dict(ldv=0), INVALID), (dict(ldo=8), INVALID),
    (dict(ldq=3588), ALIGN), (dict(ldo=3590), ALIGN), (dict(q=0x1008), ALIGN), (dict(out=0x7002), ALIGN),
    (dict(cu=0x4002), ALIGN), (dict(lens=0x5001), ALIGN), (dict(mask=0x6004), ALIGN), (dict(lse=0x8002), ALIGN),
    (dict(ws=None), WS), (dict(wsb=1000), WS), (dict(ws=0x10010), ALIGN)])
def test_arguments(L, kw, want):
    assert _call(L, **kw) == want


@pytest.mark.parametrize("cache,want", [
    (dict(dtype=q.QERL_F32), INVALID), (dict(head_dim=96), SHAPE), (dict(page_size=0), INVALID),
    (dict(k_scale=0x100), INVALID), (dict(num_pages=2 ** 31), SHAPE), (dict(ld_table=4), INVALID),
    (dict(page_table=None), INVALID), (dict(v=0x20004), ALIGN)])
def test_caches(L, cache, want):
    assert _call(L, cache) == want


def test_nothing_to_do(L):
    assert _call(L, tokens=0, ws=None) == "QERL_OK"
    assert _call(L, dict(num_seqs=0), ws=None) == "QERL_OK"


def test_workspace_size(L):
    size = q.qerl_tree_attention_workspace_size
    assert size(-1, 28, 4, 128, 1) == 0 and size(5, 28, 5, 128, 1) == 0 and size(5, 28, 4, 96, 1) == 0
    assert size(5, 28, 4, 128, -1) == 0
    sizes = [size(t, 28, 4, 128, 1) for t in (1, 5, 36, 37, 10 ** 6)]
    assert sizes == sorted(sizes) and sizes[-1] == sizes[-2]  # a partial has 256 rows at most
    needed = size(12, 28, 4, 128, 3)
    assert _call(L, wsb=needed - 1) == WS
