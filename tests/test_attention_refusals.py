"""What the attention calls refuse, on the host and before any work is enqueued."""
import ctypes

import pytest
import torch

import nvfp4_weight_quantized_03_gb300 as q

# The calls here pass pointers that are no memory: one that unexpectedly passed its checks would
# launch on them, so they run only where no GPU is visible.
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


def _append(L, cache=None, **kw):
    a = dict(q=0x1000, ldq=3584, heads=28, k=0x2000, ldk=512, v=0x3000, ldv=512, hk=4, dim=128, tokens=3, seq=None,
             pos=0x4000, freq=0x5000, rot=128, q_out=0x6000, ldqo=3584, k_out=0x7000, ldko=512, ws=0x8000, wsb=256)
    a.update(kw)
    st = L.qerl_rope_append(cache, a["q"], a["ldq"], a["heads"], a["k"], a["ldk"], a["v"], a["ldv"], a["hk"], a["dim"],
                            a["tokens"], a["seq"], a["pos"], a["freq"], a["rot"], a["q_out"], a["ldqo"], a["k_out"],
                            a["ldko"], a["ws"], a["wsb"], None)
    return q.STATUS_NAMES[st]


def _decode(L, cache, **kw):
    a = dict(q=0x1000, ldq=3584, heads=28, lens=0x2000, scale=0.1, out=0x3000, ldo=3584, lse=0x4000, ws=0x10000,
             wsb=1 << 30)
    a.update(kw)
    return q.STATUS_NAMES[L.qerl_decode_attention(cache, a["q"], a["ldq"], a["heads"], a["lens"], a["scale"], a["out"],
                                                  a["ldo"], a["lse"], a["ws"], a["wsb"], None)]


INVALID, SHAPE, ALIGN, WS = ("QERL_ERR_INVALID_ARGUMENT", "QERL_ERR_UNSUPPORTED_SHAPE", "QERL_ERR_MISALIGNED",
                             "QERL_ERR_WORKSPACE")

BAD_CACHES = [
    (dict(dtype=q.QERL_F32), INVALID), (dict(dtype=7), INVALID), (dict(k_scale=0x100), INVALID),
    (dict(v_scale=0x100), INVALID), (dict(page_size=0), INVALID), (dict(num_pages=-1), INVALID),
    (dict(num_seqs=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(ld_table=4), INVALID),
    (dict(page_size=65537), SHAPE), (dict(num_pages=2 ** 31), SHAPE), (dict(num_seqs=2 ** 20 + 1), SHAPE),
    (dict(max_pages=2 ** 27, ld_table=2 ** 27), SHAPE), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(page_table=None), INVALID), (dict(k=0x10008), ALIGN), (dict(v=0x20004), ALIGN),
    (dict(page_table=0x30002), ALIGN), (dict(dtype=q.QERL_E4M3, k_scale=0x102), ALIGN),
]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_cache_descriptors(L, kw, want):
    assert _append(L, _cache(**kw)) == want
    assert _decode(L, _cache(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), INVALID), (dict(rot=-16), INVALID), (dict(rot=144), INVALID), (dict(rot=24), SHAPE),
    (dict(dim=96, ldq=2688, ldk=384), SHAPE), (dict(heads=30), INVALID), (dict(heads=0), INVALID), (dict(hk=0), INVALID),
    (dict(k=None), INVALID), (dict(pos=None), INVALID), (dict(freq=None), INVALID), (dict(v=None), INVALID),
    (dict(q_out=None), INVALID), (dict(q=None, heads=0), INVALID), (dict(ldq=3576), INVALID), (dict(ldk=504), INVALID),
    (dict(ldv=504), INVALID), (dict(ldqo=3576), INVALID), (dict(ldko=504), INVALID), (dict(ldq=3588), ALIGN),
    (dict(q=0x1008), ALIGN), (dict(k=0x2002), ALIGN), (dict(v=0x3004), ALIGN), (dict(k_out=0x7008), ALIGN),
    (dict(pos=0x4002), ALIGN), (dict(seq=0x4001), ALIGN), (dict(freq=0x5004), ALIGN),
    (dict(q_out=0x1000, ldqo=4096), INVALID), (dict(k_out=0x2000, ldko=1024), INVALID), (dict(ws=None), WS),
    (dict(wsb=255), WS), (dict(ws=0x8080), ALIGN), (dict(hk=8, ldk=1024, ldv=1024, ldko=1024, heads=32, ldq=4096,
                                                         ldqo=4096), INVALID),
])
def test_append_arguments(L, kw, want):
    assert _append(L, _cache(), **kw) == want


def test_append_without_a_cache(L):
    assert _append(L, None, k_out=None) == INVALID
    assert _append(L, None, tokens=0) == "QERL_OK"
    assert _append(L, _cache(), tokens=0) == "QERL_OK"


@pytest.mark.parametrize("kw,want", [
    (dict(heads=27), INVALID), (dict(heads=0), INVALID), (dict(heads=-4), INVALID), (dict(q=None), INVALID),
    (dict(lens=None), INVALID), (dict(out=None), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(ldq=3576), INVALID), (dict(ldo=3576), INVALID), (dict(ldq=3585), ALIGN),
    (dict(ldo=3588), ALIGN), (dict(q=0x1004), ALIGN), (dict(out=0x3008), ALIGN), (dict(lens=0x2002), ALIGN),
    (dict(lse=0x4001), ALIGN), (dict(ws=None), WS), (dict(wsb=4096), WS), (dict(ws=0x10080), ALIGN),
    (dict(heads=1028, ldq=1028 * 128, ldo=1028 * 128), SHAPE),
])
def test_decode_arguments(L, kw, want):
    assert _decode(L, _cache(), **kw) == want


def test_decode_shapes(L):
    assert _decode(L, None) == INVALID
    assert _decode(L, _cache(head_dim=80)) == SHAPE
    assert _decode(L, _cache(num_kv_heads=0)) == INVALID
    assert _decode(L, _cache(num_seqs=0)) == "QERL_OK"
    need = L.qerl_decode_attention_workspace_size(3, 28, 4, 128)
    assert need > 0
    assert _decode(L, _cache(), wsb=need - 1) == WS
    assert L.qerl_decode_attention_workspace_size(-1, 28, 4, 128) == 0
    assert L.qerl_decode_attention_workspace_size(3, 28, 3, 128) == 0
    assert L.qerl_decode_attention_workspace_size(3, 28, 4, 100) == 0


def _prompt(L, **kw):
    a = dict(q=0x1000, ldq=3584, k=0x2000, ldk=512, v=0x3000, ldv=512, tokens=300, heads=28, hk=4, dim=128, cu=0x4000,
             n=2, scale=0.1, out=0x5000, ldo=3584, lse=0x6000, ws=0x8000, wsb=256)
    a.update(kw)
    return q.STATUS_NAMES[L.qerl_prompt_attention(a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["tokens"],
                                                  a["heads"], a["hk"], a["dim"], a["cu"], a["n"], a["scale"], a["out"],
                                                  a["ldo"], a["lse"], a["ws"], a["wsb"], None)]


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), INVALID), (dict(n=-1), INVALID), (dict(heads=27), INVALID), (dict(hk=0), INVALID),
    (dict(dim=96), SHAPE), (dict(dim=256), SHAPE), (dict(tokens=2 ** 30 + 1), SHAPE), (dict(n=2 ** 20 + 1), SHAPE),
    (dict(scale=float("nan")), INVALID), (dict(scale=-float("inf")), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(out=None), INVALID), (dict(cu=None), INVALID),
    (dict(ldq=3576), INVALID), (dict(ldk=504), INVALID), (dict(ldv=504), INVALID), (dict(ldo=3576), INVALID),
    (dict(ldq=3588), ALIGN), (dict(ldv=516), ALIGN), (dict(q=0x1008), ALIGN), (dict(k=0x2002), ALIGN),
    (dict(v=0x3004), ALIGN), (dict(out=0x5008), ALIGN), (dict(cu=0x4002), ALIGN), (dict(lse=0x6002), ALIGN),
    (dict(ldq=2 ** 36), SHAPE), (dict(ldk=2 ** 36), SHAPE), (dict(ws=None), WS), (dict(wsb=255), WS),
    (dict(ws=0x8080), ALIGN), (dict(tokens=0), "QERL_OK"), (dict(n=0), "QERL_OK"),
])
def test_prompt_arguments(L, kw, want):
    assert _prompt(L, **kw) == want


def test_descriptor_layout():
    """KvCache mirrors the C struct: 13 fields, 8-byte aligned, no padding but what C has."""
    assert ctypes.sizeof(q.KvCache) == 4 * 4 + 9 * 8
    assert q.KvCache.num_pages.offset == 32 and q.KvCache.ld_table.offset == 80


def test_python_checks_types():
    cpu = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        q.kv_cache(cpu, cpu, torch.zeros((1, 1), dtype=torch.int32))
    with pytest.raises(TypeError):
        q.kv_cache(cpu.float(), cpu.float(), torch.zeros((1, 1), dtype=torch.int32))
