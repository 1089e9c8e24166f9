"""What the window calls refuse, on the host and before any work is enqueued."""
import pytest
import torch

import nvfp4_weight_quantized_03_gb300 as q

INVALID = "QERL_ERR_INVALID_ARGUMENT"

# Pointers that are no memory: only calls that are refused (or have nothing to do) may be made with them.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer calls run only without a GPU")


@pytest.fixture(scope="module")
def L():
    from nvfp4_weight_quantized_03_gb300 import build
    build.build()
    return q.lib()


def _decode(L, **kw):
    a = dict(window=10, sinks=4, heads=28, scale=0.1, num_seqs=3, ws=0x10000, wsb=1 << 30, q=0x1000, out=0x3000)
    a.update(kw)
    c = q.KvCache()
    for name, value in dict(k=0x10000, v=0x20000, dtype=q.QERL_BF16, num_kv_heads=4, head_dim=128, page_size=16,
                            num_pages=10, page_table=0x30000, num_seqs=a["num_seqs"], max_pages=5, ld_table=5).items():
        setattr(c, name, value)
    return q.STATUS_NAMES[L.qerl_window_decode_attention(c, a["q"], 3584, a["heads"], 0x2000, a["window"], a["sinks"],
                                                         a["scale"], a["out"], 3584, 0x4000, a["ws"], a["wsb"], None)]


def _prompt(L, **kw):
    a = dict(window=10, sinks=4, tokens=5, dim=128, scale=0.1, q=0x1000, out=0x4000, ws=0x10000, wsb=1 << 30)
    a.update(kw)
    return q.STATUS_NAMES[L.qerl_window_prompt_attention(a["q"], 512, 0x2000, 512, 0x3000, 512, a["tokens"], 4, 4,
                                                         a["dim"], 0x5000, 2, a["window"], a["sinks"], a["scale"],
                                                         a["out"], 512, 0x6000, a["ws"], a["wsb"], None)]


@pytest.mark.parametrize("kw", [dict(window=0), dict(window=-1), dict(window=-2 ** 31), dict(sinks=-1),
                                dict(scale=float("nan")), dict(q=None), dict(out=None)])
def test_refused(L, kw):
    assert _decode(L, **kw) == INVALID
    assert _prompt(L, **kw) == INVALID


def test_workspace_shape_and_alignment(L):
    assert _decode(L, wsb=255) == "QERL_ERR_WORKSPACE" and _prompt(L, wsb=255) == "QERL_ERR_WORKSPACE"
    assert _decode(L, q=0x1004) == "QERL_ERR_MISALIGNED" and _prompt(L, q=0x1004) == "QERL_ERR_MISALIGNED"
    assert _prompt(L, dim=96) == "QERL_ERR_UNSUPPORTED_SHAPE"


def test_nothing_to_do(L):
    assert _decode(L, num_seqs=0) == "QERL_OK" and _prompt(L, tokens=0) == "QERL_OK"
    # the window is looked at all the same
    assert _decode(L, num_seqs=0, window=0) == INVALID and _prompt(L, tokens=0, sinks=-1) == INVALID


@pytest.mark.parametrize("window,sinks", [(2 ** 31, 0), (5, 2 ** 32), (-2 ** 31 - 1, 0)])
def test_binding_refuses_wider_numbers(window, sinks):
    with pytest.raises(ValueError):
        q.qerl_window_decode_attention(None, None, None, window, sinks, 1.0, None, None, None)
    with pytest.raises(ValueError):
        q.qerl_window_prompt_attention(None, None, None, None, window, sinks, 1.0, None, None, None)
