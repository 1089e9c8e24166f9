"""The window, tree and page calls refuse memory that their launch could not reach, and tensors of another shape or
type.  Run on stand-ins for tensors, with a library that notes whether it was called, so nothing reaches a GPU."""
import pytest
import torch

import nvfp4_weight_quantized_03_gb300 as q
from test_attention_memory_checks import BF, F32, I32, Stand, _cache, lib  # noqa: F401 (lib is a fixture)


def _calls(dev=0):
    """name -> (function, its arguments by name)."""
    rows = lambda n, h: Stand((n, h, 64), BF, dev)
    ws = lambda: Stand((1 << 20,), torch.uint8, dev)
    ints = lambda *shape: Stand(shape, I32, dev)
    return {
        "window_decode": (q.qerl_window_decode_attention, dict(
            cache=_cache(dev), q=rows(3, 4), lengths=ints(3), window=7, sinks=2, scale=0.1, out=rows(3, 4),
            lse=Stand((3, 4), F32, dev), workspace=ws())),
        "window_prompt": (q.qerl_window_prompt_attention, dict(
            q=rows(9, 4), k=rows(9, 2), v=rows(9, 2), cu_seqlens=ints(3), window=7, sinks=2, scale=0.1, out=rows(9, 4),
            lse=Stand((9, 4), F32, dev), workspace=ws())),
        "tree": (q.qerl_tree_attention, dict(
            cache=_cache(dev), q=rows(9, 4), k=rows(9, 2), v=rows(9, 2), cu_tokens=ints(4), lengths=ints(3),
            mask=Stand((9, 2), torch.int64, dev), scale=0.1, out=rows(9, 4), lse=Stand((9, 4), F32, dev),
            workspace=ws())),
        "fork": (q.qerl_kv_fork, dict(
            cache=_cache(dev), parents=ints(2), children=ints(2), lengths=ints(2), new_pages=ints(2), workspace=ws())),
        "compact": (q.qerl_kv_compact, dict(
            cache=_cache(dev), lengths=ints(3), new_table=ints(3, 4), live_pages=ints(1), workspace=ws())),
    }


TENSORS = [(call, name) for call, (_, kw) in _calls().items() for name, x in kw.items() if isinstance(x, Stand)]


@pytest.mark.parametrize("call", list(_calls()))
def test_good_calls_go_through(lib, call):
    f, kw = _calls()[call]
    assert f(**kw) == 0 and lib.calls == 1


@pytest.mark.parametrize("dev", [-1, 1])
@pytest.mark.parametrize("call,name", TENSORS)
def test_memory_of_the_host_or_another_device(lib, call, name, dev):
    f, kw = _calls()[call]
    x = kw[name]
    with pytest.raises((TypeError, ValueError)):
        f(**{**kw, name: Stand(x.shape, x.dtype, dev)})
    assert lib.calls == 0


@pytest.mark.parametrize("call", list(_calls()))
def test_everything_on_another_device_than_the_current_one(lib, call):
    f, kw = _calls(dev=1)[call]
    with pytest.raises(ValueError):
        f(**kw)
    assert lib.calls == 0


@pytest.mark.parametrize("call", ["window_decode", "tree", "fork", "compact"])
def test_a_cache_on_another_device(lib, call):
    f, kw = _calls()[call]
    with pytest.raises(ValueError):
        f(**{**kw, "cache": _cache(1)})
    assert lib.calls == 0


@pytest.mark.parametrize("call", list(_calls()))
def test_a_workspace_in_pieces(lib, call):
    f, kw = _calls()[call]
    with pytest.raises(ValueError):
        f(**{**kw, "workspace": Stand((1 << 20,), torch.uint8, 0, contiguous=False)})
    assert lib.calls == 0


@pytest.mark.parametrize("call,name", [x for x in TENSORS if x[1] != "workspace"])
def test_another_type_or_shape(lib, call, name):
    f, kw = _calls()[call]
    x = kw[name]
    for bad in (Stand(x.shape, torch.float16), Stand((x.shape[0] + 1, *x.shape[1:]), x.dtype),
                Stand((*x.shape, 1), x.dtype)):
        if name == "cu_seqlens" and bad.dtype is x.dtype and bad.dim() == 1:
            continue  # another number of sequences
        if call == "fork" and name == "parents" and bad.dtype is x.dtype and bad.dim() == 1:
            continue  # the count is taken from it; the others then differ
        with pytest.raises((TypeError, ValueError)):
            f(**{**kw, name: bad})
        assert lib.calls == 0


@pytest.mark.parametrize("call,name", [("tree", "mask"), ("fork", "lengths"), ("compact", "lengths"), ("tree", "cu_tokens")])
def test_entries_in_pieces(lib, call, name):
    f, kw = _calls()[call]
    x = kw[name]
    with pytest.raises((TypeError, ValueError)):
        f(**{**kw, name: Stand(x.shape, x.dtype, 0, contiguous=False)})
    assert lib.calls == 0


def test_lse_and_mask_may_be_left_out(lib):
    for call in ("window_decode", "window_prompt", "tree"):
        f, kw = _calls()[call]
        assert f(**{**kw, "lse": None}) == 0
    f, kw = _calls()["tree"]
    assert f(**{**kw, "mask": None}) == 0 and lib.calls == 4
